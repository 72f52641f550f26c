// Host-only driver for the sanitizer test of attention over a paged cache, the reads
// and appends of a cache in 8 bits, and the step between two blocks (tplinear_cache.cpp,
// attn.cpp, tplinear_norm.cpp): linked against recording launchers, it checks which
// kernel a call takes, how its work is cut and the addresses and strides it is given,
// that the workspace holds every plan of its sizes, and runs the refusals.  Built with
// AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_host_sanitizers_cache_norm.py.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "attn.h"
#include "attn_plan.h"
#include "heads.h"
#include "kernels.h"
#include "norm.h"
#include "tplinear.h"

namespace {
const char *last = "";
tpl::AttnArgs la;
tpl::AttnPlan lp;
tpl::ReadArgs lr;
tpl::HeadArgs lh;
tpl::NormArgs ln;
bool ldma = false;
int les = 0, launches = 0, failures = 0;
hipError_t note(const char *name, int es) { last = name; les = es; ++launches; return hipSuccess; }
hipError_t attention(const char *name, const tpl::AttnArgs &a, const tpl::AttnPlan &p, bool dma) {
    la = a; lp = p; ldma = dma;
    return note(name, 0);
}
}  // namespace
#define CHECK(c) do { if (!(c)) { std::fprintf(stderr, "check failed: %s (line %d, last %s)\n", #c, __LINE__, last); ++failures; } } while (0)

namespace tpl {
// the 16-bit layers: not reached here
hipError_t launch_gemm_tile(const GemmArgs &, int, const GemmExtra *, hipStream_t) { std::abort(); }
hipError_t launch_gemm_narrow(const GemmArgs &, int, const GemmExtra *, hipStream_t) { std::abort(); }
bool gemm_tile_supported(const GemmArgs &, const GemmExtra *) { std::abort(); }
hipError_t launch_gemm_skinny(const GemmArgs &, int, const FoldArgs *, const GemmExtra *, hipStream_t) { std::abort(); }
bool gemm_skinny_supported(const GemmArgs &, const GemmExtra *) { std::abort(); }
hipError_t launch_gemm_generic(const GemmArgs &, int, int, const GemmExtra *, hipStream_t) { std::abort(); }
hipError_t launch_shard_fold(const ReduceArgs &, int, hipStream_t) { std::abort(); }
hipError_t launch_gemm_rowfold(const GemmArgs &, const ReduceArgs &, hipStream_t) { std::abort(); }
bool gemm_rowfold_supported(const GemmArgs &, const ReduceArgs &) { std::abort(); }
hipError_t launch_embedding(const EmbedArgs &, int, hipStream_t) { std::abort(); }
hipError_t launch_fill_zero(void *, size_t, hipStream_t) { std::abort(); }
int device_cu_count() { return 256; }

hipError_t launch_attention_any(const AttnArgs &a, int es, hipStream_t) { la = a; return note("any", es); }
hipError_t launch_attention_bf16(const AttnArgs &a, const AttnPlan &p, bool d, hipStream_t) { return attention("bf16", a, p, d); }
hipError_t launch_attention_f32(const AttnArgs &a, const AttnPlan &p, bool d, hipStream_t) { return attention("f32", a, p, d); }
hipError_t launch_attention_bf16_int8(const AttnArgs &a, const AttnPlan &p, bool d, hipStream_t) { return attention("bf16 int8", a, p, d); }
hipError_t launch_attention_f32_int8(const AttnArgs &a, const AttnPlan &p, bool d, hipStream_t) { return attention("f32 int8", a, p, d); }
hipError_t launch_kv_read(const ReadArgs &a, int es, hipStream_t) { lr = a; return note("read", es); }
hipError_t launch_kv_append_quant(const HeadArgs &a, int es, hipStream_t) { lh = a; return note("append", es); }
hipError_t launch_residual_norm(const NormArgs &a, int es, hipStream_t) { ln = a; return note("norm", es); }
hipError_t launch_residual_norm_backward(const NormArgs &a, int es, hipStream_t) { ln = a; return note("backward", es); }
int64_t norm_backward_blocks(int64_t, int64_t) { return 256; }
}  // namespace tpl

static bool is(const char *a) {
    for (const char *b = last; *a || *b; ++a, ++b)
        if (*a != *b) return false;
    return true;
}

static void *at(int64_t i) { return (void *)(uintptr_t)(0x100000 * i); }
static const int32_t *const CU = (const int32_t *)at(1), *const PAST = (const int32_t *)at(2), *const TABLE = (const int32_t *)at(3);

// An attention call with sizes that a test changes one at a time.
struct Call {
    int64_t T = 64, B = 64, Hq = 32, Hkv = 8, D = 128, page = 64, pages = 1000, max_pages = 256, window = 0, ldq = 0, sp = -1, ss = -1, sh = -1;
    int32_t dtype = TP_BF16;
    bool int8 = false;
    uintptr_t shift = 0;
    float scale = 0.1f;
    size_t less = 0;
    tp_status go() const {
        const int64_t h = sh < 0 ? D : sh, s = ss < 0 ? Hkv * D : ss, p = sp < 0 ? page * Hkv * D : sp;
        const size_t n = tp_kv_attention_workspace_bytes(T, B, Hq, Hkv, D);
        const char *k = (const char *)at(4) + shift;
        return tp_kv_attention(at(6), ldq ? ldq : Hq * D, CU, PAST, B, TABLE, max_pages, max_pages, k, at(5), pages, page, p, s, h,
                               int8 ? (const float *)at(7) : nullptr, int8 ? (const float *)at(8) : nullptr, page * Hkv, Hkv, 1, scale, window, at(9), Hq * D,
                               nullptr, 0, n ? at(10) : nullptr, n - (n ? less : 0), T, Hq, Hkv, D, dtype, nullptr, nullptr);
    }
};

static uint64_t seed = 1;
static int64_t draw(int64_t lo, int64_t hi) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return lo + (int64_t)((seed >> 33) % (uint64_t)(hi - lo + 1));
}

int main() {
    // Which kernel, and how it is cut.
    auto taken = [](const Call &c, const char *want) { CHECK(c.go() == TP_OK); CHECK(is(want)); };
    Call c;
    taken(c, "bf16");
    CHECK(lp.few && lp.stream && ldma && lp.row_tiles == 64 * 4 / 32 + 64 && lp.groups == 1024 && lp.last_pos == 256 * 64);
    CHECK(lp.window == 2 * tpl::PLAN_FAR && la.G == 4 && la.c.shift == 6 && la.c.s_page == 64 * 1024 && la.c.s_slot == 1024 && la.c.s_head == 128);
    c.int8 = true;
    taken(c, "bf16 int8");
    CHECK(ldma && lp.groups == 2048 && la.c.ss_page == 512 && la.c.ss_slot == 8 && la.c.ss_head == 1);
    c.dtype = TP_F32;
    taken(c, "f32 int8");
    c.int8 = false;
    taken(c, "f32");
    CHECK(lp.groups == 512);
    c = Call(); c.T = 4096;
    taken(c, "bf16");
    CHECK(!lp.few && lp.stream && lp.row_tiles == 4096 * 4 / 128 + 64);
    c.T = 20000;
    taken(c, "bf16");
    CHECK(!lp.few && !lp.stream && tp_kv_attention_workspace_bytes(c.T, c.B, c.Hq, c.Hkv, c.D) == 0);
    c.T = 2048; c.B = 1; c.Hq = 64; c.max_pages = 32;    // a prompt from its first token on
    taken(c, "bf16");
    CHECK(!lp.few && !lp.stream);
    c.max_pages = 128;                              // or the end of a longer one
    taken(c, "bf16");
    CHECK(lp.stream);
    c.max_pages = 32; c.window = 500;
    taken(c, "bf16");
    CHECK(lp.stream);
    c.window = 0; c.Hq = 4; c.Hkv = 1;
    taken(c, "bf16");
    CHECK(lp.stream);
    // What goes to LDS without a stop: rows at multiples of 16 bytes.
    for (const bool q : {false, true}) {
        const int64_t n = q ? 16 : 8;
        c = Call(); c.int8 = q;
        c.shift = 8; taken(c, q ? "bf16 int8" : "bf16"); CHECK(!ldma); c.shift = 0;
        c.sh = 128 + n - 1; c.ss = 2000 - 2000 % n; c.sp = 64 * c.ss; taken(c, q ? "bf16 int8" : "bf16"); CHECK(!ldma);
        c.sh = 128 + n; taken(c, q ? "bf16 int8" : "bf16"); CHECK(ldma);
        c.ss += 1; c.sp = 64 * c.ss; taken(c, q ? "bf16 int8" : "bf16"); CHECK(!ldma);
        c = Call(); c.int8 = q; c.D = 72;
        taken(c, q ? "bf16 int8" : "bf16"); CHECK(ldma == !q);
    }
    // What 32 bits, or the tiles, do not hold.
    for (const int64_t d : {1, 7, 257, 264, 1000}) { c = Call(); c.D = d; taken(c, "any"); }
    for (const int64_t d : {9, 12, 100, 127, 250}) {
        c = Call(); c.D = d; taken(c, "bf16"); CHECK(!ldma);
        c.int8 = true; taken(c, "bf16 int8"); CHECK(!ldma);
    }
    c = Call(); c.max_pages = int64_t(1) << 30; taken(c, "any");
    c = Call(); c.max_pages = 1 << 20; c.page = 1 << 12; taken(c, "any");                       // 2^32 positions
    c = Call(); c.page = int64_t(1) << 33; c.max_pages = 1; c.ss = 1; c.sp = 0; taken(c, "any"); // one page of all
    CHECK(la.c.page == 0xFFFFFFFFu && la.c.shift == -1);
    c = Call(); c.window = (int64_t)tpl::PLAN_FAR; taken(c, "any");                              // with the positions past 2^29
    c = Call(); c.window = 2 * (int64_t)tpl::PLAN_FAR; taken(c, "bf16"); CHECK(lp.window == 2 * tpl::PLAN_FAR);
    c = Call(); c.window = INT64_MAX; taken(c, "bf16"); CHECK(lp.window == 2 * tpl::PLAN_FAR);
    c = Call(); c.window = 77; taken(c, "bf16"); CHECK(lp.window == 77);
    c = Call(); c.T = INT32_MAX; c.B = 1; taken(c, "any");
    c = Call(); c.T = 1000; c.B = 1000; c.max_pages = 1 << 18; taken(c, "bf16"); CHECK(!lp.stream);   // units of all runs past 2^31
    c = Call(); c.page = 48; taken(c, "bf16"); CHECK(la.c.shift == -1 && la.c.page == 48);

    for (int64_t G = 1; G <= 65536; ++G) {
        const tpl::AttnPlan p = tpl::attention_plan(64, 1, 1, (int32_t)G, 64, 2, false);
        for (const uint32_t x : {0u, (uint32_t)G - 1, (uint32_t)G, (uint32_t)(INT32_MAX / G * G), (uint32_t)(INT32_MAX / G * G - 1), (uint32_t)INT32_MAX})
            CHECK((uint32_t)((uint64_t)x * p.g.by >> p.g.shift) == x / (uint32_t)G);
    }
    for (int i = 0; i < 100000; ++i) {
        const int64_t d = i < 2 ? 0xFFFFFFFFll - i : draw(1, i % 2 ? 5000 : 0xFFFFFFFFll);
        const tpl::Divisor v = tpl::divisor(d);
        for (const int64_t x : {(int64_t)0, d - 1, d, draw(0, INT32_MAX), INT32_MAX / d * d, (int64_t)INT32_MAX})
            CHECK(x > INT32_MAX || (int64_t)((uint64_t)x * v.by >> v.shift) == x / d);
    }
    // The workspace of the sizes holds the plan of every type.
    for (int i = 0; i < 200000; ++i) {
        const int64_t G = draw(1, 16), Hkv = draw(1, 16), D = i % 4 ? draw(1, 264) : 8 * draw(1, 33), B = draw(1, i % 3 ? 64 : 4000), T = draw(1, i % 2 ? 200 : 1 << 20);
        const size_t n = tp_kv_attention_workspace_bytes(T, B, Hkv * G, Hkv, D);
        const int64_t d = D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : 256;
        for (int k = 0; k < 4 && D >= 8 && D <= 256; ++k) {
            const tpl::AttnPlan p = tpl::attention_plan(T, B, Hkv, (int32_t)G, D, k & 1 ? 4 : 2, k & 2);
            CHECK(p.groups >= 8 && p.groups % 8 == 0);
            for (const uint32_t x : {0u, 1u, (uint32_t)G - 1, (uint32_t)G, (uint32_t)draw(0, INT32_MAX), (uint32_t)(draw(0, INT32_MAX / G) * G), (uint32_t)INT32_MAX})
                CHECK((uint32_t)((uint64_t)x * p.g.by >> p.g.shift) == x / (uint32_t)G);
            if (p.stream) CHECK(n >= (size_t)(tpl::plan_desc_bytes(p.groups) + tpl::plan_stats_bytes(p.groups) + 2 * p.groups * (p.few ? 32 : 128) * d * 4));
        }
        CHECK(n <= 300u << 20);
    }

    // Refusals queue nothing.
    const int before = launches;
    c = Call(); c.less = 1; CHECK(c.go() == TP_ERR_WORKSPACE);
    c = Call(); c.ldq = INT64_MAX; CHECK(c.go() == TP_ERR_SHAPE);
    c = Call(); c.sp = INT64_MAX; CHECK(c.go() == TP_ERR_SHAPE);
    c = Call(); c.ss = INT64_MAX / 32; CHECK(c.go() == TP_ERR_SHAPE);
    c = Call(); c.sh = INT64_MAX / 4; CHECK(c.go() == TP_ERR_SHAPE);
    c = Call(); c.pages = INT64_MAX; CHECK(c.go() == TP_ERR_SHAPE);
    c = Call(); c.max_pages = INT64_MAX; CHECK(c.go() == TP_ERR_SHAPE);
    c = Call(); c.window = INT64_MIN; CHECK(c.go() == TP_ERR_SHAPE);
    c = Call(); c.T = INT64_MAX; CHECK(c.go() == TP_ERR_SHAPE);
    c = Call(); c.B = INT64_MAX; CHECK(c.go() == TP_ERR_SHAPE);
    c = Call(); c.Hq = INT64_MAX; c.ldq = 1; CHECK(tp_kv_attention_workspace_bytes(c.T, c.B, c.Hq, c.Hkv, c.D) == 0);
    c = Call(); c.scale = -1.0f; CHECK(c.go() == TP_ERR_SHAPE);
    CHECK(tp_kv_read(CU, PAST, 2, TABLE, 8, 8, at(4), at(5), 100, 16, 16 * 512, 512, 128, nullptr, nullptr, 0, 0, 0, at(6), 511, at(7), 512, 9, 4, 128, TP_BF16,
                     nullptr, nullptr) == TP_ERR_SHAPE);
    CHECK(tp_residual_norm(at(1), INT64_MAX, nullptr, 0, nullptr, 0, nullptr, nullptr, 1, 1, 0, at(2), 8, nullptr, 0, nullptr, 3, 8, TP_BF16, nullptr) == TP_ERR_SHAPE);
    CHECK(tp_residual_norm(at(1), 8, nullptr, 0, nullptr, 0, nullptr, nullptr, 1, 1, 0, at(2), 8, nullptr, 0, nullptr, INT64_MAX, 8, TP_BF16, nullptr) == TP_ERR_SHAPE);
    CHECK(launches == before);

    // The other calls' strides.
    CHECK(tp_kv_read(CU, PAST, 2, TABLE, 8, 8, at(4), at(5), 100, 16, 16 * 512, 512, 128, (const float *)at(8), (const float *)at(9), 64, 1, 16, at(6), 520, nullptr, 0,
                     9, 4, 128, TP_F32, nullptr, nullptr) == TP_OK && is("read") && les == 4);
    CHECK(lr.c.ss_page == 64 && lr.c.ss_slot == 1 && lr.c.ss_head == 16 && lr.ldk == 520 && !lr.V && lr.ldv == 0 && lr.c.B == 2 && lr.c.T == 9);
    const auto append = [&](int64_t ssp, int64_t sss, int64_t ssh) {
        return tp_kv_append_quant(at(11), 2048, TP_Y_CONCAT, (const float *)at(12), (const float *)at(13), 9, 128, TP_ROPE_HALVES, nullptr, nullptr, 0.0f, CU, PAST, 2,
                                  TABLE, 8, 8, (int8_t *)at(4), (int8_t *)at(5), 10, 16, 16 * 512, 512, 128, (float *)at(8), (float *)at(9), ssp, sss, ssh, nullptr, 0, 7,
                                  8, 4, 128, 4, TP_BF16, nullptr, nullptr);
    };
    CHECK(append(64, 4, 1) == TP_OK && is("append") && les == 2 && lh.ss_page == 64 && lh.ss_slot == 4 && lh.ss_head == 1 && lh.x_shard == 512);
    CHECK(append(64, 1, 16) == TP_OK && append(4, 40, 1) == TP_OK && append(1000, 33, 8) == TP_OK);
    CHECK(append(63, 4, 1) == TP_ERR_SHAPE && append(64, 3, 1) == TP_ERR_SHAPE && append(64, 4, 0) == TP_ERR_SHAPE && append(INT64_MAX, 4, 1) == TP_ERR_SHAPE);
    CHECK(tp_residual_norm(at(1), 8, at(3), 9, at(4), 0, at(5), nullptr, 0.5f, 2.0f, 1e-6f, at(2), 10, at(6), 11, (float *)at(7), 3, 8, TP_F32, nullptr) == TP_OK && is("norm"));
    CHECK(ln.ldy == 8 && ln.ldr == 9 && ln.ldg == 0 && ln.ldh == 10 && ln.ldn == 11 && ln.post == at(5) && !ln.pre && ln.scale == at(7) && les == 4);
    CHECK(tp_residual_norm_workspace_bytes(3, 8) == 256 * 3 * 8 * 4);
    const auto backward = [&](size_t n) {
        return tp_residual_norm_backward(at(1), 8, at(3), 9, at(4), 12, nullptr, at(5), 1, 1, 0, at(6), 13, nullptr, 0, at(7), 14, nullptr, 0, at(8), 15, nullptr,
                                         (float *)at(9), at(10), n, 3, 8, TP_BF16, nullptr);
    };
    CHECK(backward(256 * 3 * 8 * 4) == TP_OK && is("backward") && ln.lddh == 13 && ln.lddn == 0 && ln.lddy == 14 && ln.lddr == 0 && ln.lddg == 15 && ln.partials == at(10));
    CHECK(backward(256 * 3 * 8 * 4 - 1) == TP_ERR_WORKSPACE);
    if (failures) return 1;
    std::printf("cache and norm driver ok (%d launches)\n", launches);
    return 0;
}
