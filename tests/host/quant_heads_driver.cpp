// Host-only driver for the sanitizer test of the 8-bit layers' and the head
// steps' entry points (tplinear_quant.cpp, tplinear_heads.cpp): linked against
// recording launchers, it checks which kernel a call takes and the addresses it
// is given, and runs every refusal.  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_host_sanitizers_quant.py.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "heads.h"
#include "kernels.h"
#include "quant.h"
#include "tplinear.h"

namespace {
const char *last = "";
tpl::GemmArgs lg;
tpl::ReduceArgs lr;
tpl::QuantArgs lq;
tpl::GemmExtra lex;
tpl::HeadArgs lh;
int lout = -1, launches = 0;
int failures = 0;
hipError_t note(const char *name) { last = name; ++launches; return hipSuccess; }
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

static hipError_t gemm(const char *name, const GemmArgs &g, int out, const GemmExtra &ex, const QuantArgs &q) {
    lg = g; lout = out; lex = ex; lq = q;
    return note(name);
}
hipError_t launch_quant_generic(const GemmArgs &g, int o, const GemmExtra &ex, const QuantArgs &q, hipStream_t) { return gemm("generic", g, o, ex, q); }
hipError_t launch_quant_tile(const GemmArgs &g, int o, const GemmExtra &ex, const QuantArgs &q, hipStream_t) { return gemm("tile", g, o, ex, q); }
hipError_t launch_quant_narrow(const GemmArgs &g, int o, const GemmExtra &ex, const QuantArgs &q, hipStream_t) { return gemm("narrow", g, o, ex, q); }
hipError_t launch_quant_skinny(const GemmArgs &g, int o, const FoldArgs *f, const GemmExtra &ex, const QuantArgs &q, hipStream_t) {
    return gemm(f ? "skinny fold" : "skinny", g, o, ex, q);
}
// the launchers' own rules on alignment, restated
bool quant_dma_supported(const GemmArgs &g, const GemmExtra &, int) {
    return g.K > 0 && g.K % 16 == 0 && g.lda % 16 == 0 && g.ldb % 16 == 0 && g.a_shard % 16 == 0 && g.b_shard % 16 == 0 &&
           (uintptr_t)g.A % 16 == 0 && (uintptr_t)g.B % 16 == 0;
}
bool quant_skinny_supported(const GemmArgs &g, const GemmExtra &ex) { return g.M <= (ex.act == ACT_SWIGLU ? 48 : 32) && quant_dma_supported(g, ex, 0); }
bool quant_rowfold_supported(const GemmArgs &g, const ReduceArgs &r, const QuantArgs &) {
    return quant_dma_supported(g, GemmExtra{}, 0) && (r.slice_rows >= g.M || r.slice_rows % 256 == 0);
}
hipError_t launch_quant_rowfold(const GemmArgs &g, const ReduceArgs &r, const QuantArgs &q, int o, hipStream_t) {
    lg = g; lr = r; lq = q; lout = o;
    return note("rowfold");
}
hipError_t launch_quant_fold(const ReduceArgs &r, const QuantArgs &q, bool per_shard, int o, hipStream_t) {
    lr = r; lq = q; lout = o;
    return note(per_shard ? "partials + fold" : "partials + integer fold");
}
hipError_t launch_quantize_rows(const QuantizeArgs &, int, hipStream_t) { return note("quantize"); }
hipError_t launch_qk_norm_rope(const HeadArgs &a, int, hipStream_t) { lh = a; return note("qk"); }
hipError_t launch_kv_append(const HeadArgs &a, int, hipStream_t) { lh = a; return note("append"); }
hipError_t launch_qk_norm_rope_backward(const HeadArgs &a, int, hipStream_t) { lh = a; return note("backward"); }
int64_t qk_backward_blocks(int64_t) { return 768; }
}  // namespace tpl

static bool is(const char *a) {
    for (const char *b = last; *a || *b; ++a, ++b)
        if (*a != *b) return false;
    return true;
}

static int8_t *const X = (int8_t *)0x100000, *const W = (int8_t *)0x200000;
static float *const SX = (float *)0x300000, *const SW = (float *)0x400000;
static void *const Y = (void *)0x500000, *const WS = (void *)0x600000;

static void column(int64_t M, int64_t N, int64_t K, int32_t P, int act, const char *want) {
    const int64_t on = act ? N / 2 : N;
    CHECK(tp_linear_column_quant(X, K, SX, 1, W, K, SW, nullptr, Y, on, TP_Y_CONCAT, act, M, N, K, P, TP_BF16, nullptr) == TP_OK);
    CHECK(is(want));
    CHECK(lg.b_shard == N / P * K && lg.c_shard == on / P && lg.N == on / P && lg.P == P && lq.w_shard == N / P && lq.x_shard == 0);
}
static void row(int64_t M, int64_t N, int64_t K, int32_t P, int32_t G, int mode, const char *want) {
    const size_t need = tp_row_workspace_bytes(mode, M, N, P);
    CHECK(tp_linear_row_quant(X, K, SX, G, G, W, K, SW, nullptr, Y, nullptr, N, 0, mode, WS, need, M, N, K, P, TP_BF16, nullptr) == TP_OK);
    CHECK(is(want));
}

int main() {
    // Which kernel a column layer takes, around each threshold (256 CUs).
    column(16, 28672, 8192, 8, 0, "skinny");
    column(32, 28672, 8192, 8, 0, "skinny");
    column(33, 10240, 8192, 8, 0, "narrow");
    column(32, 28672, 8192, 8, 1, "skinny");
    column(48, 8192, 8192, 8, 1, "skinny");        // gated: 64 tiles of 128 W rows, a quarter of the CUs
    column(48, 8320, 8192, 8, 1, "narrow");        // 65
    column(49, 8192, 8192, 8, 1, "narrow");
    column(256, 28672, 4096, 8, 0, "narrow");      // 112 tiles of 256 x 256
    column(257, 28672, 4096, 8, 0, "tile");        // 224
    column(768, 10240, 8192, 8, 0, "narrow");
    column(769, 10240, 8192, 8, 0, "tile");
    column(4096, 28672, 4096, 8, 1, "tile");
    column(4096, 28672, 4097, 8, 0, "generic");    // K not a multiple of 16
    // And a row layer.
    row(16, 8192, 28672, 8, 8, TP_ROW_FUSED, "skinny fold");
    row(17, 8192, 28672, 8, 8, TP_ROW_FUSED, "partials + fold");
    row(16, 2048, 28672, 8, 8, TP_ROW_SUM, "partials + fold");     // few workgroups, a long K
    row(16, 2048, 4096, 8, 8, TP_ROW_SUM, "skinny fold");
    row(4096, 4096, 14336, 8, 8, TP_ROW_FUSED, "rowfold");
    CHECK(lg.a_shard == 1792 && lg.b_shard == 1792 && lg.K == 1792 && lg.P == 8 && lq.x_shard == 1 && lr.Y == Y);
    row(1024, 4096, 14336, 8, 8, TP_ROW_FUSED, "partials + fold");  // 128 tiles of 256 x 128: too few for K / P = 1792
    CHECK(lr.partials == WS && lr.shard_stride == 1024 * 4096 && lr.P == 8);
    row(1280, 4096, 14336, 8, 8, TP_ROW_FUSED, "rowfold");          // 160
    row(2048, 4096, 4096, 8, 8, TP_ROW_SCATTER, "rowfold");
    CHECK(lr.slice_rows == 256 && lr.slice_stride == 256 * 4096);
    row(2040, 4096, 4096, 8, 8, TP_ROW_SCATTER, "partials + fold"); // slices of 255 rows
    row(4096, 4096, 14336, 8, 1, TP_ROW_SUM, "tile");               // one scale a token: one product
    CHECK(lg.P == 1 && lg.K == 14336 && lg.a_shard == 0 && lg.C == Y && lq.x_shard == 0 && lout == tpl::OUT_BF16);
    row(256, 4096, 14336, 8, 1, TP_ROW_SUM, "partials + integer fold");
    row(200, 2048, 4096, 8, 1, TP_ROW_SUM, "narrow");
    row(2048, 4096, 4096, 8, 1, TP_ROW_SCATTER, "narrow");          // the slices as shards in M
    CHECK(lg.P == 8 && lg.M == 256 && lg.a_shard == 256 * 4096 && lg.b_shard == 0 && lg.c_shard == 256 * 4096 && lq.x_shard == 256);
    row(300, 520, 512, 4, 4, TP_ROW_PARTIAL, "narrow");
    CHECK(lout == tpl::OUT_F32 && lg.c_shard == 300 * 520 && lq.x_shard == 1 && lq.w_shard == 0);
    setenv("TPLINEAR_ROW_FOLD", "gemm", 1);
    row(32, 8192, 28672, 8, 8, TP_ROW_FUSED, "skinny fold");
    row(33, 8192, 28672, 8, 8, TP_ROW_FUSED, "rowfold");
    row(128, 4096, 14336, 8, 8, TP_ROW_FUSED, "rowfold");
    row(64, 4096, 14336, 8, 1, TP_ROW_FUSED, "narrow");
    unsetenv("TPLINEAR_ROW_FOLD");

    // Refusals queue nothing.
    const int before = launches;
    CHECK(tp_linear_column_quant(X, 131072, SX, 1, W, 131072, SW, nullptr, Y, 16, TP_Y_CONCAT, 0, 4, 16, 131072, 1, TP_BF16, nullptr) == TP_ERR_SHAPE);
    CHECK(tp_linear_row_quant(X, 64, SX, 2, 2, W, 64, SW, nullptr, Y, nullptr, 16, 0, TP_ROW_SUM, WS, 1 << 20, 4, 16, 64, 4, TP_BF16, nullptr) == TP_ERR_SHAPE);
    CHECK(tp_linear_row_quant(X, 64, SX, 4, 4, W, 64, SW, nullptr, Y, nullptr, 16, 0, TP_ROW_SUM, WS, 16, 4, 16, 64, 4, TP_BF16, nullptr) == TP_ERR_WORKSPACE);
    CHECK(tp_linear_row_quant(X, INT64_MAX, SX, 4, 4, W, 64, SW, nullptr, Y, nullptr, 16, 0, TP_ROW_SUM, WS, 1 << 20, 4, 16, 64, 4, TP_BF16, nullptr) == TP_ERR_SHAPE);
    CHECK(tp_quantize_rows(X, INT64_MAX, W, 8, SX, 1, 4, 8, 1, TP_BF16, nullptr) == TP_ERR_SHAPE);
    CHECK(tp_quantize_rows(X, 8, W, 8, SX, 1, INT64_MAX, 8, 1, TP_BF16, nullptr) == TP_ERR_SHAPE);
    CHECK(launches == before);
    CHECK(tp_quantize_rows(X, 8, W, 8, SX, 2, 4, 8, 2, TP_F32, nullptr) == TP_OK && is("quantize"));

    // Heads: the shards' places in either layout, and the cache's strides.
    const float *C = SX, *S = SW;
    CHECK(tp_qk_norm_rope(X, 2048, TP_Y_CONCAT, (const int64_t *)W, C, S, 9, 128, TP_ROPE_HALVES, nullptr, nullptr, 0.0f, Y, 1024, nullptr, 0, 7, 8, 4, 128, 4,
                          TP_BF16, nullptr, nullptr) == TP_OK && is("qk"));
    CHECK(lh.x_shard == 512 && lh.hq == 2 && lh.hk == 1);
    CHECK(tp_qk_norm_rope(X, 520, TP_Y_SHARDS, (const int64_t *)W, C, S, 9, 128, TP_ROPE_PAIRS, nullptr, nullptr, 0.0f, Y, 1024, nullptr, 0, 7, 8, 4, 128, 4,
                          TP_BF16, nullptr, nullptr) == TP_OK);
    CHECK(lh.x_shard == 7 * 520 && lh.pairs == 1);
    auto append = [&](int64_t pages, int64_t sp, int64_t page, int64_t ss, int64_t sh) {
        return tp_kv_append(X, 2048, TP_Y_CONCAT, C, S, 9, 128, TP_ROPE_HALVES, nullptr, nullptr, 0.0f, (const int32_t *)W, (const int32_t *)W, 2,
                            (const int32_t *)W, 8, 8, Y, WS, pages, page, sp, ss, sh, nullptr, 0, 7, 8, 4, 128, 4, TP_BF16, nullptr, nullptr);
    };
    CHECK(append(10, 16 * 512, 16, 512, 128) == TP_OK && is("append"));           // [page, slot, head]
    CHECK(append(10, 16 * 512, 16, 128, 16 * 128) == TP_OK);                      // [page, head, slot]
    CHECK(append(10, 512, 16, 10 * 512, 128) == TP_OK);                           // pages inside slots
    CHECK(append(10, 16 * 1024, 16, 1024, 128) == TP_OK);                         // keys and values side by side
    CHECK(append(1, 0, 16, 512, 128) == TP_OK);                                   // one page: any stride
    const int n = launches;
    CHECK(append(10, 16 * 512 - 1, 16, 512, 128) == TP_ERR_SHAPE);
    CHECK(append(10, 16 * 512, 16, 511, 128) == TP_ERR_SHAPE);
    CHECK(append(10, 16 * 512, 16, 512, 127) == TP_ERR_SHAPE);
    CHECK(append(10, INT64_MAX, 16, 512, 128) == TP_ERR_SHAPE);
    CHECK(append(10, -512, 16, 512, 128) == TP_ERR_SHAPE);
    CHECK(append(INT64_MAX, 16 * 512, 16, 512, 128) == TP_ERR_SHAPE);
    CHECK(append(10, 16 * 512, 0, 512, 128) == TP_ERR_SHAPE);
    CHECK(launches == n);
    CHECK(tp_qk_norm_rope_backward(X, 2048, TP_Y_CONCAT, (const int64_t *)W, C, S, 9, 128, TP_ROPE_HALVES, SX, SX, 0.0f, Y, 1024, Y, 512, nullptr, 0, WS, 2056, SX, SW,
                                   WS, tp_qk_norm_rope_workspace_bytes(7, 128), 7, 8, 4, 128, 4, TP_BF16, nullptr, nullptr) == TP_OK && is("backward"));
    CHECK(lh.x_shard == 512 && lh.dx_shard == 512 && lh.lddx == 2056 && lh.partials == (float *)WS);
    if (failures) return 1;
    std::printf("quant and heads driver ok (%d launches)\n", launches);
    return 0;
}
