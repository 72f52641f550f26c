// Host-only driver: which form an attention call takes and how its work is cut
// (attn.cpp), for windows of any length and for calls whose items fill the GPU by
// themselves: the cases of tests/test_gpu_attention_windows.py and
// tests/test_gpu_attention_items.py, which compare what those forms compute.  Built with
// AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_host_sanitizers_form.py.
#include <cstdint>
#include <cstdio>

#include "attn.h"
#include "attn_plan.h"

namespace {
const char *last = "";
tpl::AttnPlan lp;
int failures = 0;
hipError_t note(const char *name, const tpl::AttnPlan &p) { last = name; lp = p; return hipSuccess; }
}  // namespace
#define CHECK(c) do { if (!(c)) { std::fprintf(stderr, "check failed: %s (line %d, last %s)\n", #c, __LINE__, last); ++failures; } } while (0)

namespace tpl {
hipError_t launch_attention_any(const AttnArgs &, int, hipStream_t) { return note("any", AttnPlan{}); }
hipError_t launch_attention_bf16(const AttnArgs &, const AttnPlan &p, bool, hipStream_t) { return note("tile", p); }
hipError_t launch_attention_f32(const AttnArgs &, const AttnPlan &p, bool, hipStream_t) { return note("tile", p); }
hipError_t launch_attention_bf16_int8(const AttnArgs &, const AttnPlan &p, bool, hipStream_t) { return note("tile", p); }
hipError_t launch_attention_f32_int8(const AttnArgs &, const AttnPlan &p, bool, hipStream_t) { return note("tile", p); }
}  // namespace tpl

static bool tile() { return last[0] == 't'; }

static void call(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_pages, int64_t page, int64_t window, int es = 2, bool int8 = false) {
    static const float one = 1.0f;
    tpl::AttnArgs a{};
    a.c.T = T; a.c.B = B; a.c.Hkv = (int32_t)Hkv; a.c.D = (int32_t)D;
    a.c.max_pages = max_pages; a.c.page = (uint32_t)page; a.c.n_pages = 1000;
    a.c.ks = a.c.vs = int8 ? &one : nullptr;
    a.G = (int32_t)(Hq / Hkv);
    a.window = window;
    CHECK(tpl::launch_kv_attention(a, es, nullptr) == hipSuccess);
}

int main() {
    constexpr int64_t FAR = tpl::PLAN_FAR, ALL = int64_t(1) << 62;
    // Windows: the tiles take all but those between FAR less the table's positions and FAR.
    const int64_t held = 1000 * 16;
    for (const int64_t w : {(int64_t)1, (int64_t)4096, FAR - held, FAR + 1, (int64_t)1000000000, 2 * FAR - 1, 2 * FAR, 2 * FAR + 1, (int64_t)INT32_MAX, ALL}) {
        call(64, 64, 32, 8, 128, 1000, 16, w);
        CHECK(tile() && lp.window == (w < 2 * FAR ? w : 2 * FAR) && lp.excess == (w == ALL ? UINT32_MAX : (uint32_t)(w - lp.window)));
    }
    for (const int64_t w : {FAR - held + 1, FAR}) { call(64, 64, 32, 8, 128, 1000, 16, w); CHECK(!tile()); }
    // no table of 2^29 positions, whatever the window
    for (const int64_t w : {(int64_t)5, FAR + 1, ALL}) { call(64, 64, 32, 8, 128, FAR / 16, 16, w); CHECK(!tile()); }
    // Calls whose items take a workgroup each (tests/test_gpu_attention_items.py).
    int64_t T = 8;
    for (int i = 0; i < 2100; ++i) { const int n[10] = {1, 1, 1, 0, 1, 3, 1, 1, 20, 1}; T += n[i % 10]; }
    const auto own = [&](bool few) {
        CHECK(tile() && !lp.stream && lp.few == few && tpl::attention_workspace(T, 2100, 2, 1, 32) == 0);
    };
    for (const bool int8 : {false, true})
        for (const int es : {2, 4}) {
            call(T, 2100, 2, 1, 32, 9, 16, ALL, es, int8); own(true);
            call(T, 2100, 4, 2, 64, 9, 8, 33, es, int8); own(true);
            call(T, 2100, 3, 1, 50, 9, 16, ALL, es, int8); own(true);
            call(T, 2100, 2, 1, 256, 9, 16, 40, es, int8); own(true);
        }
    int64_t C = 8;
    for (int i = 0; i < 540; ++i) { const int n[7] = {1, 0, 37, 9, 60, 5, 0}; C += n[i % 7]; }
    int64_t H = 1;
    for (int i = 0; i < 300; ++i) { const int n[5] = {33, 0, 70, 34, 31}; H += n[i % 5]; }
    for (const bool int8 : {false, true})
        for (const int es : {2, 4}) {
            call(C, 540, 8, 1, 64, 10, 16, ALL, es, int8); own(false);
            call(C, 540, 16, 2, 32, 10, 16, 50, es, int8); own(false);
            call(C, 540, 8, 1, 36, 30, 5, ALL, es, int8); own(false);
            CHECK(tpl::attention_workspace(C, 540, 8, 1, 64) == 0);
            call(H, 300, 8, 8, 32, 7, 16, ALL, es, int8); own(false);
            CHECK(lp.row_tiles <= 512 && tpl::attention_workspace(H, 300, 8, 8, 32) == 0);
            // prompts from their first tokens on, and with a wider table
            for (const int64_t Hq : {8, 4}) {
                call(440, 4, Hq, Hq / 4, 128, 13, 16, ALL, es, int8); own(false);
                call(539, 3, Hq, Hq / 4, 128, 13, 16, ALL, es, int8); own(false);
                call(440, 4, Hq, Hq / 4, 128, 3013, 16, ALL, es, int8); CHECK(tile() && lp.stream && !lp.few);
            }
        }
    if (failures) return 1;
    std::printf("attention form driver ok\n");
    return 0;
}
