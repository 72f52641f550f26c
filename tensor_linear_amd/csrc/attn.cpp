// Which kernels an attention call takes, and its workspace (host code only).
#include "attn.h"

#include <cstdint>

#include "attn_plan.h"

namespace tpl {

namespace {

constexpr int64_t MAX_TILE_D = 256;     // largest head of the matrix-core form

// What the matrix-core form takes: heads of 8 to 256; rows and positions of the table that
// 32 bits hold, with room for their sums; windows of any length but those, far longer than
// any sequence, from FAR less the table's positions to FAR.
constexpr int64_t FAR = PLAN_FAR;
bool tile_ok(int64_t T, int64_t B, int64_t G, int64_t D) { return D >= 8 && D <= MAX_TILE_D && T < FAR && B < FAR && T * G < INT32_MAX - 128; }
bool positions_ok(const AttnArgs &a) {
    const int64_t last = a.c.max_pages * (int64_t)a.c.page;
    return a.c.max_pages < FAR && last < FAR && (a.window > FAR || last + a.window <= FAR);
}

// A cache whose rows lie at multiples of 16 bytes goes to LDS without a stop.
bool dma_ok(const AttnArgs &a, int es) {
    const int64_t n = 16 / (a.c.ks ? 1 : es);
    return a.c.D % n == 0 && (uintptr_t)a.c.kc % 16 == 0 && (uintptr_t)a.c.vc % 16 == 0 && a.c.s_page % n == 0 && a.c.s_slot % n == 0 && a.c.s_head % n == 0;
}

}  // namespace

AttnPlan attention_plan(int64_t T, int64_t B, int64_t Hkv, int32_t G, int64_t D, int es, bool quant) {
    AttnPlan p{};
    p.g = divisor(G);
    // 32 rows a workgroup where the sequences have no more on average.  One form for the whole
    // call: 64 single tokens behind 8000 at most (214 us) and a chunk of 256 behind 2000 (70),
    // 8 query heads a key head, are 2560 rows and take 290 us in workgroups of 128; 200 behind
    // 2000 at most (189) and a chunk of 512 (89) 326 us in ones of 32.
    p.few = T * G <= 32 * B;
    const int64_t rows = p.few ? 32 : 128;
    p.row_tiles = T * G / rows + B;
    // Equal runs while adding up the sequences' tiles in every workgroup is cheap and the
    // items are too few to even out by themselves: 200 tokens of pasts up to 1000, 8 key
    // heads, 108 us for 126, 1500 309 for 325, but 3000 over int8 270 for 240; 12 chunks
    // over a window of 1024 121 us for 133, but a prompt of 4 x 1024 tokens 172 for 143.
    p.stream = p.few ? p.row_tiles <= 2048 : p.row_tiles <= 512 && p.row_tiles * Hkv <= 2048;
    // As many as 256 CUs hold at once, by LDS (two stages of 32 keys, one wavefront) and by
    // registers (two wavefronts a SIMD, one for the longest heads).  Not taken from the
    // device: the workspace's size and the order of the sums depend on the call alone.
    const int64_t row = (D <= 64 ? 64 : D <= 128 ? 128 : 256) * (quant ? 1 : es);
    p.groups = 256 * (!p.few ? (D <= 128 ? 2 : 1) : row <= 128 ? 8 : row <= 256 ? 4 : row <= 512 ? 2 : 1);
    return p;
}

size_t attention_workspace(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
    if (T == 0 || B == 0 || !tile_ok(T, B, Hq / Hkv, D)) return 0;
    // the most runs that any type of cache has
    const AttnPlan p = attention_plan(T, B, Hkv, (int32_t)(Hq / Hkv), D, 2, true);
    if (!p.stream) return 0;
    const int64_t d = D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : 256, rows = p.few ? 32 : 128;
    return (size_t)(plan_desc_bytes(p.groups) + plan_stats_bytes(p.groups) + 2 * p.groups * rows * d * 4);
}

hipError_t launch_kv_attention(const AttnArgs &a, int es, hipStream_t s) {
    if (!tile_ok(a.c.T, a.c.B, a.G, a.c.D) || !positions_ok(a)) return launch_attention_any(a, es, s);
    AttnPlan p = attention_plan(a.c.T, a.c.B, a.c.Hkv, a.G, a.c.D, es, a.c.ks != nullptr);
    p.last_pos = (int32_t)(a.c.max_pages * (int64_t)a.c.page);
    p.window = (int32_t)(a.window < 2 * FAR ? a.window : 2 * FAR);
    p.excess = (uint32_t)(a.window - p.window < (int64_t)UINT32_MAX ? a.window - p.window : (int64_t)UINT32_MAX);
    p.page = divisor(a.c.page);
    p.n_pages = (uint32_t)(a.c.n_pages < (int64_t)1 << 31 ? a.c.n_pages : (int64_t)1 << 31);
    // units of a run: tiles of 32 keys and changes of items, counted in 32 bits
    if (p.stream && p.row_tiles * (p.last_pos / 32 + 8) * a.c.Hkv >= INT32_MAX) p.stream = 0;
    if (!p.stream && p.row_tiles * a.c.Hkv > (1 << 23)) return launch_attention_any(a, es, s);   // more than one launch holds
    // Prompts from their first tokens on: the items' lengths go from one tile of 64 keys to
    // L, which taking a prompt's longest first evens out.  By themselves they then take the
    // time of 3/4 L tiles or all tiles' share of a workgroup, the runs that share and 6 tiles
    // more, the sums' way by the workspace (64 query and 8 key heads of 128, one prompt of
    // 512, 1024 and 2048 tokens: 31, 54 and 125 us for 42, 65 and 142; but with 8 query heads
    // and one key head 4096 tokens 146 for 78).  All that the host knows of the lengths is the
    // table's width: prompts with a table of more than twice their mean take the runs.
    if (p.stream && !p.few && p.window >= p.last_pos && 2 * a.c.T >= a.c.B * (int64_t)p.last_pos) {
        const int64_t L = p.last_pos / 64, items = p.row_tiles * a.c.Hkv;
        if (L * (3 * p.groups - 2 * items) <= 24 * (int64_t)p.groups) p.stream = 0;
    }
    const bool dma = dma_ok(a, es);
    if (a.c.ks) return es == 2 ? launch_attention_bf16_int8(a, p, dma, s) : launch_attention_f32_int8(a, p, dma, s);
    return es == 2 ? launch_attention_bf16(a, p, dma, s) : launch_attention_f32(a, p, dma, s);
}

}  // namespace tpl
