// Device code shared by the kernels that read a paged cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "attn_plan.h"

namespace tpl {
namespace {

// The sequence that owns row t of a call, by a 64-way search of cu; -1 for none.
__device__ __forceinline__ int64_t sequence_of(const CacheArgs &a, int64_t t, int lane) {
    // the number of sequences s in [0, B) with cu[s] <= t, for non-decreasing cu
    int64_t lo = 0, n = a.B;
    while (n > 0) {
        const int64_t step = (n + 63) / 64;
        const int64_t i = lo + lane * step;
        const bool below = lane * step < n && a.cu[i] <= t;
        const int c = __popcll(__ballot(below));
        if (c == 0) { n = 0; break; }
        const int64_t base = (int64_t)(c - 1) * step;      // the last such probe
        lo += base + 1;
        n = (n - base < step ? n - base : step) - 1;
    }
    const int64_t s = lo - 1;
    return s >= 0 && t < a.cu[s + 1] ? s : -1;
}

// Page and slot of position p >= 0 of a sequence whose table begins at `table`; the
// page is -1 where the position or its page is outside the cache.  Nothing read from
// the caller's arrays is used as an index before it is checked.
struct Row { int64_t page; uint32_t slot; };
__device__ __forceinline__ Row row_of(const CacheArgs &a, const int32_t *table, uint32_t p) {
    const uint32_t i = a.shift >= 0 ? p >> a.shift : p / a.page;
    Row r{-1, p - (a.shift >= 0 ? i << a.shift : i * a.page)};
    if ((int64_t)i < a.max_pages) {
        const int64_t id = table[i];
        if (id >= 0 && id < a.n_pages) r.page = id;
    }
    return r;
}

// One value of a cache: bf16 (2 bytes), fp32 (4) or int8 (1).
template <int CS>
__device__ __forceinline__ float cached(const void *p, int64_t i) {
    if (CS == 1) return (float)((const int8_t *)p)[i];
    return CS == 2 ? (float)((const __bf16 *)p)[i] : ((const float *)p)[i];
}

template <int ES>
__device__ __forceinline__ float value(const void *p, int64_t i) {
    return ES == 2 ? (float)((const __bf16 *)p)[i] : ((const float *)p)[i];
}
template <int ES>
__device__ __forceinline__ void store(void *p, int64_t i, float v) {
    if (ES == 2) ((__bf16 *)p)[i] = (__bf16)v;
    else ((float *)p)[i] = v;
}

// ---- the plan on the device

__device__ __forceinline__ PlanDesc *plan_desc(void *ws) { return (PlanDesc *)ws; }
__device__ __forceinline__ float *plan_stats(void *ws, int W) { return (float *)((char *)ws + plan_desc_bytes(W)); }
typedef float plan_f32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ plan_f32x4 *plan_sums(void *ws, int W) {
    return (plan_f32x4 *)((char *)ws + plan_desc_bytes(W) + plan_stats_bytes(W));
}

// 32 bits hold what the matrix-core form takes (attn.cpp): rows of tokens and heads,
// positions of the table and tokens below FAR, windows to 2 FAR.  A past before -FAR may be
// taken for -FAR, whose rows are all before the table.  Beyond FAR, where rows are behind the
// table, it counts for the first position that a row sees alone, past - window + 1: so a
// window that is `excess` longer than 2 FAR brings it nearer by as much, and it is held
// between FAR, whose rows see all of the table if the window is 2 FAR, and 3 FAR - 2, whose
// rows see nothing of it (and whose positions, of FAR - 2 tokens on, are below 2^31 - 1).
constexpr int FAR = PLAN_FAR;

// A sequence's first row and number of rows among the call's T, and the position of the
// first of them.  Rows outside the call do not count, whatever cu says.
struct Sequence { int first, n, past; };
__device__ __forceinline__ int plan_clamp(int v, int T) { return v < 0 ? 0 : v > T ? T : v; }
__device__ __forceinline__ Sequence plan_sequence(const CacheArgs &c, uint32_t excess, int s) {
    const int from = c.cu[s], to = c.cu[s + 1], T = (int)c.T;
    Sequence q;
    q.first = plan_clamp(from, T);
    const int end = plan_clamp(to, T);
    q.n = end > q.first ? end - q.first : 0;
    // rows before the call's first count: the past is past + FAR - most, of up to 33 bits
    const int past = c.past[s], most = from < 0 ? FAR + from : FAR;
    const uint32_t beyond = (uint32_t)past - (uint32_t)most, behind = beyond > excess ? beyond - excess : 0;
    if (past > most) q.past = FAR + (int)(behind < 2 * FAR - 2 ? behind : 2 * FAR - 2);
    else q.past = past + (FAR - most) > -FAR ? past + (FAR - most) : -FAR;
    return q;
}

// Index of a sequence's first row tile where sequence s begins at cu[s] G / ROWS + s:
// floor(x / ROWS) + 1 - floor(y / ROWS) tiles are enough for the rows y .. x - 1.
__device__ __forceinline__ int plan_index(const CacheArgs &c, int s, int G, int ROWS) {
    return plan_clamp(c.cu[s], (int)c.T) * G / ROWS + s;
}

// Row tile r of a sequence: the positions of its first and last row, the positions that
// its rows see (those of the table), and the tiles of BK that hold them; at least one, so
// that rows that see nothing are written.
struct Span { int pos0, pos1, begin, end, first, tiles; };
__device__ __forceinline__ int plan_divide(uint32_t x, const Divisor &d) { return (int)((uint64_t)x * d.by >> d.shift); }
__device__ __forceinline__ Span plan_span(const AttnPlan &p, const Sequence &q, int r, int G, int ROWS, int BK) {
    const int window = p.window, last_pos = p.last_pos;
    Span s;
    const uint32_t row = (uint32_t)r * ROWS, all = (uint32_t)(q.n * G), rows = all - row < (uint32_t)ROWS ? all - row : ROWS;
    s.pos0 = q.past + plan_divide(row, p.g);
    s.pos1 = q.past + plan_divide(row + rows - 1, p.g);
    s.begin = s.pos0 - window + 1 > 0 ? s.pos0 - window + 1 : 0;
    s.end = s.pos1 + 1 < last_pos ? s.pos1 + 1 : last_pos;
    if (s.end < 0) s.end = 0;
    s.first = s.begin / BK;
    const int n = (s.end + BK - 1) / BK - s.first;
    s.tiles = n > 0 ? n : 1;
    return s;
}

// Four features of a row, d .. d + 3 of D, divided by the row's sum.  ENDS: a row may end
// inside them; FULL: it does not before them either.
enum { ROW_FULL = 0, ROW_FOURS = 1, ROW_ENDS = 2 };
template <int ES, int ROW>
__device__ __forceinline__ void write_out(void *O, int64_t at, int d, int D, plan_f32x4 v, bool none, float inv) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = none ? 0.0f : v[e] * inv;
    if (ROW == ROW_FULL || d + 4 <= D) {
        if constexpr (ES == 2) {
            typedef __bf16 bf16x4_ __attribute__((ext_vector_type(4)));
            typedef uint32_t u32x2_at __attribute__((ext_vector_type(2), aligned(1)));
            bf16x4_ h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = (__bf16)y[e];
            typedef uint32_t u32x2_ __attribute__((ext_vector_type(2)));
            *(u32x2_at *)((char *)O + (at + d) * 2) = __builtin_bit_cast(u32x2_, h);
        } else {
            typedef float f32x4_at __attribute__((ext_vector_type(4), aligned(4)));
            *(f32x4_at *)((float *)O + at + d) = f32x4_at{y[0], y[1], y[2], y[3]};
        }
    } else if (ROW == ROW_ENDS && d < D) {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (d + e < D) store<ES>(O, at + d + e, y[e]);
    }
}

}  // namespace
}  // namespace tpl
