// Device code shared by the kernels on heads and paged caches: a lane's 16 values of
// a head, their loads, stores and rotation, and a token's place in the cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "heads.h"

namespace tpl {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// in memory: at any address (the same instructions as for aligned ones)
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));

constexpr int HT = 256;

// Ordinary stores: past the caches they are faster by themselves (8192 tokens of 64 +
// 8 heads of 128 60.1 us for 64.5), but the step that reads the result then pays more
// (with a pass over the queries and keys behind it 124.5 us for 115.8).
template <int ES, bool FINE>
__device__ __forceinline__ void put8(void *p, int64_t i, int a, int b, const float *v) {
    char *q = (char *)p + (i + a) * ES, *q2 = (char *)p + (i + b) * ES;
    if constexpr (ES == 2) {
        typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
        bf16x8 h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (__bf16)v[e];
        const u32x4 w = __builtin_bit_cast(u32x4, h);
        if constexpr (FINE) {
            *(u32x2_any *)q = u32x2{w[0], w[1]};
            *(u32x2_any *)q2 = u32x2{w[2], w[3]};
        } else {
            *(u32x4_any *)q = w;
        }
    } else {
        u32x4 c, d;
#pragma unroll
        for (int e = 0; e < 4; ++e) { c[e] = __float_as_uint(v[e]); d[e] = __float_as_uint(v[4 + e]); }
        *(u32x4_any *)q = c;
        *(u32x4_any *)(FINE ? q2 : q + 16) = d;
    }
}

template <int ES>
__device__ __forceinline__ float get1(const void *p, int64_t i) {
    return ES == 2 ? (float)((const __bf16 *)p)[i] : ((const float *)p)[i];
}
template <int ES>
__device__ __forceinline__ void put1(void *p, int64_t i, float v) {
    if (ES == 2) ((__bf16 *)p)[i] = (__bf16)v;
    else ((float *)p)[i] = v;
}

// 8 consecutive values as they are, and widened.
template <int ES>
struct Raw8 { u32x4 w[ES / 2]; };
// Those at i + a .. + 3 and i + b .. + 3; not FINE: b is a + 4.
template <int ES, bool FINE>
__device__ __forceinline__ Raw8<ES> raw8(const void *p, int64_t i, int a, int b) {
    Raw8<ES> r;
    const char *q = (const char *)p + (i + a) * ES;
    if constexpr (!FINE) {
#pragma unroll
        for (int h = 0; h < ES / 2; ++h) r.w[h] = *(const u32x4_any *)(q + 16 * h);
    } else if constexpr (ES == 2) {
        const u32x2 lo = *(const u32x2_any *)q, hi = *(const u32x2_any *)((const char *)p + (i + b) * ES);
        r.w[0] = u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
        r.w[0] = *(const u32x4_any *)q;
        r.w[ES / 4] = *(const u32x4_any *)((const char *)p + (i + b) * ES);
    }
    return r;
}
template <int ES>
__device__ __forceinline__ void widen8(const Raw8<ES> &r, float *v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (ES == 2) v[e] = __uint_as_float((e & 1) ? r.w[0][e / 2] & 0xFFFF0000u : r.w[0][e / 2] << 16);
        else v[e] = __uint_as_float(r.w[ES / 2 * e / 8][e % 4]);
    }
}

enum { HEAD_Q = 0, HEAD_K = 1, HEAD_V = 2 };

// Where a token goes: its position and, for the append, the element offset of
// its slot, its page and the row in it.  ok: the position is in the table (and the
// slot in the cache).
struct Place { int64_t pos, slot; bool mine, ok; int64_t page, row; };

// Token t's sequence by a 64-way search of cu, its position, page and slot.
// mine: some sequence owns the token.  Nothing read from the caller's arrays is
// used as an index before it is checked.
__device__ __forceinline__ Place find_place(const HeadArgs &a, int64_t t, int lane) {
    Place p{0, 0, false, false, 0, 0};
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
    if (s < 0) return p;
    if (t >= a.cu[s + 1]) return p;
    p.mine = true;
    p.pos = (int64_t)a.past[s] + (t - a.cu[s]);
    if (p.pos < 0 || p.pos >= a.max_pages * a.page || (a.R > 0 && p.pos >= a.n_pos)) return p;
    const int64_t pg = p.pos / a.page;
    const int64_t id = a.table[s * a.ldt + pg];
    if (id < 0 || id >= a.n_pages) return p;
    p.page = id;
    p.row = p.pos - pg * a.page;
    p.slot = id * a.s_page + p.row * a.s_slot;
    p.ok = true;
    return p;
}

__device__ __forceinline__ Place given_place(const HeadArgs &a, int64_t t) {
    Place p{0, 0, true, true, 0, 0};
    if (a.R > 0) {
        p.pos = a.pos[t];
        p.ok = p.pos >= 0 && p.pos < a.n_pos;
    }
    return p;
}

// A lane's 16 values: four runs of 4 from a, a2, b, b2 on, of which the elements of
// a and a2 pair with those of b and b2 (halves), or neighbours pair (pairs).
// turn, turn2: whether the pairs of the values 0-3 and 4-7 of either half (pairs:
// the first and the last 8 values) rotate.  Where R is a multiple of 16 both do or
// neither, and a2 = a + 4, b2 = b + 4; where it is only one of 8 (FINE), R / 2 pairs
// end inside a lane, and the loads are of 4 values.
struct Runs { int a, a2, b, b2; bool on, turn, turn2; };
template <bool FINE>
__device__ __forceinline__ Runs runs_of(int unit, int D, int R, int pairs) {
    Runs r;
    r.on = unit * 16 < D;
    r.turn = unit * 16 < R;
    r.turn2 = FINE ? unit * 16 + 8 < R : r.turn;
    r.a = r.turn && !pairs ? unit * 8 : unit * 16;
    r.b = r.turn && !pairs ? R / 2 + unit * 8 : unit * 16 + (FINE && !pairs ? 4 : 8);
    if (!FINE || pairs) {
        r.a2 = r.a + 4;
        r.b2 = r.b + 4;
    } else {
        r.a2 = r.turn2 ? unit * 8 + 4 : unit * 16 + 8;
        r.b2 = r.turn2 ? R / 2 + unit * 8 + 4 : unit * 16 + 12;
    }
    return r;
}
// Element e of them.
__device__ __forceinline__ int run_at(const Runs &r, int e) {
    return e < 4 ? r.a + e : e < 8 ? r.a2 + e - 4 : e < 12 ? r.b + e - 8 : r.b2 + e - 12;
}

// 16 values of a row, raw and stored.
template <int ES, bool FINE>
__device__ __forceinline__ void load16(const void *p, int64_t i, const Runs &r, Raw8<ES> (&x)[2]) {
    x[0] = raw8<ES, FINE>(p, i, r.a, r.a2);
    x[1] = raw8<ES, FINE>(p, i, r.b, r.b2);
}
template <int ES, bool FINE>
__device__ __forceinline__ void store16(void *p, int64_t i, const Runs &r, const float *v) {
    put8<ES, FINE>(p, i, r.a, r.a2, v);
    put8<ES, FINE>(p, i, r.b, r.b2, v + 8);
}

// The cosines and sines of a lane's 8 pairs at table row `pos`.
template <bool FINE>
__device__ __forceinline__ void load_angles(const HeadArgs &a, int64_t pos, int unit, const Runs &r, float *c, float *s) {
    const int64_t i = pos * (a.R / 2) + unit * 8;
    const int last = FINE && !r.turn2 ? 0 : 4;   // past the table's row: the first four again
    const Raw8<4> cr = raw8<4, FINE>(a.cos, i, 0, last), sr = raw8<4, FINE>(a.sin, i, 0, last);
    widen8<4>(cr, c);
    widen8<4>(sr, s);
}

// The rotation of a lane's pairs by +angle (back: by -angle).
template <bool FINE>
__device__ __forceinline__ void turn16(float *v, const float *c, const float *s, const Runs &r, bool pairs, bool back) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (FINE && e >= 4 && !r.turn2) continue;
        const int ia = pairs ? 2 * e : e, ib = pairs ? 2 * e + 1 : e + 8;
        const float x = v[ia], y = v[ib], sn = back ? -s[e] : s[e];
        v[ia] = x * c[e] - y * sn;
        v[ib] = y * c[e] + x * sn;
    }
}

__device__ __forceinline__ float lanes_sum(float v, int width) {
    for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// The heads of a shard that a call handles, of its hq q, hk k and hk v heads in
// the order of X: `per` of them from `first` on.
struct Span { int first, per; };
__device__ __host__ __forceinline__ Span span_of(const HeadArgs &a, bool q, bool k, bool v) {
    const int first = q ? 0 : k ? a.hq : a.hq + a.hk;
    return Span{first, (v ? a.hq + 2 * a.hk : k ? a.hq + a.hk : a.hq) - first};
}

// Slot s of a token's heads: shard, then the heads of the span.
struct Head { int kind, head, shard, col; bool on; };
__device__ __forceinline__ Head head_of(const HeadArgs &a, int slot, const Span &sp, int slots) {
    Head h;
    h.on = slot < slots;
    h.shard = (h.on ? slot : 0) / sp.per;
    const int j = (h.on ? slot : 0) - h.shard * sp.per + sp.first;
    h.kind = j < a.hq ? HEAD_Q : j < a.hq + a.hk ? HEAD_K : HEAD_V;
    h.head = h.kind == HEAD_Q ? h.shard * a.hq + j
                              : h.shard * a.hk + (j - a.hq - (h.kind == HEAD_V ? a.hk : 0));
    h.col = j * a.D;
    return h;
}

// Position of pair j's two elements, or of the single elements from R on:
// j counts R/2 pairs, then D - R singles (b < 0).
__device__ __forceinline__ void pair_at(const HeadArgs &a, int j, int &x, int &y) {
    if (j >= a.R / 2) { x = a.R + (j - a.R / 2); y = -1; return; }
    x = a.pairs ? 2 * j : j;
    y = a.pairs ? 2 * j + 1 : j + a.R / 2;
}

// Whether the 16-values-a-lane form takes the heads.
inline bool vec_ok(const HeadArgs &a) { return a.D % 16 == 0 && a.R % 8 == 0 && a.D <= 512; }

inline int lanes_per_head(int D) {
    int l = 1;
    while (l * 16 < D) l <<= 1;
    return l;
}

// Launches with `waves` wavefronts for each token: as many as the tokens need, since
// one launch has fewer than 2^32 threads.
template <class Launch>
inline hipError_t launch_tokens(HeadArgs a, int64_t waves, Launch launch) {
    const int64_t T = a.T, most = waves < (1 << 25) ? (1 << 25) / waves : 1;
    for (a.t0 = 0; a.t0 < T; a.t0 = a.T) {
        a.T = T - a.t0 < most ? T : a.t0 + most;
        launch(a, (unsigned)(((a.T - a.t0) * waves + HT / 64 - 1) / (HT / 64)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace
}  // namespace tpl
