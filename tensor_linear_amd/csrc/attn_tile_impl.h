// Attention of new tokens over a paged cache on the matrix cores.
//
// The new tokens of a sequence and the G query heads that read one key head are the
// rows of one matrix (row = token * G + head), so the keys and values of a head are
// read once for all of them.  A workgroup takes 32 WR such rows, 32 a wavefront, and walks
// the keys they see in tiles of BK = 32 KB, with the softmax's running maximum and sum:
//   m' = max(m, max x),  f = 2^(m - m'),  p = 2^(x - m'),  l' = f l + sum p,
//   o' = f o + p V;   at the end O = o / l,  lse = m ln 2 + log l,
// x the products times softmax_scale * log2(e).
//
// Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T, with 32x32 matrix
// instructions: a lane then has ONE row (its column l % 32 of S^T and O^T) and 16 of the
// 32 keys, so that a row's maximum and sum need one exchange (with lane l ^ 32), its
// factors are the lane's own, and the lane's 16 weights are, in order, what the second
// product takes of it: no weight leaves its lane.  (The order of the keys within an
// instruction is free as long as the values come in the same one.)
//
// K and V tiles lie in LDS as rows of 64, 128 or 256 values, their 16-byte chunks
// permuted by the row so that reads meet no bank twice: K by chunks of 32 rows, bf16
// values by the transposing read (4 keys x 16 features a 16-lane group, 8 keys in int8),
// fp32 values by words.  Two stages: the next tile is fetched while this one is worked on,
// straight into LDS (16 bytes a lane) where the cache is 16-byte aligned, else by way of
// registers.  int8 becomes bf16 or fp32 (exactly; a key's scale multiplies its products, a
// value's scale its weight) as a wavefront reads it from LDS where it is alone, on the way
// into LDS where four read the same keys.
//
// What a row does not see must not touch it: keys and values of no position are zeros,
// products that a row does not see are minus infinity before the maximum, and a tile at
// the edge of what its rows see is looked through for values that are not finite, which
// then go their own way (weight zero times infinity would be NaN).
//
// Work: `items` are (sequence, rows, key head).  Where there are many, a workgroup takes
// one, the longest first, neighbours in the grid on other key heads (an XCD, every 8th
// workgroup, then keeps to few heads, whose keys its L2 holds).  Else the tiles of all
// items in a row are cut into equal runs, one for each workgroup: a run's whole items are
// finished, the others' sums go to the workspace and are joined by a second launch in the
// order of the tiles.  The lengths are on the device: each workgroup adds them up itself.
// One thread then reads an item's lengths and tells the others, so that a workgroup stays
// together and in bounds whatever is in those arrays, were they to change under it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_device.h"
#include "attn_plan.h"

namespace tpl {
namespace {

#define LDS_PTR(T) __attribute__((address_space(3))) T *

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// in memory: at any address (the same instructions as for aligned ones)
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// Source of the chunks of no position.
static __device__ __attribute__((aligned(16))) const uint32_t no_key[4] = {0, 0, 0, 0};

// A lane's operand: 16 bytes, chunk 2 s + l / 32 of row l % 32 for step s.
template <int ES>
__device__ __forceinline__ f32x16 product(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (ES == 2) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0, 0);
        return c;
    }
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// An item, and the part of its tiles that a run has; pieces: runs from this one to the
// item's last.  s < 0: none.
struct Item { int64_t s; Sequence q; Span sp; int r, h, k0, k1, pieces; };

// Byte permutation of a row of K and of V in LDS (XOR with the byte in the row).
// K: the 16 rows of a quarter of a read on 16 chunks.  V: the rows of half a read (int8: 0-3
// and 8-11, 32 bytes each; bf16: 0-3, 64 bytes; fp32: two, 4 apart, 128 bytes) side by side.
template <int RB>
__device__ __forceinline__ uint32_t k_swizzle(uint32_t row) {
    return (RB == 64 ? (row >> 2) & 3 : RB == 128 ? (row >> 1) & 7 : row & 15) << 4;
}
template <int LS, int RB>
__device__ __forceinline__ uint32_t v_swizzle(uint32_t row) {
    if (LS == 1) return RB == 64 ? ((row >> 3) & 1) << 5 : RB == 128 ? ((row >> 1) & 1) << 5 | ((row >> 3) & 1) << 6
                                                                     : (row & 3) << 5 | ((row >> 3) & 1) << 7;
    if (LS == 4) return ((row >> 2) & 1) << 7;
    return RB == 128 ? ((row >> 1) & 1) << 6 : (row & 3) << 6;
}

// int8 values to operands: four words of two bf16 (8 values) or of one fp32 (4).
template <int ES>
__device__ __forceinline__ u32x4 from_int8(uint32_t lo, uint32_t hi) {
    const uint32_t w[2] = {lo, hi};
    if constexpr (ES == 2) {
        bf16x8 h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (__bf16)(float)((int32_t)(w[e / 4] << (24 - 8 * (e & 3))) >> 24);
        return __builtin_bit_cast(u32x4, h);
    } else {
        u32x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __float_as_uint((float)((int32_t)(lo << (24 - 8 * e)) >> 24));
        return y;
    }
}

__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32); }

// A value that all lanes have, as a scalar.
__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// What lies in LDS: rows of the call's type by way of registers, the same straight from
// the cache, or int8 straight from the cache.
enum { STAGE_REGS = 0, STAGE_DMA = 1, STAGE_INT8 = 2 };

template <int ES, int CS, int NB, int WR, int KB, int ST, int OCC>
__global__ __launch_bounds__(64 * WR, OCC)
void attention_tile(AttnArgs a, AttnPlan plan) {
    constexpr int NW = WR, NTH = 64 * NW, ROWS = 32 * WR, BK = 32 * KB;
    constexpr int LS = ST == STAGE_INT8 ? 1 : ES;                       // bytes of a value in LDS
    constexpr bool DMA = ST != STAGE_REGS;
    constexpr int DP = NB == 3 ? 128 : NB * 32, RB = DP * LS;          // a row in LDS
    constexpr int KS = NB * ES;                                         // steps of the first product
    constexpr int CH = RB / 16, LI = BK * CH / NTH;                     // chunks of a row; of a thread and tile
    constexpr int STAGE = 2 * BK * RB;
    constexpr bool QUANT = CS == 1;
    static_assert(BK <= NTH, "a thread a row of the tile");
    __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
    __shared__ int64_t row_at[2][BK];                 // element offsets of the tiles' rows, -1 for none
    __shared__ float row_scale[2][2][QUANT ? BK : 1];
    __shared__ uint64_t row_mask[2][(BK + 63) / 64];
    __shared__ int64_t scan[NW + 2];
    __shared__ int found[2];
    __shared__ Item next_item;
    LDS_PTR(char) lds = (LDS_PTR(char))smem;
    const uint32_t lds_u = (uint32_t)(uintptr_t)lds;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave, half = lane >> 5, col = lane & 31;
    const CacheArgs &c = a.c;
    const int D = c.D, G = a.G;
    const float cs = a.scale * 1.44269504088896340736f;
    const int64_t last_pos = c.max_pages * (int64_t)c.page;             // positions of the table
    const int chunks = D * LS / 16;                                     // of a row in LDS that hold features

    auto sequence = [&](int64_t s) { return plan_sequence(c, s); };
    auto span = [&](const Sequence &q, int r) { return plan_span(q, r, G, ROWS, BK, a.window, last_pos); };
    auto count = [&](const Sequence &q) {
        const int nr = (int)((q.n * G + ROWS - 1) / ROWS);
        int64_t n = 0;
        for (int r = 0; r < nr; ++r) n += span(q, r).tiles;
        return n;
    };

    // ---- the run of tiles of this workgroup
    int64_t all = 0, u = 0, u1 = 0, base = 0, seq = 0;   // units in all, the run [u, u1); the first one of sequence seq
    int W = plan.groups;                                 // runs that have tiles
    int w = blockIdx.x;
    if (plan.stream) {
        const int64_t q = (c.B + NTH - 1) / NTH, sb = tid * q;
        int64_t mine = 0;
        for (int64_t i = sb; i < sb + q && i < c.B; ++i) mine += count(sequence(i));
        int64_t run = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t v = __shfl_up(run, o);
            if (lane >= o) run += v;
        }
        if (lane == 63) scan[wave] = run;
        if (tid == 0) scan[NW] = c.B;
        __syncthreads();
        int64_t before = 0;
        for (int i = 0; i < NW; ++i) {
            if (i < wave) before += scan[i];
            all += scan[i];
        }
        all = uniform(all) * c.Hkv;
        if (all < W) W = (int)all;
        else w = (w & 7) * (W / 8) + (w >> 3);          // runs next to each other on one XCD
        if (tid == 0) plan_desc(a.ws)[w].pieces = 0;
        if (w >= W) return;
        u = all * w / W;
        u1 = all * (w + 1) / W;
        int64_t at = (before + run - mine) * c.Hkv;
        if (u >= at && u < (before + run) * c.Hkv) {    // one thread
            for (int64_t i = sb; i < sb + q && i < c.B; ++i) {
                const int64_t n = count(sequence(i)) * c.Hkv;
                if (u < at + n) {
                    scan[NW] = i;
                    scan[NW + 1] = at;
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        seq = scan[NW];
        base = scan[NW + 1];
    }
    int stamp = 0;
    if (tid < 2) found[tid] = -1;

    // The next item and the part of its tiles, by one thread (one wavefront).
    auto find_item = [&]() {
        Item m{};
        m.s = -1;
        if (plan.stream) {
            while (u < u1 && seq < c.B) {
                const Sequence q = sequence(seq);
                const int64_t n = count(q);
                if (u >= base + n * c.Hkv) { base += n * c.Hkv; ++seq; continue; }
                const int64_t rel = u - base;
                m.h = (int)(rel / n);
                int64_t rem = rel - m.h * n;
                const int nr = (int)((q.n * G + ROWS - 1) / ROWS);
                Span sp = span(q, 0);
                int r = 0;
                while (rem >= sp.tiles && r + 1 < nr) { rem -= sp.tiles; sp = span(q, ++r); }
                const int64_t item_u = u - rem;
                m.s = seq; m.q = q; m.sp = sp; m.r = r;
                m.k0 = (int)rem;
                m.k1 = (int)(u1 - item_u < sp.tiles ? u1 - item_u : sp.tiles);
                if (m.k1 <= m.k0) { m.s = -1; break; }
                int64_t to = ((item_u + sp.tiles) * W - 1) / all;               // the run with the item's last tile
                if (to >= W) to = W - 1;
                m.pieces = (int)(to - w + 1);
                u = item_u + m.k1;
                break;
            }
        } else {
            const int64_t i = plan.row_tiles - 1 - w / c.Hkv;
            // sequence s has the indices from cu[s] G / ROWS + s on, enough for its rows
            int64_t lo = 0, n = c.B;
            while (n > 0) {
                const int64_t step = (n + 63) / 64;
                const int64_t j = lo + lane * step;
                const bool below = lane * step < n && plan_index(c, j, G, ROWS) <= i;
                const int k = __popcll(__ballot(below));
                if (k == 0) break;
                const int64_t b = (int64_t)(k - 1) * step;
                lo += b + 1;
                n = (n - b < step ? n - b : step) - 1;
            }
            const int64_t s = uniform(lo) - 1;
            if (s >= 0) {
                const Sequence q = sequence(s);
                const int64_t r = i - plan_index(c, s, G, ROWS);
                if (r >= 0 && r < (q.n * G + ROWS - 1) / ROWS) {
                    m.s = s; m.q = q; m.r = (int)r; m.h = w % c.Hkv;
                    m.sp = span(q, (int)r);
                    m.k1 = m.sp.tiles;
                }
            }
        }
        return m;
    };

    while (true) {
        if (wave == 0) {
            const Item m = find_item();
            if (lane == 0) next_item = m;
        }
        __syncthreads();
        const int64_t s = uniform(next_item.s);
        if (s < 0) return;
        Sequence q;
        q.first = uniform(next_item.q.first); q.n = uniform(next_item.q.n); q.past = uniform(next_item.q.past);
        Span sp;
        sp.pos0 = uniform(next_item.sp.pos0); sp.pos1 = uniform(next_item.sp.pos1);
        sp.begin = uniform(next_item.sp.begin); sp.end = uniform(next_item.sp.end); sp.first = uniform(next_item.sp.first);
        sp.tiles = uniform(next_item.sp.tiles); sp.outside = next_item.sp.outside;
        const int item_r = uniform(next_item.r), item_h = uniform(next_item.h), pieces = uniform(next_item.pieces);
        const int k0 = uniform(next_item.k0), k1 = uniform(next_item.k1);
        if (sp.outside && c.bad && tid == 0) *c.bad = 1;

        // ---- this lane's row
        const uint32_t R = (uint32_t)item_r * ROWS + wr * 32 + col;         // T G < 2^31
        const bool live = R < (uint32_t)(q.n * G);
        const uint32_t tok = live ? R / (uint32_t)G : 0;
        const int head = item_h * G + (int)(live ? R - tok * G : 0);
        const int64_t pos = q.past + tok, row = q.first + tok;
        const int64_t hi = live ? pos : -1;
        const int64_t lo = pos - a.window + 1;
        u32x4 qf[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            qf[k] = u32x4{0, 0, 0, 0};
            // the features that a lane's k-th operand of K has
            const int ch = ST == STAGE_INT8 ? (2 * (k / ES) + half) * ES + k % ES : 2 * k + half;
            if (live && ch < D * ES / 16) qf[k] = *(const u32x4_any *)((const char *)a.Q + (row * a.ldq + (int64_t)head * D) * ES + ch * 16);
        }
        f32x16 o[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[b][i] = 0.0f;
        float mx = -INFINITY, l = 0.0f;

        // ---- rows of a tile: where they are, and which there are
        const int32_t *table = c.table + s * c.ldt;
        struct Look { int32_t id; uint32_t slot; bool want; };
        auto look = [&](int k) {
            Look e{-1, 0, false};
            const int64_t p = ((int64_t)sp.first + k) * BK + tid;
            if (tid < BK && k < k1 && p >= sp.begin && p < sp.end) {
                const uint32_t x = (uint32_t)p, i = c.shift >= 0 ? x >> c.shift : x / c.page;
                e.slot = x - (c.shift >= 0 ? i << c.shift : i * c.page);
                e.id = table[i];                       // i < max_pages: p < last_pos
                e.want = true;
            }
            return e;
        };
        auto place = [&](const Look &e, int k) {
            if (wave * 64 >= BK) return;
            const bool ok = e.want && e.id >= 0 && e.id < c.n_pages;
            if (e.want && !ok && c.bad) *c.bad = 1;
            const uint64_t m = __ballot(ok);
            if (tid < BK) row_at[k & 1][tid] = ok ? e.id * c.s_page + (int64_t)e.slot * c.s_slot + item_h * c.s_head : -1;
            if (lane == 0) row_mask[k & 1][wave] = m;
        };
        struct Scales { float k, v; };
        auto scales = [&](const Look &e) {
            Scales z{0.0f, 0.0f};
            if (QUANT && e.want && e.id >= 0 && e.id < c.n_pages) {
                const int64_t i = e.id * c.ss_page + (int64_t)e.slot * c.ss_slot + item_h * c.ss_head;
                z.k = c.ks[i];
                z.v = c.vs[i];
            }
            return z;
        };
        auto put_scales = [&](const Scales &z, int k) {
            if (QUANT && tid < BK) { row_scale[k & 1][0][tid] = z.k; row_scale[k & 1][1][tid] = z.v; }
        };

        // ---- a tile's chunks: thread tid has chunk i NTH + tid of K and of V
        u32x4 kr[DMA ? 1 : LI], vr[DMA ? 1 : LI];
        auto fetch = [&](int k) __attribute__((always_inline)) {
            const int st = k & 1;
#pragma unroll
            for (int i = 0; i < LI; ++i) {
                const int n = i * NTH + tid, r = n / CH, ch = n % CH;
                const int64_t at = row_at[st][r];
                if constexpr (DMA) {
                    const uint32_t dst = lds_u + st * STAGE + (i * NTH + wave * 64) * 16;
                    const int kc = ch ^ (k_swizzle<RB>(r) >> 4), vc = ch ^ (v_swizzle<LS, RB>(r) >> 4);
                    const char *ka = at >= 0 && kc < chunks ? (const char *)c.kc + at * CS + kc * 16 : (const char *)no_key;
                    const char *va = at >= 0 && vc < chunks ? (const char *)c.vc + at * CS + vc * 16 : (const char *)no_key;
                    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" :: "v"(ka), "s"(dst) : "memory", "m0");
                    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" :: "v"(va), "s"(dst + BK * RB) : "memory", "m0");
                } else {
                    kr[i] = vr[i] = u32x4{0, 0, 0, 0};
                    if (at >= 0 && ch < chunks) {
                        const char *ka = (const char *)c.kc + at * CS + ch * (16 / ES) * CS;
                        const char *va = (const char *)c.vc + at * CS + ch * (16 / ES) * CS;
                        if constexpr (!QUANT) {
                            kr[i] = *(const u32x4_any *)ka;
                            vr[i] = *(const u32x4_any *)va;
                        } else if constexpr (ES == 2) {
                            const u32x2 x = *(const u32x2_any *)ka, y = *(const u32x2_any *)va;
                            kr[i][0] = x[0]; kr[i][1] = x[1];
                            vr[i][0] = y[0]; vr[i][1] = y[1];
                        } else {
                            kr[i][0] = *(const u32_any *)ka;
                            vr[i][0] = *(const u32_any *)va;
                        }
                    }
                }
            }
        };
        auto settle = [&](int k) __attribute__((always_inline)) {      // the fetched tile is in LDS, this thread's part
            if constexpr (DMA) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            } else {
#pragma unroll
                for (int i = 0; i < LI; ++i) {
                    const int n = i * NTH + tid, r = n / CH, ch = n % CH;
                    const uint32_t at = (k & 1) * STAGE + r * RB;
                    *(LDS_PTR(u32x4))(lds + at + ((ch * 16) ^ k_swizzle<RB>(r))) = QUANT ? from_int8<ES>(kr[i][0], kr[i][1]) : kr[i];
                    *(LDS_PTR(u32x4))(lds + at + BK * RB + ((ch * 16) ^ v_swizzle<LS, RB>(r))) = QUANT ? from_int8<ES>(vr[i][0], vr[i][1]) : vr[i];
                }
            }
        };

        // ---- one tile
        const int64_t see_all = sp.pos0, see_from = sp.pos1 - a.window + 1;      // keys that every row sees
        auto tile = [&](int k) __attribute__((always_inline)) {
            const int st = k & 1;
            const int64_t t0 = ((int64_t)sp.first + k) * BK;
            const bool edge = t0 + BK - 1 > see_all || t0 < see_from;
            // values that are not finite, where rows see different keys
            bool dirty = false;
            if (!QUANT && edge && sp.pos1 > sp.pos0) {
                bool any = false;
#pragma unroll
                for (int i = 0; i < LI; ++i) {
                    const u32x4 x = *(LDS_PTR(u32x4))(lds + st * STAGE + BK * RB + (i * NTH + tid) * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (ES == 2) any |= (x[e] & 0x7F80) == 0x7F80 || (x[e] & 0x7F800000) == 0x7F800000;
                        else any |= (x[e] & 0x7F800000) == 0x7F800000;
                    }
                }
                ++stamp;
                if (any) found[stamp & 1] = stamp;
                __syncthreads();
                dirty = found[stamp & 1] == stamp;
            }
            f32x16 x[KB];
            uint32_t seen[KB];
            const uint32_t kl = st * STAGE + col * RB, ks = (half * 16) ^ k_swizzle<RB>(col);
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) x[b][i] = 0.0f;
#pragma unroll
            for (int s2 = 0; s2 < KS; s2 += ES / LS)
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    const u32x4 kf = *(LDS_PTR(u32x4))(lds + kl + b * 32 * RB + ((s2 * LS / ES * 32) ^ ks));
                    if constexpr (ST != STAGE_INT8) {
                        x[b] = product<ES>(kf, qf[s2], x[b]);
                    } else {
#pragma unroll
                        for (int e = 0; e < ES; ++e)
                            x[b] = product<ES>(ES == 2 ? from_int8<ES>(kf[2 * (e & 1)], kf[2 * (e & 1) + 1]) : from_int8<ES>(kf[e], 0), qf[s2 + e], x[b]);
                    }
                }
            if constexpr (QUANT) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 z = *(LDS_PTR(f32x4))(LDS_PTR(float))&row_scale[st][0][b * 32 + 8 * i + 4 * half];
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[b][4 * i + e] *= z[e];
                    }
            }
            bool masked = edge;
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                const int n = b * 32;
                seen[b] = __builtin_amdgcn_readfirstlane((uint32_t)(row_mask[st][n / 64] >> (n & 63)));
                masked |= seen[b] != 0xFFFFFFFFu;
            }
            if (masked) {
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    const int64_t n = t0 + b * 32, up = hi - n, from = lo - n;
                    uint32_t m = seen[b];
                    m &= up >= 31 ? 0xFFFFFFFFu : up < 0 ? 0u : (2u << (int)up) - 1u;
                    m &= from <= 0 ? 0xFFFFFFFFu : from > 31 ? 0u : 0xFFFFFFFFu << (int)from;
                    m >>= 4 * half;
                    seen[b] = m;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!(m >> (8 * (i / 4) + i % 4) & 1)) x[b][i] = -INFINITY;
                }
            }
            float top = x[0][0];
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, x[b][i]);
            top = fmaxf(top, other_half(top));
            const float next = fmaxf(mx, top * cs);
            const float zero = next == -INFINITY ? 0.0f : next;
            if (__any(next > mx)) {
                const float f = __builtin_amdgcn_exp2f(mx - zero);
                l *= f;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[b][i] *= f;
                mx = next;
            }
            float sum = 0.0f;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[b][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[b][i], cs, -zero));
                    sum += x[b][i];
                }
            l += sum;
            if constexpr (QUANT) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 z = *(LDS_PTR(f32x4))(LDS_PTR(float))&row_scale[st][1][b * 32 + 8 * i + 4 * half];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[b][4 * i + e] *= z[e];
                            if (masked && !(seen[b] >> (8 * i + e) & 1)) x[b][4 * i + e] = 0.0f;   // whatever the scale
                        }
                    }
            }
            const uint32_t vl = st * STAGE + BK * RB;
            auto values = [&](auto put) __attribute__((always_inline)) {
                if constexpr (ST == STAGE_INT8) {
                    // keys 16 s + 8 e + 4 half + i of a step, 4 e + i = (l % 16) / 2
                    const uint32_t r = (lane & 15) >> 1, key = (r & 3) + (r >> 2) * 8 + 4 * half;
                    const uint32_t at = vl + key * RB + ((lane >> 4) & 1) * 16 + (lane & 1) * 8, sw = v_swizzle<LS, RB>(key);
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int s2 = 0; s2 < 2; ++s2) {
                            u32x4 p[ES / 2];
                            if constexpr (ES == 2) {
                                bf16x8 h;
#pragma unroll
                                for (int e = 0; e < 8; ++e) h[e] = (__bf16)x[b][8 * s2 + e];
                                p[0] = __builtin_bit_cast(u32x4, h);
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e) p[e / 4 * (ES / 4)][e % 4] = __float_as_uint(x[b][8 * s2 + e]);
                            }
#pragma unroll
                            for (int d = 0; d < NB; ++d) {
                                typedef int i32x2 __attribute__((ext_vector_type(2)));
                                const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS_PTR(i32x2))(lds + at + (b * 32 + s2 * 16) * RB + ((d * 32) ^ sw)));
                                if constexpr (ES == 2) {
                                    put(d, b, s2, from_int8<ES>(v[0], v[1]), p[0]);
                                } else {
                                    put(d, b, 2 * s2, from_int8<ES>(v[0], 0), p[0]);
                                    put(d, b, 2 * s2 + 1, from_int8<ES>(v[1], 0), p[ES / 4]);
                                }
                            }
                        }
                } else if constexpr (ES == 2) {
                    // keys 16 s + 8 e + 4 half + r of a step, r = (l % 16) / 4; features of 16 lanes
                    const uint32_t r = (lane & 15) >> 2;
                    const uint32_t at = vl + (4 * half + r) * RB + ((lane >> 4) & 1) * 32 + (lane & 3) * 8, sw = v_swizzle<LS, RB>(r);
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int s2 = 0; s2 < 2; ++s2) {
                            bf16x8 p;
#pragma unroll
                            for (int e = 0; e < 8; ++e) p[e] = (__bf16)x[b][8 * s2 + e];
#pragma unroll
                            for (int d = 0; d < NB; ++d) {
                                LDS_PTR(char) v = lds + at + (b * 32 + s2 * 16) * RB + ((d * 64) ^ sw);
                                const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR(s16x4))v);
                                const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR(s16x4))(v + 8 * RB));
                                put(d, b, s2, __builtin_bit_cast(u32x4, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7)), __builtin_bit_cast(u32x4, p));
                            }
                        }
                } else {
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int d = 0; d < NB; ++d) {
                                u32x4 v, p;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t n = b * 32 + 8 * i + e + 4 * half;       // (n >> 2) & 1 = half
                                    v[e] = *(LDS_PTR(uint32_t))(lds + vl + n * RB + ((d * 128 + col * 4) ^ (half << 7)));
                                    p[e] = __float_as_uint(x[b][4 * i + e]);
                                }
                                put(d, b, i, v, p);
                            }
                }
            };
            if (!dirty) {
                values([&](int d, int, int, u32x4 v, u32x4 p) __attribute__((always_inline)) { o[d] = product<ES>(v, p, o[d]); });
            } else {
                // Finite values as usual; of the others, counts of those that a row sees by
                // their kind (a NaN is of both), and then the infinity itself.
#pragma unroll
                for (int dd = 0; dd < NB; ++dd) {
                    __builtin_amdgcn_sched_barrier(0);     // one block after another: few registers
                    f32x16 up, down;
#pragma unroll
                    for (int i = 0; i < 16; ++i) up[i] = down[i] = 0.0f;
                    values([&](int d, int b, int s2, u32x4 v, u32x4 p) __attribute__((always_inline)) {
                        if (d != dd) return;
                        __builtin_amdgcn_sched_barrier(0);
                        u32x4 fine, pos_, neg, one;
                        if constexpr (ES == 2) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t x16 = v[e / 2] >> (16 * (e & 1)) & 0xFFFF, sh = 16 * (e & 1);
                                const bool odd = (x16 & 0x7F80) == 0x7F80, nan = odd && (x16 & 0x7F);
                                const uint32_t keep = e & 1 ? 0xFFFF : 0;
                                fine[e / 2] = (fine[e / 2] & keep) | (odd ? 0u : x16) << sh;
                                pos_[e / 2] = (pos_[e / 2] & keep) | (odd && (nan || !(x16 & 0x8000)) ? 0x3F80u : 0u) << sh;
                                neg[e / 2] = (neg[e / 2] & keep) | (odd && (nan || (x16 & 0x8000)) ? 0x3F80u : 0u) << sh;
                                const uint32_t bit = seen[b] >> (16 * s2 + 8 * (e / 4) + e % 4) & 1;
                                one[e / 2] = (one[e / 2] & keep) | (bit ? 0x3F80u : 0u) << sh;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const bool odd = (v[e] & 0x7F800000u) == 0x7F800000u, nan = odd && (v[e] & 0x7FFFFFu);
                                fine[e] = odd ? 0u : v[e];
                                pos_[e] = odd && (nan || !(v[e] >> 31)) ? 0x3F800000u : 0u;
                                neg[e] = odd && (nan || (v[e] >> 31)) ? 0x3F800000u : 0u;
                                one[e] = seen[b] >> (8 * s2 + e) & 1 ? 0x3F800000u : 0u;
                            }
                        }
                        o[dd] = product<ES>(fine, p, o[dd]);
                        up = product<ES>(pos_, one, up);
                        down = product<ES>(neg, one, down);
                    });
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (up[i] > 0.0f) o[dd][i] += INFINITY;
                        if (down[i] > 0.0f) o[dd][i] -= INFINITY;
                    }
                }
            }
        };

        // ---- the tiles
        {
            const Look e0 = look(k0), e1 = look(k0 + 1);
            Scales z = scales(e0);
            place(e0, k0);
            place(e1, k0 + 1);
            put_scales(z, k0);
            z = scales(e1);
            __syncthreads();
            fetch(k0);
            for (int k = k0; k < k1; ++k) {
                settle(k);
                __syncthreads();
                const Look e = look(k + 2);
                if (k + 1 < k1) fetch(k + 1);
                tile(k);
                if (k + 1 < k1) {
                    put_scales(z, k + 1);
                    place(e, k + 2);
                    z = scales(e);
                }
            }
        }

        l += other_half(l);
        const bool whole = !plan.stream || (k0 == 0 && k1 == sp.tiles);
        const int slot = plan.stream ? 2 * w + (k0 == 0 ? 1 : 0) : 0;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if (live) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = o[b][4 * i + e];
                    if (whole) write_out<ES>(a.O, row * a.ldo + (int64_t)head * D, b * 32 + 8 * i + 4 * half, D, v, l == 0.0f, inv);
                    else plan_sums(a.ws, plan.groups)[(((int64_t)slot * WR + wr) * NB + b) * 256 + i * 64 + lane] = v;
                }
            if (half == 0 && !whole) {
                float *ml = plan_stats(a.ws, plan.groups) + ((int64_t)slot * ROWS + wr * 32 + col) * 2;
                ml[0] = mx;
                ml[1] = l;
            } else if (half == 0 && a.lse) {
                a.lse[row * a.ldl + head] = l == 0.0f ? -INFINITY : mx * 0.69314718055994530942f + logf(l);
            }
        }
        if (!plan.stream) return;
        if (!whole && k0 == 0 && tid == 0) {
            // this run begins the item: it names the runs that hold the rest
            plan_desc(a.ws)[w] = PlanDesc{pieces, item_r, item_h, 0, s};
        }
        __syncthreads();
    }
}

// Joins the sums of the items that more than one run holds: workgroup (w, y) the item
// that run w begins, block y of its rows and features; its first sums are in slot 2 w + 1,
// the later ones in slots 2 (w + 1), 2 (w + 2), ...
template <int ES, int NB, int WR>
__global__ __launch_bounds__(256)
void attention_join(AttnArgs a, AttnPlan plan) {
    constexpr int ROWS = 32 * WR;
    const int w = blockIdx.x, wr = blockIdx.y / NB, b = blockIdx.y % NB;
    const PlanDesc d = plan_desc(a.ws)[w];
    if (d.pieces == 0) return;
    const int lane = threadIdx.x & 63, i = threadIdx.x >> 6, half = lane >> 5, col = lane & 31;
    const Sequence q = plan_sequence(a.c, d.s);
    const uint32_t R = (uint32_t)d.r * ROWS + wr * 32 + col;
    if (R >= (uint32_t)(q.n * a.G)) return;
    const uint32_t tok = R / (uint32_t)a.G;
    const int64_t row = q.first + tok;
    const int head = d.h * a.G + (int)(R - tok * a.G);
    const float *ml = plan_stats(a.ws, plan.groups) + (int64_t)(wr * 32 + col) * 2;
    const f32x4 *sums = plan_sums(a.ws, plan.groups) + ((int64_t)wr * NB + b) * 256 + i * 64 + lane;
    auto slot = [&](int k) { return k == 0 ? (int64_t)2 * w + 1 : (int64_t)2 * (w + k); };
    float m = -INFINITY;
#pragma unroll 8
    for (int k = 0; k < d.pieces; ++k) m = fmaxf(m, ml[slot(k) * ROWS * 2]);
    const float zero = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int k = 0; k < d.pieces; ++k) {
        const float *s = ml + slot(k) * ROWS * 2;
        const float f = __builtin_amdgcn_exp2f(s[0] - zero);
        l = __builtin_fmaf(f, s[1], l);
        const f32x4 x = sums[slot(k) * WR * NB * 256];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f, x[e], v[e]);
    }
    write_out<ES>(a.O, row * a.ldo + (int64_t)head * a.c.D, b * 32 + 8 * i + 4 * half, a.c.D, v, l == 0.0f, l == 0.0f ? 0.0f : 1.0f / l);
    if (a.lse && b == 0 && i == 0 && half == 0) a.lse[row * a.ldl + head] = l == 0.0f ? -INFINITY : m * 0.69314718055994530942f + logf(l);
}

template <int ES, int CS, int NB, int WR, int KB, int ST, int OCC>
hipError_t launch_tile(const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    const unsigned grid = p.stream ? (unsigned)p.groups : (unsigned)(p.row_tiles * a.c.Hkv);
    attention_tile<ES, CS, NB, WR, KB, ST, OCC><<<dim3(grid), dim3(64 * WR), 0, s>>>(a, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.stream) return e;
    attention_join<ES, NB, WR><<<dim3((unsigned)p.groups, WR * NB), dim3(256), 0, s>>>(a, p);
    return hipGetLastError();
}

// dma: the cache goes to LDS without a stop.  Tiles by the bytes of a row in LDS.
template <int ES, int CS, int NB>
hipError_t launch_nb(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s) {
    constexpr int RB = (NB == 3 ? 128 : NB * 32) * ES;
    if (p.few) {
        if (dma) return launch_tile<ES, CS, NB, 1, 1, CS == 1 ? STAGE_INT8 : STAGE_DMA, CS == 1 && NB < 8 ? 2 : 1>(a, p, s);
        return launch_tile<ES, CS, NB, 1, 1, STAGE_REGS, 1>(a, p, s);
    }
    constexpr int KB = RB <= 256 ? 2 : 1, OCC = NB == 8 ? 1 : 2;
    if (dma && CS != 1) return launch_tile<ES, CS, NB, 4, KB, CS == 1 ? STAGE_REGS : STAGE_DMA, OCC>(a, p, s);
    return launch_tile<ES, CS, NB, 4, KB, STAGE_REGS, OCC>(a, p, s);
}

template <int ES, int CS>
hipError_t launch_by_size(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s) {
    if (a.c.D <= 64) return launch_nb<ES, CS, 2>(a, p, dma, s);
    if (a.c.D <= 96) return launch_nb<ES, CS, 3>(a, p, dma, s);
    if (a.c.D <= 128) return launch_nb<ES, CS, 4>(a, p, dma, s);
    return launch_nb<ES, CS, 8>(a, p, dma, s);
}

}  // namespace
}  // namespace tpl
