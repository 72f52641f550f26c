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
// instruction is free as long as the values come in the same one.)  That product's weights
// are of the values' type, since an instruction takes two of one type: bf16 with bf16
// values, by 2^-8 off at most (a result 1.86e-3 off where its own rounding alone makes it
// 1.65e-3), fp16 with int8 ones (1.67e-3), exact in fp32.  Their sum is not rounded.
//
// K and V tiles lie in LDS as rows of 64, 128 or 256 values, their 16-byte chunks permuted
// by the row so that reads meet no bank twice: K by chunks of 32 rows, bf16 values by the
// transposing read (4 keys x 16 features a 16-lane group, 8 keys in int8), fp32 values by
// words.  Two stages: the next tile is fetched while this one is there, straight into LDS
// (16 bytes a lane) where the cache is 16-byte aligned, else by way of registers, of rows
// that end inside a chunk too.  (But hipcc waits for every load before a tile's first
// product, since the query may have been loaded just before: a wavefront's fetch goes on
// under the work of other wavefronts, not under its own.)  int8 becomes bf16 or fp32
// (exactly; a key's scale multiplies its products, a value's scale its weight) as a
// wavefront reads it from LDS where it is alone, on the way into LDS where four read the
// same keys.
//
// What a row does not see must not touch it: keys and values of no position are zeros,
// products that a row does not see are minus infinity before the maximum, and a tile at
// the edge of what its rows see is looked through for values that are not finite: those
// become zeros there (weight zero times infinity would be NaN), and the rows that do see
// them get the infinity afterwards.
//
// Work: `items` are (sequence, rows, key head).  Where there are many, a workgroup takes
// one, the last rows of the last sequence first (a sequence's longest item; a long first
// sequence comes last: one of 2048 tokens behind 6000 before 300 of 128 730 us, behind
// them 712), neighbours in the grid on other key heads (an XCD, every 8th workgroup, then
// keeps to few heads, whose keys its L2 holds).  Else the tiles of all items in a row are
// cut into equal runs, one for each workgroup: a run's whole items are finished, the
// others' sums go to the workspace and are joined by a second launch in the order of the
// tiles.  The lengths are on the device: each workgroup adds them up itself. A run's tiles
// are one stream, across its items: wavefront 0 looks up the rows of the tile after next
// (and the next item, when one ends), which all need a tile later, so that the fetches
// never wait for it.  It alone reads the lengths, and the others go by what it leaves in
// LDS: a workgroup stays together and in bounds whatever is in those arrays, were they to
// change under it.
//
// Measured (both launches, a captured graph; inputs that no cache holds).  One token each
// of 64 sequences of 8000 at most, 64 query and 8 key heads of 128: 214 us, 5.0 TB/s, the
// rate of a copy; 16000 at most of 32 query heads over int8 213 us, 4.6 TB/s, where a
// tile's 500 vector instructions (its values become bf16 and fp16 in each wavefront) take
// 52% of the cycles.  A prompt of 4096 tokens, the same heads: 385-425 us by the chip's
// temperature, 650-700 TFLOP/s: the matrix cores are busy 29% and the vector units 44% of
// the cycles; the rest are the wait for the next tile above and four wavefronts' for each
// other every 64 keys (wavefront 0's look-ups 8%).  12 chunks of 600 tokens at most, 24
// query and 8 key heads of 96, a window of 1024 over int8: 114 us, 251 TFLOP/s, 630 vector
// instructions for 24 products a wavefront and tile, and 11 us the join.  4 sequences of
// 300 keys: 16 us, where the first tile is worked on after 9, lengths, page table, rows
// and keys read one after another. Split: 64 keys a tile instead of 32 where four
// wavefronts share them (fewer meetings), two workgroups a CU.  One wavefront a workgroup
// for 32 rows: four wavefronts that cut the keys of one tile among them and joined their
// sums in LDS took 257 us for the first case.  Heads past 128 are 256 features here, whose sums
// and query do not fit the registers (38 to 702 of them spilled), and take the time of 256: 64
// sequences of 8000 at most, 32 + 8 heads of 160, 192, 256 534, 551, 562 us.
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
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Source of the rows of no position (a row is 1 KB at most).
static __device__ __attribute__((aligned(16))) const uint32_t no_key[256] = {};

// A chunk of 16, or a word of 4 bytes a lane from the cache to LDS, at `lds` + lane * its
// size: instructions that the compiler does not track; the waits for them are written out
// below.
__device__ __forceinline__ void dma16(const char *from, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" :: "v"(from), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const char *from, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" :: "v"(from), "s"(lds) : "memory", "m0");
}

// The WR wavefronts meet: what each wrote to LDS before is there after it.  Written out,
// since hipcc leaves out the wait for LDS before a __syncthreads() that comes right behind
// a wait in inline assembly: rows looked up by wavefront 0 were then read by the others
// before they were there.
template <int WR>
__device__ __forceinline__ void meet() {
    if constexpr (WR > 1) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

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

// The second product of an int8 cache in a bf16 call: values and weights in fp16.
__device__ __forceinline__ f32x16 product_half(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// A value that all lanes have, as a scalar.
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
}
template <int N> struct Const { static constexpr int value = N; };
template <int ES> struct Bits { typedef uint32_t T; };
template <> struct Bits<2> { typedef uint16_t T; };
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// An item, and the part of its tiles that a run has; pieces: runs from this one to the
// item's last.  s < 0: none.
struct Item { int s; Sequence q; Span sp; int r, h, k0, k1, pieces; };

// A tile of a run: its rows that hold keys, the position of the first; what: its item's
// place in a ring, with BEGINS in the first tile of the item's part and ENDS in its last
// (-1: there is none).
struct __attribute__((aligned(16))) Tile { uint64_t rows; int first, what; };
enum { ITEMS = 4, BEGINS = 4, ENDS = 8 };

// Tiles that the change from one item to the next costs a run in time (a wavefront by
// itself: the query's loads, the sums' way out, the next item's lengths).
constexpr int CHANGE = 2;

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

// int8 values to fp16, 8 of them: a byte with its sign flipped is v + 128, below the
// exponent of 1024 it makes 1152 + v.
__device__ __forceinline__ u32x4 half_from_int8(uint32_t lo, uint32_t hi) {
    const uint32_t w[2] = {lo ^ 0x80808080u, hi ^ 0x80808080u};
    u32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        y[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w[e / 2], e & 1 ? 0x04030402u : 0x04010400u)) - f16x2{1152, 1152});
    return y;
}

// The bytes of x from bit n on (0 .. 120), zeros behind them.
__device__ __forceinline__ u32x4 shift_down(u32x4 x, int n) {
    const uint64_t lo = (uint64_t)x[1] << 32 | x[0], hi = (uint64_t)x[3] << 32 | x[2];
    const uint64_t l = n >= 64 ? hi >> (n & 63) : n > 0 ? lo >> n | hi << (64 - n) : lo, h = n >= 64 ? 0 : hi >> n;
    return u32x4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
}

__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32); }

// What lies in LDS: rows of the call's type by way of registers, the same straight from
// the cache, or int8 straight from the cache.  ODD: as REGS, of rows that end inside a chunk;
// the last is loaded so that it ends with the row, and moved to its place.
enum { STAGE_REGS = 0, STAGE_DMA = 1, STAGE_INT8 = 2, STAGE_ODD = 3 };

// FULL: D is 32 NB, all of a row in LDS.
template <int ES, int CS, int NB, int WR, int KB, int ST, int OCC, bool FULL>
__global__ __launch_bounds__(64 * WR, OCC)
void attention_tile(AttnArgs a, AttnPlan plan) {
    constexpr bool DMA = ST == STAGE_DMA || ST == STAGE_INT8, ALONE = WR == 1 && DMA;   // see the loop at the end
    constexpr int NW = WR, NTH = 64 * NW, ROWS = 32 * WR, BK = 32 * KB;
    constexpr int LS = ST == STAGE_INT8 ? 1 : ES;                       // bytes of a value in LDS
    constexpr int DP = NB == 3 ? 128 : NB * 32, RB = DP * LS;          // a row in LDS
    constexpr int KS = NB * ES;                                         // steps of the first product
    constexpr int CH = RB / 16, LI = BK * CH / NTH;                     // chunks of a row; of a thread and tile
    constexpr int STAGE = 2 * BK * RB;
    constexpr bool QUANT = CS == 1;
    constexpr bool HALF = QUANT && ES == 2;                             // values and weights in fp16: see below
    static_assert(BK <= NTH, "a thread a row of the tile");
    __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
    __shared__ struct { const char *k, *v; } row_at[2][BK];          // where the tiles' rows are
    __shared__ __attribute__((aligned(256))) float row_scale[2][2][QUANT ? 64 : 4];
    __shared__ Tile tiles[2];                          // the next tile and the one after it
    __shared__ Item items[ITEMS];
    __shared__ int scan[NW];
    // Where a run is (wavefront 0's, in LDS since scalar registers are short): its units
    // left, the sequence of the next with its row tiles, the next item's head and row tile;
    // of the first one the units before the sequence and those of one of its heads.
    __shared__ struct { int u, u1, all, W, first, seq, base, units, nr, h, r; Sequence q; } walk;
    __shared__ Sequence known[NTH];                    // the call's sequences, if they are no more
    __shared__ int found[2];
    __shared__ uint64_t odd[QUANT ? 1 : 2][QUANT ? 1 : DP];   // keys whose value of a feature is not finite: up, down
    LDS_PTR(char) lds = (LDS_PTR(char))smem;
    const uint32_t lds_u = (uint32_t)(uintptr_t)lds, scale_u = (uint32_t)(uintptr_t)(LDS_PTR(float))&row_scale[0][0][0];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave, half = lane >> 5, col = lane & 31;
    const CacheArgs &c = a.c;
    const int D = c.D, G = a.G;
    const float cs = a.scale * 1.44269504088896340736f;
    const int last_pos = plan.last_pos, window_of = plan.window;         // positions of the table; FAR: all
    const int chunks = ST == STAGE_ODD ? (D * LS + 15) / 16 : D * LS / 16;      // of a row in LDS that hold features
    constexpr int CB = 16 / ES * CS;                                    // bytes of a chunk in the cache (by way of registers)
    // where this thread's chunk, always the same of a row, is loaded
    const int load_at = ST == STAGE_ODD && (tid % CH + 1) * CB > D * CS ? D * CS - CB : tid % CH * CB;

    auto sequence = [&](int s) { return plan_sequence(c, plan.excess, s); };
    auto span = [&](const Sequence &q, int r) { return plan_span(plan, q, r, G, ROWS, BK); };
    auto row_tiles = [&](const Sequence &q) { return (q.n * G + ROWS - 1) / ROWS; };
    // Units of one head of each lane's sequence (its tiles, and the changes between its
    // items): by the lane where they are few, else by all lanes for one after another.
    auto count = [&](const Sequence &q) {
        const int nr = row_tiles(q);
        int n = nr * CHANGE;
        if (!__any(nr > 16)) {
            for (int r = 0; r < nr; ++r) n += span(q, r).tiles;
            return n;
        }
        for (uint64_t todo = __ballot(nr > 0); todo; todo &= todo - 1) {
            const int j = __builtin_ctzll(todo);
            const Sequence p{0, __shfl(q.n, j), __shfl(q.past, j)};
            int v = 0;
            for (int r = lane; r < row_tiles(p); r += 64) v += span(p, r).tiles;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
            if (lane == j) n += v;
        }
        return n;
    };

    // ---- the run of units of this workgroup
    int w = blockIdx.x;
    const int B = (int)c.B;
    if (plan.stream) {
        int all = 0, W = plan.groups;                   // units in all, runs that have any
        const int per = B <= NTH ? 1 : (B + NTH - 1) / NTH, sb = tid * per;
        int mine = 0;
        for (int i = sb; i < sb + per; ++i) {           // in step: count() takes whole wavefronts
            Sequence q{};
            if (i < B) q = sequence(i);
            const int n = count(q);
            mine += n;
            if (per == 1) known[tid] = q;
        }
        int run = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(run, o);
            if (lane >= o) run += v;
        }
        if (lane == 63) scan[wave] = run;
        meet<WR>();
        int before = 0;
        for (int i = 0; i < NW; ++i) {
            if (i < wave) before += scan[i];
            all += scan[i];
        }
        all = uniform(all) * c.Hkv;
        if (all < W) W = all;
        else w = (w & 7) * (W / 8) + (w >> 3);          // runs next to each other on one XCD
        if (tid == 0) plan_desc(a.ws)[w].pieces = 0;
        if (w >= W) return;
        auto cut = [&](int i) { return W < plan.groups ? i : (int)((int64_t)all * i / plan.groups); };
        const int u = cut(w);
        if (tid == 0) {
            walk.u = u;
            walk.u1 = cut(w + 1);
            walk.all = all;
            walk.W = W;
            walk.seq = B;
            walk.first = 1;
        }
        meet<WR>();
        int at = (before + run - mine) * c.Hkv;
        const bool here = u >= at && u < (before + run) * c.Hkv;       // one thread
        if (per == 1) {
            if (here) {
                walk.seq = tid;
                walk.base = at;
                walk.units = mine;
            }
        } else {
            bool open = here;
            for (int i = sb; i < sb + per && __any(open); ++i) {
                Sequence q{};
                if (i < B) q = sequence(i);
                const int n = count(q);
                if (open && u < at + n * c.Hkv) {
                    walk.seq = i;
                    walk.base = at;
                    walk.units = n;
                    open = false;
                }
                at += n * c.Hkv;
            }
        }
        meet<WR>();
    }
    int stamp = 0;
    if (tid < 2) found[tid] = -1;

    // The next item and the part of its tiles (wavefront 0): the run's first by search, the
    // ones after it in order.
    bool first_item = true;
    auto known_sequence = [&](int i) {
        Sequence q;
        if (B <= NTH) q = known[i];
        else q = sequence(i);
        return Sequence{uniform(q.first), uniform(q.n), uniform(q.past)};
    };
    auto find_item = [&]() {
        Item m{};
        m.s = -1;
        if (plan.stream) {
            int u = uniform(walk.u), seq = uniform(walk.seq), h = uniform(walk.h), r = uniform(walk.r), nr = uniform(walk.nr);
            const int u1 = uniform(walk.u1);
            Sequence q{uniform(walk.q.first), uniform(walk.q.n), uniform(walk.q.past)};
            bool begin = uniform(walk.first);
            while (u < u1 && seq < B) {
                int rem = 0;
                if (begin) {
                    begin = false;
                    const int units = uniform(walk.units);
                    q = known_sequence(seq);
                    nr = row_tiles(q);
                    rem = u - uniform(walk.base);
                    if (units <= 0 || rem < 0) break;       // sums past 32 bits, of lengths that no call has
                    h = (uint32_t)rem / (uint32_t)units;
                    if (h >= c.Hkv) break;
                    rem -= h * units;
                    // the row tile in which the units up to `rem` end, of 64 at a time
                    bool got = false;
                    for (int r0 = 0; r0 < nr && !got; r0 += 64) {
                        const int t = r0 + lane < nr ? CHANGE + span(q, r0 + lane).tiles : 0;
                        int v = t;
#pragma unroll
                        for (int o = 1; o < 64; o <<= 1) {
                            const int y = __shfl_up(v, o);
                            if (lane >= o) v += y;
                        }
                        const uint64_t beyond = __ballot(rem < v && t > 0);
                        got = beyond != 0;
                        const int j = got ? __builtin_ctzll(beyond) : 63;
                        r = r0 + j;
                        rem -= uniform(__shfl(got ? v - t : v, j));
                    }
                    if (!got) break;
                } else if (++r >= nr) {
                    r = 0;
                    if (++h >= c.Hkv) {
                        h = 0;
                        r = -1;                             // the next step's is the sequence's first, if it has rows
                        if (++seq >= B) break;
                        q = known_sequence(seq);
                        nr = row_tiles(q);
                        if (nr == 0) h = c.Hkv;
                        continue;
                    }
                }
                const Span sp = span(q, r);
                const int item_u = u - rem, end = item_u + CHANGE + sp.tiles;       // the item's units
                m.q = q; m.sp = sp; m.r = r; m.h = h;
                m.k0 = rem > CHANGE ? rem - CHANGE : 0;
                m.k1 = (u1 < end ? u1 : end) - item_u - CHANGE;
                u = end;
                if (m.k1 <= m.k0) continue;                 // none of its tiles: all in the next run
                m.s = seq;
                m.pieces = 1;
                if (end > u1) {
                    const int W = uniform(walk.W);
                    int to = (int)(((int64_t)end * W - 1) / uniform(walk.all));     // the run with the item's last tile
                    if (to >= W) to = W - 1;
                    m.pieces = to - w + 1;
                }
                break;
            }
            walk.u = u;
            walk.seq = seq;
            walk.h = h;
            walk.r = r;
            walk.nr = nr;
            walk.q = q;
            walk.first = 0;
        } else if (first_item) {
            first_item = false;
            const int i = (int)plan.row_tiles - 1 - w / c.Hkv;
            // sequence s has the indices from cu[s] G / ROWS + s on, enough for its rows
            int lo = 0, n = B;
            while (n > 0) {
                const int step = (n + 63) / 64;
                const int j = lo + lane * step;
                const bool below = lane * step < n && plan_index(c, j, G, ROWS) <= i;
                const int k = __popcll(__ballot(below));
                if (k == 0) break;
                const int b = (k - 1) * step;
                lo += b + 1;
                n = (n - b < step ? n - b : step) - 1;
            }
            const int s = uniform(lo) - 1;
            if (s >= 0) {
                const Sequence q = sequence(s);
                const int r = i - plan_index(c, s, G, ROWS);
                if (r >= 0 && r < row_tiles(q)) {
                    m.s = s; m.q = q; m.r = r; m.h = w % c.Hkv;
                    m.sp = span(q, r);
                    m.k1 = m.sp.tiles;
                    m.pieces = 1;
                }
            }
        }
        return m;
    };

    // ---- rows of a tile: where they are, and which there are (wavefront 0, in the order
    // of the run's tiles; numbers of tiles and items go round in rings)
    int ahead_s = -1, ahead_begin = 0, ahead_end = 0, ahead_t0 = 0, ahead_left = 0, ahead_item = -1;
    int64_t ahead_at = 0, ahead_sat = 0;               // of the head in the cache's rows, and among the scales
    // Entries of the table: lane i has entry `window + i` of the sequence's, so that a tile
    // needs a load only where it leaves them.
    int32_t entry = -1;
    int window = 0;
    const char *scale_k = (const char *)no_key, *scale_v = (const char *)no_key;     // of this lane's row of the last tile looked up
    auto look = [&](int n) {
        const bool begins = ahead_left == 0;
        if (!begins) {
            --ahead_left;
            ahead_t0 += BK;
        } else {
            const Item m = find_item();
            ahead_item = (ahead_item + 1) % ITEMS;
            if (lane == 0) items[ahead_item] = m;
            ahead_s = uniform(m.s);
            ahead_begin = uniform(m.sp.begin);
            ahead_end = ahead_s >= 0 ? uniform(m.sp.end) : 0;       // of no item no position is looked up
            ahead_t0 = (uniform(m.sp.first) + uniform(m.k0)) * BK;
            ahead_at = uniform(m.h) * c.s_head;
            ahead_sat = uniform(m.h) * c.ss_head;
            ahead_left = ahead_s >= 0 ? uniform(m.k1) - uniform(m.k0) - 1 : 0;
            window = -64;                               // another sequence's
        }
        const int t0 = ahead_t0, p = t0 + lane;
        const bool want = lane < BK && p >= ahead_begin && p < ahead_end;
        const int i = plan_divide(p, plan.page);
        if (__any(want && (uint32_t)(i - window) >= 64)) {
            // from the tile's first position that counts on; its last is in less than BK pages
            window = uniform(plan_divide(t0 > ahead_begin ? t0 : ahead_begin, plan.page));
            entry = window + lane < (int)c.max_pages ? c.table[ahead_s * c.ldt + window + lane] : -1;
            // waited for here, once in 64 pages, and not by every use below
            asm volatile("s_waitcnt vmcnt(0)" : "+v"(entry) :: "memory");
        }
        const uint32_t id = (uint32_t)__builtin_amdgcn_ds_bpermute((i - window) * 4, entry);     // of lane (i - window) % 64
        const uint32_t slot = (uint32_t)p - (uint32_t)i * c.page;
        const bool ok = want && id < plan.n_pages;
        if (__any(want && !ok) && c.bad) *c.bad = 1;
        const uint64_t rows = __ballot(ok);
        if (lane < BK) {
            const int64_t at = ((int64_t)((uint64_t)id * (uint64_t)c.s_page + (uint64_t)slot * (uint64_t)c.s_slot) + ahead_at) * CS;
            row_at[n & 1][lane].k = ok ? (const char *)c.kc + at : (const char *)no_key;
            row_at[n & 1][lane].v = ok ? (const char *)c.vc + at : (const char *)no_key;
        }
        if (lane == 0) tiles[n & 1] = Tile{rows, t0, ahead_s < 0 ? -1 : ahead_item | (begins ? BEGINS : 0) | (ahead_left == 0 ? ENDS : 0)};
        if (QUANT) {
            const int64_t at = (int64_t)((uint64_t)id * (uint64_t)c.ss_page + (uint64_t)slot * (uint64_t)c.ss_slot) + ahead_sat;
            scale_k = ok ? (const char *)(c.ks + at) : (const char *)no_key;
            scale_v = ok ? (const char *)(c.vs + at) : (const char *)no_key;
        }
    };

    // ---- a tile's chunks: thread tid has chunk i NTH + tid of K and of V
    u32x4 kr[DMA ? 1 : LI], vr[DMA ? 1 : LI];
    float scale_kr = 0.0f, scale_vr = 0.0f;
    auto place = [&](int n) { return (n & 1) * STAGE; };                     // of tile n in LDS
    // K (or V) of tile n: K with the scales of the tile that was looked up last.
    auto fetch = [&](int n, auto is_v) __attribute__((always_inline)) {
        constexpr bool V = decltype(is_v)::value;
        const int st = n & 1;
        const char *from[LI];
#pragma unroll
        for (int i = 0; i < LI; ++i) from[i] = V ? row_at[st][(i * NTH + tid) / CH].v : row_at[st][(i * NTH + tid) / CH].k;
#pragma unroll
        for (int i = 0; i < LI; ++i) {
            const int k = i * NTH + tid, r = k / CH, ch = k % CH;
            if constexpr (DMA) {
                const int at = ch ^ ((V ? v_swizzle<LS, RB>(r) : k_swizzle<RB>(r)) >> 4);
                dma16(FULL || at < chunks ? from[i] + at * 16 : (const char *)no_key, lds_u + place(n) + (V ? BK * RB : 0) + (i * NTH + wave * 64) * 16);
            } else {
                u32x4 &x = V ? vr[i] : kr[i];
                x = u32x4{0, 0, 0, 0};
                if (ch < chunks) {
                    const char *p = from[i] + load_at;
                    if constexpr (!QUANT) {
                        x = *(const u32x4_any *)p;
                    } else if constexpr (ES == 2) {
                        const u32x2 y = *(const u32x2_any *)p;
                        x[0] = y[0]; x[1] = y[1];
                    } else {
                        x[0] = *(const u32_any *)p;
                    }
                }
            }
        }
        if (QUANT && !V && wave == 0) {
            if constexpr (DMA) {
                dma4(scale_k, scale_u + st * 512);
                dma4(scale_v, scale_u + st * 512 + 256);
            } else {
                scale_kr = *(const float *)scale_k;
                scale_vr = *(const float *)scale_v;
            }
        }
    };
    // What was fetched is in LDS, this thread's part.
    auto settle_all = [&](int n) __attribute__((always_inline)) {
        if constexpr (DMA) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
#pragma unroll
            for (int i = 0; i < LI; ++i) {
                const int k = i * NTH + tid, r = k / CH, ch = k % CH;
                const uint32_t at = (n & 1) * STAGE + r * RB;
                if (ST == STAGE_ODD) {
                    kr[i] = shift_down(kr[i], ch < chunks ? 8 * (ch * CB - load_at) : 0);
                    vr[i] = shift_down(vr[i], ch < chunks ? 8 * (ch * CB - load_at) : 0);
                }
                *(LDS_PTR(u32x4))(lds + at + ((ch * 16) ^ k_swizzle<RB>(r))) = QUANT ? from_int8<ES>(kr[i][0], kr[i][1]) : kr[i];
                *(LDS_PTR(u32x4))(lds + at + BK * RB + ((ch * 16) ^ v_swizzle<LS, RB>(r))) = HALF ? half_from_int8(vr[i][0], vr[i][1]) : QUANT ? from_int8<ES>(vr[i][0], vr[i][1]) : vr[i];
            }
            if (QUANT && wave == 0) {
                row_scale[n & 1][0][QUANT ? lane : 0] = scale_kr;
                row_scale[n & 1][1][QUANT ? lane : 0] = scale_vr;
            }
        }
    };
    // Of this tile, while the next one's instructions are under way (64 at most; the counter
    // holds 63).
    auto settle_first = [&]() __attribute__((always_inline)) {
        constexpr int LATER = 2 * LI + (QUANT ? 2 : 0);
        asm volatile("s_waitcnt vmcnt(%0)" :: "n"(LATER < 63 ? LATER : 63) : "memory");
    };

    // ---- the item that a tile belongs to: this lane's row, its query and its sums
    bool live = false, several = false, whole = false;
    int item_r = 0, item_h = 0, pieces = 0, slot = 0, head = 0;
    int rows = 0, first = 0, row = 0, hi = 0, lo = 0, see_all = 0, see_from = 0;
    bool begins_split = false;
    u32x4 qf[KS];
    f32x16 o[NB];
    float mx = -INFINITY, l = 0.0f;
    // HALF: weights times scales go into the second product as fp16, which rounds them by
    // 2^-11 at most (bf16: 2^-8, as much as the output's own rounding) where they are its normal
    // numbers, and smaller ones to multiples of 2^-24: all weights are 2^shift times the
    // softmax's, o with them, so that the largest of a row (top_w) is between 2^4 and 2^15.  The
    // shift begins at 2^16, for scales of values of order one, and hardly ever changes.  As far
    // as it is in 0 .. NEAR it is in the exponential's argument, where it costs nothing (l has it
    // too), and what is missing of it (far) is put in behind the product with the scale.  A row
    // that sees scales past MOST_SCALE, where that product might not be finite, has none of it in
    // the argument for that tile.  With a shift of MOST fp32's smallest values are fp16's.
    constexpr float NEAR = 60.0f, MOST = 125.0f, MOST_SCALE = 0x1p67f;
    float shift = 16.0f, top_w = 0.0f;
    uint64_t far = 0;                                                       // the lanes whose shift is not in 0 .. NEAR
    auto near_of = [&](float v) { return fminf(fmaxf(v, 0.0f), NEAR); };
    auto enter = [&](int i) __attribute__((always_inline)) {
        const Item &m = items[i];
        first = uniform(m.q.first);
        const int past = uniform(m.q.past), pos0 = uniform(m.sp.pos0), pos1 = uniform(m.sp.pos1);
        rows = uniform(m.q.n) * G;
        item_r = uniform(m.r);
        item_h = uniform(m.h);
        pieces = uniform(m.pieces);
        const int k0 = uniform(m.k0), k1 = uniform(m.k1), n = uniform(m.sp.tiles);
        whole = k0 == 0 && k1 == n;
        begins_split = k0 == 0 && k1 < n;
        slot = 2 * w + (k0 == 0 ? 1 : 0);
        if ((pos0 < 0 || pos1 >= last_pos) && c.bad && tid == 0) *c.bad = 1;
        const int R = item_r * ROWS + wr * 32 + col;
        live = R < rows;
        const int tok = live ? plan_divide(R, plan.g) : 0;
        head = item_h * G + (live ? R - tok * G : 0);
        row = first + tok;
        hi = live ? past + tok : -1;
        lo = past + tok - window_of + 1;
        see_all = pos0;                                                     // keys that every row sees
        see_from = pos1 - window_of + 1;
        several = pos1 > pos0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            // the features that a lane's k-th operand of K has
            const int ch = ST == STAGE_INT8 ? (2 * (k / ES) + half) * ES + k % ES : 2 * k + half;
            qf[k] = u32x4{0, 0, 0, 0};
            const char *p = (const char *)a.Q + ((int64_t)row * a.ldq + (int64_t)head * D) * ES;
            if (live && ch < D * ES / 16) qf[k] = *(const u32x4_any *)(p + ch * 16);
            else if (ST == STAGE_ODD && live && ch < chunks) qf[k] = shift_down(*(const u32x4_any *)(p + D * ES - 16), 8 * ((ch + 1) * 16 - D * ES));
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[b][e] = 0.0f;
        mx = -INFINITY;
        l = 0.0f;
        shift = 16.0f;
        top_w = 0.0f;
        far = 0;
    };

    // ---- one tile
    auto tile = [&](int n, int t0, uint64_t valid) __attribute__((always_inline)) {
        const int st = n & 1;
        const bool edge = t0 + BK - 1 > see_all || t0 < see_from;
        f32x16 x[KB];
        const uint32_t kl = place(n) + col * RB, ks = (half * 16) ^ k_swizzle<RB>(col);
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
        uint64_t apart = 0;         // HALF: where scales are that they and the shift may take past fp32, or shifts that are far
        if constexpr (QUANT) {
            if constexpr (HALF) apart = far | __ballot(!(fabsf(row_scale[st][1][lane & (BK - 1)]) <= MOST_SCALE));
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 z = *(LDS_PTR(f32x4))(LDS_PTR(float))&row_scale[st][0][b * 32 + 8 * i + 4 * half];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[b][4 * i + e] *= z[e];
                }
        }
        // the keys that this lane's row sees
        uint64_t seen = valid;
        const bool masked = edge || valid != (BK == 64 ? ~0ull : (1ull << (BK & 63)) - 1);
        if (masked) {
            const int up = hi - t0, from = lo - t0;
            seen &= up >= 63 ? ~0ull : up < 0 ? 0ull : (2ull << up) - 1;
            seen &= from <= 0 ? ~0ull : from > 63 ? 0ull : ~0ull << from;
            const uint64_t mine = seen >> (4 * half);
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!((uint32_t)(mine >> (32 * b)) >> (8 * (i / 4) + i % 4) & 1)) x[b][i] = -INFINITY;
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
            if (HALF) top_w *= f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][i] *= f;
            mx = next;
        }
        float held = shift;                                                 // HALF: the shift in the exponents
        if constexpr (HALF) {
            if (__builtin_expect(apart != 0, 0)) {
                const uint64_t mine = seen >> (4 * half);
                float z = 0.0f;                                             // of the scales that the row sees
                for (int i = 0; i < 16 * KB; ++i)
                    if (mine >> (8 * (i / 4) + i % 4) & 1) z = fmaxf(z, fabsf(row_scale[st][1][8 * (i / 4) + i % 4 + 4 * half]));
                held = fmaxf(z, other_half(z)) > MOST_SCALE ? 0.0f : near_of(shift);
            }
        }
        const float less = HALF ? held - zero : -zero;
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[b][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[b][i], cs, less));
                sum += x[b][i];
            }
        if constexpr (QUANT) {
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 z = *(LDS_PTR(f32x4))(LDS_PTR(float))&row_scale[st][1][b * 32 + 8 * i + 4 * half];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[b][4 * i + e] *= z[e];
                }
            if (masked) {                                   // whatever the scale
                const uint64_t mine = seen >> (4 * half);
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!((uint32_t)(mine >> (32 * b)) >> (8 * (i / 4) + i % 4) & 1)) x[b][i] = 0.0f;
            }
        }
        if constexpr (HALF) {
            float most = fabsf(x[0][0]);
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(x[b][i]));
            most = fmaxf(most, other_half(most));
            const float was = top_w;
            top_w = fmaxf(was, most);
            if (__builtin_expect((apart | __ballot((top_w >= 32768.0f) | ((top_w < 16.0f) & (top_w > 0.0f)))) != 0, 0)) {
                // the row's largest to 2^12 (an infinite scale stays infinite)
                const int old = (int)shift;
                const float largest = fmaxf(__builtin_amdgcn_ldexpf(was, -old), __builtin_amdgcn_ldexpf(most, -(int)held));
                const float there = __builtin_amdgcn_ldexpf(largest, old);
                const bool off = (largest > 0.0f) & (largest < INFINITY) & ((there >= 32768.0f) | (there < 16.0f));
                shift = off ? fminf((float)(13 - __builtin_amdgcn_frexp_expf(largest)), MOST) : shift;
                const int by = (int)shift - old, lacks = (int)(shift - held);
                top_w = __builtin_amdgcn_ldexpf(largest, (int)shift);
                l = __builtin_amdgcn_ldexpf(l, (int)(near_of(shift) - near_of((float)old)));
                sum = __builtin_amdgcn_ldexpf(sum, (int)(near_of(shift) - held));
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[b][i] = __builtin_amdgcn_ldexpf(x[b][i], lacks);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[b][i] = __builtin_amdgcn_ldexpf(o[b][i], by);
                far = __ballot(near_of(shift) != shift);
            }
        }
        l += sum;
        // values that are not finite, where rows see different keys
        bool dirty = false;
        if (!QUANT && edge && several) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < LI; ++i) {
                const u32x4 x = *(LDS_PTR(u32x4))(lds + place(n) + BK * RB + (i * NTH + tid) * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (ES == 2) any |= (x[e] & 0x7F80) == 0x7F80 || (x[e] & 0x7F800000) == 0x7F800000;
                    else any |= (x[e] & 0x7F800000) == 0x7F800000;
                }
            }
            ++stamp;
            if (any) found[stamp & 1] = stamp;
            meet<WR>();
            dirty = uniform(found[stamp & 1]) == stamp;
            if (dirty) {
                // zeros in their place, and for each feature the keys: a NaN is up and down
                for (int i = tid; i < 2 * DP; i += NTH) odd[i / DP][i % DP] = 0;
                meet<WR>();
                for (int i = 0; i < LI; ++i) {
                    const int k = i * NTH + tid, r = k / CH;
                    const int d = ((k % CH) * 16 ^ v_swizzle<LS, RB>(r)) / ES;
                    for (int e = 0; e < 16 / ES; ++e) {
                        typedef typename Bits<ES>::T B;
                        LDS_PTR(B) v = (LDS_PTR(B))(lds + place(n) + BK * RB + k * 16) + e;
                        const uint32_t y = ES == 2 ? (uint32_t)*v << 16 : (uint32_t)*v;
                        if ((y & 0x7F800000) != 0x7F800000) continue;
                        *v = 0;
                        const bool nan = (y & 0x7FFFFF) != 0;
                        if (nan || !(y >> 31)) atomicOr((unsigned long long *)&odd[0][d + e], 1ull << r);
                        if (nan || y >> 31) atomicOr((unsigned long long *)&odd[QUANT ? 0 : 1][d + e], 1ull << r);
                    }
                }
                meet<WR>();
            }
        }
        const uint32_t vl = place(n) + BK * RB;
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
                        f16x8 h;
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = (_Float16)x[b][8 * s2 + e];
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
                            o[d] = product_half(half_from_int8(v[0], v[1]), p[0], o[d]);
                        } else {
                            o[d] = product<ES>(from_int8<ES>(v[0], 0), p[0], o[d]);
                            o[d] = product<ES>(from_int8<ES>(v[1], 0), p[ES / 4], o[d]);
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
                    u32x4 p;
                    if constexpr (HALF) {
                        f16x8 h;
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = (_Float16)x[b][8 * s2 + e];
                        p = __builtin_bit_cast(u32x4, h);
                    } else {
                        bf16x8 h;
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = (__bf16)x[b][8 * s2 + e];
                        p = __builtin_bit_cast(u32x4, h);
                    }
#pragma unroll
                    for (int d = 0; d < NB; ++d) {
                        LDS_PTR(char) v = lds + at + (b * 32 + s2 * 16) * RB + ((d * 64) ^ sw);
                        const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR(s16x4))v);
                        const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_PTR(s16x4))(v + 8 * RB));
                        const u32x4 y = __builtin_bit_cast(u32x4, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
                        o[d] = HALF ? product_half(y, p, o[d]) : product<ES>(y, p, o[d]);
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
                            const uint32_t k = b * 32 + 8 * i + e + 4 * half;           // (k >> 2) & 1 = half
                            v[e] = *(LDS_PTR(uint32_t))(lds + vl + k * RB + ((d * 128 + col * 4) ^ (half << 7)));
                            p[e] = __float_as_uint(x[b][4 * i + e]);
                        }
                        o[d] = product<ES>(v, p, o[d]);
                    }
        }
        if (dirty) {
#pragma unroll
            for (int d = 0; d < NB; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    __builtin_amdgcn_sched_barrier(0);
                    const int f = d * 32 + 8 * (i / 4) + 4 * half + i % 4;
                    if (odd[0][QUANT ? 0 : f] & seen) o[d][i] += INFINITY;
                    if (odd[QUANT ? 0 : 1][QUANT ? 0 : f] & seen) o[d][i] -= INFINITY;
                }
        }
    };

    // ---- the end of an item's part: rows, or sums for the join
    auto leave = [&]() __attribute__((always_inline)) {
        l += other_half(l);
        if constexpr (HALF) l = __builtin_amdgcn_ldexpf(l, -(int)near_of(shift));
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float unshift = HALF ? __builtin_amdgcn_ldexpf(1.0f, -(int)shift) : 1.0f;
        if (live) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4 v;
                    // HALF, of all of a row: the quotient first, which is finite where the sum may not be
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = HALF ? o[b][4 * i + e] * (whole ? inv : unshift) : o[b][4 * i + e];
                    if (whole) write_out<ES, FULL ? ROW_FULL : ST == STAGE_ODD ? ROW_ENDS : ROW_FOURS>(a.O, (int64_t)row * a.ldo + (int64_t)head * D, b * 32 + 8 * i + 4 * half, D, v, l == 0.0f, HALF ? unshift : inv);
                    else plan_sums(a.ws, plan.groups)[(((int64_t)slot * WR + wr) * NB + b) * 256 + i * 64 + lane] = v;
                }
            if (half == 0 && !whole) {
                float *ml = plan_stats(a.ws, plan.groups) + ((int64_t)slot * ROWS + wr * 32 + col) * 2;
                ml[0] = mx;
                ml[1] = l;
            } else if (half == 0 && a.lse) {
                a.lse[(int64_t)row * a.ldl + head] = l == 0.0f ? -INFINITY : mx * 0.69314718055994530942f + logf(l);
            }
        }
        // a run that begins an item names the runs that hold the rest of it
        if (begins_split && tid == 0) plan_desc(a.ws)[w] = PlanDesc{pieces, item_r, item_h, rows, first};
    };

    // ---- the tiles.  In one loop, so that each step is there once (a launch begins without
    // instructions in the caches): tile n + 2 is looked up, tile n + 1 fetched, tile n worked
    // on.  A wavefront by itself (ALONE) asks for the next tile before this one is there, as
    // soon as its place in LDS is free; four wait for theirs first, and then for each other.
    Tile now{0, 0, -1}, next{0, 0, -1};
    for (int n = -2;; ++n) {
        if (!ALONE && n >= 0) settle_all(n);
        meet<WR>();                                     // also: this wavefront's reads of the last tile are done
        bool more = true;
        if (n >= -1) {
            const Tile t = tiles[(n + 1) & 1];
            next = Tile{uniform64(t.rows), uniform(t.first), uniform(t.what)};
            more = next.what >= 0;
            if (n < 0 && !more) return;
            if (more) {
                fetch(n + 1, Const<0>());
                fetch(n + 1, Const<1>());
            }
        }
        if (ALONE && n >= 0) {
            if (more) settle_first();
            else settle_all(n);
        }
        if (more && wave == 0) look(n + 2);
        if (n >= 0) {
            if (now.what & BEGINS) enter(now.what % ITEMS);
            tile(n, now.first, now.rows);
            if (now.what & ENDS) leave();
            if (!more) return;
        }
        now = next;
    }
}

// Joins the sums of the items that more than one run holds: workgroup (w, y) 32 rows and 32
// features of the item that run w begins; its first sums are in slot 2 w + 1, the later ones
// in slots 2 (w + 1), 2 (w + 2), ...  Of few runs a wavefront adds up 8 of the features, in
// the runs' order; of many (a long sequence with few heads) it takes every fourth run with
// all of the features, and then the four are added in order.
constexpr int JOIN = 256, JOIN_ALONE = 8;
template <int N> struct JoinSums { float m, l; f32x4 x[N]; };

template <int N>
__device__ __forceinline__ void join_add(JoinSums<N> &s, float m, float l, const f32x4 (&y)[N]) {
    const float top = fmaxf(s.m, m), zero = top == -INFINITY ? 0.0f : top;
    const float f0 = __builtin_amdgcn_exp2f(s.m - zero), f1 = __builtin_amdgcn_exp2f(m - zero);
    s.m = top;
    s.l = __builtin_fmaf(f1, l, s.l * f0);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s.x[i][e] = __builtin_fmaf(f1, y[i][e], s.x[i][e] * f0);
}

template <int ES, int NB, int WR, bool ODD>
__global__ __launch_bounds__(JOIN)
void attention_join(AttnArgs a, AttnPlan plan) {
    constexpr int ROWS = 32 * WR, JW = JOIN / 64;
    __shared__ JoinSums<4> parts[JW][64];
    const int w = blockIdx.x, wr = blockIdx.y / NB, b = blockIdx.y % NB;
    const PlanDesc d = plan_desc(a.ws)[w];
    if (d.pieces == 0) return;
    const int lane = threadIdx.x & 63, v = threadIdx.x >> 6, half = lane >> 5, col = lane & 31;
    const int R = d.r * ROWS + wr * 32 + col;
    const bool live = R < d.rows;
    const int tok = live ? (int)((uint32_t)R / (uint32_t)a.G) : 0, head = d.h * a.G + (live ? R - tok * a.G : 0);
    const int64_t row = d.first + tok;
    const float *ml = plan_stats(a.ws, plan.groups) + (int64_t)(wr * 32 + col) * 2;
    auto slot = [&](int k) { return k == 0 ? (int64_t)2 * w + 1 : (int64_t)2 * (w + k); };
    const f32x4 *sums = plan_sums(a.ws, plan.groups) + ((int64_t)wr * NB + b) * 256 + lane;
    const bool few = d.pieces <= JOIN_ALONE;
    JoinSums<4> s{-INFINITY, 0.0f, {}};
    JoinSums<1> t{-INFINITY, 0.0f, {}};
    if (live && few) {
        // four runs at a time, whose loads leave together
        for (int k0 = 0; k0 < d.pieces; k0 += 4) {
            f32x4 y[4][1];
            float m[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[j] = -INFINITY;
                l[j] = 0.0f;
                y[j][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                if (k0 + j < d.pieces) {
                    const float *p = ml + slot(k0 + j) * ROWS * 2;
                    m[j] = p[0];
                    l[j] = p[1];
                    y[j][0] = sums[slot(k0 + j) * WR * NB * 256 + v * 64];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) join_add<1>(t, m[j], l[j], y[j]);
        }
    } else if (live) {
#pragma unroll 4
        for (int k = v; k < d.pieces; k += JW) {
            const float *p = ml + slot(k) * ROWS * 2;
            f32x4 y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = sums[slot(k) * WR * NB * 256 + i * 64];
            join_add<4>(s, p[0], p[1], y);
        }
    }
    if (!few) {
        parts[v][lane] = s;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < JW; ++k) {
            const f32x4 y[1] = {parts[k][lane].x[v]};
            join_add<1>(t, parts[k][lane].m, parts[k][lane].l, y);
        }
    }
    if (!live) return;
    const bool none = t.l == 0.0f;
    write_out<ES, ODD ? ROW_ENDS : ROW_FOURS>(a.O, row * a.ldo + (int64_t)head * a.c.D, b * 32 + 8 * v + 4 * half, a.c.D, t.x[0], none, none ? 0.0f : 1.0f / t.l);
    if (a.lse && b == 0 && v == 0 && half == 0) a.lse[row * a.ldl + head] = none ? -INFINITY : t.m * 0.69314718055994530942f + logf(t.l);
}

template <int ES, int CS, int NB, int WR, int KB, int ST, int OCC, bool FULL>
hipError_t launch_tile(const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    const unsigned grid = p.stream ? (unsigned)p.groups : (unsigned)(p.row_tiles * a.c.Hkv);
    attention_tile<ES, CS, NB, WR, KB, ST, OCC, FULL><<<dim3(grid), dim3(64 * WR), 0, s>>>(a, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.stream) return e;
    attention_join<ES, NB, WR, ST == STAGE_ODD><<<dim3((unsigned)p.groups, WR * NB), dim3(JOIN), 0, s>>>(a, p);
    return hipGetLastError();
}

// dma: the cache goes to LDS without a stop.  Tiles by the bytes of a row in LDS.
template <int ES, int CS, int NB, bool FULL>
hipError_t launch_full(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s) {
    constexpr int RB = (NB == 3 ? 128 : NB * 32) * ES, OCC = NB == 8 ? 1 : 2;
    const bool odd = a.c.D % (16 / ES);
    if (p.few) {
        if (odd) return launch_tile<ES, CS, NB, 1, 1, STAGE_ODD, 1, false>(a, p, s);
        if (dma) return launch_tile<ES, CS, NB, 1, 1, CS == 1 ? STAGE_INT8 : STAGE_DMA, OCC, FULL>(a, p, s);
        return launch_tile<ES, CS, NB, 1, 1, STAGE_REGS, 1, false>(a, p, s);
    }
    constexpr int KB = RB <= 256 ? 2 : 1;
    if (odd) return launch_tile<ES, CS, NB, 4, KB, STAGE_ODD, OCC, false>(a, p, s);
    if (dma && CS != 1) return launch_tile<ES, CS, NB, 4, KB, CS == 1 ? STAGE_REGS : STAGE_DMA, OCC, CS != 1 && FULL>(a, p, s);
    return launch_tile<ES, CS, NB, 4, KB, STAGE_REGS, OCC, false>(a, p, s);
}
template <int ES, int CS, int NB>
hipError_t launch_nb(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s) {
    if (NB != 3 && a.c.D == 32 * NB) return launch_full<ES, CS, NB, NB != 3>(a, p, dma, s);
    return launch_full<ES, CS, NB, false>(a, p, dma, s);
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
