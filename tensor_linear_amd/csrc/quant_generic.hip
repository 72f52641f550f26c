// Int8 shard GEMM for any M, N, K, leading dimension and alignment ("模型并行",
// "Tensor Parallel": the per-shard products Y_i = X W_i and X_i W_i, the
// operands held in 8 bits): acc[m, n] = sum_k x[m, k] w[n, k] exactly in int32
// on v_mfma_i32_16x16x64_i8, scaled in the epilogue.
//
// Tiles 128 x 128 (four waves of 64 x 64) or 64 x 64 (four of 16 x 64), 128 bytes of K
// a stage: each thread loads its 16-byte chunks of the next stage into registers
// while the current one is multiplied, and then writes them to the other of two
// LDS buffers, rows of 144 bytes (the 16 padding bytes turn the 16 rows of a
// fragment read into different banks).  Chunks past K and rows past M or N are
// zeros, which add nothing to an integer sum.  It serves what the DMA kernels
// cannot load (K or strides not a multiple of 16, unaligned views) and is bound by
// its unaligned loads, which often take two lines each: 4096 tokens of 4097 -> 28672
// 779-827 us (1.2 POP/s; the DMA kernels with K = 4096 373-387), three shards of 1999 ->
// 1112 at 333 tokens 23 us (10.8).  256 bytes a stage for the small tile were slower
// (1999: 33 us).
#include "quant.h"
#include "quant_epilogue.h"

namespace tpl {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int QGROUP = 8;       // tile rows visited as a group

// 16 bytes from p (any alignment), of which the first `n` are in the row.
__device__ __forceinline__ i32x4 load16(const int8_t *p, int64_t n) {
    i32x4 v = {0, 0, 0, 0};
    if (n >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else {
        for (int b = 0; b < n; ++b) v[b >> 2] |= (int)((uint32_t)(uint8_t)p[b] << (8 * (b & 3)));
    }
    return v;
}

template <int OUT, bool SWIGLU, int T>
__global__ __launch_bounds__(256, 2)
void quant_generic_kernel(GemmArgs g, int tiles_m, int tiles_n, int tiles, int vec, GemmExtra ex, QuantArgs qa) {
    constexpr int ON = SWIGLU ? T / 2 : T;     // output columns per tile
    constexpr int QK = 128;                    // K bytes per stage
    constexpr int QROW = QK + 16;              // LDS bytes per row
    constexpr int CPR = QK / 16;               // 16-byte chunks of a row's stage
    constexpr int NC = T * CPR / 256;          // chunks a thread loads of either operand
    constexpr int NJ = T == 128 ? 4 : 1;       // a wave's 16-row blocks of X; it has 4 of W
    __shared__ __attribute__((aligned(16))) char smem[2][2][T * QROW];

    // Tiles in contiguous ranges on the XCDs, a shard's tile rows in groups.
    const int per = (tiles + 7) / 8, logical = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (logical >= tiles || (int)(blockIdx.x >> 3) >= per) return;
    const int per_shard = tiles_m * tiles_n, shard = logical / per_shard, t = logical - shard * per_shard;
    const int first_m = t / (QGROUP * tiles_n) * QGROUP, gsz = min(tiles_m - first_m, QGROUP);
    const int tr = t - first_m * tiles_n;
    const int64_t m0 = (int64_t)(first_m + tr % gsz) * T, n0 = (int64_t)(tr / gsz) * ON;
    const int8_t *A = (const int8_t *)g.A + (int64_t)shard * g.a_shard;
    const int8_t *B = (const int8_t *)g.B + (int64_t)shard * g.b_shard;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = T == 128 ? wave >> 1 : wave, wn = T == 128 ? wave & 1 : 0;

    // Chunk c of this thread: tile row (tid + 256 c) / CPR, 16-byte column tid % CPR
    // of the stage.  W rows are placed for the epilogue
    // (quant_w_row); for the gated unit, of each 64 the last 32 are the up rows.
    const int8_t *xrow[NC], *wrow[NC];
    bool xin[NC], win[NC];
    const int kc = tid % CPR * 16;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int r = (tid + 256 * c) / CPR;
        xin[c] = m0 + r < g.M;
        xrow[c] = A + (xin[c] ? m0 + r : 0) * g.lda + kc;
        int64_t n = n0 + (SWIGLU ? (r >> 6) * 32 + quant_w_row(r & 31) : quant_w_row(r));
        win[c] = n < g.N;
        if (!win[c]) n = 0;
        if (SWIGLU && (r & 32)) n += ex.up_off;
        wrow[c] = B + n * g.ldb + kc;
    }
    i32x4 xv[NC], wv[NC];
    auto load = [&](int64_t k0) {
        const int64_t left = g.K - k0 - kc;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            xv[c] = wv[c] = i32x4{0, 0, 0, 0};
            if (xin[c] && left > 0) xv[c] = load16(xrow[c] + k0, left);
            if (win[c] && left > 0) wv[c] = load16(wrow[c] + k0, left);
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int at = (tid + 256 * c) / CPR * QROW + kc;
            *(i32x4 *)(smem[buf][0] + at) = xv[c];
            *(i32x4 *)(smem[buf][1] + at) = wv[c];
        }
    };

    i32x4 acc[4][NJ] = {};
    load(0);
    put(0);
    __syncthreads();
    int buf = 0;
    for (int64_t k0 = 0; k0 < g.K; k0 += QK) {
        const bool more = k0 + QK < g.K;
        if (more) load(k0 + QK);
#pragma unroll
        for (int h = 0; h < QK / 64; ++h) {
            const int kb = h * 64 + (lane >> 4) * 16;
            i32x4 a[4], b[NJ];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = *(const i32x4 *)(smem[buf][1] + (wn * 64 + i * 16 + (lane & 15)) * QROW + kb);
#pragma unroll
            for (int j = 0; j < NJ; ++j) b[j] = *(const i32x4 *)(smem[buf][0] + ((wm * NJ + j) * 16 + (lane & 15)) * QROW + kb);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
        }
        buf ^= 1;
        if (more) put(buf);
        __syncthreads();
    }
    const int64_t mw = m0 + wm * NJ * 16, nw = n0 + wn * (SWIGLU ? 32 : 64);
    if constexpr (SWIGLU)
        quant_store_gated<OUT, 4, NJ>(g, ex.bias, ex.bias_shard, ex.up_off, qa, vec, shard, mw, nw, lane, acc);
    else
        quant_store<OUT, 4, NJ>(g, ex.bias, ex.bias_shard, qa, vec, shard, mw, nw, lane, acc);
}

// One launch has fewer than 2^32 threads: more tiles go by shards, then by halves
// of the rows or columns.
template <int OUT, bool SW, int T>
hipError_t launch_pieces(const GemmArgs &g, const GemmExtra &ex, const QuantArgs &q, hipStream_t s) {
    constexpr int ON = SW ? T / 2 : T, OS = OUT == OUT_BF16 ? 2 : 4;
    constexpr int64_t MOST = (1 << 24) - 8;
    const int64_t tm = (g.M + T - 1) / T, tn = (g.N + ON - 1) / ON;
    if (tm > MOST || tn > MOST || tm * tn > MOST / g.P) {
        // rows x cols outputs from row m, column n of shard i on
        auto part = [&](int32_t i, int64_t m, int64_t n, int64_t rows, int64_t cols) {
            GemmArgs h = g;
            GemmExtra e = ex;
            QuantArgs r = q;
            h.A = (const char *)g.A + i * g.a_shard + m * g.lda;
            h.B = (const char *)g.B + i * g.b_shard + n * g.ldb;
            h.C = (char *)g.C + (i * g.c_shard + m * g.ldc + n) * OS;
            h.M = rows; h.N = cols; h.P = 1;
            if (ex.bias) e.bias = (const char *)ex.bias + (i * ex.bias_shard + n) * OS;
            if (OUT != OUT_I32) {
                r.x_scale = q.x_scale + i * q.x_shard + m * q.x_ld;
                r.w_scale = q.w_scale + i * q.w_shard + n;
            }
            return launch_pieces<OUT, SW, T>(h, e, r, s);
        };
        hipError_t e = hipSuccess;
        if (g.P > 1) {
            for (int32_t i = 0; i < g.P && e == hipSuccess; ++i) e = part(i, 0, 0, g.M, g.N);
        } else if (tm > 1) {
            const int64_t m = tm / 2 * T;
            e = part(0, 0, 0, m, g.N);
            if (e == hipSuccess) e = part(0, m, 0, g.M - m, g.N);
        } else {
            const int64_t n = tn / 2 * ON;
            e = part(0, 0, 0, g.M, n);
            if (e == hipSuccess) e = part(0, 0, n, g.M, g.N - n);
        }
        return e;
    }
    const int tiles = (int)(tm * tn * g.P);
    const int vw = OUT == OUT_BF16 ? 8 : 4;
    const int vec = g.ldc % vw == 0 && g.c_shard % vw == 0 && (uintptr_t)g.C % 16 == 0;
    quant_generic_kernel<OUT, SW, T><<<dim3((tiles + 7) / 8 * 8), dim3(256), 0, s>>>(g, (int)tm, (int)tn, tiles, vec, ex, q);
    return hipGetLastError();
}

template <int OUT, bool SW>
hipError_t launch_t(const GemmArgs &g, const GemmExtra &ex, const QuantArgs &q, hipStream_t s) {
    const int on = SW ? 2 : 1;
    auto count = [&](int T) { return ((g.M + T - 1) / T) * ((g.N + T / on - 1) / (T / on)); };
    // The larger tile where it fills the CUs.  Same box, 8 shards, us, 128 vs 64: 4097
    // -> 28672 at 4096 tokens 779 vs 1357, 517 -> 4096 at 1000 (256 tiles of 128) 15.0 vs
    // 15.0, 3000 -> 8192 at 300 (192) 36.6 vs 30.1, 1001 -> 10240 at 128 (80) 21.6 vs 14.5.
    const int T = count(128) * g.P >= device_cu_count() ? 128 : 64;
    return T == 128 ? launch_pieces<OUT, SW, 128>(g, ex, q, s) : launch_pieces<OUT, SW, 64>(g, ex, q, s);
}

}  // namespace

hipError_t launch_quant_generic(const GemmArgs &g, int out_type, const GemmExtra &ex,
                                const QuantArgs &q, hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    const bool sw = ex.act == ACT_SWIGLU;
    if (ex.x_rows > 0 || (out_type == OUT_I32 && (sw || ex.bias))) return hipErrorInvalidValue;
    if (out_type == OUT_I32) return launch_t<OUT_I32, false>(g, ex, q, s);
    if (out_type == OUT_BF16) return sw ? launch_t<OUT_BF16, true>(g, ex, q, s) : launch_t<OUT_BF16, false>(g, ex, q, s);
    return sw ? launch_t<OUT_F32, true>(g, ex, q, s) : launch_t<OUT_F32, false>(g, ex, q, s);
}

}  // namespace tpl
