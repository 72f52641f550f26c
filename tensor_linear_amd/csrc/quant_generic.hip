// Int8 shard GEMM for any M, N, K, leading dimension and alignment ("模型并行",
// "Tensor Parallel": the per-shard products Y_i = X W_i and X_i W_i, the
// operands held in 8 bits): acc[m, n] = sum_k x[m, k] w[n, k] exactly in int32
// on v_mfma_i32_16x16x64_i8, scaled in the epilogue.
//
// Tile 64 (M) x 64 (N), four waves in a 2 x 2 grid of 32 x 32 outputs, 128
// bytes of K a stage: each thread loads two 16-byte chunks of either operand
// into registers while the stage before is multiplied, and writes them to LDS
// rows of 144 bytes (the 16 padding bytes turn the 16 rows of a fragment read
// into different banks).  Chunks past K and rows past M or N are zeros, which
// add nothing to an integer sum.  It serves what the DMA kernels cannot load
// (K or strides not a multiple of 16, unaligned views); bound by its loads'
// latency (one stage ahead).
#include "quant.h"
#include "quant_math.h"

namespace tpl {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int QB = 64;     // tile edge in M and N
constexpr int QK = 128;    // K bytes per stage
constexpr int QROW = QK + 16;

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

template <int OUT>
__device__ __forceinline__ float bias_value(const void *b, int64_t i) {
    if (OUT == OUT_BF16) return (float)((const __bf16 *)b)[i];
    return ((const float *)b)[i];
}

template <int OUT, bool SWIGLU>
__global__ __launch_bounds__(256)
void quant_generic_kernel(GemmArgs g, int tiles_m, int tiles_n, GemmExtra ex, QuantArgs qa) {
    constexpr int ON = SWIGLU ? QB / 2 : QB;   // output columns per tile
    __shared__ __attribute__((aligned(16))) char Xs[QB * QROW];
    __shared__ __attribute__((aligned(16))) char Ws[QB * QROW];

    const int per_shard = tiles_m * tiles_n;
    const int shard = blockIdx.x / per_shard;
    const int t = blockIdx.x - shard * per_shard;
    const int64_t m0 = (int64_t)(t / tiles_n) * QB;
    const int64_t n0 = (int64_t)(t % tiles_n) * ON;
    const int8_t *A = (const int8_t *)g.A + (int64_t)shard * g.a_shard;
    const int8_t *B = (const int8_t *)g.B + (int64_t)shard * g.b_shard;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;

    // Chunk c (0, 1) of this thread: tile row (tid + 256 c) / 8, 16-byte
    // column (tid + 256 c) % 8 of the stage.  For the gated unit W tile rows
    // 16-31 of each 32 are the up rows of the units in rows 0-15.
    const int8_t *xrow[2], *wrow[2];
    int kc[2], at[2];
    bool xin[2], win[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int r = (tid + 256 * c) >> 3;
        kc[c] = ((tid + 256 * c) & 7) * 16;
        at[c] = r * QROW + kc[c];
        xin[c] = m0 + r < g.M;
        xrow[c] = A + (xin[c] ? m0 + r : 0) * g.lda;
        int64_t n = SWIGLU ? n0 + (r >> 5) * 16 + (r & 15) : n0 + r;
        win[c] = n < g.N;
        if (!win[c]) n = 0;
        if (SWIGLU && ((r >> 4) & 1)) n += ex.up_off;
        wrow[c] = B + n * g.ldb;
    }
    i32x4 xv[2], wv[2];
    auto load = [&](int64_t k0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int64_t k = k0 + kc[c], left = g.K - k;
            xv[c] = wv[c] = i32x4{0, 0, 0, 0};
            if (xin[c] && left > 0) xv[c] = load16(xrow[c] + k, left);
            if (win[c] && left > 0) wv[c] = load16(wrow[c] + k, left);
        }
    };

    i32x4 acc[2][2] = {};
    load(0);
    for (int64_t k0 = 0; k0 < g.K; k0 += QK) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            *(i32x4 *)(Xs + at[c]) = xv[c];
            *(i32x4 *)(Ws + at[c]) = wv[c];
        }
        __syncthreads();
        if (k0 + QK < g.K) load(k0 + QK);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kb = h * 64 + (lane >> 4) * 16;
            i32x4 a[2], b[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                a[u] = *(const i32x4 *)(Ws + (wn * 32 + u * 16 + (lane & 15)) * QROW + kb);
                b[u] = *(const i32x4 *)(Xs + (wm * 32 + u * 16 + (lane & 15)) * QROW + kb);
            }
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int mb = 0; mb < 2; ++mb)
                    acc[nb][mb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[nb], b[mb], acc[nb][mb], 0, 0, 0);
        }
        __syncthreads();
    }

    // acc[nb][mb][r]: row m = lane % 16, column n = 4 (lane / 16) + r of the block.
    const int64_t cbase = (int64_t)shard * g.c_shard, bsh = (int64_t)shard * ex.bias_shard;
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
        const int64_t m = m0 + wm * 32 + mb * 16 + (lane & 15);
        if (m >= g.M) continue;
        const float sx = OUT == OUT_I32 ? 1.0f : qa.x_scale[m * qa.x_ld + (int64_t)shard * qa.x_shard];
        const float *sw = qa.w_scale + (int64_t)shard * qa.w_shard;
#pragma unroll
        for (int nb = 0; nb < (SWIGLU ? 1 : 2); ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t n = n0 + (SWIGLU ? wn * 16 : wn * 32 + nb * 16) + 4 * (lane >> 4) + r;
                if (n >= g.N) continue;
                const int64_t o = cbase + m * g.ldc + n;
                if constexpr (OUT == OUT_I32) {
                    ((int32_t *)g.C)[o] = acc[nb][mb][r];
                } else {
                    float v = quant_value(acc[nb][mb][r], sx, sw[n],
                                          ex.bias ? bias_value<OUT>(ex.bias, bsh + n) : 0.0f);
                    if (SWIGLU)
                        v = quant_silu(v) * quant_value(acc[1][mb][r], sx, sw[ex.up_off + n],
                                                      ex.bias ? bias_value<OUT>(ex.bias, bsh + ex.up_off + n) : 0.0f);
                    if (OUT == OUT_BF16) ((__bf16 *)g.C)[o] = (__bf16)v;
                    else ((float *)g.C)[o] = v;
                }
            }
    }
}

}  // namespace

hipError_t launch_quant_generic(const GemmArgs &g, int out_type, const GemmExtra &ex,
                                const QuantArgs &q, hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    const bool sw = ex.act == ACT_SWIGLU;
    if (ex.x_rows > 0 || (out_type == OUT_I32 && (sw || ex.bias))) return hipErrorInvalidValue;
    const int on = sw ? QB / 2 : QB;
    const int64_t tm = (g.M + QB - 1) / QB, tn = (g.N + on - 1) / on;
    if (tm > 0x7FFFFFFFll || tn > 0x7FFFFFFFll || tm * tn > 0x7FFFFFFFll ||
        tm * tn * g.P > 0xFFFFFFFFll / 256)   // 2^32 threads a launch
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(tm * tn * g.P)), block(256);
    const int a = (int)tm, b = (int)tn;
    if (out_type == OUT_I32) quant_generic_kernel<OUT_I32, false><<<grid, block, 0, s>>>(g, a, b, ex, q);
    else if (out_type == OUT_BF16 && sw) quant_generic_kernel<OUT_BF16, true><<<grid, block, 0, s>>>(g, a, b, ex, q);
    else if (out_type == OUT_BF16) quant_generic_kernel<OUT_BF16, false><<<grid, block, 0, s>>>(g, a, b, ex, q);
    else if (sw) quant_generic_kernel<OUT_F32, true><<<grid, block, 0, s>>>(g, a, b, ex, q);
    else quant_generic_kernel<OUT_F32, false><<<grid, block, 0, s>>>(g, a, b, ex, q);
    return hipGetLastError();
}

}  // namespace tpl
