// Epilogues of the int8 shard GEMM kernels: int32 sums staged in LDS by a wave,
// read back row by row, scaled (quant_value), and stored as whole row pieces.
#pragma once

#include "kernels.h"
#include "quant.h"

namespace tpl {

typedef int q_i32x4 __attribute__((ext_vector_type(4)));
typedef float q_f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 q_bf16x8 __attribute__((ext_vector_type(8)));

// N values of fp32 `p` from n on, those past `end` read as element 0.
template <int N>
__device__ __forceinline__ void quant_load_f32(const float *p, int64_t n, int64_t end, float *v) {
    if (n + N <= end) {
        __builtin_memcpy(v, p + n, N * 4);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = p[n + e < end ? n + e : 0];
    }
}

// N bias values of the output type from n on (0 without a bias).
template <int OUT, int N>
__device__ __forceinline__ void quant_load_bias(const void *b, int64_t base, int64_t n, int64_t end, float *v) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int64_t i = base + (n + e < end ? n + e : 0);
        v[e] = !b ? 0.0f : OUT == OUT_BF16 ? (float)((const __bf16 *)b)[i] : ((const float *)b)[i];
    }
}

// Eight outputs of one row from column n on.
template <int OUT>
__device__ __forceinline__ void quant_put8(void *C, int64_t row, int64_t n, int64_t N, bool vec, const float *v) {
    if (OUT == OUT_BF16) {
        q_bf16x8 h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (__bf16)v[e];
        __bf16 *dst = (__bf16 *)C + row + n;
        if (vec && n + 8 <= N) {
            __builtin_nontemporal_store(h, (q_bf16x8 *)dst);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n + e < N) dst[e] = h[e];
        }
    } else {
        float *dst = (float *)C + row + n;
        if (vec && n + 8 <= N) {
            __builtin_nontemporal_store(q_f32x4{v[0], v[1], v[2], v[3]}, (q_f32x4 *)dst);
            __builtin_nontemporal_store(q_f32x4{v[4], v[5], v[6], v[7]}, (q_f32x4 *)(dst + 4));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n + e < N) dst[e] = v[e];
        }
    }
}

// A wave's block of JN * R rows x IP * LPR8 * 8 columns at (m0, n0) of shard
// `shard`: stage(j, ip) writes the int32 sums of rows R j.. and columns 8 LPR8
// ip.. to LDS, and addr(row, s) is the 16 bytes of its columns 4 s..4 s + 3.
template <int OUT, int JN, int IP, int R, int LPR8, class Stage, class Addr>
__device__ __forceinline__ void quant_store(const GemmArgs &g, const GemmExtra &ex, const QuantArgs &qa,
                                            bool vec, int shard, int64_t m0, int64_t n0, int lane,
                                            Stage stage, Addr addr) {
    const int64_t cbase = (int64_t)shard * g.c_shard;
    if constexpr (OUT == OUT_I32) {
        // lane: 4 columns of a row, so that a 256-byte row leaves as whole lines
        constexpr int LPR = 2 * LPR8, RP = 64 / LPR;
        const int c = lane % LPR, r0 = lane / LPR;
#pragma unroll
        for (int j = 0; j < JN; ++j)
#pragma unroll
            for (int ip = 0; ip < IP; ++ip) {
                __builtin_amdgcn_sched_barrier(0);
                stage(j, ip);
                q_i32x4 a[R / RP];
#pragma unroll
                for (int p = 0; p < R / RP; ++p) a[p] = *addr(p * RP + r0, c);
#pragma unroll
                for (int p = 0; p < R / RP; ++p) {
                    const int64_t m = m0 + j * R + p * RP + r0, n = n0 + ip * LPR8 * 8 + c * 4;
                    if (m >= g.M) continue;
                    int32_t *dst = (int32_t *)g.C + cbase + m * g.ldc + n;
                    if (vec && n + 4 <= g.N) {
                        __builtin_nontemporal_store(a[p], (q_i32x4 *)dst);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < g.N) dst[e] = a[p][e];
                    }
                }
            }
    } else {
        constexpr int RP = 64 / LPR8;                     // rows per pass
        const int c8 = lane % LPR8, r0 = lane / LPR8;
        const float *xs = qa.x_scale + (int64_t)shard * qa.x_shard;
        const float *ws = qa.w_scale + (int64_t)shard * qa.w_shard;
        float sw[IP][8], bv[IP][8], sx[JN][R / RP];
#pragma unroll
        for (int ip = 0; ip < IP; ++ip) {
            quant_load_f32<8>(ws, n0 + ip * LPR8 * 8 + c8 * 8, g.N, sw[ip]);
            quant_load_bias<OUT, 8>(ex.bias, (int64_t)shard * ex.bias_shard, n0 + ip * LPR8 * 8 + c8 * 8, g.N, bv[ip]);
        }
#pragma unroll
        for (int j = 0; j < JN; ++j)
#pragma unroll
            for (int p = 0; p < R / RP; ++p) {
                const int64_t m = m0 + j * R + p * RP + r0;
                sx[j][p] = xs[(m < g.M ? m : 0) * qa.x_ld];
            }
#pragma unroll
        for (int j = 0; j < JN; ++j)
#pragma unroll
            for (int ip = 0; ip < IP; ++ip) {
                __builtin_amdgcn_sched_barrier(0);
                stage(j, ip);
                q_i32x4 a0[R / RP], a1[R / RP];
#pragma unroll
                for (int p = 0; p < R / RP; ++p) {
                    a0[p] = *addr(p * RP + r0, 2 * c8);
                    a1[p] = *addr(p * RP + r0, 2 * c8 + 1);
                }
#pragma unroll
                for (int p = 0; p < R / RP; ++p) {
                    const int64_t m = m0 + j * R + p * RP + r0;
                    if (m >= g.M) continue;
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = quant_value(e < 4 ? a0[p][e & 3] : a1[p][e & 3], sx[j][p], sw[ip][e], bv[ip][e]);
                    quant_put8<OUT>(g.C, cbase + m * g.ldc, n0 + ip * LPR8 * 8 + c8 * 8, g.N, vec, v);
                }
            }
    }
}

// The gated unit: a block of JN * 16 rows x LPR8 * 8 hidden units; stage(j)
// writes 16 rows, gate sums in slots 0 .. 2 LPR8 - 1 and up sums in the next.
template <int OUT, int JN, int LPR8, class Stage, class Addr>
__device__ __forceinline__ void quant_store_gated(const GemmArgs &g, const GemmExtra &ex, const QuantArgs &qa,
                                                  bool vec, int shard, int64_t m0, int64_t n0, int lane,
                                                  Stage stage, Addr addr) {
    constexpr int RP = 64 / LPR8;
    const int c8 = lane % LPR8, r0 = lane / LPR8;
    const int64_t n = n0 + c8 * 8, cbase = (int64_t)shard * g.c_shard, b0 = (int64_t)shard * ex.bias_shard;
    const float *xs = qa.x_scale + (int64_t)shard * qa.x_shard;
    const float *ws = qa.w_scale + (int64_t)shard * qa.w_shard;
    float swg[8], swu[8], bg[8], bu[8], sx[JN][16 / RP];
    quant_load_f32<8>(ws, n, g.N, swg);
    quant_load_f32<8>(ws + ex.up_off, n, g.N, swu);
    quant_load_bias<OUT, 8>(ex.bias, b0, n, g.N, bg);
    quant_load_bias<OUT, 8>(ex.bias, b0 + ex.up_off, n, g.N, bu);
#pragma unroll
    for (int j = 0; j < JN; ++j)
#pragma unroll
        for (int p = 0; p < 16 / RP; ++p) {
            const int64_t m = m0 + j * 16 + p * RP + r0;
            sx[j][p] = xs[(m < g.M ? m : 0) * qa.x_ld];
        }
#pragma unroll
    for (int j = 0; j < JN; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        stage(j);
        q_i32x4 gq[16 / RP][2], uq[16 / RP][2];
#pragma unroll
        for (int p = 0; p < 16 / RP; ++p)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                gq[p][h] = *addr(p * RP + r0, 2 * c8 + h);
                uq[p][h] = *addr(p * RP + r0, 2 * LPR8 + 2 * c8 + h);
            }
#pragma unroll
        for (int p = 0; p < 16 / RP; ++p) {
            const int64_t m = m0 + j * 16 + p * RP + r0;
            if (m >= g.M) continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gg = quant_value(gq[p][e >> 2][e & 3], sx[j][p], swg[e], bg[e]);
                v[e] = silu_f32(gg) * quant_value(uq[p][e >> 2][e & 3], sx[j][p], swu[e], bu[e]);
            }
            quant_put8<OUT>(g.C, cbase + m * g.ldc, n, g.N, vec, v);
        }
    }
}

}  // namespace tpl
