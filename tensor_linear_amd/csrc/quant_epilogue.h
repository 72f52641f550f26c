// Epilogues of the int8 shard GEMM kernels: a wave's int32 sums, scaled
// (quant_value) and stored from its registers.
#pragma once

#include <type_traits>

#include "kernels.h"
#include "quant.h"
#include "quant_math.h"

namespace tpl {

typedef int q_i32x4 __attribute__((ext_vector_type(4)));
typedef int q_i32x4_any __attribute__((ext_vector_type(4), aligned(1)));   // in memory, at any address

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

// Eight bias values of the output type from n on, as they are held (zeros
// without a bias), and one of them in fp32.
template <int OUT>
struct QuantBias { uint32_t w[OUT == OUT_BF16 ? 4 : 8]; };
template <int OUT>
__device__ __forceinline__ QuantBias<OUT> quant_load_bias(const void *b, int64_t base, int64_t n, int64_t end) {
    QuantBias<OUT> r = {};
    constexpr int ES = OUT == OUT_BF16 ? 2 : 4;
    if (!b) return r;
    const char *p = (const char *)b + base * ES;
    if (n + 8 <= end) {
        __builtin_memcpy(r.w, p + n * ES, 8 * ES);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t i = n + e < end ? n + e : 0;
            if (ES == 2) r.w[e / 2] |= (uint32_t)((const uint16_t *)p)[i] << (16 * (e & 1));
            else r.w[e] = ((const uint32_t *)p)[i];
        }
    }
    return r;
}
template <int OUT>
__device__ __forceinline__ float quant_bias(const QuantBias<OUT> &b, int e) {
    return __uint_as_float(OUT != OUT_BF16 ? b.w[e] : (e & 1) ? b.w[e / 2] & 0xFFFF0000u : b.w[e / 2] << 16);
}

// 16 bytes of outputs: 8 (bf16) or 4 (fp32, int32) columns of a row from n on.
template <int OUT>
__device__ __forceinline__ void quant_put16(void *C, int64_t row, int64_t n, int64_t N, bool vec, q_i32x4 v) {
    typedef typename std::conditional<OUT == OUT_BF16, uint16_t, uint32_t>::type T;
    constexpr int E = OUT == OUT_BF16 ? 8 : 4;
    T *dst = (T *)C + row + n;
    if (n + E <= N) {
        // rows that straddle lines go through the cache, which puts the lines together
        if (vec) __builtin_nontemporal_store(v, (q_i32x4 *)dst);
        else *(q_i32x4_any *)dst = v;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (n + e < N) dst[e] = (T)((uint32_t)v[e * 4 / E] >> (E == 8 ? 16 * (e & 1) : 0));
    }
}

// Lanes 0-7 of each 16 give b and take the others' a; lanes 8-15 give a and take
// the others' b: with a and b two 16-byte pieces of a lane's output row, v1 is
// a piece of rows 0-7 and v2 of rows 8-15, the same piece for eight lanes each.
__device__ __forceinline__ void quant_swap8(bool hi, q_i32x4 a, q_i32x4 b, q_i32x4 &v1, q_i32x4 &v2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int y = __builtin_amdgcn_mov_dpp(hi ? a[e] : b[e], 0x128 /* row_ror:8 */, 0xf, 0xf, false);
        v1[e] = hi ? y : a[e];
        v2[e] = hi ? b[e] : y;
    }
}

// Stores NP pairs of blocks of one 16-row block: val(p, e) is the lane's output in
// column n0 + 8 (lane / 16) + 32 p + e of row m0 + lane % 16, as fp32 or int32 bits.  The lanes exchange 16-byte pieces first,
// so that a store instruction writes eight rows of 128 bytes (two pairs of bf16,
// one of fp32) and not sixteen of 64.  (n0: the wave's first column.)
// FAST: every output is inside M x N and 16-byte aligned; the stores are a uniform
// row address and a 32-bit offset of the lane.
template <bool FAST, int OUT, int NP, class Val>
__device__ __forceinline__ void quant_put_rows(void *C, int64_t ld, int64_t m0, int64_t M, int64_t n0, int64_t N,
                                               bool vec, int lane, Val val) {
    constexpr int ES = OUT == OUT_BF16 ? 2 : 4;
    const bool hi = lane & 8;
    const int64_t r1 = m0 + (lane & 7);
    const int64_t n1 = n0 + (lane >> 4) * 8;
    auto pack = [&](int p) {
        q_i32x4 d;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            d[e] = __builtin_bit_cast(int, bf16x2{(__bf16)__builtin_bit_cast(float, val(p, 2 * e)),
                                                  (__bf16)__builtin_bit_cast(float, val(p, 2 * e + 1))});
        }
        return d;
    };
    // this lane's place among the piece's rows 0-7, `far` columns on in the upper half
    char *const base = (char *)C + (m0 * ld + n0) * ES;
    const uint32_t at = (uint32_t)(((int)(lane & 7) * (int)ld + (lane >> 4) * 8 + (hi ? (OUT == OUT_BF16 ? 32 : 4) : 0)) * ES);
    auto put2 = [&](q_i32x4 a, q_i32x4 b, int64_t n, int p) {
        q_i32x4 v1, v2;
        quant_swap8(hi, a, b, v1, v2);
        if constexpr (FAST) {
            __builtin_nontemporal_store(v1, (q_i32x4 *)(base + p * (32 * ES) + at));
            __builtin_nontemporal_store(v2, (q_i32x4 *)(base + 8 * ld * ES + p * (32 * ES) + at));
            return;
        }
        if (r1 < M) quant_put16<OUT>(C, r1 * ld, n, N, vec, v1);
        if (r1 + 8 < M) quant_put16<OUT>(C, (r1 + 8) * ld, n, N, vec, v2);
    };
    if constexpr (OUT == OUT_BF16) {
#pragma unroll
        for (int p = 0; p + 1 < NP; p += 2) put2(pack(p), pack(p + 1), n1 + 32 * p + (hi ? 32 : 0), p);
        if (NP & 1) {
            const int64_t m = m0 + (lane & 15);
            if (m < M) quant_put16<OUT>(C, m * ld, n1 + 32 * (NP - 1), N, vec, pack(NP - 1));
        }
    } else {
#pragma unroll
        for (int p = 0; p < NP; ++p)
            put2(q_i32x4{val(p, 0), val(p, 1), val(p, 2), val(p, 3)}, q_i32x4{val(p, 4), val(p, 5), val(p, 6), val(p, 7)},
                 n1 + 32 * p + (hi ? 4 : 0), p);
    }
}

// The int8 kernels place W rows in LDS so that two neighbouring 16-row blocks of
// MFMA results hold 8 consecutive output columns in a lane: LDS row r of such a
// pair of blocks (32 rows) takes W row quant_w_row(r).  Lane l of blocks 2p, 2p + 1
// then has columns 32 p + 8 (l / 16) .. + 7 of output row l % 16, scaled and stored
// without a pass through LDS (which the bf16 forms take for whole-line stores).
__device__ __forceinline__ int quant_w_row(int r) {
    return (r & ~31) + ((r >> 2) & 3) * 8 + ((r >> 4) & 1) * 4 + (r & 3);
}

// Whether a wave's block that ends before row m and column n takes the FAST form.
__device__ __forceinline__ bool quant_inside(const GemmArgs &g, bool vec, int64_t m, int64_t n) {
    return vec && m <= g.M && n <= g.N && g.ldc < (1 << 24);
}

// A wave's NI x NJ blocks (NI even) at rows m0, columns n0 of shard `shard`; two
// pairs of blocks at a time, so that their scales and bias stay in registers.
template <int OUT, int NI, int NJ, class AccT>
__device__ __forceinline__ void quant_store(const GemmArgs &g, const void *bias, int64_t bias_shard,
                                            const QuantArgs &qa, bool vec, int shard, int64_t m0,
                                            int64_t n0, int lane, const AccT (&acc)[NI][NJ]) {
    constexpr int NP = NI >= 4 ? 2 : 1;
    const int64_t n1 = n0 + (lane >> 4) * 8;
    char *C = (char *)g.C + (int64_t)shard * g.c_shard * (OUT == OUT_BF16 ? 2 : 4);
    const bool inside = quant_inside(g, vec, m0 + NJ * 16, n0 + NI * 16);
    float sx[NJ];
    if constexpr (OUT != OUT_I32) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int64_t m = m0 + j * 16 + (lane & 15);
            sx[j] = qa.x_scale[(int64_t)shard * qa.x_shard + (m < g.M ? m : 0) * qa.x_ld];
        }
    }
#pragma unroll
    for (int i0 = 0; i0 < NI / 2; i0 += NP) {
        float sw[NP][8];
        QuantBias<OUT> bv[NP];
        if constexpr (OUT != OUT_I32) {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                quant_load_f32<8>(qa.w_scale + (int64_t)shard * qa.w_shard, n1 + (i0 + p) * 32, g.N, sw[p]);
                bv[p] = quant_load_bias<OUT>(bias, (int64_t)shard * bias_shard, n1 + (i0 + p) * 32, g.N);
            }
        }
        auto rows = [&](auto fast) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                __builtin_amdgcn_sched_barrier(0);
                quant_put_rows<decltype(fast)::value, OUT, NP>(C, g.ldc, m0 + j * 16, g.M, n0 + i0 * 32, g.N, vec, lane, [&](int p, int e) __attribute__((always_inline)) {
                    const int v = acc[2 * (i0 + p) + (e >> 2)][j][e & 3];
                    if constexpr (OUT == OUT_I32) return v;
                    else return __builtin_bit_cast(int, quant_value(v, sx[j], sw[p][e], quant_bias<OUT>(bv[p], e)));
                });
            }
        };
        if (inside) rows(std::true_type{});
        else rows(std::false_type{});
    }
}

// The gated unit: blocks 0 .. NI/2 - 1 gate sums, the rest the up sums of the same
// hidden units (16 NI / 2 of them from n0 on).
template <int OUT, int NI, int NJ, class AccT>
__device__ __forceinline__ void quant_store_gated(const GemmArgs &g, const void *bias, int64_t bias_shard,
                                                  int64_t up_off, const QuantArgs &qa, bool vec, int shard,
                                                  int64_t m0, int64_t n0, int lane, const AccT (&acc)[NI][NJ]) {
    constexpr int U = NI / 2, NP = U / 2;            // gate blocks, pairs of them
    const int64_t n1 = n0 + (lane >> 4) * 8, b0 = (int64_t)shard * bias_shard;
    const float *ws = qa.w_scale + (int64_t)shard * qa.w_shard;
    char *C = (char *)g.C + (int64_t)shard * g.c_shard * (OUT == OUT_BF16 ? 2 : 4);
    float swg[NP][8], swu[NP][8], sx[NJ];
    QuantBias<OUT> bg[NP], bu[NP];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int64_t m = m0 + j * 16 + (lane & 15);
        sx[j] = qa.x_scale[(int64_t)shard * qa.x_shard + (m < g.M ? m : 0) * qa.x_ld];
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        quant_load_f32<8>(ws, n1 + p * 32, g.N, swg[p]);
        quant_load_f32<8>(ws + up_off, n1 + p * 32, g.N, swu[p]);
        bg[p] = quant_load_bias<OUT>(bias, b0, n1 + p * 32, g.N);
        bu[p] = quant_load_bias<OUT>(bias, b0 + up_off, n1 + p * 32, g.N);
    }
    auto rows = [&](auto fast) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            __builtin_amdgcn_sched_barrier(0);
            quant_put_rows<decltype(fast)::value, OUT, NP>(C, g.ldc, m0 + j * 16, g.M, n0, g.N, vec, lane, [&](int p, int e) __attribute__((always_inline)) {
                const float gg = quant_value(acc[2 * p + (e >> 2)][j][e & 3], sx[j], swg[p][e], quant_bias<OUT>(bg[p], e));
                const float uu = quant_value(acc[U + 2 * p + (e >> 2)][j][e & 3], sx[j], swu[p][e], quant_bias<OUT>(bu[p], e));
                return __builtin_bit_cast(int, quant_silu(gg) * uu);
            });
        }
    };
    if (quant_inside(g, vec, m0 + NJ * 16, n0 + U * 16)) rows(std::true_type{});
    else rows(std::false_type{});
}

}  // namespace tpl
