// Skinny shard GEMM for decode-shaped inputs (M <= 48 tokens): C_i = A_i B_i^T
// where the weight dominates the bytes, so the kernel is bound by how fast
// it streams W from HBM ("模型并行", "Tensor Parallel": Y_i = X W_i for the
// column form, the partials X_i W_i for the row form).
//
// Work unit: one workgroup owns BN = 16*NB rows of W (NB blocks of 16 output
// columns) and one shard -- or, in the fused row form, all P shards in
// ascending order; the NB blocks share the staged X rows.
// W and X move global -> LDS with global_load_lds_dwordx4 in NST stages of
// KB columns of K; each 1 KB load instruction covers one contiguous KB*2-byte
// run of one row, so HBM sees long sequential runs rather than 64-byte
// pieces of many rows.  In LDS, 16-byte chunk c of row r sits at slot
// c ^ (r % 16), so the 16 rows of an MFMA fragment read hit 16 different
// bank groups.  The shard's K is cut into 32-column blocks; wave w takes the
// blocks whose index is w mod 4, in ascending order, and multiplies on
// v_mfma_f32_16x16x32_bf16 (W rows as the row operand).  The four wave sums
// are added through LDS in the fixed order ((w0 + w1) + w2) + w3 when a
// shard ends.  Since a stage holds a multiple of four blocks, which blocks
// each wave adds, and in which order, does not depend on the stage size:
// every instantiation gives the same fp32 result for the same shard.
//
// Fused fold (row form, decode): the shard partials are added into a
// running fp32 sum in ascending shard order, one add at a time, and the sum
// is rounded once -- the same operations, in the same order, as writing the
// partials and running the fold kernel, so the result is bitwise equal to
// that unfused sequence.  No workspace, counter or cross-workgroup signal is
// needed.
//
// Epilogue options: the column bias (Shard(0)) is added to each output in
// fp32 before rounding; the row bias (Partial(), the whole layer's bias) is
// added once to the fused sum after the last shard.  The gated unit of a
// fused gate+up column layer (SWIGLU) takes 16 gate rows and the 16 up rows
// of the same hidden units per workgroup (NB = 2), so both products of an
// output land in the same thread's reduction: silu(g + bg) * (u + bu).
#pragma once

#include <type_traits>

#include "kernels.h"
#include "mfma_ops.h"
#include "quant.h"
#include "quant_math.h"

namespace tpl {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

#define LDS_PTR(T) __attribute__((address_space(3))) T *

constexpr int SK_THREADS = 256;

template <int OUT>
__device__ __forceinline__ void store_out(void *Y, int64_t o, float v) {
    if (OUT == OUT_BF16) ((__bf16 *)Y)[o] = (__bf16)v;
    else ((float *)Y)[o] = v;
}

// A bias value of the output type (0 without a bias).
template <int OUT>
__device__ __forceinline__ float skinny_bias(const void *b, int64_t i) {
    if (!b) return 0.0f;
    return OUT == OUT_BF16 ? (float)((const __bf16 *)b)[i] : ((const float *)b)[i];
}

// NB: 16-row blocks of W.  MB: 16-row blocks of M.  KB: K columns per stage (int8:
// twice as many; the stage's bytes are the same).  NST: stages.  OP: the
// operands' type (mfma_ops.h).
template <int NB, int MB, int KB, int NST, int OUT, bool FOLD, bool SWIGLU, class OP = OpBf16>
__global__ __launch_bounds__(SK_THREADS)
void gemm_skinny_kernel(GemmArgs g, FoldArgs f, GemmExtra ex, QuantArgs qa) {
    typedef typename OP::Frag Frag;
    typedef typename OP::Acc Acc;
    typedef typename std::conditional<OP::INT8, int32_t, float>::type Sum;
    constexpr int ES = OP::ES;
    constexpr int EC = 16 / ES;            // elements per chunk
    static_assert(!SWIGLU || (NB == 2 && !FOLD), "gated unit: 16 gate + 16 up rows, column form");
    constexpr int BN = 16 * NB;            // W rows per workgroup
    constexpr int ON = SWIGLU ? 16 : BN;   // output columns per workgroup
    constexpr int XR = 16 * MB;            // X rows staged
    constexpr int ROWB = KB * 2;           // bytes per staged row
    constexpr int CPR = ROWB / 16;         // 16-byte chunks per row
    static_assert(CPR >= 16, "rows of at least 256 bytes");
    constexpr int STB = (BN + XR) * ROWB;  // bytes per stage (rows back to back)
    constexpr int NI = STB / 1024;         // 1 KB load instructions per stage
    static_assert(STB % 4096 == 0, "loads split over 4 waves");
    constexpr int LPW = NI / 4;            // per wave
    constexpr int SUBS = KB / 32 / 4;      // k32 sub-steps per wave per stage
    static_assert(SUBS >= 1, "KB >= 128");
    __shared__ __attribute__((aligned(1024))) char smem[NST * STB];
    __shared__ Acc red[4][NB][MB][64];
    LDS_PTR(char) lds = (LDS_PTR(char))smem;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    int tn, s_begin, s_count;
    if (FOLD) {
        tn = blockIdx.x; s_begin = 0; s_count = g.P;
    } else {
        tn = blockIdx.x / g.P; s_begin = blockIdx.x - tn * g.P; s_count = 1;
    }
    const int64_t n0 = (int64_t)tn * ON;
    const int64_t Ks = g.K;
    constexpr int KE = KB * 2 / ES;        // K elements per stage
    const int nks = (int)((Ks + KE - 1) / KE);  // stages per shard
    const int total = s_count * nks;

    // ---- load cursor: stage t -> (shard, k stage).  Load instruction q
    // (= j*4 + wave) fills bytes [q KB, (q+1) KB) of the stage; lane takes
    // 16-byte unit idx = 64q + lane: row idx / CPR (W rows first, then X
    // rows), slot idx % CPR, which holds chunk slot ^ (row % 16).
    int ls = 0, lk = 0;
    // int8, fused fold: the workgroups walk K in step, and rows a multiple of 4 KB
    // apart put their reads of one moment on few memory channels.  The sum does not
    // depend on the order of K, so each workgroup then begins a shard at a stage of
    // its own and wraps: 16 tokens, weights from HBM, 28672 -> 8192 49.5 -> 47.3 us, 32768
    // -> 8192 58.2 -> 56.9, 8192 -> 8192 20.6 -> 20.1.  Without such a stride it costs a
    // little (14336 -> 4096 after a flush 24.4 -> 24.8), and the column form, whose
    // workgroups are not in step, gains nothing.
    const int rot = OP::INT8 && FOLD && g.ldb % 4096 == 0 ? (int)(blockIdx.x % (unsigned)nks) : 0;
    auto turned = [&](int k) { return OP::INT8 && FOLD ? (k + rot < nks ? k + rot : k + rot - nks) : k; };
    auto issue = [&](int t) {
        if (t >= total) return;  // uniform
        const int shard = s_begin + ls;
        const int64_t kb = (int64_t)turned(lk) * KE;
        LDS_PTR(char) dst = lds + (t % NST) * STB;
#pragma unroll
        for (int j = 0; j < LPW; ++j) {
            const int q = j * 4 + wave;
            const int idx = q * 64 + lane;
            const int row = idx / CPR, slot = idx % CPR;
            const int chunk = slot ^ (row & 15);
            int64_t k = kb + chunk * EC;
            // K tail: chunks past the shard's K are loaded from column 0 of
            // the row (in bounds) and zeroed after the fragment read.
            if (k >= Ks) k = 0;
            const char *src;
            if (row < BN) {
                int64_t n = n0 + (SWIGLU ? (row & 15) : row);
                if (n > g.N - 1) n = g.N - 1;
                if (SWIGLU && row >= 16) n += ex.up_off;   // the up row of the same unit
                src = (const char *)g.B + ((int64_t)shard * g.b_shard + n * g.ldb + k) * ES;
            } else {
                int64_t m = row - BN;
                if (m > g.M - 1) m = g.M - 1;
                src = (const char *)g.A + ((int64_t)shard * g.a_shard + m * g.lda + k) * ES;
            }
            // Written as an instruction the compiler does not track: its own
            // wait analysis would drain every load in flight before the next
            // LDS read (it cannot tell which stage a load writes), which
            // leaves no stage of lead; the waits the pipeline needs are the
            // explicit ones at the top of each stage.
            const uint32_t m0v = (uint32_t)(uintptr_t)(dst + q * 1024);
            asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                         :: "v"(src), "s"(m0v) : "memory", "m0");
        }
        if (++lk == nks) { lk = 0; ++ls; }
    };

#pragma unroll
    for (int t = 0; t < NST - 1; ++t) issue(t);

    Acc acc[NB][MB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = Acc{};
    float run[NB][MB];  // running fused sum, output mapping (see below)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) run[nb][mb] = 0.f;

    const int frow = lane & 15;   // fragment row
    const int fk = lane >> 4;     // fragment 8-column group
    int cs = 0, ck = 0;           // compute cursor (shard index, k stage)
    for (int t = 0; t < total; ++t) {
        // Stage t's loads were issued NST-1 stages ago; the loads of the
        // later stages issued since (NST-2 of them, fewer in the last stages,
        // where nothing is issued past the end) may stay in flight.
        const int later = total - 1 - t;
        if (later >= NST - 2) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LPW * (NST - 2)) : "memory");
        } else {
#pragma unroll
            for (int r = 0; r < NST - 2; ++r)
                if (later == r) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LPW * r) : "memory");
        }
        __syncthreads();
        issue(t + NST - 1);
        LDS_PTR(char) st = lds + (t % NST) * STB;
        const int64_t kb = (int64_t)turned(ck) * KE;
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub) {
            const int c = (sub * 4 + wave) * 4 + fk;  // chunk within the stage
            const bool valid = kb + c * EC < Ks;
            Frag wv[NB], xv[MB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                wv[nb] = *(LDS_PTR(Frag))(st + (nb * 16 + frow) * ROWB + ((c ^ frow) << 4));
                if (!valid) wv[nb] = Frag{};
            }
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                const int xr = BN + mb * 16 + frow;
                xv[mb] = *(LDS_PTR(Frag))(st + xr * ROWB + ((c ^ (xr & 15)) << 4));
                if (!valid) xv[mb] = Frag{};
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                acc[nb][mb] = OP::mfma(wv[nb], xv[mb], acc[nb][mb]);
        }
        if (++ck < nks) continue;

        // ---- shard finished: add the four waves' partials in fixed order.
        // Output (n, m) of the tile sits in lane 16*(n/4) + m%16, register
        // n%4, block m/16 (16x16 D layout, W rows as the row operand).
        // Thread tid takes n = tid % 16, m = tid / 16 + 16*mb.
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            red[wave][nb][mb][lane] = acc[nb][mb];
            acc[nb][mb] = Acc{};
        }
        __syncthreads();
        const int on = tid & 15, om = tid >> 4;
        const int src_lane = 16 * (on >> 2) + om, src_r = on & 3;
        const int shard = s_begin + cs;
        const __bf16 *bb = (const __bf16 *)ex.bias;
        if (SWIGLU) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                Sum gv = red[0][0][mb][src_lane][src_r];
                gv = gv + red[1][0][mb][src_lane][src_r];
                gv = gv + red[2][0][mb][src_lane][src_r];
                gv = gv + red[3][0][mb][src_lane][src_r];
                Sum uv = red[0][1][mb][src_lane][src_r];
                uv = uv + red[1][1][mb][src_lane][src_r];
                uv = uv + red[2][1][mb][src_lane][src_r];
                uv = uv + red[3][1][mb][src_lane][src_r];
                const int64_t m = om + 16 * mb, n = n0 + on;
                if (m < g.M && n < g.N) {
                    float gf, uf;
                    if constexpr (OP::INT8) {
                        const float sx = qa.x_scale[m * qa.x_ld + (int64_t)shard * qa.x_shard];
                        const float *sw = qa.w_scale + (int64_t)shard * qa.w_shard;
                        const int64_t b0 = (int64_t)shard * ex.bias_shard;
                        gf = quant_value(gv, sx, sw[n], skinny_bias<OUT>(ex.bias, b0 + n));
                        uf = quant_value(uv, sx, sw[ex.up_off + n], skinny_bias<OUT>(ex.bias, b0 + ex.up_off + n));
                    } else {
                        if (bb) {
                            const __bf16 *bs = bb + (int64_t)shard * ex.bias_shard;
                            gv = gv + (float)bs[n];
                            uv = uv + (float)bs[ex.up_off + n];
                        }
                        gf = gv;
                        uf = uv;
                    }
                    store_out<OUT>(g.C, (int64_t)shard * g.c_shard + m * g.ldc + n,
                                   (OP::INT8 ? quant_silu(gf) : silu_f32(gf)) * uf);
                }
            }
        } else {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                Sum v = red[0][nb][mb][src_lane][src_r];
                v = v + red[1][nb][mb][src_lane][src_r];
                v = v + red[2][nb][mb][src_lane][src_r];
                v = v + red[3][nb][mb][src_lane][src_r];
                const int64_t m = om + 16 * mb, n = n0 + nb * 16 + on;
                if constexpr (OP::INT8) {
                    if (m >= g.M || n >= g.N) continue;
                    if (OUT == OUT_I32) {
                        ((int32_t *)g.C)[(int64_t)shard * g.c_shard + m * g.ldc + n] = v;
                        continue;
                    }
                    const float sx = qa.x_scale[m * qa.x_ld + (int64_t)shard * qa.x_shard];
                    if (FOLD) {
                        run[nb][mb] = cs == 0 ? (float)v * sx : __builtin_fmaf((float)v, sx, run[nb][mb]);
                        if (cs == s_count - 1)
                            store_out<OUT>(f.Y, m * f.ldy + n,
                                           __builtin_fmaf(run[nb][mb], qa.w_scale[n], skinny_bias<OUT>(ex.bias, n)));
                    } else {
                        store_out<OUT>(g.C, (int64_t)shard * g.c_shard + m * g.ldc + n,
                                       quant_value(v, sx, qa.w_scale[(int64_t)shard * qa.w_shard + n],
                                                   skinny_bias<OUT>(ex.bias, (int64_t)shard * ex.bias_shard + n)));
                    }
                } else if (FOLD) {
                    run[nb][mb] = cs == 0 ? v : run[nb][mb] + v;
                    if (cs == s_count - 1 && m < g.M && n < g.N) {
                        float y = run[nb][mb];
                        if (bb) y = y + (float)bb[n];     // row bias: once, after the fold
                        store_out<OUT>(f.Y, m * f.ldy + n, y);
                    }
                } else if (m < g.M && n < g.N) {
                    if (bb) v = v + (float)bb[(int64_t)shard * ex.bias_shard + n];
                    store_out<OUT>(g.C, (int64_t)shard * g.c_shard + m * g.ldc + n, v);
                }
            }
        }
        ck = 0;
        ++cs;
        // `red` is written again only after at least one more barrier.
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

}  // namespace
}  // namespace tpl
