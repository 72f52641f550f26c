// Fold of the P int32 partials of an int8 row layer ("模型并行", "Row parallel":
// Y = sum_i X_i W_i; the all-reduce done on device) into the scaled output.
//
// The partials are exact integers, so nothing is lost before the scales: with
// one scale for each token and shard the fold is the chain
//   S = p_0 x_0;  S = fma(p_i, x_i, S), i ascending;  Y = fma(S, w_n, bias_n),
// the operations the fold inside a GEMM does, in their order; with one scale
// a token the p_i are added as integers first, which no order changes.
//
// HBM-bound as shard_fold: a wavefront folds 1024 columns of one row, 16 bytes
// per lane and load, all loads of eight shards in flight before their adds.
// The row's scales are uniform over the wavefront.  It serves row layers of few
// output tiles for their K (rowfold_faster): 256 tokens of 14336 -> 4096 in 8 shards
// 33.7 us, products and fold together (P M N 4 + M N 2 = 36 MB read and written here).
#include "quant.h"

namespace tpl {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int QF_THREADS = 128;
constexpr int QF_BATCH = 8;                // shards loaded before their adds
constexpr int QF_G = 4;                    // 4-column groups per lane
constexpr int QF_WCOLS = 64 * 4 * QF_G;    // columns per wavefront

template <int ES>
__device__ __forceinline__ char *out_ptr(const ReduceArgs &r, int64_t m, int64_t n) {
    const int64_t j = m / r.slice_rows;
    const int64_t row = m - j * r.slice_rows;
    if (r.use_slices) return (char *)r.y_slice[j] + (row * r.ldy + n) * ES;
    return (char *)r.Y + (j * r.slice_stride + row * r.ldy + n) * ES;
}

template <int OUT>
__device__ __forceinline__ float bias_at(const void *b, int64_t n) {
    if (OUT == OUT_BF16) return (float)((const __bf16 *)b)[n];
    return ((const float *)b)[n];
}

// first: the launch's first wavefront.
template <int OUT, bool PER_SHARD>
__global__ __launch_bounds__(QF_THREADS)
void quant_fold_vec(ReduceArgs r, QuantArgs qa, int64_t first) {
    const int64_t wpr = (r.N + QF_WCOLS - 1) / QF_WCOLS;   // wavefronts per row
    const int64_t wid = first + (int64_t)blockIdx.x * (QF_THREADS / 64) +
                        __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (wid >= r.M * wpr) return;
    const int64_t m = wid / wpr;
    const int64_t nw = (wid - m * wpr) * QF_WCOLS;
    const float *sx = qa.x_scale + m * qa.x_ld;
    bool in[QF_G];
#pragma unroll
    for (int h = 0; h < QF_G; ++h) in[h] = nw + h * 256 + 4 * lane < r.N;
    const int32_t *p = (const int32_t *)r.partials + m * r.ldp + nw + 4 * lane;

    f32x4 a[QF_G] = {};
    i32x4 sum[QF_G] = {};
    for (int i0 = 0; i0 < r.P; i0 += QF_BATCH) {
        i32x4 v[QF_BATCH][QF_G];
        const int cnt = min(QF_BATCH, r.P - i0);
#pragma unroll
        for (int u = 0; u < QF_BATCH; ++u) {
            if (u < cnt) {
                const int32_t *q = p + (int64_t)(i0 + u) * r.shard_stride;
#pragma unroll
                for (int h = 0; h < QF_G; ++h)
                    if (in[h]) v[u][h] = __builtin_nontemporal_load((const i32x4 *)(q + h * 256));
            }
        }
#pragma unroll
        for (int u = 0; u < QF_BATCH; ++u) {
            if (u < cnt) {
                const float x = PER_SHARD ? sx[i0 + u] : 0.0f;
#pragma unroll
                for (int h = 0; h < QF_G; ++h) {
                    if (!PER_SHARD) { sum[h] += v[u][h]; continue; }
#pragma unroll
                    for (int e = 0; e < 4; ++e)   // the first product has no add: -0 stays -0
                        a[h][e] = i0 + u == 0 ? (float)v[u][h][e] * x : __builtin_fmaf((float)v[u][h][e], x, a[h][e]);
                }
            }
        }
    }
    const float x0 = PER_SHARD ? 0.0f : sx[0];
#pragma unroll
    for (int h = 0; h < QF_G; ++h) {
        if (!in[h]) continue;
        const int64_t n = nw + h * 256 + 4 * lane;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float S = PER_SHARD ? a[h][e] : (float)sum[h][e] * x0;
            y[e] = __builtin_fmaf(S, qa.w_scale[n + e], r.bias ? bias_at<OUT>(r.bias, n + e) : 0.0f);
        }
        if (OUT == OUT_BF16) {
            bf16x4 hv;
#pragma unroll
            for (int e = 0; e < 4; ++e) hv[e] = (__bf16)y[e];
            __builtin_nontemporal_store(hv, (bf16x4 *)out_ptr<2>(r, m, n));
        } else {
            __builtin_nontemporal_store(f32x4{y[0], y[1], y[2], y[3]}, (f32x4 *)out_ptr<4>(r, m, n));
        }
    }
}

// Any N, stride and alignment: one thread per output, from `first` on.
template <int OUT, bool PER_SHARD>
__global__ __launch_bounds__(QF_THREADS)
void quant_fold_scalar(ReduceArgs r, QuantArgs qa, int64_t first) {
    const int64_t idx = first + (int64_t)blockIdx.x * QF_THREADS + threadIdx.x;
    if (idx >= r.M * r.N) return;
    const int64_t m = idx / r.N;
    const int64_t n = idx - m * r.N;
    const int32_t *p = (const int32_t *)r.partials + m * r.ldp + n;
    const float *sx = qa.x_scale + m * qa.x_ld;
    float S;
    if (PER_SHARD) {
        S = (float)p[0] * sx[0];
        for (int i = 1; i < r.P; ++i) S = __builtin_fmaf((float)p[(int64_t)i * r.shard_stride], sx[i], S);
    } else {
        int32_t sum = p[0];
        for (int i = 1; i < r.P; ++i) sum += p[(int64_t)i * r.shard_stride];
        S = (float)sum * sx[0];
    }
    const float y = __builtin_fmaf(S, qa.w_scale[n], r.bias ? bias_at<OUT>(r.bias, n) : 0.0f);
    if (OUT == OUT_BF16) *(__bf16 *)out_ptr<2>(r, m, n) = (__bf16)y;
    else *(float *)out_ptr<4>(r, m, n) = y;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

template <int OUT, bool PER_SHARD>
void launch_t(bool vec, dim3 grid, const ReduceArgs &r, const QuantArgs &q, int64_t first, hipStream_t s) {
    if (vec) quant_fold_vec<OUT, PER_SHARD><<<grid, dim3(QF_THREADS), 0, s>>>(r, q, first);
    else quant_fold_scalar<OUT, PER_SHARD><<<grid, dim3(QF_THREADS), 0, s>>>(r, q, first);
}

}  // namespace

hipError_t launch_quant_fold(const ReduceArgs &r, const QuantArgs &q, bool per_shard, int out_type,
                             hipStream_t s) {
    if (r.M == 0 || r.N == 0) return hipSuccess;
    // Vector path: 16-byte partial loads, stores of 4 values.
    auto out_ok = [&](const void *p) {
        return out_type == OUT_BF16 ? ((uintptr_t)p % 8 == 0) : aligned16(p);
    };
    bool vec = r.N % 4 == 0 && r.ldp % 4 == 0 && r.shard_stride % 4 == 0 && aligned16(r.partials) &&
               r.ldy % 4 == 0;
    if (r.use_slices) {
        for (int64_t j = 0; j * r.slice_rows < r.M; ++j) vec = vec && out_ok(r.y_slice[j]);
    } else {
        vec = vec && out_ok(r.Y) && r.slice_stride % 4 == 0;
    }
    // As many launches as the outputs need, since one has fewer than 2^32 threads.
    const int64_t unit = vec ? 64 : 1;                     // threads of a wavefront's part of a row, or of an output
    const int64_t units = vec ? r.M * ((r.N + QF_WCOLS - 1) / QF_WCOLS) : r.M * r.N, most = ((int64_t)1 << 31) / unit;
    for (int64_t first = 0; first < units; first += most) {
        const int64_t n = units - first < most ? units - first : most;
        const dim3 grid((unsigned)((n * unit + QF_THREADS - 1) / QF_THREADS));
        if (out_type == OUT_BF16 && per_shard) launch_t<OUT_BF16, true>(vec, grid, r, q, first, s);
        else if (out_type == OUT_BF16) launch_t<OUT_BF16, false>(vec, grid, r, q, first, s);
        else if (per_shard) launch_t<OUT_F32, true>(vec, grid, r, q, first, s);
        else launch_t<OUT_F32, false>(vec, grid, r, q, first, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tpl
