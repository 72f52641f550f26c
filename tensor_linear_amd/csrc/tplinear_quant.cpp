// Host side of the 8-bit integer Linear: argument checks and the choice of
// kernel.  Declarations and the meaning of every argument are in
// include/tplinear.h.
#include "tplinear.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "host_checks.h"
#include "kernels.h"
#include "quant.h"

namespace {

using namespace tpl;

// Longest product whose int32 sum cannot overflow: 2^14 (-128 * -128) times
// this many terms stays below 2^31.
constexpr int64_t MAX_QUANT_K = 131071;

hipError_t run_quant(const GemmArgs &g, int out, const GemmExtra &ex, const QuantArgs &q,
                     hipStream_t s) {
    if (quant_dma_supported(g, ex, 256) && g.M > 32) {
        const bool sw = ex.act == ACT_SWIGLU;
        const int64_t t256 = ((g.M + 255) / 256) * ((g.N + (sw ? 127 : 255)) / (sw ? 128 : 256)) * g.P;
        if (2 * t256 <= device_cu_count()) return launch_quant_narrow(g, out, ex, q, s);
        return launch_quant_tile(g, out, ex, q, s);
    }
    return launch_quant_generic(g, out, ex, q, s);
}

}  // namespace

extern "C" {

tp_status tp_quantize_rows(const void *X, int64_t ldx, int8_t *Q, int64_t ldq, float *scale,
                           int64_t lds, int64_t M, int64_t K, int32_t G, int32_t dtype,
                           void *stream) {
    if (M < 0 || K < 0 || G < 1 || G > TP_MAX_SHARDS) return TP_ERR_SHAPE;
    if (ldx < K || ldq < K || ldx < 1 || ldq < 1 || lds < G) return TP_ERR_SHAPE;
    if (!extent_ok(M, ldx) || !extent_ok(M, ldq) || !extent_ok(M, lds)) return TP_ERR_SHAPE;
    if (!valid_dtype(dtype)) return TP_ERR_DTYPE;
    if (K % G != 0) return TP_ERR_INDIVISIBLE;
    if (M == 0) return TP_OK;
    if (!scale || (K > 0 && (!X || !Q))) return TP_ERR_NULL;
    const QuantizeArgs a{X, ldx, Q, ldq, scale, lds, M, K / G, G};
    return hip_status(launch_quantize_rows(a, dtype == TP_BF16 ? IN_BF16 : IN_F32, (hipStream_t)stream));
}

tp_status tp_linear_column_quant(const int8_t *X, int64_t ldx, const float *x_scale, int64_t ldxs,
                                 const int8_t *W, int64_t ldw, const float *w_scale,
                                 const void *bias, void *Y, int64_t ldy, int32_t y_mode,
                                 int32_t act, int64_t M, int64_t N, int64_t K, int32_t P,
                                 int32_t out_dtype, void *stream) {
    const tp_status st = check_gemm_shape(M, N, K, P, ldx, ldw);
    if (st != TP_OK) return st;
    if (K > MAX_QUANT_K || ldxs < 1 || !extent_ok(M, ldxs)) return TP_ERR_SHAPE;
    if (!valid_dtype(out_dtype)) return TP_ERR_DTYPE;
    if (y_mode != TP_Y_CONCAT && y_mode != TP_Y_SHARDS) return TP_ERR_MODE;
    if (act != TP_ACT_NONE && act != TP_ACT_SWIGLU) return TP_ERR_MODE;
    if (N % P != 0) return TP_ERR_INDIVISIBLE;
    const int64_t Ns = N / P;                                   // W rows per shard
    const bool swiglu = act == TP_ACT_SWIGLU;
    if (swiglu && Ns % 2 != 0) return TP_ERR_INDIVISIBLE;
    const int64_t On = swiglu ? Ns / 2 : Ns;                     // outputs per shard
    if (y_mode == TP_Y_CONCAT ? ldy < On * P : ldy < On) return TP_ERR_SHAPE;
    if (ldy < 1) return TP_ERR_SHAPE;
    if (!extent_ok(M, ldy, y_mode == TP_Y_SHARDS ? P : 1)) return TP_ERR_SHAPE;
    if (M == 0 || N == 0) return TP_OK;
    if (!Y || !x_scale || !w_scale || (K > 0 && (!X || !W))) return TP_ERR_NULL;

    // Shard strides from the placements, as in tp_linear_column_ex; the
    // channels' scales are Shard(0) as the bias is.
    const int64_t w_stride = view_stride(N, K, ldw, TP_SHARD, 0, P);
    const int64_t y_stride = y_mode == TP_Y_CONCAT ? view_stride(M, P * On, ldy, TP_SHARD, 1, P)
                                                   : view_stride(P * M, On, ldy, TP_SHARD, 0, P);
    const int64_t b_stride = view_stride(N, 1, 1, TP_SHARD, 0, P);
    if (w_stride < 0 || y_stride < 0 || b_stride < 0) return TP_ERR_SHAPE;
    GemmArgs g;
    g.A = X; g.lda = ldx; g.a_shard = 0;
    g.B = W; g.ldb = ldw; g.b_shard = w_stride;
    g.C = Y; g.ldc = ldy; g.c_shard = y_stride;
    g.M = M; g.N = On; g.K = K; g.P = P;
    GemmExtra ex{};
    ex.bias = bias; ex.bias_shard = b_stride;
    ex.act = swiglu ? ACT_SWIGLU : ACT_NONE; ex.up_off = swiglu ? On : 0;
    const QuantArgs q{x_scale, ldxs, 0, w_scale, b_stride};
    return hip_status(run_quant(g, out_dtype == TP_BF16 ? OUT_BF16 : OUT_F32, ex, q, (hipStream_t)stream));
}

tp_status tp_linear_row_quant(const int8_t *X, int64_t ldx, const float *x_scale, int64_t ldxs,
                              int32_t x_groups, const int8_t *W, int64_t ldw,
                              const float *w_scale, const void *bias, void *Y,
                              void *const *y_slices, int64_t ldy, int64_t y_slice_stride,
                              int32_t mode, void *workspace, size_t ws_bytes, int64_t M,
                              int64_t N, int64_t K, int32_t P, int32_t out_dtype, void *stream) {
    const tp_status st = check_gemm_shape(M, N, K, P, ldx, ldw);
    if (st != TP_OK) return st;
    if (x_groups != 1 && x_groups != P) return TP_ERR_SHAPE;
    if (ldxs < x_groups || !extent_ok(M, ldxs)) return TP_ERR_SHAPE;
    if (!valid_dtype(out_dtype)) return TP_ERR_DTYPE;
    if (mode < TP_ROW_PARTIAL || mode > TP_ROW_SCATTER) return TP_ERR_MODE;
    if (bias && mode == TP_ROW_PARTIAL) return TP_ERR_MODE;
    if (y_slices && mode != TP_ROW_SCATTER) return TP_ERR_MODE;
    if (K % P != 0) return TP_ERR_INDIVISIBLE;
    // The sums that stay integers: over a shard's columns, or with one scale
    // a token over all of them.
    const bool per_shard = x_groups > 1;
    if ((per_shard || mode == TP_ROW_PARTIAL ? K / P : K) > MAX_QUANT_K) return TP_ERR_SHAPE;
    if (mode == TP_ROW_SCATTER && M % P != 0) return TP_ERR_INDIVISIBLE;
    if (ldy < N || ldy < 1 || y_slice_stride < 0) return TP_ERR_SHAPE;
    if (!extent_ok(M, ldy, mode == TP_ROW_PARTIAL ? P : 1) ||
        !extent_ok(M, N, (int64_t)P * (int64_t)sizeof(float)) || !extent_ok(P, y_slice_stride))
        return TP_ERR_SHAPE;
    if (mode == TP_ROW_SCATTER && !y_slices && !slice_stride_ok(y_slice_stride, M / P, N, ldy))
        return TP_ERR_SHAPE;
    if (M == 0 || N == 0) return TP_OK;
    if (y_slices) {
        for (int32_t j = 0; j < P; ++j)
            if (!y_slices[j]) return TP_ERR_NULL;
    } else if (!Y) {
        return TP_ERR_NULL;
    }
    if (!x_scale || !w_scale || (K > 0 && (!X || !W))) return TP_ERR_NULL;
    const size_t need = tp_row_workspace_bytes(mode, M, N, P);
    if (need > 0 && (!workspace || ws_bytes < need || ((uintptr_t)workspace % WS_ALIGN) != 0))
        return TP_ERR_WORKSPACE;

    const hipStream_t s = (hipStream_t)stream;
    const int out = out_dtype == TP_BF16 ? OUT_BF16 : OUT_F32;
    const int64_t x_stride = view_stride(M, K, ldx, TP_SHARD, 1, P);
    const int64_t w_stride = view_stride(N, K, ldw, TP_SHARD, 1, P);
    const int64_t p_stride = view_stride(M, N, mode == TP_ROW_PARTIAL ? ldy : N, TP_PARTIAL, 0, P);
    const int64_t s_stride = mode == TP_ROW_SCATTER ? view_stride(M, N, ldy, TP_SHARD, 0, P) : 0;
    if (x_stride < 0 || w_stride < 0 || p_stride < 0 || s_stride < 0) return TP_ERR_SHAPE;
    GemmArgs g;
    g.A = X; g.lda = ldx; g.a_shard = x_stride;
    g.B = W; g.ldb = ldw; g.b_shard = w_stride;
    g.M = M; g.N = N; g.K = K / P; g.P = P;
    GemmExtra ex{};
    QuantArgs q{x_scale, ldxs, per_shard ? 1 : 0, w_scale, 0};
    if (mode == TP_ROW_PARTIAL) {
        g.C = Y; g.ldc = ldy; g.c_shard = p_stride;
        return hip_status(run_quant(g, OUT_F32, ex, q, s));
    }
    g.C = workspace; g.ldc = N; g.c_shard = p_stride;
    ReduceArgs r;
    r.partials = (const float *)workspace; r.shard_stride = p_stride; r.ldp = N;
    r.Y = Y; r.ldy = ldy; r.M = M; r.N = N; r.P = P;
    r.bias = bias;
    set_out_slices(r, y_slices, P);
    r.slice_rows = mode == TP_ROW_SCATTER ? M / P : M;
    r.slice_stride = mode == TP_ROW_SCATTER ? (y_slice_stride ? y_slice_stride : s_stride) : 0;
    if (per_shard && M > 64 && quant_rowfold_supported(g, r, q)) {
        const int64_t tiles = ((M + 255) / 256) * ((N + 127) / 128);
        if (tiles >= device_cu_count()) return hip_status(launch_quant_rowfold(g, r, q, out, s));
    }
    const hipError_t e = run_quant(g, OUT_I32, ex, q, s);
    if (e != hipSuccess) return TP_ERR_HIP;
    return hip_status(launch_quant_fold(r, q, per_shard, out, s));
}

}  // extern "C"
