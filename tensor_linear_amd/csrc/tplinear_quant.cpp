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

// The kernel for an int8 shard GEMM.  All give the same bits, so the choice is
// by speed; same box, 8 shards, us after a read-only 1 GiB flush / warm:
//  - skinny (streams W) up to 32 tokens: 16 tokens skinny vs narrow 4096 -> 28672
//    28.1 / 20.9 vs 28.6 / 20.7, 8192 -> 28672 45.9 / 37.7 vs 52.1 / 36.3, 32 tokens 8192
//    -> 10240 24.3 / 19.9 vs 27.4 / 21.1; above that narrow, whose halves of K
//    stream as well: 48 tokens 8192 -> 10240 31.5 / 26.1 vs 27.8 / 20.2, 1024 -> 4096 8.0 /
//    7.2 vs 6.9 / 6.2.  The gated unit, which has no such halves, up to 48 where 128
//    W rows a tile would fill at most a quarter of the CUs: 48 tokens 4096 -> 2 x
//    4096 14.2 / 12.4 vs 19.0 / 16.8, 8192 -> 2 x 8192 (half) 49.7 / 41.0 vs 43.1 / 31.6;
//  - narrow tiles where the 256 x 256 ones would fill at most half of the CUs:
//    narrow vs tile 4096 -> 28672, 256 tokens (112 tiles) 40.2 / 32.2 vs 53.1 /
//    47.6, 512 tokens (224) 68.2 / 60.9 vs 61.1 / 53.9; 8192 -> 10240, 768 tokens
//    (120) 64.8 / 61.3 vs 90.1 / 82.8, 1024 tokens (160) 114.2 / 102.1 vs 91.1 / 81.1;
//  - generic where K, a stride or an address is not a multiple of 16 (three shards
//    of 2000 -> 1112 at 333 tokens, narrow 10.8, generic with K = 1999 23.2).
hipError_t run_quant(const GemmArgs &g, int out, const GemmExtra &ex, const QuantArgs &q,
                     hipStream_t s) {
    const bool sw = ex.act == ACT_SWIGLU;
    const int64_t cus = device_cu_count();
    if (quant_skinny_supported(g, ex) && (g.M <= 32 || 4 * ((g.N * g.P + 63) / 64) <= cus))
        return launch_quant_skinny(g, out, nullptr, ex, q, s);
    if (quant_dma_supported(g, ex, 256)) {
        const int64_t t256 = ((g.M + 255) / 256) * ((g.N + (sw ? 127 : 255)) / (sw ? 128 : 256)) * g.P;
        if (2 * t256 <= cus) return launch_quant_narrow(g, out, ex, q, s);
        return launch_quant_tile(g, out, ex, q, s);
    }
    return launch_quant_generic(g, out, ex, q, s);
}

// One scale a token: one product over all of K, or P int32 partials and their
// fold (the same integer sums).  The product has P times fewer workgroups to
// hide its longer loop; the partials cost 8 P M N bytes.  8 shards, us, product vs
// partials, weights from HBM (several in turn that no cache holds, in a graph): 16
// tokens 14336 -> 4096 16.3 vs 21.1, 8192 -> 8192 15.2 vs 23.5, 28672 -> 8192 47.5 vs
// 53.0, but 28672 -> 2048 28.2 vs 20.6; 32 tokens 8192 -> 8192 24.4 vs 25.3, 14336 ->
// 4096 31.9 vs 22.2; above, with r = P M N / K: 14336 -> 4096 at 128 tokens (r = 293) 50.8
// vs 23.8, 4096 -> 2048 at 128 (512) 16.5 vs 12.4, at 200 (800) 15.5 vs 14.1 (warm 13.1 vs
// 14.7), 8192 -> 2048 at 300 (600) 28.5 vs 22.2, 28672 -> 8192 at 256 (585) 104 vs 81, at
// 384 (878) 140 vs 129 (warm 103 vs 125), 8192 -> 8192 at 128 (1024) 32.3 vs 36.1: around
// the threshold of 800 the partials win with cold weights and the product with warm ones.
// The second launch itself is about 1.2e6 of P M N (1024 -> 1024 at 64 tokens 6.6 vs 9.4).
// The rule holds for one output.  Token slices (TP_ROW_SCATTER) take it as well, though
// each slice is then a product of its own that reads all of W: 8192 -> 8192 after a
// flush, in slices vs in one output, 16 tokens 77.6 vs 18.0 (partials 26.6), 64 tokens 36.4
// vs 36.2, 256 tokens 85.7 vs 34.7.
bool one_product_faster(int64_t M, int64_t N, int64_t K, int32_t P) {
    if (P == 1) return true;
    if (M <= 16 && N >= 16 * (int64_t)device_cu_count()) return true;
    if (M <= 32) return K <= 8192;
    return (double)P * M * N + 1.2e6 >= 800.0 * K;
}

// A scale for each token and shard: the fold inside the product, or int32
// partials and their fold (the same bits).  8 shards, us, fold inside vs partials,
// weights from HBM as above.  Up to 16 tokens (skinny): 28672 -> 8192 47.3 vs 54.4, 8192
// -> 8192 20.1 vs 23.7, 14336 -> 4096 20.7 vs 21.3 (warm 20.5 vs 19.0), 4096 -> 2048 8.6 vs
// 10.4, 1024 -> 1024 7.6 vs 8.0, but 28672 -> 2048 30.4 vs 20.8 and 14080 -> 2000 19.8 vs 16.1
// (fewer workgroups than CUs and a long K); 32 tokens 14336 -> 4096 50.2 vs 22.2.
bool skinny_fold_faster(int64_t M, int64_t N, int64_t K) {
    return M <= 16 && (N >= 16 * (int64_t)device_cu_count() || K <= 4096);
}

// 256 x 128 tiles with the fold in registers walk the shards of a tile in turn,
// so they need enough tiles, the more the longer the shard's K (us, fold vs partials,
// weights from HBM as above): K/P = 512 at 48 tiles 37.6 vs 30.0, at 64 37.7 vs 36.3, at 96
// 37.6 vs 55.0; 1024 at 64 61.7 vs 41.8, at 128 61.2 vs 75.4; 1792 at 128 103.6 vs 94.2, at
// 160 103.6 vs 123.7; 3584 at 192 194.5 vs 197.5, at 256 216 vs 257; 4096 tokens 14336 -> 4096
// 219 vs 344, 28672 -> 8192 810 vs 1080.
bool rowfold_faster(int64_t M, int64_t N, int64_t Ks) {
    if (M <= 64) return false;   // its 256-row tile would be three-quarters empty
    const int64_t tiles = ((M + 255) / 256) * ((N + 127) / 128), cus = device_cu_count();
    return tiles >= cus || tiles * 6400 >= cus * (1536 + Ks);
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
    // Inside the product where that is faster, or with TPLINEAR_ROW_FOLD=gemm
    // wherever a kernel takes the call.
    const bool forced = row_fold_in_gemm_forced();
    ex.bias = bias;
    if (!per_shard) {
        if (!y_slices && (forced || one_product_faster(M, N, K, P))) {
            GemmArgs d = g;
            d.K = K; d.P = 1; d.a_shard = d.b_shard = 0;
            d.C = Y; d.ldc = ldy; d.c_shard = 0;
            if (mode == TP_ROW_SCATTER) {
                // the token slices as shards in M: row block j of X into slice j
                d.M = M / P; d.P = P;
                d.a_shard = (M / P) * ldx; d.c_shard = r.slice_stride;
                q.x_shard = (M / P) * ldxs;
            }
            return hip_status(run_quant(d, out, ex, q, s));
        }
    } else if (mode != TP_ROW_SCATTER && quant_skinny_supported(g, ex) &&
               (forced || skinny_fold_faster(M, N, K))) {
        const FoldArgs f{Y, ldy, out};
        return hip_status(launch_quant_skinny(g, out, &f, ex, q, s));
    } else if (quant_rowfold_supported(g, r, q) && (forced || rowfold_faster(M, N, K / P))) {
        return hip_status(launch_quant_rowfold(g, r, q, out, s));
    }
    ex.bias = nullptr;
    const hipError_t e = run_quant(g, OUT_I32, ex, q, s);
    if (e != hipSuccess) return TP_ERR_HIP;
    return hip_status(launch_quant_fold(r, q, per_shard, out, s));
}

}  // extern "C"
