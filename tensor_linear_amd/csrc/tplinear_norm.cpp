// Host side of the step between two blocks: argument checks.  Declarations and the
// meaning of every argument are in include/tplinear.h.
#include "tplinear.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "host_checks.h"
#include "norm.h"

namespace {

using namespace tpl;

constexpr int64_t MAX_F = 1 << 20;

bool rows_ok(const void *p, int64_t ld, int64_t T, int64_t F) { return !p || (ld >= F && ld >= 1 && extent_ok(T, ld)); }

tp_status check_norm(const void *Y, int64_t ldy, const void *R, int64_t ldr, const void *gate, int64_t ldg,
                     float eps, int64_t T, int64_t F, int32_t dtype) {
    if (T < 0 || F < 0 || F > MAX_F || !(eps >= 0.0f)) return TP_ERR_SHAPE;
    if (!valid_dtype(dtype)) return TP_ERR_DTYPE;
    if (!rows_ok(Y, ldy, T, F) || !rows_ok(R, ldr, T, F) || (ldg != 0 && !rows_ok(gate, ldg, T, F))) return TP_ERR_SHAPE;
    return TP_OK;
}

NormArgs norm_args(const void *Y, int64_t ldy, const void *R, int64_t ldr, const void *gate, int64_t ldg,
                   const void *post, const void *pre, float alpha, float beta, float eps, int64_t T, int64_t F) {
    NormArgs a{};
    a.Y = Y; a.ldy = ldy; a.R = R; a.ldr = R ? ldr : 0; a.gate = gate; a.ldg = gate ? ldg : 0;
    a.post = post; a.pre = pre; a.alpha = alpha; a.beta = beta; a.eps = eps; a.T = T; a.F = F;
    return a;
}

}  // namespace

extern "C" {

tp_status tp_residual_norm(const void *Y, int64_t ldy, const void *R, int64_t ldr, const void *gate,
                           int64_t ldg, const void *post_weight, const void *pre_weight,
                           float residual_scale, float branch_scale, float eps, void *H, int64_t ldh,
                           void *N, int64_t ldn, float *n_scale, int64_t T, int64_t F, int32_t dtype,
                           void *stream) {
    const tp_status st = check_norm(Y, ldy, R, ldr, gate, ldg, eps, T, F, dtype);
    if (st != TP_OK) return st;
    if (!rows_ok(H, ldh, T, F) || !rows_ok(N, ldn, T, F)) return TP_ERR_SHAPE;
    if (n_scale && !N && F > 0) return TP_ERR_NULL;
    if (T == 0 || (F == 0 && !n_scale)) return TP_OK;
    if (F > 0 && (!Y || (!H && !N))) return TP_ERR_NULL;
    NormArgs a = norm_args(Y, ldy, R, ldr, gate, ldg, post_weight, pre_weight, residual_scale, branch_scale, eps, T, F);
    a.H = H; a.ldh = H ? ldh : 0; a.N = N; a.ldn = N ? ldn : 0; a.scale = n_scale;
    return hip_status(launch_residual_norm(a, dtype == TP_BF16 ? 2 : 4, (hipStream_t)stream));
}

size_t tp_residual_norm_workspace_bytes(int64_t T, int64_t F) {
    if (T < 0 || F < 0 || F > MAX_F) return 0;
    return round_up((size_t)norm_backward_blocks(T, F) * 3 * (size_t)F * sizeof(float), WS_ALIGN);
}

tp_status tp_residual_norm_backward(const void *Y, int64_t ldy, const void *R, int64_t ldr,
                                    const void *gate, int64_t ldg, const void *post_weight,
                                    const void *pre_weight, float residual_scale,
                                    float branch_scale, float eps, const void *dH, int64_t lddh,
                                    const void *dN, int64_t lddn, void *dY, int64_t lddy, void *dR,
                                    int64_t lddr, void *dgate, int64_t lddg, float *dpost_weight,
                                    float *dpre_weight, void *workspace, size_t ws_bytes, int64_t T,
                                    int64_t F, int32_t dtype, void *stream) {
    const tp_status st = check_norm(Y, ldy, R, ldr, gate, ldg, eps, T, F, dtype);
    if (st != TP_OK) return st;
    if (!rows_ok(dH, lddh, T, F) || !rows_ok(dN, lddn, T, F) || !rows_ok(dY, lddy, T, F) || !rows_ok(dR, lddr, T, F)) return TP_ERR_SHAPE;
    if (ldg != 0 && !rows_ok(dgate, lddg, T, F)) return TP_ERR_SHAPE;
    if ((dgate && !gate) || (dpost_weight && !post_weight) || (dpre_weight && !pre_weight) || (dR && !R)) return TP_ERR_NULL;
    if (!dY && !dR && !dgate && !dpost_weight && !dpre_weight) return TP_ERR_NULL;
    const bool sums = (dgate && ldg == 0) || dpost_weight || dpre_weight;
    if (F == 0 || (T == 0 && !sums)) return TP_OK;
    if (T > 0 && (!Y || (!dH && !dN))) return TP_ERR_NULL;
    if (sums && (!workspace || ws_bytes < tp_residual_norm_workspace_bytes(T, F) || (uintptr_t)workspace % WS_ALIGN)) return TP_ERR_WORKSPACE;
    NormArgs a = norm_args(Y, ldy, R, ldr, gate, ldg, post_weight, pre_weight, residual_scale, branch_scale, eps, T, F);
    a.dH = dH; a.lddh = dH ? lddh : 0; a.dN = dN; a.lddn = dN ? lddn : 0;
    a.dY = dY; a.lddy = dY ? lddy : 0; a.dR = dR; a.lddr = dR ? lddr : 0;
    a.dgate = dgate; a.lddg = dgate ? lddg : 0; a.dpost = dpost_weight; a.dpre = dpre_weight;
    a.partials = sums ? (float *)workspace : nullptr;
    return hip_status(launch_residual_norm_backward(a, dtype == TP_BF16 ? 2 : 4, (hipStream_t)stream));
}

}  // extern "C"
