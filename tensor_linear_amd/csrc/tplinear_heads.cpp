// Host side of the per-head steps on a fused QKV layer's output: argument
// checks.  Declarations and the meaning of every argument are in
// include/tplinear.h.
#include "tplinear.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "heads.h"
#include "host_checks.h"

namespace {

using namespace tpl;

constexpr int64_t MAX_HEADS = 1 << 16;   // heads of all shards together
constexpr int64_t MAX_D = 1024;          // the backward for odd sizes keeps a head's sums in LDS

// The QKV matrix, heads and rotation, common to the three entry points.
tp_status check_heads(int64_t ldx, int32_t x_mode, const float *cos_t, const float *sin_t,
                      int64_t n_pos, int64_t R, int32_t style, float eps, int64_t T, int64_t Hq,
                      int64_t Hkv, int64_t D, int32_t P, int32_t dtype) {
    if (T < 0 || Hq < 0 || Hkv < 0 || D < 1 || D > MAX_D || P < 1 || P > TP_MAX_SHARDS) return TP_ERR_SHAPE;
    if (Hq > MAX_HEADS || Hkv > MAX_HEADS || n_pos < 0 || R < 0 || R > D || R % 2) return TP_ERR_SHAPE;
    if (!(eps >= 0.0f)) return TP_ERR_SHAPE;
    if (!valid_dtype(dtype)) return TP_ERR_DTYPE;
    if (x_mode != TP_Y_CONCAT && x_mode != TP_Y_SHARDS) return TP_ERR_MODE;
    if (style != TP_ROPE_HALVES && style != TP_ROPE_PAIRS) return TP_ERR_MODE;
    if (Hq % P || Hkv % P) return TP_ERR_INDIVISIBLE;
    const int64_t per = (Hq + 2 * Hkv) / P * D;
    if (ldx < 1 || ldx < (x_mode == TP_Y_CONCAT ? per * P : per)) return TP_ERR_SHAPE;
    if (!extent_ok(T, ldx, x_mode == TP_Y_SHARDS ? P : 1) || !extent_ok(n_pos, R ? R : 1)) return TP_ERR_SHAPE;
    if (T > 0 && R > 0 && (!cos_t || !sin_t)) return TP_ERR_NULL;
    return TP_OK;
}

// No two rows of a cache share elements: in the order of their strides, each
// stride is at least what the rows below it span.  Dimensions of one entry may
// have any stride.
bool cache_strides_ok(int64_t pages, int64_t s_page, int64_t page, int64_t s_slot, int64_t heads,
                      int64_t s_head, int64_t D) {
    int64_t n[3] = {pages, page, heads}, st[3] = {s_page, s_slot, s_head};
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0 || !extent_ok(n[i], st[i])) return false;
        for (int j = i; j > 0 && st[j] < st[j - 1]; --j) {
            const int64_t a = n[j], b = st[j];
            n[j] = n[j - 1]; st[j] = st[j - 1];
            n[j - 1] = a; st[j - 1] = b;
        }
    }
    int64_t span = D;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < span) return false;
        span += (n[i] - 1) * st[i];
    }
    return true;
}

HeadArgs head_args(const void *X, int64_t ldx, int32_t x_mode, const float *cos_t,
                   const float *sin_t, int64_t n_pos, int64_t R, int32_t style, const void *wq,
                   const void *wk, float eps, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                   int32_t P, int32_t *bad) {
    HeadArgs a{};
    a.X = X; a.ldx = ldx;
    // shard i's block: column block i of the concatenated output (Shard(1)),
    // or block i of the P stacked ones (Shard(0)), as the column layer writes it
    const int64_t per = (Hq + 2 * Hkv) / P * D;
    a.x_shard = x_mode == TP_Y_CONCAT ? view_stride(T, per * P, ldx, TP_SHARD, 1, P)
                                      : view_stride(P * T, per, ldx, TP_SHARD, 0, P);
    a.T = T; a.P = P; a.hq = (int32_t)(Hq / P); a.hk = (int32_t)(Hkv / P);
    a.D = (int32_t)D; a.R = (int32_t)R; a.pairs = style == TP_ROPE_PAIRS;
    a.cos = cos_t; a.sin = sin_t; a.n_pos = n_pos;
    a.wq = wq; a.wk = wk; a.eps = eps; a.bad = bad;
    return a;
}

}  // namespace

extern "C" {

tp_status tp_qk_norm_rope(const void *X, int64_t ldx, int32_t x_mode, const int64_t *pos,
                          const float *cos_t, const float *sin_t, int64_t n_pos, int64_t R,
                          int32_t style, const void *q_weight, const void *k_weight, float eps,
                          void *Q, int64_t ldq, void *K, int64_t ldk, int64_t T, int64_t Hq,
                          int64_t Hkv, int64_t D, int32_t P, int32_t dtype, int32_t *bad_flag,
                          void *stream) {
    const tp_status st = check_heads(ldx, x_mode, cos_t, sin_t, n_pos, R, style, eps, T, Hq, Hkv, D, P, dtype);
    if (st != TP_OK) return st;
    if ((Q && ldq < Hq * D) || (K && ldk < Hkv * D)) return TP_ERR_SHAPE;
    if ((Q && !extent_ok(T, ldq)) || (K && !extent_ok(T, ldk))) return TP_ERR_SHAPE;
    if (T == 0 || Hq + Hkv == 0) return TP_OK;
    if (!X || (!Q && !K) || (R > 0 && !pos)) return TP_ERR_NULL;
    HeadArgs a = head_args(X, ldx, x_mode, cos_t, sin_t, n_pos, R, style, q_weight, k_weight, eps,
                           T, Hq, Hkv, D, P, bad_flag);
    a.pos = pos;
    a.Q = Q; a.ldq = Q ? ldq : 0; a.K = K; a.ldk = K ? ldk : 0;
    return hip_status(launch_qk_norm_rope(a, dtype == TP_BF16 ? 2 : 4, (hipStream_t)stream));
}

tp_status tp_kv_append(const void *X, int64_t ldx, int32_t x_mode, const float *cos_t,
                       const float *sin_t, int64_t n_pos, int64_t R, int32_t style,
                       const void *q_weight, const void *k_weight, float eps, const int32_t *cu,
                       const int32_t *past, int64_t B, const int32_t *table, int64_t ldt,
                       int64_t max_pages, void *k_cache, void *v_cache, int64_t n_pages,
                       int64_t page_size, int64_t page_stride, int64_t slot_stride,
                       int64_t head_stride, void *Q, int64_t ldq, int64_t T, int64_t Hq,
                       int64_t Hkv, int64_t D, int32_t P, int32_t dtype, int32_t *bad_flag,
                       void *stream) {
    const tp_status st = check_heads(ldx, x_mode, cos_t, sin_t, n_pos, R, style, eps, T, Hq, Hkv, D, P, dtype);
    if (st != TP_OK) return st;
    if (B < 0 || max_pages < 0 || n_pages < 0 || page_size < 1 || ldt < 1 || ldt < max_pages) return TP_ERR_SHAPE;
    if (Q && (ldq < Hq * D || !extent_ok(T, ldq))) return TP_ERR_SHAPE;
    if (!extent_ok(B, ldt) || !extent_ok(max_pages, page_size)) return TP_ERR_SHAPE;
    if (!cache_strides_ok(n_pages, page_stride, page_size, slot_stride, Hkv, head_stride, D)) return TP_ERR_SHAPE;
    if (T == 0 || B == 0 || Hq + Hkv == 0) return TP_OK;
    if (!X || !cu || !past || (max_pages > 0 && !table)) return TP_ERR_NULL;
    if (Hkv > 0 && n_pages > 0 && (!k_cache || !v_cache)) return TP_ERR_NULL;
    HeadArgs a = head_args(X, ldx, x_mode, cos_t, sin_t, n_pos, R, style, q_weight, k_weight, eps,
                           T, Hq, Hkv, D, P, bad_flag);
    a.cu = cu; a.past = past; a.B = B;
    a.table = table; a.ldt = ldt; a.max_pages = max_pages;
    a.n_pages = n_pages; a.page = page_size;
    a.kc = k_cache; a.vc = v_cache;
    a.s_page = page_stride; a.s_slot = slot_stride; a.s_head = head_stride;
    a.Q = Q; a.ldq = Q ? ldq : 0;
    return hip_status(launch_kv_append(a, dtype == TP_BF16 ? 2 : 4, (hipStream_t)stream));
}

size_t tp_qk_norm_rope_workspace_bytes(int64_t T, int64_t D) {
    if (T < 0 || D < 1 || D > MAX_D) return 0;
    return round_up((size_t)qk_backward_blocks(T) * 2 * (size_t)D * sizeof(float), WS_ALIGN);
}

tp_status tp_qk_norm_rope_backward(const void *X, int64_t ldx, int32_t x_mode, const int64_t *pos,
                                   const float *cos_t, const float *sin_t, int64_t n_pos,
                                   int64_t R, int32_t style, const void *q_weight,
                                   const void *k_weight, float eps, const void *dQ, int64_t lddq,
                                   const void *dK, int64_t lddk, const void *dV, int64_t lddv,
                                   void *dX, int64_t lddx, float *dq_weight, float *dk_weight,
                                   void *workspace, size_t ws_bytes, int64_t T, int64_t Hq,
                                   int64_t Hkv, int64_t D, int32_t P, int32_t dtype,
                                   int32_t *bad_flag, void *stream) {
    const tp_status st = check_heads(ldx, x_mode, cos_t, sin_t, n_pos, R, style, eps, T, Hq, Hkv, D, P, dtype);
    if (st != TP_OK) return st;
    const int64_t per = (Hq + 2 * Hkv) / P * D;
    if (lddx < 1 || lddx < (x_mode == TP_Y_CONCAT ? per * P : per)) return TP_ERR_SHAPE;
    if (!extent_ok(T, lddx, x_mode == TP_Y_SHARDS ? P : 1)) return TP_ERR_SHAPE;
    if ((dQ && lddq < Hq * D) || (dK && lddk < Hkv * D) || (dV && lddv < Hkv * D)) return TP_ERR_SHAPE;
    if ((dQ && !extent_ok(T, lddq)) || (dK && !extent_ok(T, lddk)) || (dV && !extent_ok(T, lddv))) return TP_ERR_SHAPE;
    // A weight's gradient exists where there is a norm, and is the sum over the
    // heads whose output gradient is given.
    if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return TP_ERR_NULL;
    const bool grads = dq_weight || dk_weight;
    if (grads && (!workspace || ws_bytes < tp_qk_norm_rope_workspace_bytes(T, D) ||
                  ((uintptr_t)workspace % WS_ALIGN) != 0))
        return TP_ERR_WORKSPACE;
    if (T > 0 && Hq + Hkv > 0) {
        if (!dQ && !dK && !dV) return TP_ERR_NULL;
        if (!dX || (R > 0 && !pos) || ((q_weight || k_weight) && !X)) return TP_ERR_NULL;
    } else if (!grads) {
        return TP_OK;
    }
    HeadArgs a = head_args(X, ldx, x_mode, cos_t, sin_t, n_pos, R, style, q_weight, k_weight, eps,
                           T, Hq, Hkv, D, P, bad_flag);
    a.pos = pos;
    a.dQ = dQ; a.lddq = dQ ? lddq : 0; a.dK = dK; a.lddk = dK ? lddk : 0; a.dV = dV; a.lddv = dV ? lddv : 0;
    a.dX = dX; a.lddx = lddx;
    a.dx_shard = x_mode == TP_Y_CONCAT ? view_stride(T, per * P, lddx, TP_SHARD, 1, P)
                                       : view_stride(P * T, per, lddx, TP_SHARD, 0, P);
    a.dwq = dq_weight; a.dwk = dk_weight;
    a.partials = grads ? (float *)workspace : nullptr;
    return hip_status(launch_qk_norm_rope_backward(a, dtype == TP_BF16 ? 2 : 4, (hipStream_t)stream));
}

}  // extern "C"
