// Host side of the calls on a cache in 8 bits and of those that read a paged cache:
// argument checks.  Declarations and the meaning of every argument are in
// include/tplinear.h.
#include "tplinear.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn.h"
#include "heads_checks.h"

namespace {

using namespace tpl;

// Sequences, table and strides of a cache that is read.
tp_status check_cache(int64_t B, int64_t ldt, int64_t max_pages, int64_t n_pages, int64_t page_size,
                      int64_t sp, int64_t ss, int64_t sh, int64_t T, int64_t Hkv, int64_t D,
                      int32_t dtype) {
    if (T < 0 || Hkv < 0 || Hkv > MAX_HEADS || D < 1 || D > MAX_D) return TP_ERR_SHAPE;
    if (B < 0 || max_pages < 0 || n_pages < 0 || page_size < 1 || ldt < 1 || ldt < max_pages) return TP_ERR_SHAPE;
    if (!valid_dtype(dtype)) return TP_ERR_DTYPE;
    if (sp < 0 || ss < 0 || sh < 0) return TP_ERR_SHAPE;
    if (!extent_ok(B, ldt) || !extent_ok(max_pages, page_size)) return TP_ERR_SHAPE;
    if (!extent_ok(n_pages, sp) || !extent_ok(page_size, ss) || !extent_ok(Hkv, sh)) return TP_ERR_SHAPE;
    return TP_OK;
}

CacheArgs cache_args(const int32_t *cu, const int32_t *past, int64_t B, const int32_t *table,
                     int64_t ldt, int64_t max_pages, const void *kc, const void *vc, int64_t n_pages,
                     int64_t page_size, int64_t sp, int64_t ss, int64_t sh, const float *ks,
                     const float *vs, int64_t ssp, int64_t sss, int64_t ssh, int64_t T, int64_t Hkv,
                     int64_t D, int32_t *bad) {
    CacheArgs c{};
    c.cu = cu; c.past = past; c.B = B; c.table = table; c.ldt = ldt;
    c.max_pages = max_pages; c.n_pages = n_pages;
    // positions are below 2^32 - 1: in a larger page all lie in the first
    c.page = page_size < 0xFFFFFFFF ? (uint32_t)page_size : 0xFFFFFFFFu;
    c.shift = (c.page & (c.page - 1)) == 0 ? __builtin_ctz(c.page) : -1;
    c.kc = kc; c.vc = vc; c.s_page = sp; c.s_slot = ss; c.s_head = sh;
    c.ks = ks; c.vs = vs; c.ss_page = ssp; c.ss_slot = sss; c.ss_head = ssh;
    c.T = T; c.Hkv = (int32_t)Hkv; c.D = (int32_t)D; c.bad = bad;
    return c;
}

bool scale_strides_ok(int64_t n_pages, int64_t page_size, int64_t Hkv, int64_t sp, int64_t ss, int64_t sh) {
    return sp >= 0 && ss >= 0 && sh >= 0 && extent_ok(n_pages, sp) && extent_ok(page_size, ss) && extent_ok(Hkv, sh);
}

}  // namespace

extern "C" {

tp_status tp_kv_append_quant(const void *X, int64_t ldx, int32_t x_mode, const float *cos_t,
                             const float *sin_t, int64_t n_pos, int64_t R, int32_t style,
                             const void *q_weight, const void *k_weight, float eps,
                             const int32_t *cu, const int32_t *past, int64_t B,
                             const int32_t *table, int64_t ldt, int64_t max_pages,
                             int8_t *k_cache, int8_t *v_cache, int64_t n_pages, int64_t page_size,
                             int64_t page_stride, int64_t slot_stride, int64_t head_stride,
                             float *k_scale, float *v_scale, int64_t scale_page_stride,
                             int64_t scale_slot_stride, int64_t scale_head_stride, void *Q,
                             int64_t ldq, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int32_t P,
                             int32_t dtype, int32_t *bad_flag, void *stream) {
    const tp_status st = check_heads(ldx, x_mode, cos_t, sin_t, n_pos, R, style, eps, T, Hq, Hkv, D, P, dtype);
    if (st != TP_OK) return st;
    if (B < 0 || max_pages < 0 || n_pages < 0 || page_size < 1 || ldt < 1 || ldt < max_pages) return TP_ERR_SHAPE;
    if (Q && (ldq < Hq * D || !extent_ok(T, ldq))) return TP_ERR_SHAPE;
    if (!extent_ok(B, ldt) || !extent_ok(max_pages, page_size)) return TP_ERR_SHAPE;
    if (!cache_strides_ok(n_pages, page_stride, page_size, slot_stride, Hkv, head_stride, D)) return TP_ERR_SHAPE;
    if (!cache_strides_ok(n_pages, scale_page_stride, page_size, scale_slot_stride, Hkv, scale_head_stride, 1)) return TP_ERR_SHAPE;
    if (T == 0 || B == 0 || Hq + Hkv == 0) return TP_OK;
    if (!X || !cu || !past || (max_pages > 0 && !table)) return TP_ERR_NULL;
    if (Hkv > 0 && n_pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale)) return TP_ERR_NULL;
    HeadArgs a = head_args(X, ldx, x_mode, cos_t, sin_t, n_pos, R, style, q_weight, k_weight, eps,
                           T, Hq, Hkv, D, P, bad_flag);
    a.cu = cu; a.past = past; a.B = B;
    a.table = table; a.ldt = ldt; a.max_pages = max_pages;
    a.n_pages = n_pages; a.page = page_size;
    a.kc = k_cache; a.vc = v_cache;
    a.s_page = page_stride; a.s_slot = slot_stride; a.s_head = head_stride;
    a.ks = k_scale; a.vs = v_scale;
    a.ss_page = scale_page_stride; a.ss_slot = scale_slot_stride; a.ss_head = scale_head_stride;
    a.Q = Q; a.ldq = Q ? ldq : 0;
    return hip_status(launch_kv_append_quant(a, dtype == TP_BF16 ? 2 : 4, (hipStream_t)stream));
}

tp_status tp_kv_read(const int32_t *cu, const int32_t *past, int64_t B, const int32_t *table,
                     int64_t ldt, int64_t max_pages, const void *k_cache, const void *v_cache,
                     int64_t n_pages, int64_t page_size, int64_t page_stride, int64_t slot_stride,
                     int64_t head_stride, const float *k_scale, const float *v_scale,
                     int64_t scale_page_stride, int64_t scale_slot_stride,
                     int64_t scale_head_stride, void *K, int64_t ldk, void *V, int64_t ldv,
                     int64_t T, int64_t Hkv, int64_t D, int32_t dtype, int32_t *bad_flag,
                     void *stream) {
    const tp_status st = check_cache(B, ldt, max_pages, n_pages, page_size, page_stride, slot_stride, head_stride, T, Hkv, D, dtype);
    if (st != TP_OK) return st;
    const bool quant = k_scale || v_scale;
    if (quant && !scale_strides_ok(n_pages, page_size, Hkv, scale_page_stride, scale_slot_stride, scale_head_stride)) return TP_ERR_SHAPE;
    if ((K && (ldk < Hkv * D || !extent_ok(T, ldk))) || (V && (ldv < Hkv * D || !extent_ok(T, ldv)))) return TP_ERR_SHAPE;
    if (T == 0 || B == 0 || Hkv == 0) return TP_OK;
    if (!cu || !past || (max_pages > 0 && !table) || (!K && !V)) return TP_ERR_NULL;
    if (n_pages > 0 && ((K && !k_cache) || (V && !v_cache))) return TP_ERR_NULL;
    if (quant && ((K && !k_scale) || (V && !v_scale))) return TP_ERR_NULL;
    ReadArgs a{};
    a.c = cache_args(cu, past, B, table, ldt, max_pages, k_cache, v_cache, n_pages, page_size, page_stride, slot_stride, head_stride,
                     k_scale, v_scale, scale_page_stride, scale_slot_stride, scale_head_stride, T, Hkv, D, bad_flag);
    a.K = K; a.V = V; a.ldk = K ? ldk : 0; a.ldv = V ? ldv : 0;
    return hip_status(launch_kv_read(a, dtype == TP_BF16 ? 2 : 4, (hipStream_t)stream));
}

size_t tp_kv_attention_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
    if (T < 0 || B < 0 || T > INT32_MAX || B > INT32_MAX || Hq < 1 || Hkv < 1 || Hq > MAX_HEADS || Hkv > MAX_HEADS || Hq % Hkv || D < 1 || D > MAX_D) return 0;
    return round_up(attention_workspace(T, B, Hq, Hkv, D), WS_ALIGN);
}

tp_status tp_kv_attention(const void *Q, int64_t ldq, const int32_t *cu, const int32_t *past,
                          int64_t B, const int32_t *table, int64_t ldt, int64_t max_pages,
                          const void *k_cache, const void *v_cache, int64_t n_pages,
                          int64_t page_size, int64_t page_stride, int64_t slot_stride,
                          int64_t head_stride, const float *k_scale, const float *v_scale,
                          int64_t scale_page_stride, int64_t scale_slot_stride,
                          int64_t scale_head_stride, float softmax_scale, int64_t window, void *O,
                          int64_t ldo, float *lse, int64_t ldl, void *workspace, size_t ws_bytes,
                          int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int32_t dtype,
                          int32_t *bad_flag, void *stream) {
    const tp_status st = check_cache(B, ldt, max_pages, n_pages, page_size, page_stride, slot_stride, head_stride, T, Hkv, D, dtype);
    if (st != TP_OK) return st;
    if (T > INT32_MAX || B > INT32_MAX || Hq < 0 || Hq > MAX_HEADS || (Hq > 0 && Hkv == 0)) return TP_ERR_SHAPE;
    if (!(softmax_scale > 0.0f) || std::isinf(softmax_scale) || window < 0) return TP_ERR_SHAPE;
    if (ldq < Hq * D || ldo < Hq * D || !extent_ok(T, ldq) || !extent_ok(T, ldo)) return TP_ERR_SHAPE;
    if (lse && (ldl < Hq || !extent_ok(T, ldl))) return TP_ERR_SHAPE;
    if (Hkv > 0 && Hq % Hkv) return TP_ERR_INDIVISIBLE;
    if ((k_scale == nullptr) != (v_scale == nullptr)) return TP_ERR_NULL;
    if (k_scale && !scale_strides_ok(n_pages, page_size, Hkv, scale_page_stride, scale_slot_stride, scale_head_stride)) return TP_ERR_SHAPE;
    if (T == 0 || B == 0 || Hq == 0) return TP_OK;
    if (!Q || !O || !cu || !past || (max_pages > 0 && !table) || (n_pages > 0 && (!k_cache || !v_cache))) return TP_ERR_NULL;
    const size_t need = tp_kv_attention_workspace_bytes(T, B, Hq, Hkv, D);
    if (need > 0 && (!workspace || ws_bytes < need || (uintptr_t)workspace % WS_ALIGN)) return TP_ERR_WORKSPACE;
    AttnArgs a{};
    a.c = cache_args(cu, past, B, table, ldt, max_pages, k_cache, v_cache, n_pages, page_size, page_stride, slot_stride, head_stride,
                     k_scale, v_scale, scale_page_stride, scale_slot_stride, scale_head_stride, T, Hkv, D, bad_flag);
    a.Q = Q; a.ldq = ldq; a.O = O; a.ldo = ldo; a.lse = lse; a.ldl = lse ? ldl : 0;
    const int64_t all = (int64_t)1 << 62;
    a.scale = softmax_scale; a.window = window > 0 && window < all ? window : all;
    a.G = (int32_t)(Hq / Hkv);
    a.ws = workspace;
    return hip_status(launch_kv_attention(a, dtype == TP_BF16 ? 2 : 4, (hipStream_t)stream));
}

}  // extern "C"
