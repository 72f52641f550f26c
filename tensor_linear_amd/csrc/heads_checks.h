// Argument checks shared by the entry points on heads and caches (host code only).
#pragma once

#include "heads.h"
#include "host_checks.h"

namespace tpl {

constexpr int64_t MAX_HEADS = 1 << 16;   // heads of all shards together
constexpr int64_t MAX_D = 1024;          // the backward for odd sizes keeps a head's sums in LDS

// The QKV matrix, heads and rotation, common to the three entry points.
inline tp_status check_heads(int64_t ldx, int32_t x_mode, const float *cos_t, const float *sin_t,
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
inline bool cache_strides_ok(int64_t pages, int64_t s_page, int64_t page, int64_t s_slot, int64_t heads,
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

inline HeadArgs head_args(const void *X, int64_t ldx, int32_t x_mode, const float *cos_t,
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

}  // namespace tpl
