// Launch interface of the per-head steps on a fused QKV column layer's output:
// norm and position rotation of queries and keys, their gradients, and the
// append to a paged cache.  Internal, as kernels.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tpl {

// The QKV matrix: shard i's columns start at X + i * x_shard, row stride ldx,
// and hold hq query heads, then hk key heads, then hk value heads of D values.
// Head j of shard i is head i * hq + j (queries) or i * hk + j (keys, values).
// cos, sin: [n_pos, R / 2] fp32.  wq, wk: [D] of the data's type, or NULL for
// no norm.  An invalid token sets *bad when bad != NULL.
struct HeadArgs {
    const void *X; int64_t ldx, x_shard;
    int64_t T, t0;                          // tokens; the first one of a launch
    int32_t P, hq, hk, D, R, pairs;
    const float *cos, *sin; int64_t n_pos;
    const void *wq, *wk; float eps;
    int32_t *bad;
    const int64_t *pos;                     // token positions (not for the append)
    void *Q; int64_t ldq;                   // queries [T, P * hq * D], or NULL
    void *K; int64_t ldk;                   // keys [T, P * hk * D], or NULL
    // append: sequence s has the tokens cu[s] .. cu[s + 1] - 1 at the positions
    // from past[s] on; position p lies in slot p % page of cache page
    // table[s * ldt + p / page]; element strides of page, slot and head.
    const int32_t *cu, *past, *table; int64_t ldt, B, max_pages, n_pages, page;
    void *kc, *vc; int64_t s_page, s_slot, s_head;
    // backward: gradients of the outputs (NULL: that part of dX is left) and
    // dX with the strides of X; weight gradients by way of `partials`.
    const void *dQ, *dK, *dV; int64_t lddq, lddk, lddv;
    void *dX; int64_t lddx, dx_shard;
    float *dwq, *dwk;
    float *partials;
};

hipError_t launch_qk_norm_rope(const HeadArgs &a, int elem_bytes, hipStream_t s);
hipError_t launch_kv_append(const HeadArgs &a, int elem_bytes, hipStream_t s);
hipError_t launch_qk_norm_rope_backward(const HeadArgs &a, int elem_bytes, hipStream_t s);

// Most workgroups that leave weight-gradient sums of either kind (D floats each)
// in `partials`.
int64_t qk_backward_blocks(int64_t T);

}  // namespace tpl
