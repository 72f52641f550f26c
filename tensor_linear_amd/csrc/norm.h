// Launch interface of the step between two blocks: norm after a block, gate, residual,
// norm before the next.  Internal, as kernels.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tpl {

// u = norm(Y) post;  h = alpha R + beta gate u;  n = norm(h) pre.  NULL: no such part.
struct NormArgs {
    const void *Y, *R, *gate, *post, *pre; int64_t ldy, ldr, ldg;   // ldg 0: one gate [F]
    float alpha, beta, eps;
    void *H, *N; int64_t ldh, ldn;
    float *scale;                        // N is int8, with a scale a token
    int64_t T, F;
    // backward
    const void *dH, *dN; int64_t lddh, lddn;
    void *dY, *dR, *dgate; int64_t lddy, lddr, lddg;   // dgate: rows of the gate's type, or fp32 [F]
    float *dpost, *dpre;
    float *partials;                     // [workgroup][gate, post, pre][F]
};

hipError_t launch_residual_norm(const NormArgs &a, int elem_bytes, hipStream_t s);
hipError_t launch_residual_norm_backward(const NormArgs &a, int elem_bytes, hipStream_t s);

// Most workgroups that leave sums in `partials`.
int64_t norm_backward_blocks(int64_t T, int64_t F);

}  // namespace tpl
