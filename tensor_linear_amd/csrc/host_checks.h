// Argument checks shared by the host files of the C ABI (host code only).
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime.h>

#include "kernels.h"
#include "tplinear.h"

namespace tpl {

constexpr size_t WS_ALIGN = 256;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool valid_dtype(int32_t d) { return d == TP_F32 || d == TP_BF16; }

inline tp_status hip_status(hipError_t e) { return e == hipSuccess ? TP_OK : TP_ERR_HIP; }

// Largest element (or byte) count the library accepts for one buffer: every
// offset and size it derives then fits in int64 / size_t without wrapping.
constexpr int64_t MAX_EXTENT = (int64_t)1 << 60;

// a * b * c <= MAX_EXTENT for non-negative a, b, c, without overflow.
inline bool extent_ok(int64_t a, int64_t b, int64_t c = 1) {
    int64_t ab, abc;
    return !__builtin_mul_overflow(a, b, &ab) && !__builtin_mul_overflow(ab, c, &abc) &&
           abc <= MAX_EXTENT;
}

// Common size checks of the Linear entry points.
inline tp_status check_gemm_shape(int64_t M, int64_t N, int64_t K, int32_t P, int64_t ldx,
                                  int64_t ldw) {
    if (M < 0 || N < 0 || K < 0) return TP_ERR_SHAPE;
    if (P < 1 || P > TP_MAX_SHARDS) return TP_ERR_SHAPE;
    if (ldx < K || ldw < K || ldx < 1 || ldw < 1) return TP_ERR_SHAPE;
    if (!extent_ok(M, ldx) || !extent_ok(N, ldw)) return TP_ERR_SHAPE;
    return TP_OK;
}

// A reduce-scatter's slice stride: 0 (the slices are the row blocks of Y)
// or at least the extent of one slice, (rows - 1) * ldy + N elements, so that
// no two slices share an element (shared elements would be written by two
// workgroups in no fixed order).
inline bool slice_stride_ok(int64_t stride, int64_t rows, int64_t N, int64_t ldy) {
    if (stride == 0 || rows == 0 || N == 0) return true;
    return stride >= (rows - 1) * ldy + N;
}

// Element distance between consecutive shard views of a placement over a
// [rows, cols] tensor with row stride ld.  The launch path addresses shard i
// at base + i * stride, so the stride is read off tp_shard_layout's own views
// (and checked to be uniform): the views the kernels touch are exactly the
// ones the layout entry point reports.  -1 if the layout rejects the shape.
inline int64_t view_stride(int64_t rows, int64_t cols, int64_t ld, int32_t kind, int32_t dim,
                           int32_t P) {
    tp_view v[TP_MAX_SHARDS];
    if (tp_shard_layout(rows, cols, ld, tp_placement{kind, dim}, P, v) != TP_OK) return -1;
    const int64_t stride = P > 1 ? v[1].elem_offset - v[0].elem_offset : 0;
    for (int32_t i = 0; i < P; ++i)
        if (v[i].elem_offset != i * stride) return -1;
    return stride;
}

// Fill the slice table of r from a host array (nullptr: the strided layout).
inline void set_out_slices(ReduceArgs &r, void *const *y_slices, int32_t P) {
    r.use_slices = y_slices ? 1 : 0;
    for (int j = 0; j < MAX_SLICES; ++j) r.y_slice[j] = (y_slices && j < P) ? y_slices[j] : nullptr;
}

}  // namespace tpl
