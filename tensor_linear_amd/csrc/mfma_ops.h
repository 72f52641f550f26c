// Operand types of the DMA-fed shard GEMM kernels.  A fragment is 16 rows x 64
// bytes of K for either type: lane l holds 16 bytes of row l % 16, the (l / 16)th
// of the 64-byte run, and a 16x16 matrix instruction takes 16 cycles for 32 bf16
// or 64 int8 values of K.  So a K step of 128 bytes is the same pipeline, with the
// same loads, LDS reads and instruction count, for both.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tpl {

struct OpBf16 {
    typedef __bf16 Frag __attribute__((ext_vector_type(8)));
    typedef float Acc __attribute__((ext_vector_type(4)));
    static constexpr int ES = 2;          // bytes per element
    static constexpr bool INT8 = false;
    static __device__ __forceinline__ Acc mfma(Frag a, Frag b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

struct OpI8 {
    typedef int Frag __attribute__((ext_vector_type(4)));
    typedef int Acc __attribute__((ext_vector_type(4)));
    static constexpr int ES = 1;
    static constexpr bool INT8 = true;
    static __device__ __forceinline__ Acc mfma(Frag a, Frag b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    }
};

// Source of the W chunks past the end of K (an int8 sum takes zeros there).
static __device__ __attribute__((aligned(16))) const uint32_t zero_chunk[4] = {0, 0, 0, 0};

}  // namespace tpl
