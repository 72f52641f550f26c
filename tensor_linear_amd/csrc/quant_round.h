// Rounding of a group of values to int8 with one scale, shared by the quantizer, the
// append to a cache in 8 bits and the norm before an 8-bit layer (device code).  The
// mathematics is described in quantize.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tpl {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// How a group is rounded: s and 1/s after an exact power-of-two shift that
// keeps 1/s finite for groups of tiny values.
struct Step { float up, s, inv, half; bool zero; };

__device__ __forceinline__ Step step_of(uint32_t amax, float &scale) {
    Step t;
    const float a = __uint_as_float(amax);
    scale = amax >= 0x7F800000u ? __builtin_nanf("") : a / 127.0f;
    t.zero = amax >= 0x7F800000u || scale == 0.0f;
    t.up = a < 0x1p-60f ? 0x1p66f : 1.0f;
    t.s = t.zero ? 1.0f : scale * t.up;
    t.inv = 1.0f / t.s;
    t.half = 0.5f * t.s;
    return t;
}

__device__ __forceinline__ int round_one(uint32_t bits, const Step &t) {
    if (t.zero) return 0;
    const float x = __uint_as_float(bits) * t.up;
    const float r = __builtin_rintf(x * t.inv);
    const float e = __builtin_fmaf(-r, t.s, x);
    int q = (int)r;
    const float d = __builtin_fabsf(e);
    if (d > t.half || (d == t.half && (q & 1))) q += e > 0.0f ? 1 : -1;
    return min(max(q, -127), 127);
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (a & 255) | (b & 255) << 8 | (c & 255) << 16 | (uint32_t)d << 24;
}

// The whole numbers' low bytes: bytes 0-3 of a permutation select from its second word.
__device__ __forceinline__ u32x2 low_bytes(const uint32_t (&u)[8]) {
    const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400), b = __builtin_amdgcn_perm(u[3], u[2], 0x0c0c0400);
    const uint32_t c = __builtin_amdgcn_perm(u[5], u[4], 0x0c0c0400), d = __builtin_amdgcn_perm(u[7], u[6], 0x0c0c0400);
    return u32x2{__builtin_amdgcn_perm(b, a, 0x05040100), __builtin_amdgcn_perm(d, c, 0x05040100)};
}

// Eight values a lane to bytes; t is uniform over the wavefront.
__device__ __forceinline__ u32x2 round8(const uint32_t (&v)[8], const Step &t) {
    constexpr float MAGIC = 12582912.0f;   // 1.5 * 2^23: the sum's ulp is 1
    if (!t.zero && t.up == 1.0f) {
        uint32_t u[8];
        float worst = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = __uint_as_float(v[e]), w = __builtin_fmaf(x, t.inv, MAGIC);
            worst = __builtin_fmaxf(worst, __builtin_fabsf(__builtin_fmaf(x, t.inv, MAGIC - w)));
            u[e] = __float_as_uint(w);
        }
        if (!__any(worst >= 0.5f - 0x1p-15f)) {
            return low_bytes(u);
        }
    }
    int q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = round_one(v[e], t);
    return u32x2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
}

// The same where the lanes of a wavefront have groups of their own.
__device__ __forceinline__ u32x2 round8_mixed(const uint32_t (&v)[8], const Step &t) {
    constexpr float MAGIC = 12582912.0f;
    uint32_t u[8];
    float worst = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = __uint_as_float(v[e]), w = __builtin_fmaf(x, t.inv, MAGIC);
        worst = __builtin_fmaxf(worst, __builtin_fabsf(__builtin_fmaf(x, t.inv, MAGIC - w)));
        u[e] = __float_as_uint(w);
    }
    if (!__any(!t.zero && (t.up != 1.0f || worst >= 0.5f - 0x1p-15f))) {
        const u32x2 q = low_bytes(u);
        return t.zero ? u32x2{0, 0} : q;
    }
    int q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = round_one(v[e], t);
    return u32x2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
}

}  // namespace
}  // namespace tpl
