// Rows to 8-bit integers: for each row m and each of its G equal column groups
//   a = max |x|,  s = a / 127 rounded to fp32,  q = x / s rounded to the nearest
// whole number (halves to even), at most 127 in size.  G = 1 gives a token's or
// an output channel's scale; G = P the scale of each shard's column block of a
// row layer's input, which P ranks would each find for their own slice.
//
// The quotient is rounded as the real number x / s, not as its fp32 rounding:
// with r = rint(x * (1/s)) off by at most one, e = x - r s is exact in one fused
// multiply-add (r has 7 bits; the difference is a multiple of the smaller ulp
// and at most about s / 2), and comparing |e| with s / 2 settles the last step.
// That costs four instructions more than rounding x * (1/s), and keeps results
// the same wherever the quotient is computed (bf16 inputs hit halves often: x =
// a / 2 is 63.5).
//
// HBM-bound, one read and one write: a wavefront (or a workgroup of four, for
// groups over 2048 columns) holds its group in registers between the maximum and
// the rounding, 16-byte loads, so X is read once.  Groups of more than 8192
// columns, or odd sizes and alignments, are read twice (the second time mostly
// from cache).
//
// The maximum is taken over the bit patterns without their sign, which order as
// the values do, with infinities and NaN on top: a group that holds one gets the
// scale NaN and zeros, so that every product of that row comes out NaN.
#include "quant.h"

namespace tpl {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int QT = 256;

// The fp32 bit patterns of 8 consecutive inputs.
template <int IN>
__device__ __forceinline__ void load8(const void *p, int64_t i, uint32_t (&v)[8]) {
    if (IN == IN_BF16) {
        const u32x4 h = __builtin_nontemporal_load((const u32x4 *)((const uint16_t *)p + i));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = h[e] << 16;
            v[2 * e + 1] = h[e] & 0xFFFF0000u;
        }
    } else {
        const u32x4 a = __builtin_nontemporal_load((const u32x4 *)((const float *)p + i));
        const u32x4 b = __builtin_nontemporal_load((const u32x4 *)((const float *)p + i + 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
    }
}

template <int IN>
__device__ __forceinline__ uint32_t load1(const void *p, int64_t i) {
    if (IN == IN_BF16) return (uint32_t)((const uint16_t *)p)[i] << 16;
    return ((const uint32_t *)p)[i];
}

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

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// W: wavefronts per group (1: four groups per workgroup; 4: one).  NV: chunks
// of 8 columns that a lane holds.
template <int IN, int W, int NV>
__global__ __launch_bounds__(QT)
void quantize_vec(QuantizeArgs a) {
    __shared__ uint32_t red[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t grp = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    if (W == 1 && grp >= a.M * a.G) return;
    const int64_t m = grp / a.G;
    const int g = (int)(grp - m * a.G);
    const int64_t x0 = m * a.ldx + g * a.Kg, q0 = m * a.ldq + g * a.Kg;
    const int first = (W == 1 ? lane : (int)threadIdx.x) * 8;
    uint32_t v[NV][8];
    uint32_t mx = 0;
#pragma unroll
    for (int c = 0; c < NV; ++c)
        if (first + c * W * 512 < a.Kg) load8<IN>(a.X, x0 + first + c * W * 512, v[c]);
#pragma unroll
    for (int c = 0; c < NV; ++c)
        if (first + c * W * 512 < a.Kg)
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = max(mx, v[c][e] & 0x7FFFFFFFu);
    mx = wave_max(mx);
    if (W > 1) {
        if (lane == 0) red[wave] = mx;
        __syncthreads();
        mx = max(max(red[0], red[1]), max(red[2], red[3]));
    }
    float scale;
    const Step t = step_of(mx, scale);
    if (first == 0) a.scale[m * a.lds + g] = scale;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int k = first + c * W * 512;
        if (k >= a.Kg) continue;
        int q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = round_one(v[c][e], t);
        *(u32x2 *)(a.Q + q0 + k) = u32x2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
    }
}

// Any size and alignment: a workgroup per group, read twice.
template <int IN>
__global__ __launch_bounds__(QT)
void quantize_any(QuantizeArgs a) {
    __shared__ uint32_t red[4];
    const int64_t grp = blockIdx.x;
    const int64_t m = grp / a.G;
    const int g = (int)(grp - m * a.G);
    const int64_t x0 = m * a.ldx + g * a.Kg, q0 = m * a.ldq + g * a.Kg;
    uint32_t mx = 0;
    for (int64_t k = threadIdx.x; k < a.Kg; k += QT) mx = max(mx, load1<IN>(a.X, x0 + k) & 0x7FFFFFFFu);
    mx = wave_max(mx);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
    __syncthreads();
    mx = max(max(red[0], red[1]), max(red[2], red[3]));
    float scale;
    const Step t = step_of(mx, scale);
    if (threadIdx.x == 0) a.scale[m * a.lds + g] = scale;
    for (int64_t k = threadIdx.x; k < a.Kg; k += QT) a.Q[q0 + k] = (int8_t)round_one(load1<IN>(a.X, x0 + k), t);
}

template <int IN>
hipError_t launch_t(const QuantizeArgs &a, hipStream_t s) {
    const int64_t groups = a.M * a.G;
    if (groups > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    constexpr int ES = IN == IN_BF16 ? 2 : 4;
    const bool vec = a.Kg % 8 == 0 && (a.ldx * ES) % 16 == 0 && (uintptr_t)a.X % 16 == 0 &&
                     a.ldq % 8 == 0 && (uintptr_t)a.Q % 8 == 0 && a.Kg <= 8192;
    const dim3 one((unsigned)groups), four((unsigned)((groups + 3) / 4)), block(QT);
    if (!vec) quantize_any<IN><<<one, block, 0, s>>>(a);
    else if (a.Kg <= 512) quantize_vec<IN, 1, 1><<<four, block, 0, s>>>(a);
    else if (a.Kg <= 1024) quantize_vec<IN, 1, 2><<<four, block, 0, s>>>(a);
    else if (a.Kg <= 2048) quantize_vec<IN, 1, 4><<<four, block, 0, s>>>(a);
    else if (a.Kg <= 4096) quantize_vec<IN, 4, 2><<<one, block, 0, s>>>(a);
    else quantize_vec<IN, 4, 4><<<one, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const QuantizeArgs &a, int in_type, hipStream_t s) {
    if (a.M == 0 || a.G == 0) return hipSuccess;
    return in_type == IN_BF16 ? launch_t<IN_BF16>(a, s) : launch_t<IN_F32>(a, s);
}

}  // namespace tpl
