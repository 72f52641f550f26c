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
// That keeps results the same wherever the quotient is computed (bf16 inputs hit
// halves often: x = a / 2 is 63.5).  Most values need none of it: a wavefront
// first rounds 8 values a lane by adding 1.5 * 2^23 in one multiply-add (the sum's
// low byte is the whole number), and only where some lane's distance from its
// whole number is within 2^-15 of a half -- x * (1/s) is off by less than 2^-16 --
// does it go through those 8 again exactly.
//
// HBM-bound, one read and one write: a wavefront (or a workgroup of four or
// sixteen, for groups over 2048 columns) holds its group in registers between the
// maximum and the rounding, 16-byte loads, so X is read once: 4096 x 14336 bf16 in
// 8 groups or in one 36.6 us (4.8 TB/s; 47 when read twice).  Only groups of
// more than 32768 columns are read twice.  The loads need no alignment, and a
// group's last columns past a multiple of 8 go one by one (4096 x 14342 38 us, with
// a value a lane 109).  Loads past the caches, ordinary stores: the product that
// comes next reads Q, not X.  Stores past the caches are faster by themselves (4096
// x 4096 12.4 us for 14.7), but with the product behind them 256 x 8192 -> 10240 takes
// 46.8 us for 42.8, 4096 x 14336 -> 4096 266 for 263.
//
// The maximum is taken over the bit patterns without their sign, which order as
// the values do, with infinities and NaN on top: a group that holds one gets the
// scale NaN and zeros, so that every product of that row comes out NaN.
#include "quant.h"

namespace tpl {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// in memory: at any address (the same instructions as for aligned ones)
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));

constexpr int QT = 256;

// 8 consecutive inputs as they are: four words of two bf16, or eight fp32.
template <int IN>
struct Raw8 { uint32_t w[IN == IN_BF16 ? 4 : 8]; };

// Those of the 8 from element i on that are among the first n (TAIL: n may be less
// than 8), the rest zeros.
template <int IN, bool TAIL>
__device__ __forceinline__ Raw8<IN> load8(const void *p, int64_t i, int64_t n) {
    Raw8<IN> r = {};
    if (n <= 0) return r;
    if (!TAIL || n >= 8) {
        const u32x4_any *q = (const u32x4_any *)((const char *)p + i * (IN == IN_BF16 ? 2 : 4));
        const u32x4 a = __builtin_nontemporal_load(q);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.w[e] = a[e];
        if constexpr (IN == IN_F32) {
            const u32x4 b = __builtin_nontemporal_load(q + 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) r.w[4 + e] = b[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e) {
            if (e >= n) break;
            if constexpr (IN == IN_BF16) r.w[e / 2] |= (uint32_t)((const uint16_t *)p)[i + e] << (16 * (e & 1));
            else r.w[e] = ((const uint32_t *)p)[i + e];
        }
    }
    return r;
}

template <bool TAIL>
__device__ __forceinline__ void store8(int8_t *p, int64_t n, u32x2 q) {
    if (n <= 0) return;
    if (!TAIL || n >= 8) {
        *(u32x2_any *)p = q;
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) p[e] = (int8_t)(q[e / 4] >> (8 * (e & 3)));
    }
}

// Running maximum of the patterns without their signs (bf16: of the low and the
// high halves apart), and its fp32 pattern.
template <int IN>
__device__ __forceinline__ uint32_t max8(uint32_t m, const Raw8<IN> &r) {
    if constexpr (IN == IN_BF16) {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 a = __builtin_bit_cast(u16x2, m);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            a = __builtin_elementwise_max(a, __builtin_bit_cast(u16x2, r.w[e] & 0x7FFF7FFFu));
        return __builtin_bit_cast(uint32_t, a);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, r.w[e] & 0x7FFFFFFFu);
        return m;
    }
}
template <int IN>
__device__ __forceinline__ uint32_t max_bits(uint32_t m) {
    return IN == IN_BF16 ? max(m << 16, m & 0xFFFF0000u) : m;
}

// The fp32 patterns of 8 inputs.
template <int IN>
__device__ __forceinline__ void widen8(const Raw8<IN> &r, uint32_t (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = IN == IN_F32 ? r.w[e % (IN == IN_F32 ? 8 : 4)] : (e & 1) ? r.w[e / 2] & 0xFFFF0000u : r.w[e / 2] << 16;
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
            // the low bytes: bytes 0-3 of a permutation select from its second word
            const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400), b = __builtin_amdgcn_perm(u[3], u[2], 0x0c0c0400);
            const uint32_t c = __builtin_amdgcn_perm(u[5], u[4], 0x0c0c0400), d = __builtin_amdgcn_perm(u[7], u[6], 0x0c0c0400);
            return u32x2{__builtin_amdgcn_perm(b, a, 0x05040100), __builtin_amdgcn_perm(d, c, 0x05040100)};
        }
    }
    int q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = round_one(v[e], t);
    return u32x2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// W: wavefronts per group (1: four groups per workgroup; else one).  NV: chunks
// of 8 columns that a lane holds.  TAIL: the groups are no multiple of 8 columns.
template <int IN, int W, int NV, bool TAIL>
__global__ __launch_bounds__(W == 1 ? QT : W * 64)
void quantize_vec(QuantizeArgs a) {
    __shared__ uint32_t red[W];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t grp = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    if (W == 1 && grp >= a.M * a.G) return;
    const int64_t m = grp / a.G;
    const int g = (int)(grp - m * a.G);
    const int64_t x0 = m * a.ldx + g * a.Kg, q0 = m * a.ldq + g * a.Kg;
    const int first = (W == 1 ? lane : (int)threadIdx.x) * 8;
    Raw8<IN> raw[NV] = {};
    uint32_t mx = 0;
#pragma unroll
    for (int c = 0; c < NV; ++c)
        raw[c] = load8<IN, TAIL>(a.X, x0 + first + c * W * 512, a.Kg - (first + c * W * 512));
#pragma unroll
    for (int c = 0; c < NV; ++c) mx = max8<IN>(mx, raw[c]);
    mx = wave_max(max_bits<IN>(mx));
    if (W > 1) {
        if (lane == 0) red[wave] = mx;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) mx = max(mx, red[w]);
    }
    float scale;
    const Step t = step_of(mx, scale);
    if (first == 0) a.scale[m * a.lds + g] = scale;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int k = first + c * W * 512;
        uint32_t v[8];
        widen8<IN>(raw[c], v);
        const u32x2 q = round8(v, t);       // every lane takes part: past the group's end on zeros
        store8<TAIL>(a.Q + q0 + k, a.Kg - k, q);
    }
}

// Longer groups: a workgroup per group, read twice.
template <int IN, bool TAIL>
__global__ __launch_bounds__(QT)
void quantize_long(QuantizeArgs a) {
    __shared__ uint32_t red[4];
    const int64_t grp = blockIdx.x;
    const int64_t m = grp / a.G;
    const int g = (int)(grp - m * a.G);
    const int64_t x0 = m * a.ldx + g * a.Kg, q0 = m * a.ldq + g * a.Kg;
    uint32_t mx = 0;
#pragma unroll 4
    for (int64_t k = threadIdx.x * 8; k < a.Kg; k += QT * 8) mx = max8<IN>(mx, load8<IN, TAIL>(a.X, x0 + k, a.Kg - k));
    mx = wave_max(max_bits<IN>(mx));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
    __syncthreads();
    mx = max(max(red[0], red[1]), max(red[2], red[3]));
    float scale;
    const Step t = step_of(mx, scale);
    if (threadIdx.x == 0) a.scale[m * a.lds + g] = scale;
#pragma unroll 2
    for (int64_t k0 = 0; k0 < a.Kg; k0 += QT * 8) {       // whole wavefronts, for round8
        const int64_t k = k0 + threadIdx.x * 8;
        uint32_t v[8];
        widen8<IN>(load8<IN, TAIL>(a.X, x0 + k, a.Kg - k), v);
        const u32x2 q = round8(v, t);
        store8<TAIL>(a.Q + q0 + k, a.Kg - k, q);
    }
}

template <int IN, bool TAIL>
hipError_t launch_t(const QuantizeArgs &a, hipStream_t s) {
    const int64_t groups = a.M * a.G;
    const dim3 one((unsigned)groups), four((unsigned)((groups + 3) / 4)), block(QT), large(1024);
    // Long groups take sixteen wavefronts in place of four where they are few: us of 4
    // vs 16, bf16: 16 x 8192 5.5 vs 3.9, 256 x 4096 4.3 vs 3.8 (512: 4.6 vs 4.9), 512 x 8192
    // 7.3 vs 6.2 (1024: 10.6 vs 11.1), 512 x 14336 11.4 vs 9.0 (2048: 23.4 vs 25.5);
    // above 16384 columns always (16 x 28672 11.6 vs 6.5, 4096 x 28672 73.6 vs 71.1, fp32
    // 111.5 vs 106.9).
    const int64_t cus = device_cu_count();
    if (a.Kg <= 512) quantize_vec<IN, 1, 1, TAIL><<<four, block, 0, s>>>(a);
    else if (a.Kg <= 1024) quantize_vec<IN, 1, 2, TAIL><<<four, block, 0, s>>>(a);
    else if (a.Kg <= 2048) quantize_vec<IN, 1, 4, TAIL><<<four, block, 0, s>>>(a);
    else if (a.Kg <= 4096 && groups > cus) quantize_vec<IN, 4, 2, TAIL><<<one, block, 0, s>>>(a);
    else if (a.Kg <= 8192 && groups > 2 * cus) quantize_vec<IN, 4, 4, TAIL><<<one, block, 0, s>>>(a);
    else if (a.Kg <= 8192) quantize_vec<IN, 16, 1, TAIL><<<one, large, 0, s>>>(a);
    else if (a.Kg <= 16384 && groups > 2 * cus) quantize_vec<IN, 4, 8, TAIL><<<one, block, 0, s>>>(a);
    else if (a.Kg <= 16384) quantize_vec<IN, 16, 2, TAIL><<<one, large, 0, s>>>(a);
    else if (a.Kg <= 32768) quantize_vec<IN, 16, 4, TAIL><<<one, large, 0, s>>>(a);
    else quantize_long<IN, TAIL><<<one, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const QuantizeArgs &a, int in_type, hipStream_t s) {
    if (a.M == 0 || a.G == 0) return hipSuccess;
    // One launch has fewer than 2^32 threads: pieces of at most 2^21 groups.
    const int64_t most = (1 << 21) / a.G;
    for (int64_t m = 0; m < a.M; m += most) {
        QuantizeArgs b = a;
        b.M = a.M - m < most ? a.M - m : most;
        b.X = (const char *)a.X + m * a.ldx * (in_type == IN_BF16 ? 2 : 4);
        b.Q = a.Q + m * a.ldq;
        b.scale = a.scale + m * a.lds;
        const bool tail = a.Kg % 8 != 0;
        const hipError_t e = in_type == IN_BF16 ? (tail ? launch_t<IN_BF16, true>(b, s) : launch_t<IN_BF16, false>(b, s))
                                                : (tail ? launch_t<IN_F32, true>(b, s) : launch_t<IN_F32, false>(b, s));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tpl
