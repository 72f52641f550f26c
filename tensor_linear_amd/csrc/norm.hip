// The step between two blocks: the norm after a block, its gate, the residual sum and
// the norm before the next block, in one pass, and its gradients.
//   u = y r1 post, r1 = rsqrt(mean(y^2) + eps);  h = alpha R + beta g u;
//   n = h r2 pre,  r2 = rsqrt(mean(h^2) + eps)
// and backwards, with m = h r2, v = y r1:
//   dpre = sum_t dn m;  z = dn pre;  dh' = dh + r2 (z - m mean(z m));  dR = alpha dh';
//   dg = beta dh' u;  du = beta g dh';  dpost = sum_t du v;
//   dy = r1 (w - v mean(w v)), w = du post.
// All in fp32, h not rounded before its norm, one rounding to the output's type.
#include "heads_device.h"
#include "kernels.h"
#include "norm.h"
#include "quant_round.h"

namespace tpl {
namespace {

constexpr int NT = 256;

template <int ES>
__device__ __forceinline__ float at(const void *p, int64_t i) { return get1<ES>(p, i); }

// The sum, or the maximum, of a value of every thread.
template <int T>
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = lanes_sum(v, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) s += red[w];
    return s;
}
template <int T>
__device__ __forceinline__ uint32_t block_max(uint32_t v, float *red) {
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = __uint_as_float(v);
    __syncthreads();
    uint32_t s = __float_as_uint(red[0]);
#pragma unroll
    for (int w = 1; w < T / 64; ++w) s = max(s, __float_as_uint(red[w]));
    return s;
}

template <int ES>
struct RowOf {
    const NormArgs &a;
    int64_t t;
    float r1;
    __device__ __forceinline__ float y(int64_t i) const { return at<ES>(a.Y, t * a.ldy + i); }
    __device__ __forceinline__ float gate(int64_t i) const { return a.gate ? at<ES>(a.gate, t * a.ldg + i) : 1.0f; }
    __device__ __forceinline__ float u(int64_t i) const { return a.post ? y(i) * r1 * at<ES>(a.post, i) : y(i); }
    __device__ __forceinline__ float h(int64_t i) const {
        const float b = a.beta * gate(i) * u(i);
        return a.R ? __builtin_fmaf(a.alpha, at<ES>(a.R, t * a.ldr + i), b) : b;
    }
};

// Any length: a workgroup a row, read again for each sum.
template <int ES>
__global__ __launch_bounds__(NT)
void norm_any(NormArgs a, int64_t t0) {
    __shared__ float red[NT / 64];
    const int64_t t = t0 + blockIdx.x;
    RowOf<ES> row{a, t, 1.0f};
    if (a.post) {
        float s = 0.0f;
        for (int64_t i = threadIdx.x; i < a.F; i += NT) s = __builtin_fmaf(row.y(i), row.y(i), s);
        row.r1 = rsqrtf(block_sum<NT>(s, red) / (float)a.F + a.eps);
    }
    float r2 = 1.0f;
    if (a.pre && a.N) {
        float s = 0.0f;
        for (int64_t i = threadIdx.x; i < a.F; i += NT) s = __builtin_fmaf(row.h(i), row.h(i), s);
        r2 = rsqrtf(block_sum<NT>(s, red) / (float)a.F + a.eps);
    }
    auto n = [&](int64_t i) { return a.pre ? row.h(i) * r2 * at<ES>(a.pre, i) : row.h(i); };
    Step st{};
    if (a.scale) {
        uint32_t m = 0;
        for (int64_t i = threadIdx.x; i < a.F; i += NT) m = max(m, __float_as_uint(n(i)) & 0x7FFFFFFFu);
        float scale;
        st = step_of(block_max<NT>(m, red), scale);
        if (threadIdx.x == 0) a.scale[t] = scale;
    }
    for (int64_t i = threadIdx.x; i < a.F; i += NT) {
        if (a.H) put1<ES>(a.H, t * a.ldh + i, row.h(i));
        if (a.scale) ((int8_t *)a.N)[t * a.ldn + i] = (int8_t)round_one(__float_as_uint(n(i)), st);
        else if (a.N) put1<ES>(a.N, t * a.ldn + i, n(i));
    }
}

// Any length: a workgroup's rows one after another, its sums in its part of the
// workspace.
template <int ES>
__global__ __launch_bounds__(NT)
void norm_backward_any(NormArgs a) {
    __shared__ float red[NT / 64];
    const bool sum_gate = a.dgate && a.ldg == 0;
    float *part = a.partials ? a.partials + (int64_t)blockIdx.x * 3 * a.F : nullptr;
    bool first = true;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, first = false) {
        RowOf<ES> row{a, t, 1.0f};
        if (a.post) {
            float s = 0.0f;
            for (int64_t i = threadIdx.x; i < a.F; i += NT) s = __builtin_fmaf(row.y(i), row.y(i), s);
            row.r1 = rsqrtf(block_sum<NT>(s, red) / (float)a.F + a.eps);
        }
        auto dn = [&](int64_t i) { return a.dN ? at<ES>(a.dN, t * a.lddn + i) : 0.0f; };
        auto z = [&](int64_t i) { return a.pre ? dn(i) * at<ES>(a.pre, i) : dn(i); };
        float r2 = 1.0f, mean = 0.0f;
        if (a.pre && a.dN) {
            float s = 0.0f, d = 0.0f;
            for (int64_t i = threadIdx.x; i < a.F; i += NT) {
                const float h = row.h(i);
                s = __builtin_fmaf(h, h, s);
                d = __builtin_fmaf(z(i), h, d);
            }
            r2 = rsqrtf(block_sum<NT>(s, red) / (float)a.F + a.eps);
            mean = block_sum<NT>(d, red) * r2 / (float)a.F;
        }
        auto dh = [&](int64_t i) {
            float g = a.dH ? at<ES>(a.dH, t * a.lddh + i) : 0.0f;
            if (a.dN) g += a.pre ? r2 * (z(i) - row.h(i) * r2 * mean) : dn(i);
            return g;
        };
        float mean1 = 0.0f;
        if (a.post && a.dY) {
            float d = 0.0f;
            for (int64_t i = threadIdx.x; i < a.F; i += NT)
                d = __builtin_fmaf(a.beta * row.gate(i) * dh(i) * at<ES>(a.post, i), row.y(i) * row.r1, d);
            mean1 = block_sum<NT>(d, red) / (float)a.F;
        }
        for (int64_t i = threadIdx.x; i < a.F; i += NT) {
            const float g = dh(i), du = a.beta * row.gate(i) * g, v = row.y(i) * row.r1;
            const float dg = a.beta * g * row.u(i);
            if (a.dR) put1<ES>(a.dR, t * a.lddr + i, a.alpha * g);
            if (a.dY) put1<ES>(a.dY, t * a.lddy + i, a.post ? row.r1 * (du * at<ES>(a.post, i) - v * mean1) : du);
            if (a.dgate && !sum_gate) put1<ES>(a.dgate, t * a.lddg + i, dg);
            if (part) {
                if (sum_gate) part[i] = (first ? 0.0f : part[i]) + dg;
                if (a.dpost) part[a.F + i] = (first ? 0.0f : part[a.F + i]) + du * v;
                if (a.dpre) part[2 * a.F + i] = (first ? 0.0f : part[2 * a.F + i]) + dn(i) * row.h(i) * r2;
            }
        }
    }
}

// ---- rows in registers ----------------------------------------------------------

// The values i + e of the first F, e < 8, raw; the rest zeros.
template <int ES, bool TAIL>
__device__ __forceinline__ Raw8<ES> row8(const void *p, int64_t base, int i, int F) {
    Raw8<ES> r = {};
    if (i >= F) return r;
    if (!TAIL || i + 8 <= F) return raw8<ES, false>(p, base + i, 0, 4);
#pragma unroll
    for (int e = 0; e < 7; ++e) {
        if (i + e >= F) break;
        if constexpr (ES == 2) r.w[0][e / 2] |= (uint32_t)((const uint16_t *)p)[base + i + e] << (16 * (e & 1));
        else r.w[e / 4][e % 4] = ((const uint32_t *)p)[base + i + e];
    }
    return r;
}
template <int ES, bool TAIL>
__device__ __forceinline__ void put_row8(void *p, int64_t base, int i, int F, const float *v) {
    if (i >= F) return;
    if (!TAIL || i + 8 <= F) {
        put8<ES, false>(p, base + i, 0, 4, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (i + e < F) put1<ES>(p, base + i + e, v[e]);
}

// The sums of N values over the W wavefronts of a row; `red` alternates between two
// parts, so that one barrier a sum is enough.  Rows of one wavefront need none.
template <int W, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[16][2], int &turn) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = lanes_sum(v[n], 64);
    if constexpr (W > 1) {
        const int wave = threadIdx.x >> 6, group = wave / W * W;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) red[turn][wave][n] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = red[turn][group][n];
#pragma unroll
            for (int w = 1; w < W; ++w) s += red[turn][group + w][n];
            v[n] = s;
        }
        turn ^= 1;
    }
}
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float (*red)[16][2], int &turn) {
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    if constexpr (W > 1) {
        const int wave = threadIdx.x >> 6, group = wave / W * W;
        if ((threadIdx.x & 63) == 0) red[turn][wave][0] = __uint_as_float(v);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) v = max(v, __float_as_uint(red[turn][group + w][0]));
        turn ^= 1;
    }
    return v;
}

// W wavefronts a row (1: four rows a workgroup), C chunks of 8 values a lane.  All of a
// row's loads leave at once and its values stay in registers between the sums: each byte
// moves once, at the rate of a copy (4096 x 8192 bf16 with both norms and a gate 53 us, 5.0
// TB/s; 16 x 8192 into 8 bits 5 us, the latency of two sums over 16 wavefronts).
template <int ES, int W, int C, bool TAIL>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64)
void norm_rows(NormArgs a, int64_t t0) {
    __shared__ float red[2][16][2];
    int turn = 0;
    const int64_t t = W == 1 ? t0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : t0 + blockIdx.x;
    if (W == 1 && t >= a.T) return;
    const int F = (int)a.F, lane = W == 1 ? threadIdx.x & 63 : threadIdx.x;
    constexpr int STEP = W * 512;
    Raw8<ES> y[C], r[C], g[C], wp[C], wn[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = c * STEP + lane * 8;
        y[c] = row8<ES, TAIL>(a.Y, t * a.ldy, i, F);
        if (a.R) r[c] = row8<ES, TAIL>(a.R, t * a.ldr, i, F);
        if (a.post) wp[c] = row8<ES, TAIL>(a.post, 0, i, F);
        if (a.gate) g[c] = row8<ES, TAIL>(a.gate, t * a.ldg, i, F);
        if (a.pre) wn[c] = row8<ES, TAIL>(a.pre, 0, i, F);
    }
    float r1 = 1.0f;
    if (a.post) {
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[8];
            widen8<ES>(y[c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(v[e], v[e], s[0]);
        }
        row_sum<W, 1>(s, red, turn);
        r1 = rsqrtf(s[0] / (float)F + a.eps);
    }
    float h[C][8], s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float v[8];
        widen8<ES>(y[c], h[c]);
        if (a.post) {
            widen8<ES>(wp[c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] = h[c][e] * r1 * v[e];
        }
        if (a.gate) {
            widen8<ES>(g[c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] = a.beta * v[e] * h[c][e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] = a.beta * h[c][e];
        }
        if (a.R) {
            widen8<ES>(r[c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] = __builtin_fmaf(a.alpha, v[e], h[c][e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(h[c][e], h[c][e], s[0]);
        if (a.H) put_row8<ES, TAIL>(a.H, t * a.ldh, c * STEP + lane * 8, F, h[c]);
    }
    if (!a.N && !a.scale) return;       // rows of no features may have a scale alone
    if (a.pre) {
        row_sum<W, 1>(s, red, turn);
        const float r2 = rsqrtf(s[0] / (float)F + a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[8];
            widen8<ES>(wn[c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] = h[c][e] * r2 * v[e];
        }
    }
    if (!a.scale) {
#pragma unroll
        for (int c = 0; c < C; ++c) put_row8<ES, TAIL>(a.N, t * a.ldn, c * STEP + lane * 8, F, h[c]);
        return;
    }
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e)     // nothing past the row's end, whatever its factors
            if (c * STEP + lane * 8 + (TAIL ? e : 0) < F) m = max(m, __float_as_uint(h[c][e]) & 0x7FFFFFFFu);
    float scale;
    const Step st = step_of(row_max<W>(m, red, turn), scale);
    if (lane == 0) a.scale[t] = scale;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = c * STEP + lane * 8;
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(h[c][e]);
        const u32x2 q = round8(u, st);      // every lane takes part
        int8_t *p = (int8_t *)a.N + t * a.ldn + i;
        if (i + 8 <= F) {
            *(u32x2_any *)p = q;
        } else if (TAIL) {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (i + e < F) p[e] = (int8_t)(q[e / 4] >> (8 * (e & 3)));
        }
    }
}

// Gradients, bound by latency and HBM: two wavefronts a SIMD, whose registers hold the
// weights widened and the sums, with three sums over the row one after another (4096 x
// 4096 bf16 with both norms and a gate 52 us with the second launch, 3.9 TB/s; 8192 x 2048
// 49; 2048 x 8192 64).  G groups of W wavefronts a workgroup, each with rows of its own one after
// another; the next row's values are loaded while the current ones are worked on.  The
// features' sums of a lane stay in registers; at the end the groups' are added in LDS in
// order and leave as the workgroup's part of the workspace, which a second kernel adds in
// an order of its own: the result does not depend on scheduling.
// Rows that no 8 divides load their last chunk value by value, each waited for before the
// next, the row ahead with it: 4096 x 4093 122 us for 4096 x 4096's 52.  Past 8192 features
// 16 wavefronts leave 128 registers a lane, 35 to 88 too few: 1024 x 16384 104 us.
template <int ES, int W, int G, int C, bool AHEAD, bool LONG, bool TAIL>
__global__ __launch_bounds__(W * G * 64)
void norm_backward_rows(NormArgs a) {
    constexpr int STEP = W * 512;
    __shared__ float red[2][16][2];
    __shared__ __attribute__((aligned(16))) float sums[G > 1 || LONG ? W * 512 * C * (LONG ? 2 : 1) : 1];
    int turn = 0;
    const int F = (int)a.F, group = threadIdx.x / (W * 64), lane = threadIdx.x % (W * 64);
    const bool sum_gate = a.dgate && a.ldg == 0;
    struct Vals { Raw8<ES> y[C], r[C], dh[C], dn[C], g[C]; };
    auto load = [&](int64_t t) {
        Vals v = {};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = c * STEP + lane * 8;
            v.y[c] = row8<ES, TAIL>(a.Y, t * a.ldy, i, F);
            if (a.R) v.r[c] = row8<ES, TAIL>(a.R, t * a.ldr, i, F);
            if (a.dH) v.dh[c] = row8<ES, TAIL>(a.dH, t * a.lddh, i, F);
            if (a.dN) v.dn[c] = row8<ES, TAIL>(a.dN, t * a.lddn, i, F);
            if (a.gate && a.ldg) v.g[c] = row8<ES, TAIL>(a.gate, t * a.ldg, i, F);
        }
        return v;
    };
    // the weights, and the gate with the branch's factor
    // (LONG: loaded again for each row, and the weights' sums are in LDS)
    constexpr int CK = LONG ? 1 : C;
    float wp_[CK][8], wn_[CK][8], wg_[CK][8], dg[C][8] = {}, dp[CK][8] = {}, dw[CK][8] = {};
    auto weight = [&](const void *w, int c, float *v) {
        Raw8<ES> p = {};
        if (w) p = row8<ES, TAIL>(w, 0, c * STEP + lane * 8, F);
        widen8<ES>(p, v);
    };
    auto gates = [&](const Raw8<ES> *g, int c, float *v) {
        if (a.gate && a.ldg) widen8<ES>(g[c], v);
        else weight(a.gate, c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = a.gate ? a.beta * v[e] : a.beta;
    };
    if constexpr (LONG) {
        for (int i = threadIdx.x; i < 2 * W * 512 * C; i += W * G * 64) sums[i] = 0.0f;      // each lane its own, below
        __syncthreads();
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            weight(a.post, c, wp_[c]);
            weight(a.pre, c, wn_[c]);
            if (!(a.gate && a.ldg)) gates(nullptr, c, wg_[c]);
        }
    }
    auto get = [&](const float (&kept)[CK][8], const void *w, int c, float *v) __attribute__((always_inline)) {
        if constexpr (LONG) weight(w, c, v);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = kept[c][e];
    };
    // adds to the sums of a weight's gradient
    auto add = [&](float (&kept)[CK][8], int kind, int c, const float *v) __attribute__((always_inline)) {
        if constexpr (LONG) {
            typedef float f32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f32x4 *p = (f32x4 *)sums + (kind * C * 2 + c * 2 + q) * W * 64 + lane;
                f32x4 x = *p;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] += v[4 * q + e];
                *p = x;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) kept[c][e] += v[e];
        }
    };
    const float inv_f = 1.0f / (float)F;
    const int64_t step = (int64_t)gridDim.x * G;
    int64_t t = (int64_t)blockIdx.x * G + group;
    Vals next = {};
    if (AHEAD && t < a.T) next = load(t);
    // every group takes part in every barrier: as many rounds for all
    for (int64_t t_all = (int64_t)blockIdx.x * G; t_all < a.T; t_all += step, t += step) {
        const bool on = t < a.T;
        Vals cur = next;
        if (!AHEAD && on) cur = load(t);
        if (AHEAD) next = t + step < a.T ? load(t + step) : Vals{};
        float r1 = 1.0f;
        if (a.post) {
            float s[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float v[8];
                widen8<ES>(cur.y[c], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(v[e], v[e], s[0]);
            }
            row_sum<W, 1>(s, red, turn);
            r1 = rsqrtf(s[0] * inv_f + a.eps);
        }
        if constexpr (!LONG)
            if (a.gate && a.ldg)
#pragma unroll
                for (int c = 0; c < C; ++c) gates(cur.g, c, wg_[c]);
        auto gate_of = [&](int c, float *v) __attribute__((always_inline)) {
            if constexpr (LONG) gates(cur.g, c, v);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = wg_[c][e];
        };
        float h[C][8], x[C][8], sd[2] = {0.0f, 0.0f};      // h; z = dn pre
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[8];
            widen8<ES>(cur.y[c], h[c]);
            if (a.post) {
                get(wp_, a.post, c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[c][e] = h[c][e] * r1 * v[e];
            }
            gate_of(c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[c][e] = v[e] * h[c][e];
            if (a.R) {
                widen8<ES>(cur.r[c], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[c][e] = __builtin_fmaf(a.alpha, v[e], h[c][e]);
            }
            widen8<ES>(cur.dn[c], x[c]);
            if (a.pre) {
                get(wn_, a.pre, c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[c][e] *= v[e];
                    sd[0] = __builtin_fmaf(h[c][e], h[c][e], sd[0]);
                    sd[1] = __builtin_fmaf(x[c][e], h[c][e], sd[1]);
                }
            }
        }
        const bool normed = a.pre && a.dN;
        float r2 = 1.0f, mean = 0.0f;
        if (normed) {
            row_sum<W, 2>(sd, red, turn);
            r2 = rsqrtf(sd[0] * inv_f + a.eps);
            mean = sd[1] * r2 * inv_f;
        }
        // the gradient of h in x; then of u
        float dot[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = c * STEP + lane * 8;
            float v[8], out[8];
            if (normed) {
                widen8<ES>(cur.dn[c], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float m = h[c][e] * r2;
                    out[e] = v[e] * m;
                    x[c][e] = r2 * (x[c][e] - m * mean);
                }
                if (on) add(dw, 1, c, out);
            }
            widen8<ES>(cur.dh[c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[c][e] += v[e];
            if (a.dR && on) {
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] = a.alpha * x[c][e];
                put_row8<ES, TAIL>(a.dR, t * a.lddr, i, F, out);
            }
            float n[8];            // y r1
            widen8<ES>(cur.y[c], n);
            if (a.post)
#pragma unroll
                for (int e = 0; e < 8; ++e) n[e] *= r1;
            get(wp_, a.post, c, v);
            if (a.dgate) {
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] = a.beta * x[c][e] * (a.post ? n[e] * v[e] : n[e]);
                if (!sum_gate) {
                    if (on) put_row8<ES, TAIL>(a.dgate, t * a.lddg, i, F, out);
                } else if (on) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dg[c][e] += out[e];
                }
            }
            float w[8];
            gate_of(c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[c][e] *= w[e];
            if (a.post) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    out[e] = x[c][e] * n[e];
                    x[c][e] *= v[e];
                    dot[0] = __builtin_fmaf(x[c][e], n[e], dot[0]);
                }
                if (on) add(dp, 0, c, out);
            }
        }
        if (a.post && a.dY) row_sum<W, 1>(dot, red, turn);
        if (a.dY && on) {
            const float mean1 = dot[0] * inv_f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (a.post) {
                    float n[8];
                    widen8<ES>(cur.y[c], n);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[c][e] = r1 * (x[c][e] - n[e] * r1 * mean1);
                }
                put_row8<ES, TAIL>(a.dY, t * a.lddy, c * STEP + lane * 8, F, x[c]);
            }
        }
    }
    if (!a.partials) return;
    float *part = a.partials + (int64_t)blockIdx.x * 3 * F;
    auto leave = [&](bool wanted, auto &v, int kind) {
        if (!wanted) return;
        constexpr bool IN_LDS = LONG && sizeof(v) != sizeof(dg);     // the weights' sums, not the gate's
        if constexpr (IN_LDS) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = sums[(((kind - 1) * C * 2 + c * 2 + e / 4) * W * 64 + lane) * 4 + e % 4];
                put_row8<4, TAIL>(part, (int64_t)kind * F, c * STEP + lane * 8, F, x);
            }
            return;
        }
        if constexpr (G > 1) {
            for (int g = 1; g < G; ++g) {
                __syncthreads();
                if (group == g)
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int e = 0; e < 8; ++e) sums[(c * 8 + e) * W * 64 + lane] = v[c][e];
                __syncthreads();
                if (group == 0)
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[c][e] += sums[(c * 8 + e) * W * 64 + lane];
            }
        }
        if constexpr (!IN_LDS)
            if (group == 0)
#pragma unroll
                for (int c = 0; c < C; ++c) put_row8<4, TAIL>(part, (int64_t)kind * F, c * STEP + lane * 8, F, v[c]);
    };
    leave(sum_gate, dg, 0);
    leave(a.dpost != nullptr, dp, 1);
    leave(a.dpre != nullptr, dw, 2);
}

// out[kind][i] = sum over blocks of partials[block][kind][i]: 64 columns by 16 strands of
// blocks a workgroup (256 bytes of a block at a time), each strand in block order, then
// the strands in order.
__global__ __launch_bounds__(NT)
void norm_grad_sum(const float *partials, int64_t blocks, int64_t F, float *dgate, float *dpost, float *dpre) {
    __shared__ float red[16][64];
    float *out = blockIdx.y == 0 ? dgate : blockIdx.y == 1 ? dpost : dpre;
    if (!out) return;
    const int q = threadIdx.x & 15, strand = threadIdx.x >> 4;
    const int64_t col = (int64_t)blockIdx.x * 64 + q * 4;
    float s[4] = {};
    const float *p = partials + blockIdx.y * F + col;
    if (col + 4 <= F) {
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll 8
        for (int64_t b = strand; b < blocks; b += 16) {
            const f32x4_any v = *(const f32x4_any *)(p + b * 3 * F);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += v[e];
        }
    } else {
        for (int e = 0; e < 4 && col + e < F; ++e)
            for (int64_t b = strand; b < blocks; b += 16) s[e] += p[b * 3 * F + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) red[strand][q * 4 + e] = s[e];
    __syncthreads();
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x < 64 && i < F) {
        float v = red[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < 16; ++k) v += red[k][threadIdx.x];
        out[i] = v;
    }
}

template <int ES, bool TAIL>
void launch_rows(const NormArgs &a, int64_t t0, int64_t n, hipStream_t s) {
    NormArgs b = a;
    b.T = t0 + n;
    const dim3 four((unsigned)((n + 3) / 4)), one((unsigned)n);
    const int64_t F = a.F;
    if (F <= 512) norm_rows<ES, 1, 1, TAIL><<<four, dim3(256), 0, s>>>(b, t0);
    else if (F <= 1024) norm_rows<ES, 1, 2, TAIL><<<four, dim3(256), 0, s>>>(b, t0);
    else if (F <= 2048) norm_rows<ES, 4, 1, TAIL><<<one, dim3(256), 0, s>>>(b, t0);
    else if (F <= 4096) norm_rows<ES, 4, 2, TAIL><<<one, dim3(256), 0, s>>>(b, t0);
    else if (F <= 8192 && n > 512) norm_rows<ES, 8, 2, TAIL><<<one, dim3(512), 0, s>>>(b, t0);
    else if (F <= 8192) norm_rows<ES, 16, 1, TAIL><<<one, dim3(1024), 0, s>>>(b, t0);
    else if (F <= 16384) norm_rows<ES, 16, 2, TAIL><<<one, dim3(1024), 0, s>>>(b, t0);
    else norm_any<ES><<<one, dim3(NT), 0, s>>>(b, t0);
}

template <int ES>
hipError_t launch_fwd(const NormArgs &a, hipStream_t s) {
    const int64_t most = 1 << 21;   // one launch has fewer than 2^32 threads
    for (int64_t t = 0; t < a.T; t += most) {
        const int64_t n = a.T - t < most ? a.T - t : most;
        if (a.F % 8) launch_rows<ES, true>(a, t, n, s);
        else launch_rows<ES, false>(a, t, n, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// blocks: the most workgroups; what the launch has of them.
template <int ES, bool TAIL>
void launch_backward(const NormArgs &a, int64_t &blocks, hipStream_t s) {
    const int64_t F = a.F;
    auto fit = [&](int g) {
        if (blocks > (a.T + g - 1) / g) blocks = (a.T + g - 1) / g;
        return dim3((unsigned)blocks);
    };
    if (F <= 512) norm_backward_rows<ES, 1, 8, 1, true, false, TAIL><<<fit(8), dim3(512), 0, s>>>(a);
    else if (F <= 1024) norm_backward_rows<ES, 2, 4, 1, true, false, TAIL><<<fit(4), dim3(512), 0, s>>>(a);
    else if (F <= 2048) norm_backward_rows<ES, 4, 2, 1, true, false, TAIL><<<fit(2), dim3(512), 0, s>>>(a);
    else if (F <= 4096) norm_backward_rows<ES, 8, 1, 1, true, false, TAIL><<<fit(1), dim3(512), 0, s>>>(a);
    else if (F <= 8192) norm_backward_rows<ES, 8, 1, 2, false, false, TAIL><<<fit(1), dim3(512), 0, s>>>(a);
    else if (F <= 16384) norm_backward_rows<ES, 16, 1, 2, false, true, TAIL><<<fit(1), dim3(1024), 0, s>>>(a);
    else norm_backward_any<ES><<<fit(1), dim3(NT), 0, s>>>(a);
}

template <int ES>
hipError_t launch_bwd(const NormArgs &a, hipStream_t s) {
    int64_t blocks = a.T == 0 ? 0 : norm_backward_blocks(a.T, a.F);
    if (blocks) {
        if (a.F % 8) launch_backward<ES, true>(a, blocks, s);
        else launch_backward<ES, false>(a, blocks, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.partials) return e;
    norm_grad_sum<<<dim3((unsigned)((a.F + 63) / 64), 3), dim3(NT), 0, s>>>(a.partials, blocks, a.F, a.ldg == 0 ? (float *)a.dgate : nullptr, a.dpost, a.dpre);
    return hipGetLastError();
}

}  // namespace

// One on each of 256 CUs, which the registers allow (with twice as many half of them wait,
// and leave twice the sums: 4096 x 4096 bf16 62 us for 54); not taken from the device: the
// workspace's size and the order of the sums depend on the call's sizes alone.
int64_t norm_backward_blocks(int64_t T, int64_t) { return T < 1 ? 1 : T < 256 ? T : 256; }

hipError_t launch_residual_norm(const NormArgs &a, int es, hipStream_t s) {
    return es == 2 ? launch_fwd<2>(a, s) : launch_fwd<4>(a, s);
}

hipError_t launch_residual_norm_backward(const NormArgs &a, int es, hipStream_t s) {
    return es == 2 ? launch_bwd<2>(a, s) : launch_bwd<4>(a, s);
}

}  // namespace tpl
