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

// out[kind][i] = sum over blocks of partials[block][kind][i]: four columns by 64 strands
// of blocks a workgroup, each strand in block order, then the strands in a tree.
__global__ __launch_bounds__(NT)
void norm_grad_sum(const float *partials, int64_t blocks, int64_t F, float *dgate, float *dpost, float *dpre) {
    __shared__ float red[4][64];
    const int c = threadIdx.x & 3, strand = threadIdx.x >> 2;
    const int64_t col = (int64_t)blockIdx.x * 4 + c;
    const int kind = blockIdx.y;
    float *out = kind == 0 ? dgate : kind == 1 ? dpost : dpre;
    if (!out) return;
    float s = 0.0f;
    if (col < F) {
        const float *p = partials + kind * F + col;
#pragma unroll 4
        for (int64_t b = strand; b < blocks; b += 64) s += p[b * 3 * F];
    }
    red[c][strand] = s;
    __syncthreads();
    const int lane = threadIdx.x & 63, k = threadIdx.x >> 6;
    const int64_t i = (int64_t)blockIdx.x * 4 + k;
    const float v = lanes_sum(red[k][lane], 64);
    if (lane == 0 && i < F) out[i] = v;
}

template <int ES>
hipError_t launch_fwd(const NormArgs &a, hipStream_t s) {
    const int64_t most = 1 << 21;   // one launch has fewer than 2^32 threads
    for (int64_t t = 0; t < a.T; t += most) {
        const int64_t n = a.T - t < most ? a.T - t : most;
        norm_any<ES><<<dim3((unsigned)n), dim3(NT), 0, s>>>(a, t);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int ES>
hipError_t launch_bwd(const NormArgs &a, hipStream_t s) {
    int64_t blocks = norm_backward_blocks(a.T, a.F);
    if (a.T == 0) blocks = 0;
    if (blocks) norm_backward_any<ES><<<dim3((unsigned)blocks), dim3(NT), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.partials) return e;
    norm_grad_sum<<<dim3((unsigned)((a.F + 3) / 4), 3), dim3(NT), 0, s>>>(a.partials, blocks, a.F, a.ldg == 0 ? (float *)a.dgate : nullptr, a.dpost, a.dpre);
    return hipGetLastError();
}

}  // namespace

int64_t norm_backward_blocks(int64_t T, int64_t) { return T < 1 ? 1 : T < 1024 ? T : 1024; }

hipError_t launch_residual_norm(const NormArgs &a, int es, hipStream_t s) {
    return es == 2 ? launch_fwd<2>(a, s) : launch_fwd<4>(a, s);
}

hipError_t launch_residual_norm_backward(const NormArgs &a, int es, hipStream_t s) {
    return es == 2 ? launch_bwd<2>(a, s) : launch_bwd<4>(a, s);
}

}  // namespace tpl
