// Rows of a paged cache as matrices: the row at each token's position, its heads'
// keys and values side by side; from a cache in 8 bits x = q s, one rounding.
// Bound by memory, each value read and written once: a wavefront for 64 chunks of 8
// values of a token.
#include "attn_device.h"
#include "kernels.h"

namespace tpl {
namespace {

typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int RT = 256;

// E values a lane: 8, or 1 where D is no multiple of 8.
template <int ES, int CS, int E>
__device__ __forceinline__ void copy_row(const void *src, int64_t i, float scale, bool ok, void *dst, int64_t o) {
    if constexpr (E == 1) {
        store<ES>(dst, o, ok ? cached<CS>(src, i) * (CS == 1 ? scale : 1.0f) : 0.0f);
    } else if constexpr (CS == 1) {
        u32x2_any q = {0, 0};
        if (ok) q = *(const u32x2_any *)((const int8_t *)src + i);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)((int32_t)(q[e / 4] << (24 - 8 * (e & 3))) >> 24) * scale;
        if constexpr (ES == 2) {
            bf16x8 h;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = (__bf16)v[e];
            *(u32x4_any *)((char *)dst + o * 2) = __builtin_bit_cast(u32x4, h);
        } else {
            u32x4 x, y;
#pragma unroll
            for (int e = 0; e < 4; ++e) { x[e] = __float_as_uint(v[e]); y[e] = __float_as_uint(v[4 + e]); }
            *(u32x4_any *)((char *)dst + o * 4) = x;
            *(u32x4_any *)((char *)dst + o * 4 + 16) = y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < ES / 2; ++k) {
            u32x4_any q = {0, 0, 0, 0};
            if (ok) q = *(const u32x4_any *)((const char *)src + i * ES + 16 * k);
            *(u32x4_any *)((char *)dst + o * ES + 16 * k) = q;
        }
    }
}

// A wavefront for part `w % parts` of a token's chunks: keys first, then values.
template <int ES, int CS, int E>
__global__ __launch_bounds__(RT)
void read_rows(ReadArgs a, int64_t w0, int64_t waves, int parts) {
    const int lane = threadIdx.x & 63;
    const int64_t w = w0 + (int64_t)blockIdx.x * (RT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (w >= waves) return;
    const int64_t t = w / parts;
    const int64_t s = sequence_of(a.c, t, lane);
    if (s < 0) return;
    const int64_t p = (int64_t)a.c.past[s] + (t - a.c.cu[s]);
    Row r{-1, 0};
    if (p >= 0) r = row_of(a.c, a.c.table + s * a.c.ldt, (uint32_t)p);
    const bool ok = r.page >= 0;
    if (!ok && a.c.bad && lane == 0) *a.c.bad = 1;
    const int64_t row = r.page * a.c.s_page + r.slot * a.c.s_slot;
    const int64_t srow = r.page * a.c.ss_page + r.slot * a.c.ss_slot;
    const int per = a.c.D / E, n = a.c.Hkv * per, all = (a.K ? n : 0) + (a.V ? n : 0);
    for (int i = (int)(w - t * parts) * 64 + lane; i < all; i += parts * 64) {
        const bool val = !a.K || i >= n;
        const int j = a.K && val ? i - n : i;
        const int h = j / per, d = (j - h * per) * E;
        float scale = 0.0f;
        if (CS == 1 && ok) scale = (val ? a.c.vs : a.c.ks)[srow + h * a.c.ss_head];
        copy_row<ES, CS, E>(val ? a.c.vc : a.c.kc, row + h * a.c.s_head + d, scale, ok, val ? a.V : a.K,
                            t * (val ? a.ldv : a.ldk) + (int64_t)h * a.c.D + d);
    }
}

template <int ES, int CS, int E>
hipError_t launch(const ReadArgs &a, hipStream_t s) {
    const int64_t chunks = (int64_t)a.c.Hkv * (a.c.D / E) * ((a.K ? 1 : 0) + (a.V ? 1 : 0));
    const int parts = (int)((chunks + 63) / 64);
    const int64_t waves = a.c.T * parts, most = 1 << 25;   // one launch has fewer than 2^32 threads
    for (int64_t w = 0; w < waves; w += most) {
        const int64_t n = waves - w < most ? waves - w : most;
        read_rows<ES, CS, E><<<dim3((unsigned)((n + RT / 64 - 1) / (RT / 64))), dim3(RT), 0, s>>>(a, w, w + n, parts);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int ES, int CS>
hipError_t launch_e(const ReadArgs &a, hipStream_t s) {
    return a.c.D % 8 ? launch<ES, CS, 1>(a, s) : launch<ES, CS, 8>(a, s);
}

}  // namespace

hipError_t launch_kv_read(const ReadArgs &a, int es, hipStream_t s) {
    if (a.c.ks || a.c.vs) return es == 2 ? launch_e<2, 1>(a, s) : launch_e<4, 1>(a, s);
    return es == 2 ? launch_e<2, 2>(a, s) : launch_e<4, 4>(a, s);
}

}  // namespace tpl
