// Rows of a paged cache as matrices: the row at each token's position, its heads'
// keys and values side by side; from a cache in 8 bits x = q s, one rounding.
// Bound by memory, each value read and written once: a wavefront for 256 chunks of 8
// values of a token, four a lane, all loaded before the first is stored, since a token's
// sequence, page and row are five loads one after another and a chunk at a time leaves too
// little under way.  12 sequences of 24000 tokens, 8 + 8 heads of 128, from int8 to bf16:
// 35 us, 4.2 TB/s (a chunk a lane: 50).
#include "attn_device.h"
#include "kernels.h"

namespace tpl {
namespace {

typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int RT = 256, AT_ONCE = 4;

// E values a lane, 8 or 1 where D is no multiple of 8: as they lie in the cache, and out.
template <int ES, int CS, int E>
struct Piece {
    uint32_t w[E == 1 ? 1 : E * CS / 4];
    __device__ __forceinline__ void load(const void *src, int64_t i) {
        if constexpr (E == 1) {
            w[0] = __float_as_uint(cached<CS>(src, i));
        } else if constexpr (CS == 1) {
            const u32x2_any q = *(const u32x2_any *)((const int8_t *)src + i);
            w[0] = q[0]; w[1] = q[1];
        } else {
#pragma unroll
            for (int k = 0; k < CS / 2; ++k) {
                const u32x4_any q = *(const u32x4_any *)((const char *)src + i * CS + 16 * k);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[4 * k + e] = q[e];
            }
        }
    }
    __device__ __forceinline__ void store_to(void *dst, int64_t o, float scale, bool ok) const {
        if constexpr (E == 1) {
            store<ES>(dst, o, ok ? __uint_as_float(w[0]) * (CS == 1 ? scale : 1.0f) : 0.0f);
        } else if constexpr (CS == 1) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = ok ? (float)((int32_t)(w[e / 4] << (24 - 8 * (e & 3))) >> 24) * scale : 0.0f;
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
            for (int k = 0; k < CS / 2; ++k) {
                u32x4 q;
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = ok ? w[4 * k + e] : 0;
                *(u32x4_any *)((char *)dst + o * CS + 16 * k) = q;
            }
        }
    }
};

// A wavefront for part `w % parts` of a token's pieces: keys first, then values.  Its lanes
// load AT_ONCE pieces before they store the first.
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
    // (a sequence that begins before the call's first row may have positions past 32 bits)
    if (p >= 0 && p < 0xFFFFFFFF) r = row_of(a.c, a.c.table + s * a.c.ldt, (uint32_t)p);
    const bool ok = r.page >= 0;
    if (!ok && a.c.bad && lane == 0) *a.c.bad = 1;
    const int64_t row = r.page * a.c.s_page + r.slot * a.c.s_slot;
    const int64_t srow = r.page * a.c.ss_page + r.slot * a.c.ss_slot;
    const uint32_t per = a.c.D / E;
    const int n = a.c.Hkv * per, all = (a.K ? n : 0) + (a.V ? n : 0);
    for (int i0 = (int)(w - t * parts) * 64 * AT_ONCE + lane; i0 < all; i0 += parts * 64 * AT_ONCE) {
        Piece<ES, CS, E> x[AT_ONCE] = {};
        float scale[AT_ONCE] = {};
        int64_t o[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int i = i0 + 64 * k;
            const bool val = !a.K || i >= n;
            const uint32_t j = a.K && val ? i - n : i, h = j / per, d = (j - h * per) * E;
            o[k] = t * (val ? a.ldv : a.ldk) + (int64_t)h * a.c.D + d;
            if (i >= all || !ok) continue;
            if (CS == 1) scale[k] = (val ? a.c.vs : a.c.ks)[srow + h * a.c.ss_head];
            x[k].load(val ? a.c.vc : a.c.kc, row + h * a.c.s_head + d);
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int i = i0 + 64 * k;
            if (i < all) x[k].store_to(!a.K || i >= n ? a.V : a.K, o[k], scale[k], ok);
        }
    }
}

template <int ES, int CS, int E>
hipError_t launch(const ReadArgs &a, hipStream_t s) {
    const int64_t chunks = (int64_t)a.c.Hkv * (a.c.D / E) * ((a.K ? 1 : 0) + (a.V ? 1 : 0));
    const int parts = (int)((chunks + 64 * AT_ONCE - 1) / (64 * AT_ONCE));
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
