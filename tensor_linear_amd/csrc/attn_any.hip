// Attention of new tokens over a paged cache, for any head size, type, strides and
// alignment: a wavefront for each row and query head walks the keys it sees, 64 at a
// time, with the softmax's running maximum and sum:
//   m' = max(m, max_j x_j),  c = exp(m - m'),  l' = c l + sum_j exp(x_j - m'),
//   o' = c o + sum_j exp(x_j - m') v_j;   at the end O = o / l, lse = m + log l.
// A lane takes a key for the products with the query and D / 64 features for the
// products with the values.  All in fp32; a key that the row does not see is never
// read into a sum.  It reads every key once for each row and head.
#include "attn_device.h"
#include "kernels.h"

namespace tpl {
namespace {

constexpr int AT = 256;
constexpr int FEATURES = 16;   // of a lane: D up to 1024

template <int ES, int CS>
__global__ __launch_bounds__(AT)
void attention_any(AttnArgs a, int64_t w0, int64_t waves) {
    const int lane = threadIdx.x & 63;
    const int64_t w = w0 + (int64_t)blockIdx.x * (AT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (w >= waves) return;
    const int Hq = a.c.Hkv * a.G;
    const int64_t t = w / Hq;
    const int h = (int)(w - t * Hq), hk = h / a.G, D = a.c.D;
    const int64_t s = sequence_of(a.c, t, lane);
    if (s < 0) return;
    const int32_t *table = a.c.table + s * a.c.ldt;
    const int64_t p = (int64_t)a.c.past[s] + (t - a.c.cu[s]);
    const int64_t first = p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    // positions of the table that 32 bits hold
    const int64_t most = 0xFFFFFFFF, all = a.c.max_pages * (int64_t)a.c.page, held = all < most ? all : most, last = p < held ? p : held - 1;
    const int64_t q0 = t * a.ldq + (int64_t)h * D;
    float m = -INFINITY, l = 0.0f, o[FEATURES] = {};
    bool bad = false;
    for (int64_t j0 = first; j0 <= last; j0 += 64) {
        const bool seen = j0 + lane <= last;
        Row r{-1, 0};
        if (seen) r = row_of(a.c, table, (uint32_t)(j0 + lane));
        bad |= seen && r.page < 0;
        const int64_t k0 = r.page * a.c.s_page + r.slot * a.c.s_slot + hk * a.c.s_head;
        float x = -INFINITY, vs = 1.0f;
        if (r.page >= 0) {
            x = 0.0f;
            for (int d = 0; d < D; ++d) x = __builtin_fmaf(value<ES>(a.Q, q0 + d), cached<CS>(a.c.kc, k0 + d), x);
            if (CS == 1) {
                const int64_t i = r.page * a.c.ss_page + r.slot * a.c.ss_slot + hk * a.c.ss_head;
                x *= a.c.ks[i];
                vs = a.c.vs[i];
            }
            x *= a.scale;
        }
        float mx = x;
        for (int i = 32; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor(mx, i));
        const float mn = fmaxf(m, mx);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float e = r.page >= 0 ? expf(x - base) : 0.0f;
        const float c = expf(m - base);
        float sum = e;
        for (int i = 32; i > 0; i >>= 1) sum += __shfl_xor(sum, i);
        l = l * c + sum;
        m = mn;
#pragma unroll
        for (int i = 0; i < FEATURES; ++i) o[i] *= c;
        uint64_t todo = __ballot(r.page >= 0);
        while (todo) {
            const int j = __builtin_ctzll(todo);
            todo &= todo - 1;
            const float ej = __shfl(e * vs, j);
            const int64_t v0 = ((int64_t)__shfl((int)(k0 >> 32), j) << 32) | (uint32_t)__shfl((int)k0, j);
#pragma unroll
            for (int i = 0; i < FEATURES; ++i)
                if (lane + 64 * i < D) o[i] = __builtin_fmaf(ej, cached<CS>(a.c.vc, v0 + lane + 64 * i), o[i]);
        }
    }
    if (p < 0 || p >= held) bad = true;
    if (__any(bad) && lane == 0 && a.c.bad) *a.c.bad = 1;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < FEATURES; ++i)
        if (lane + 64 * i < D) store<ES>(a.O, t * a.ldo + (int64_t)h * D + lane + 64 * i, l == 0.0f ? 0.0f : o[i] * inv);
    if (lane == 0 && a.lse) a.lse[t * a.ldl + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <int ES, int CS>
hipError_t launch(const AttnArgs &a, hipStream_t s) {
    const int64_t waves = a.c.T * a.c.Hkv * a.G, most = 1 << 25;   // one launch has fewer than 2^32 threads
    for (int64_t w = 0; w < waves; w += most) {
        const int64_t n = waves - w < most ? waves - w : most;
        attention_any<ES, CS><<<dim3((unsigned)((n + AT / 64 - 1) / (AT / 64))), dim3(AT), 0, s>>>(a, w, w + n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_attention_any(const AttnArgs &a, int es, hipStream_t s) {
    if (a.c.ks) return es == 2 ? launch<2, 1>(a, s) : launch<4, 1>(a, s);
    return es == 2 ? launch<2, 2>(a, s) : launch<4, 4>(a, s);
}

}  // namespace tpl
