// The append of a fused QKV layer's keys and values to a paged cache in 8 bits:
// norm and rotation of queries and keys as in heads.hip, then for each key and value
// head of D
//   s = max |x| / 127 rounded to fp32,  q = x / s rounded to the nearest whole number
// (halves to even; the mathematics of the exact rounding is in quantize.hip), where x
// is the fp32 result of the rotation, not rounded to the data's type before.
//
// Bound by memory, as the append to a cache of the data's type: the layout of the work
// is the same, 16 values a lane, D / 16 lanes a head, a wavefront for several heads of
// one token.  A head's maximum crosses its lanes as its norm's sum does, and its bytes
// leave as the lane's two runs of 8.  12 prompts, 9680 tokens of 64 + 8 + 8 heads of 128 with
// norms: 91-96 us, 4.1 TB/s of what has to move; 64 tokens 6.5 us.
#include "heads_device.h"
#include "kernels.h"
#include "quant_round.h"

namespace tpl {
namespace {

__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int width) {
    for (int o = width >> 1; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

template <int ES, int LH, bool FINE>
__global__ __launch_bounds__(HT)
void append_quant_vec(HeadArgs a, int parts) {
    const int lane = threadIdx.x & 63;
    const uint32_t w = blockIdx.x * (HT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // < 2^26
    const int64_t t = a.t0 + w / (uint32_t)parts;
    if (t >= a.T) return;
    const int part = (int)(w % (uint32_t)parts);
    const int unit = lane % LH;
    const Runs r = runs_of<FINE>(unit, a.D, a.R, a.pairs);
    const Span sp = span_of(a, a.Q != nullptr, true, true);
    const int slots = sp.per * a.P;
    constexpr int HW = 64 / LH;
    // the next heads' values are loaded while the current ones are worked on
    struct Vals { Head h; Raw8<ES> x[2]; };
    auto load = [&](int g) {
        Vals v = {};
        v.h = head_of(a, g + lane / LH, sp, slots);
        if (v.h.on && r.on) load16<ES, FINE>(a.X, v.h.shard * a.x_shard + t * a.ldx + v.h.col, r, v.x);
        return v;
    };
    Vals next = load(part * HW);
    const Place pl = find_place(a, t, lane);
    if (!pl.ok && pl.mine && a.bad && lane == 0) *a.bad = 1;
    if (!pl.mine) return;
    const int64_t srow = pl.page * a.ss_page + pl.row * a.ss_slot;
    float c[8], s[8];
    Raw8<ES> wq[2] = {}, wk[2] = {};
    if (r.on && r.turn && pl.ok) load_angles<FINE>(a, pl.pos, unit, r, c, s);
    if (a.wq && r.on) load16<ES, FINE>(a.wq, 0, r, wq);
    if (a.wk && r.on) load16<ES, FINE>(a.wk, 0, r, wk);
    for (int g = part * HW; g < slots; g += parts * HW) {
        const Vals cur = next;
        if (g + parts * HW < slots) next = load(g + parts * HW);
        const Head h = cur.h;
        const bool live = h.on && r.on;
        float v[16];
        widen8<ES>(cur.x[0], v);
        widen8<ES>(cur.x[1], v + 8);
        if (!pl.ok) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.0f;
        }
        if (a.wq || a.wk) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) sum = __builtin_fmaf(v[e], v[e], sum);
            sum = lanes_sum(sum, LH);
            if (h.kind != HEAD_V && (h.kind == HEAD_Q ? a.wq : a.wk) && pl.ok) {
                const float rr = rsqrtf(sum / (float)a.D + a.eps);
                float wt[16];
                Raw8<ES> wr[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < ES / 2; ++e) wr[i].w[e] = h.kind == HEAD_Q ? wq[i].w[e] : wk[i].w[e];
                widen8<ES>(wr[0], wt);
                widen8<ES>(wr[1], wt + 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = v[e] * rr * wt[e];
            }
        }
        if (r.turn && h.kind != HEAD_V && pl.ok) {
            if (a.pairs) turn16<FINE>(v, c, s, r, true, false);
            else turn16<FINE>(v, c, s, r, false, false);
        }
        // uniform over the wavefront: some of its heads go to the cache
        if (__any(live && h.kind != HEAD_Q && pl.ok)) {
            uint32_t u[2][8], m = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                u[e / 8][e % 8] = __float_as_uint(v[e]);
                m = max(m, u[e / 8][e % 8] & 0x7FFFFFFFu);
            }
            m = lanes_max(m, LH);
            float scale;
            const Step st = step_of(m, scale);
            const u32x2 lo = round8_mixed(u[0], st), hi = round8_mixed(u[1], st);
            if (live && h.kind != HEAD_Q && pl.ok) {
                int8_t *dst = (int8_t *)(h.kind == HEAD_K ? a.kc : a.vc) + pl.slot + h.head * a.s_head;
                typedef uint32_t u32_any __attribute__((aligned(1)));
                if (FINE) {
                    *(u32_any *)(dst + r.a) = lo[0];
                    *(u32_any *)(dst + r.a2) = lo[1];
                    *(u32_any *)(dst + r.b) = hi[0];
                    *(u32_any *)(dst + r.b2) = hi[1];
                } else {
                    *(u32x2_any *)(dst + r.a) = lo;
                    *(u32x2_any *)(dst + r.b) = hi;
                }
                if (unit == 0) (h.kind == HEAD_K ? a.ks : a.vs)[srow + h.head * a.ss_head] = scale;
            }
        }
        if (live && h.kind == HEAD_Q && a.Q) store16<ES, FINE>(a.Q, t * a.ldq + (int64_t)h.head * a.D, r, v);
    }
}

// Any D and R: a wavefront per (token, head), one element or pair a lane; the values
// are computed twice, for the maximum and to be rounded.
template <int ES>
__global__ __launch_bounds__(HT)
void append_quant_any(HeadArgs a) {
    const int lane = threadIdx.x & 63;
    const Span sp = span_of(a, a.Q != nullptr, true, true);
    const int slots = sp.per * a.P;
    const uint32_t w = blockIdx.x * (HT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // < 2^26
    const int64_t t = a.t0 + w / (uint32_t)slots;
    if (t >= a.T) return;
    const Head h = head_of(a, (int)(w % (uint32_t)slots), sp, slots);
    const Place pl = find_place(a, t, lane);
    if (!pl.ok && pl.mine && a.bad && lane == 0) *a.bad = 1;
    if (!pl.mine || (h.kind != HEAD_Q && !pl.ok)) return;
    const int64_t x0 = h.shard * a.x_shard + t * a.ldx + h.col;
    const void *wt = h.kind == HEAD_Q ? a.wq : h.kind == HEAD_K ? a.wk : nullptr;
    float rr = 1.0f;
    if (wt) {
        float sum = 0.0f;
        for (int d = lane; d < a.D; d += 64) { const float x = get1<ES>(a.X, x0 + d); sum = __builtin_fmaf(x, x, sum); }
        rr = rsqrtf(lanes_sum(sum, 64) / (float)a.D + a.eps);
    }
    // element or pair j, normed and rotated
    auto value = [&](int j, int &ia, int &ib, float &x, float &y) {
        pair_at(a, j, ia, ib);
        x = y = 0.0f;
        if (!pl.ok) return;
        x = get1<ES>(a.X, x0 + ia);
        if (ib >= 0) y = get1<ES>(a.X, x0 + ib);
        if (wt) {
            x = x * rr * get1<ES>(wt, ia);
            if (ib >= 0) y = y * rr * get1<ES>(wt, ib);
        }
        if (ib >= 0 && h.kind != HEAD_V) {
            const float c = a.cos[pl.pos * (a.R / 2) + j], s = a.sin[pl.pos * (a.R / 2) + j];
            const float p = x * c - y * s, q = y * c + x * s;
            x = p; y = q;
        }
    };
    const int items = a.D - a.R / 2;
    if (h.kind == HEAD_Q) {
        if (!a.Q) return;
        const int64_t o = t * a.ldq + (int64_t)h.head * a.D;
        for (int j = lane; j < items; j += 64) {
            int ia, ib;
            float x, y;
            value(j, ia, ib, x, y);
            put1<ES>(a.Q, o + ia, x);
            if (ib >= 0) put1<ES>(a.Q, o + ib, y);
        }
        return;
    }
    uint32_t m = 0;
    for (int j = lane; j < items; j += 64) {
        int ia, ib;
        float x, y;
        value(j, ia, ib, x, y);
        m = max(m, max(__float_as_uint(x) & 0x7FFFFFFFu, __float_as_uint(y) & 0x7FFFFFFFu));
    }
    float scale;
    const Step st = step_of(lanes_max(m, 64), scale);
    int8_t *dst = (int8_t *)(h.kind == HEAD_K ? a.kc : a.vc) + pl.slot + h.head * a.s_head;
    for (int j = lane; j < items; j += 64) {
        int ia, ib;
        float x, y;
        value(j, ia, ib, x, y);
        dst[ia] = (int8_t)round_one(__float_as_uint(x), st);
        if (ib >= 0) dst[ib] = (int8_t)round_one(__float_as_uint(y), st);
    }
    if (lane == 0) (h.kind == HEAD_K ? a.ks : a.vs)[pl.page * a.ss_page + pl.row * a.ss_slot + h.head * a.ss_head] = scale;
}

template <int ES, int LH>
hipError_t launch_vec(const HeadArgs &a, hipStream_t s) {
    const int64_t slots = (int64_t)span_of(a, a.Q != nullptr, true, true).per * a.P, hw = 64 / LH;
    const int64_t groups = (slots + hw - 1) / hw;
    // as many wavefronts as fill the chip (32 for each of 256 CUs), else one a token
    int64_t parts = (8192 + a.T - 1) / a.T;
    if (parts > groups) parts = groups;
    return launch_tokens(a, parts, [&](const HeadArgs &b, unsigned blocks) {
        if (a.R % 16) append_quant_vec<ES, LH, true><<<dim3(blocks), dim3(HT), 0, s>>>(b, (int)parts);
        else append_quant_vec<ES, LH, false><<<dim3(blocks), dim3(HT), 0, s>>>(b, (int)parts);
    });
}

template <int ES>
hipError_t launch_append(const HeadArgs &a, hipStream_t s) {
    const Span sp = span_of(a, a.Q != nullptr, true, true);
    if (a.T == 0 || sp.per == 0) return hipSuccess;
    if (!vec_ok(a)) {
        return launch_tokens(a, (int64_t)sp.per * a.P, [&](const HeadArgs &b, unsigned blocks) {
            append_quant_any<ES><<<dim3(blocks), dim3(HT), 0, s>>>(b);
        });
    }
    switch (lanes_per_head(a.D)) {
        case 1: return launch_vec<ES, 1>(a, s);
        case 2: return launch_vec<ES, 2>(a, s);
        case 4: return launch_vec<ES, 4>(a, s);
        case 8: return launch_vec<ES, 8>(a, s);
        case 16: return launch_vec<ES, 16>(a, s);
        default: return launch_vec<ES, 32>(a, s);
    }
}

}  // namespace

hipError_t launch_kv_append_quant(const HeadArgs &a, int es, hipStream_t s) {
    return es == 2 ? launch_append<2>(a, s) : launch_append<4>(a, s);
}

}  // namespace tpl
