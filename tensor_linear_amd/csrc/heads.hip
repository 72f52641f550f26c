// Per-head steps on a fused QKV column layer's output ("模型并行", "Tensor
// Parallel": the column split of the QKV weight gives each shard whole heads, so
// these need no exchange): the root-mean-square norm of each query and key head
// with the rotation of its pairs by the token's position in the same pass, the
// append of keys and values to a paged cache, and the gradients.
//
//   y = x rsqrt(mean(x^2) + eps) w          (without a weight: y = x)
//   pair j < R/2: (a, b) = (y[j], y[j + R/2]), or (y[2j], y[2j + 1]) with `pairs`
//   out = (a cos - b sin, b cos + a sin); elements from R on pass through
// and backwards, with g the gradient turned back by the same angle, r the
// reciprocal root and n = x r:
//   dw = sum over tokens and heads of g n;  h = g w;  dx = r (h - n mean(h n)).
// All in fp32, one rounding to the output's type.
//
// Bound by memory: each value is read and written once, the angles come from a
// table (cosines and sines of a far position need more than fp32 angles).  A
// lane owns 16 values of a head as two 16- (bf16) or 32-byte runs that hold
// both halves of its pairs, so the rotation stays in the lane; D / 16 lanes
// (rounded up to a power of two) share a head, and the norm's sum crosses only
// them.  A wavefront takes several heads of ONE token, so that a token's 16
// cosines and sines are loaded once per lane and used for every head: for 72
// heads of 128 the table's bytes would otherwise double the load instructions.
// With few tokens the heads of a token are spread over more wavefronts.  bf16 heads
// of 128: 8192 tokens of 64 + 8 heads 63.3 us (4.8 TB/s), 9700 such tokens with their
// values into a cache 83 us (4.8 TB/s).
#include "heads_device.h"
#include "kernels.h"

namespace tpl {
namespace {

// LH: lanes per head.  One wavefront per (token, part): part p of `parts`
// takes the groups of 64 / LH heads p, p + parts, ...
template <int ES, int LH, bool APPEND, bool FINE>
__global__ __launch_bounds__(HT)
void heads_vec(HeadArgs a, int parts) {
    const int lane = threadIdx.x & 63;
    const uint32_t w = blockIdx.x * (HT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // < 2^26
    const int64_t t = a.t0 + w / (uint32_t)parts;
    if (t >= a.T) return;
    const int part = (int)(w % (uint32_t)parts);
    const int unit = lane % LH;
    const Runs r = runs_of<FINE>(unit, a.D, a.R, a.pairs);
    const Span sp = span_of(a, a.Q != nullptr, APPEND || a.K, APPEND);
    const int slots = sp.per * a.P;
    constexpr int HW = 64 / LH;
    // The next heads' values are loaded while the current ones are worked on, the
    // first ones while the token's place is looked up.
    struct Vals { Head h; Raw8<ES> x[2]; };
    auto load = [&](int g) {
        Vals v = {};
        v.h = head_of(a, g + lane / LH, sp, slots);
        if (v.h.on && r.on) {
            const int64_t x = v.h.shard * a.x_shard + t * a.ldx + v.h.col;
            load16<ES, FINE>(a.X, x, r, v.x);
        }
        return v;
    };
    Vals next = load(part * HW);
    const Place pl = APPEND ? find_place(a, t, lane) : given_place(a, t);
    if (!pl.ok && pl.mine && a.bad && lane == 0) *a.bad = 1;
    if (APPEND && !pl.mine) return;
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
        const void *wt = h.kind == HEAD_Q ? a.wq : a.wk;
        if (a.wq || a.wk) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) sum = __builtin_fmaf(v[e], v[e], sum);
            sum = lanes_sum(sum, LH);
            if (h.kind != HEAD_V && wt && pl.ok) {   // a token without a place stays zero, whatever eps is
                const float rr = rsqrtf(sum / (float)a.D + a.eps);
                float w[16];
                Raw8<ES> wr[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < ES / 2; ++e) wr[i].w[e] = h.kind == HEAD_Q ? wq[i].w[e] : wk[i].w[e];
                widen8<ES>(wr[0], w);
                widen8<ES>(wr[1], w + 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = v[e] * rr * w[e];
            }
        }
        if (r.turn && h.kind != HEAD_V && pl.ok) {
            if (a.pairs) turn16<FINE>(v, c, s, r, true, false);
            else turn16<FINE>(v, c, s, r, false, false);
        }
        if (!live) continue;
        if (h.kind == HEAD_Q) {
            if (a.Q) store16<ES, FINE>(a.Q, t * a.ldq + (int64_t)h.head * a.D, r, v);
        } else if (APPEND) {
            if (pl.ok) store16<ES, FINE>(h.kind == HEAD_K ? a.kc : a.vc, pl.slot + h.head * a.s_head, r, v);
        } else if (a.K) {
            store16<ES, FINE>(a.K, t * a.ldk + (int64_t)h.head * a.D, r, v);
        }
    }
}

// Any D and R: a wavefront per (token, head), one element or pair a lane.
template <int ES, bool APPEND>
__global__ __launch_bounds__(HT)
void heads_any(HeadArgs a) {
    const int lane = threadIdx.x & 63;
    const Span sp = span_of(a, a.Q != nullptr, APPEND || a.K, APPEND);
    const int slots = sp.per * a.P;
    const uint32_t w = blockIdx.x * (HT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // < 2^26
    const int64_t t = a.t0 + w / (uint32_t)slots;
    if (t >= a.T) return;
    const Head h = head_of(a, (int)(w % (uint32_t)slots), sp, slots);
    const Place pl = APPEND ? find_place(a, t, lane) : given_place(a, t);
    if (!pl.ok && pl.mine && a.bad && lane == 0) *a.bad = 1;
    if (APPEND && !pl.mine) return;
    void *dst; int64_t o;
    if (h.kind == HEAD_Q) { dst = a.Q; o = t * a.ldq + (int64_t)h.head * a.D; }
    else if (APPEND) { dst = pl.ok ? (h.kind == HEAD_K ? a.kc : a.vc) : nullptr; o = pl.slot + h.head * a.s_head; }
    else { dst = a.K; o = t * a.ldk + (int64_t)h.head * a.D; }
    if (!dst) return;
    const int64_t x0 = h.shard * a.x_shard + t * a.ldx + h.col;
    const void *wt = h.kind == HEAD_Q ? a.wq : h.kind == HEAD_K ? a.wk : nullptr;
    float rr = 1.0f;
    if (wt) {
        float sum = 0.0f;
        for (int d = lane; d < a.D; d += 64) { const float x = get1<ES>(a.X, x0 + d); sum = __builtin_fmaf(x, x, sum); }
        rr = rsqrtf(lanes_sum(sum, 64) / (float)a.D + a.eps);
    }
    for (int j = lane; j < a.D - a.R / 2; j += 64) {
        int ia, ib;
        pair_at(a, j, ia, ib);
        float x = 0.0f, y = 0.0f;
        if (pl.ok) {
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
        }
        put1<ES>(dst, o + ia, x);
        if (ib >= 0) put1<ES>(dst, o + ib, y);
    }
}

// ---- gradients ---------------------------------------------------------------

// A workgroup takes the queries (the first qblocks of the grid) or the keys and
// values, so that a wavefront's weight and sums are of one kind.  Wavefront w takes
// part w % parts of the heads, 64 / LH at a time, of the tokens w / parts, w / parts
// + waves / parts, ...; with tokens enough that is one part, and a token's angles
// are loaded once.  The next heads' values and the next token's angles are loaded
// while the current ones are worked on (the sums, weights and angles leave room
// for three wavefronts a SIMD in bf16 with R a multiple of 16, 155 registers, and for
// two in fp32 or with another R, 171-195: too few to hide the loads by themselves).  The
// weights' gradient sums of a lane's 16 values stay in registers; they are added
// over the heads of a wavefront and the four wavefronts in a fixed order and left
// in partials[kind][block][D], which a second kernel adds in an order of its own:
// the result does not depend on scheduling.  4096 tokens of 32 + 8 heads of 128:
// 39.6 us in all (3.7 TB/s), 4 of them for the sums.
template <int ES, int LH, bool FINE>
__global__ __launch_bounds__(HT)
void heads_backward_vec(HeadArgs a, int qblocks, int qparts, int kparts, int64_t kind_stride) {
    __shared__ float red[4][LH * 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool isq = (int)blockIdx.x < qblocks;
    const int blk = isq ? blockIdx.x : blockIdx.x - qblocks, nblk = isq ? qblocks : gridDim.x - qblocks;
    const int unit = lane % LH;
    const Runs r = runs_of<FINE>(unit, a.D, a.R, a.pairs);
    const void *wt = isq ? a.wq : a.wk, *dy = isq ? a.dQ : a.dK;
    const int64_t ldy = isq ? a.lddq : a.lddk;
    const int nh = isq ? a.hq : a.hk, first = isq ? 0 : a.hq;     // heads of a shard, the first one's place
    float w[16] = {}, gw[16] = {};
    if (wt && r.on) {
        Raw8<ES> wr[2];
        load16<ES, FINE>(wt, 0, r, wr);
        widen8<ES>(wr[0], w);
        widen8<ES>(wr[1], w + 8);
    }
    constexpr int HW = 64 / LH;
    const int heads = nh * a.P;
    const int groups = dy ? (heads + HW - 1) / HW : 0;            // of gradients, then of value copies
    const int all = groups + (!isq && a.dV ? (heads + HW - 1) / HW : 0);
    const int parts = isq ? qparts : kparts;
    const int64_t w0 = (int64_t)blk * (HT / 64) + wave, step = (int64_t)nblk * (HT / 64) / parts;
    const int part = (int)(w0 % parts);
    int64_t t = w0 / parts;                              // waves beyond step * parts: none
    if (t >= step) t = a.T;

    // values of group g of token t: the outputs' gradients and (with a norm) X
    struct Vals { Raw8<ES> y[2], x[2]; };
    auto load = [&](int64_t t, int g) {
        Vals v = {};
        const bool val = g >= groups;
        const int h = (val ? g - groups : g) * HW + lane / LH;
        if (h < heads && r.on) {
            const void *src = val ? a.dV : dy;
            const int64_t o = t * (val ? a.lddv : ldy) + (int64_t)h * a.D;
            load16<ES, FINE>(src, o, r, v.y);
            if (wt && !val) {
                const int i = h / nh;
                const int64_t x = i * a.x_shard + t * a.ldx + (int64_t)(first + h - i * nh) * a.D;
                load16<ES, FINE>(a.X, x, r, v.x);
            }
        }
        return v;
    };
    struct Turn { float c[8], s[8]; bool ok; };
    auto angles = [&](int64_t t) {
        Turn u = {};
        const Place pl = given_place(a, t);
        u.ok = pl.ok;
        if (!pl.ok && a.bad && lane == 0) *a.bad = 1;
        if (r.on && r.turn && pl.ok) load_angles<FINE>(a, pl.pos, unit, r, u.c, u.s);
        return u;
    };
    if (t < a.T && part < all) {
        Turn now = angles(t);
        Vals cur = load(t, part);
        int g = part;
        Turn then = t + step < a.T ? angles(t + step) : Turn{};
        while (true) {
            int64_t tn = t;
            int gn = g + parts;
            if (gn >= all) { gn = part; tn = t + step; }
            Vals nxt = {};
            if (tn < a.T) nxt = load(tn, gn);
            const bool val = g >= groups;
            const int h = (val ? g - groups : g) * HW + lane / LH;
            const bool live = h < heads && r.on;
            float v[16];
            widen8<ES>(cur.y[0], v);
            widen8<ES>(cur.y[1], v + 8);
            if (!val) {
                if (!now.ok) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0.0f;
                } else {
                    if (r.turn) {
                        if (a.pairs) turn16<FINE>(v, now.c, now.s, r, true, true);
                        else turn16<FINE>(v, now.c, now.s, r, false, true);
                    }
                    if (wt) {
                        float x[16], sum = 0.0f, dot = 0.0f;
                        widen8<ES>(cur.x[0], x);
                        widen8<ES>(cur.x[1], x + 8);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            sum = __builtin_fmaf(x[e], x[e], sum);
                            dot = __builtin_fmaf(x[e], v[e] * w[e], dot);
                        }
                        sum = lanes_sum(sum, LH);
                        dot = lanes_sum(dot, LH);
                        if (live) {
                            const float rr = rsqrtf(sum / (float)a.D + a.eps);
                            const float mean = dot * rr / (float)a.D;
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float n = x[e] * rr;
                                gw[e] = __builtin_fmaf(v[e], n, gw[e]);
                                v[e] = rr * (v[e] * w[e] - n * mean);
                            }
                        }
                    }
                }
            }
            if (live) {
                const int i = h / nh;
                const int64_t o = i * a.dx_shard + t * a.lddx + (int64_t)(first + (val ? a.hk : 0) + h - i * nh) * a.D;
                store16<ES, FINE>(a.dX, o, r, v);
            }
            if (tn >= a.T) break;
            if (tn != t) {
                now = then;
                if (tn + step < a.T) then = angles(tn + step);
            }
            cur = nxt;
            t = tn;
            g = gn;
        }
    }
    if (!a.partials || !wt) return;      // uniform over the workgroup
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float q = gw[e];
        for (int o = LH; o < 64; o <<= 1) q += __shfl_xor(q, o);
        // the value's place in the head (units past D keep their own cells)
        if (lane < LH) red[wave][r.on ? run_at(r, e) : unit * 16 + e] = q;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += HT)
        a.partials[(isq ? 0 : kind_stride) + (int64_t)blk * a.D + d] = ((red[0][d] + red[1][d]) + red[2][d]) + red[3][d];
}

// Any D and R: a wavefront per token, heads one after another; its
// weight-gradient sums live in LDS (each lane its own elements).
constexpr int ANY_D = 1024;   // largest head of this form
template <int ES>
__global__ __launch_bounds__(HT)
void heads_backward_any(HeadArgs a, int64_t kind_stride) {
    __shared__ float acc[4][2][ANY_D];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int items = a.D - a.R / 2;
    for (int d = lane; d < a.D; d += 64) acc[wave][0][d] = acc[wave][1][d] = 0.0f;
    __syncthreads();
    const Span sp = span_of(a, a.dQ != nullptr, a.dK != nullptr, a.dV != nullptr);
    const int slots = sp.per * a.P;
    for (int64_t t = (int64_t)blockIdx.x * (HT / 64) + wave; t < a.T; t += (int64_t)gridDim.x * (HT / 64)) {
        const Place pl = given_place(a, t);
        if (!pl.ok && a.bad && lane == 0) *a.bad = 1;
        for (int g = 0; g < slots; ++g) {
            const Head h = head_of(a, g, sp, slots);
            const void *wt = h.kind == HEAD_Q ? a.wq : h.kind == HEAD_K ? a.wk : nullptr;
            const void *dy = h.kind == HEAD_Q ? a.dQ : h.kind == HEAD_K ? a.dK : a.dV;
            if (!dy) continue;
            const int64_t ldy = h.kind == HEAD_Q ? a.lddq : h.kind == HEAD_K ? a.lddk : a.lddv;
            const int64_t y0 = t * ldy + (int64_t)h.head * a.D, x0 = h.shard * a.x_shard + t * a.ldx + h.col;
            const int64_t o = h.shard * a.dx_shard + t * a.lddx + h.col;
            const bool in = pl.ok || h.kind == HEAD_V;
            // element or pair j's gradient, turned back
            auto grad = [&](int j, int &ia, int &ib, float &p, float &q) {
                pair_at(a, j, ia, ib);
                p = in ? get1<ES>(dy, y0 + ia) : 0.0f;
                q = in && ib >= 0 ? get1<ES>(dy, y0 + ib) : 0.0f;
                if (ib >= 0 && h.kind != HEAD_V && pl.ok) {
                    const float c = a.cos[pl.pos * (a.R / 2) + j], s = a.sin[pl.pos * (a.R / 2) + j];
                    const float u = p * c + q * s, v = q * c - p * s;
                    p = u; q = v;
                }
            };
            float rr = 1.0f, mean = 0.0f;
            if (wt && in) {
                float sum = 0.0f, dot = 0.0f;
                for (int j = lane; j < items; j += 64) {
                    int ia, ib;
                    float p, q;
                    grad(j, ia, ib, p, q);
                    const float x = get1<ES>(a.X, x0 + ia), y = ib >= 0 ? get1<ES>(a.X, x0 + ib) : 0.0f;
                    sum = __builtin_fmaf(x, x, __builtin_fmaf(y, y, sum));
                    dot = __builtin_fmaf(x, p * get1<ES>(wt, ia), dot);
                    if (ib >= 0) dot = __builtin_fmaf(y, q * get1<ES>(wt, ib), dot);
                }
                rr = rsqrtf(lanes_sum(sum, 64) / (float)a.D + a.eps);
                mean = lanes_sum(dot, 64) * rr / (float)a.D;
            }
            for (int j = lane; j < items; j += 64) {
                int ia, ib;
                float p, q;
                grad(j, ia, ib, p, q);
                if (wt && in) {
                    const float x = get1<ES>(a.X, x0 + ia) * rr;
                    acc[wave][h.kind][ia] += p * x;
                    p = rr * (p * get1<ES>(wt, ia) - x * mean);
                    if (ib >= 0) {
                        const float y = get1<ES>(a.X, x0 + ib) * rr;
                        acc[wave][h.kind][ib] += q * y;
                        q = rr * (q * get1<ES>(wt, ib) - y * mean);
                    }
                }
                put1<ES>(a.dX, o + ia, p);
                if (ib >= 0) put1<ES>(a.dX, o + ib, q);
            }
        }
    }
    if (!a.partials) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.D; i += HT) {
        const int kind = i / a.D, d = i - kind * a.D;
        a.partials[kind * kind_stride + (int64_t)blockIdx.x * a.D + d] =
            ((acc[0][kind][d] + acc[1][kind][d]) + acc[2][kind][d]) + acc[3][kind][d];
    }
}

// dw[kind][d] = sum over blocks of partials[kind][block][d]: four columns by 64
// strands of blocks a workgroup, each strand in block order, then the strands in
// a tree whose order is fixed.  Columns 0 .. D - 1 are the queries'.
__global__ __launch_bounds__(HT)
void weight_grad_sum(const float *partials, int64_t kind_stride, int64_t qblocks, int64_t kblocks, int D,
                     float *dwq, float *dwk) {
    __shared__ float red[4][64];
    const int c = threadIdx.x & 3, strand = threadIdx.x >> 2, col = blockIdx.x * 4 + c;
    float s = 0.0f;
    if (col < 2 * D) {
        const float *p = col < D ? partials + col : partials + kind_stride + col - D;
        const int64_t n = col < D ? qblocks : kblocks;
#pragma unroll 8
        for (int64_t b = strand; b < n; b += 64) s += p[b * D];
    }
    red[c][strand] = s;
    __syncthreads();
    const int lane = threadIdx.x & 63, k = threadIdx.x >> 6, at = blockIdx.x * 4 + k;   // a wavefront a column
    const float v = lanes_sum(red[k][lane], 64);
    if (lane == 0 && at < 2 * D) {
        float *dw = at < D ? dwq : dwk;
        if (dw) dw[at < D ? at : at - D] = v;
    }
}

template <int ES, int LH, bool APPEND>
hipError_t launch_vec(const HeadArgs &a, hipStream_t s) {
    const int64_t slots = (int64_t)span_of(a, a.Q != nullptr, APPEND || a.K, APPEND).per * a.P, hw = 64 / LH;
    const int64_t groups = (slots + hw - 1) / hw;
    // Enough wavefronts to fill the chip (32 for each of 256 CUs), else one
    // wavefront a token, which loads its angles and weights once.
    int64_t parts = (8192 + a.T - 1) / a.T;
    if (parts > groups) parts = groups;
    return launch_tokens(a, parts, [&](const HeadArgs &b, unsigned blocks) {
        if (a.R % 16) heads_vec<ES, LH, APPEND, true><<<dim3(blocks), dim3(HT), 0, s>>>(b, (int)parts);
        else heads_vec<ES, LH, APPEND, false><<<dim3(blocks), dim3(HT), 0, s>>>(b, (int)parts);
    });
}

template <int ES, bool APPEND>
hipError_t launch_fwd(const HeadArgs &a, hipStream_t s) {
    const Span sp = span_of(a, a.Q != nullptr, APPEND || a.K, APPEND);
    if (a.T == 0 || sp.per == 0) return hipSuccess;
    if (!vec_ok(a)) {
        return launch_tokens(a, (int64_t)sp.per * a.P, [&](const HeadArgs &b, unsigned blocks) {
            heads_any<ES, APPEND><<<dim3(blocks), dim3(HT), 0, s>>>(b);
        });
    }
    switch (lanes_per_head(a.D)) {
        case 1: return launch_vec<ES, 1, APPEND>(a, s);
        case 2: return launch_vec<ES, 2, APPEND>(a, s);
        case 4: return launch_vec<ES, 4, APPEND>(a, s);
        case 8: return launch_vec<ES, 8, APPEND>(a, s);
        case 16: return launch_vec<ES, 16, APPEND>(a, s);
        default: return launch_vec<ES, 32, APPEND>(a, s);
    }
}

// qb, kb: the most workgroups of either kind; what the launch has of them.
template <int ES, int LH>
void launch_bwd_vec(const HeadArgs &a, int64_t &qb, int64_t &kb, int64_t stride, hipStream_t s) {
    auto groups = [&](int64_t heads) { return (heads * a.P + 64 / LH - 1) / (64 / LH); };
    // Parts of the heads so that the wavefronts are as many as fit, and no more
    // workgroups than wavefronts with work.  (T = 105, 64 + 8 heads of 256: 52 us
    // with one part each, 12.9 in parts.)
    auto fit = [&](int64_t &b, int64_t g) -> int {
        if (b == 0 || g == 0) { b = 0; return 1; }
        int64_t p = b * (HT / 64) / a.T;
        p = p < 1 ? 1 : p > g ? g : p;
        const int64_t need = (a.T * p + HT / 64 - 1) / (HT / 64);
        if (b > need) b = need;
        return (int)p;
    };
    const int qp = fit(qb, a.dQ ? groups(a.hq) : 0);
    const int kp = fit(kb, groups(a.hk) * ((a.dK ? 1 : 0) + (a.dV ? 1 : 0)));
    const dim3 grid((unsigned)(qb + kb));
    if (qb + kb == 0) return;
    if (a.R % 16) heads_backward_vec<ES, LH, true><<<grid, dim3(HT), 0, s>>>(a, (int)qb, qp, kp, stride);
    else heads_backward_vec<ES, LH, false><<<grid, dim3(HT), 0, s>>>(a, (int)qb, qp, kp, stride);
}

template <int ES>
hipError_t launch_bwd(const HeadArgs &a, hipStream_t s) {
    if (a.D > ANY_D) return hipErrorInvalidValue;
    const int64_t most = qk_backward_blocks(a.T), stride = most * a.D;
    const bool q = a.dQ && a.hq > 0, k = (a.dK || a.dV) && a.hk > 0;
    int64_t qb = q ? most : 0, kb = k ? most : 0;   // workgroups that leave sums, of either kind
    if (a.T == 0) qb = kb = 0;
    if (qb + kb > 0) {
        if (!vec_ok(a)) {
            heads_backward_any<ES><<<dim3((unsigned)most), dim3(HT), 0, s>>>(a, stride);
            qb = kb = most;
        } else {
            // workgroups in proportion to the heads (a value head moves half the bytes)
            if (qb && kb) {
                const int64_t kv = (a.dK ? 2 : 0) * a.hk + (a.dV ? 1 : 0) * a.hk;
                kb = (most * kv + 2 * a.hq + kv - 1) / (2 * a.hq + kv);
                if (kb > most) kb = most;
                if (most > kb) qb = most - kb;
            }
            switch (lanes_per_head(a.D)) {
                case 1: launch_bwd_vec<ES, 1>(a, qb, kb, stride, s); break;
                case 2: launch_bwd_vec<ES, 2>(a, qb, kb, stride, s); break;
                case 4: launch_bwd_vec<ES, 4>(a, qb, kb, stride, s); break;
                case 8: launch_bwd_vec<ES, 8>(a, qb, kb, stride, s); break;
                case 16: launch_bwd_vec<ES, 16>(a, qb, kb, stride, s); break;
                default: launch_bwd_vec<ES, 32>(a, qb, kb, stride, s); break;
            }
            if (!a.dK) kb = 0;                      // value copies leave no sums
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dwq || a.dwk)   // no tokens or no gradient of a kind: zeros
        weight_grad_sum<<<dim3((unsigned)((2 * a.D + 3) / 4)), dim3(HT), 0, s>>>(a.partials, stride, qb, kb, a.D, a.dwq, a.dwk);
    return hipGetLastError();
}

}  // namespace

// Three wavefronts on each SIMD of 256 CUs (what the registers of the commonest form
// allow; 4096 tokens of 32 + 8 heads of 128, us: 512 workgroups 41.2, 768 35.6, 1024 39.6,
// 2048 39.6), fewer where a token's heads in parts are fewer.  Not taken from the
// device: the workspace's size and the order of the weights' sums depend on the call's
// sizes alone.
int64_t qk_backward_blocks(int64_t T) {
    const int64_t b = T < 64 ? 16 * T : 768;
    return b < 1 ? 1 : b > 768 ? 768 : b;
}

hipError_t launch_qk_norm_rope(const HeadArgs &a, int es, hipStream_t s) {
    return es == 2 ? launch_fwd<2, false>(a, s) : launch_fwd<4, false>(a, s);
}

hipError_t launch_kv_append(const HeadArgs &a, int es, hipStream_t s) {
    return es == 2 ? launch_fwd<2, true>(a, s) : launch_fwd<4, true>(a, s);
}

hipError_t launch_qk_norm_rope_backward(const HeadArgs &a, int es, hipStream_t s) {
    return es == 2 ? launch_bwd<2>(a, s) : launch_bwd<4>(a, s);
}

}  // namespace tpl
