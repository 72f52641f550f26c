"""Attention of new tokens over a paged cache against the definition in 64 bits on
the CPU.

Tolerances.  u = 2^-24, u_w = 2^-8 for bf16 (the weights' rounding for the product
with the values, 2^-11 where the cache is int8; none in fp32), u_out = finfo(type).eps / 2, n the keys a row sees,
A = sum w |v| / sum w.  A product with a key has D roundings of the sum of |q k|, and
three more (the scales): delta = (D + 4) u scale sum |q k| at most, plus 4 u |x - max|
for the exponential's argument and 4 u for the exponential.  Numerator and denominator
are each off by delta + n u relative to A (n additions, and a rescaling for each tile of
32 keys at least: n u in all counts both twice over), so
  |o - o*| <= 1.02 A (u_w + 2 (delta + (n + 16) u)) + u_out |o*|,
  |lse - lse*| <= 1.02 (delta + (n + 16) u) + 4 u |lse*|.
Where the cache is int8 and the type bf16, a weight times its scale is rounded to fp16,
to 2^-25 at best (half of its smallest step), in units in which the largest of the row, M,
is 2^4 or more: by 2^-29 M or less, which a value's code multiplies.  So for codes c
  |o - o*| gains 2^-29 M sum |c| / sum w,
which counts in a feature whose code is zero at the largest scales.
"""
import math

import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def workspace(T, B, Hq, Hkv, D):
    n = tl.tp_kv_attention_workspace_bytes(T, B, Hq, Hkv, D)
    return torch.full((max(n, 256),), 255, dtype=torch.uint8, device=DEV)      # NaN patterns


class Cached:
    """Sequences with `past` tokens before their `lens` new ones in a paged cache; all that no sequence holds is NaN
    (an 8-bit cache: scales).  v_scales: exponents of two, smallest and largest, of further factors of the values' scales."""

    def __init__(self, lens, past, Hkv, D, page, t, int8=False, seed=0, order="slot", pad=0, lead=0, tail=0, extra_pages=3,
                 v_scales=(0, 0)):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.past, self.Hkv, self.D, self.page, self.t, self.int8 = lens, past, Hkv, D, page, t, int8
        total = [max(0, n + p) for n, p in zip(lens, past)]
        self.cu = torch.tensor([lead] + [lead + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
        self.T = lead + sum(lens) + tail
        need = [-(-n // page) for n in total]
        self.n_pages = sum(need) + extra_pages
        ids = torch.randperm(self.n_pages, generator=g).tolist()
        self.max_pages = max(need + [1])
        self.table = torch.randint(0, self.n_pages, (len(lens), self.max_pages), generator=g).to(torch.int32)
        dims = [self.n_pages, page, Hkv, D]
        # memory order: (page, slot, head) or (page, head, slot), rows padded
        mem = [dims[0], dims[2], dims[1]] if order == "head" else dims[:3]
        view = (lambda x: x.transpose(1, 2)) if order == "head" else (lambda x: x)

        def make():
            if int8:
                c = torch.full(mem + [D + pad], 99, dtype=torch.int8)
                s = torch.full(mem, NAN)
                return view(c[..., :D]), view(s)
            return view(torch.full(mem + [D + pad], NAN).to(t)[..., :D]), None
        (self.kc, self.ks), (self.vc, self.vs) = make(), make()
        self.k, self.v = [], []       # in 64 bits, [keys, Hkv, D]
        self.v_scale = []             # int8: [keys, Hkv]
        for s, n in enumerate(total):
            mine, ids = ids[:need[s]], ids[need[s]:]
            self.table[s, :need[s]] = torch.tensor(mine, dtype=torch.int32)
            wide = []
            for c, sc in ((self.kc, self.ks), (self.vc, self.vs)):
                if int8:
                    x = torch.randint(-127, 128, (n, Hkv, D), generator=g).to(torch.int8)
                    f = (torch.rand((n, Hkv), generator=g) + 0.5) / 64
                    if c is self.vc and v_scales != (0, 0):
                        f *= 2.0 ** torch.randint(v_scales[0], v_scales[1] + 1, (n, Hkv), generator=g)
                    wide.append(x.double() * f.double()[..., None])
                else:
                    x = torch.randn((n, Hkv, D), generator=g).to(t)
                    wide.append(x.double())
                for j in range(0, n, page):
                    rows = x[j:j + page]
                    c[mine[j // page], :len(rows)] = rows
                    if int8:
                        sc[mine[j // page], :len(rows)] = f[j:j + page]
            self.k.append(wide[0])
            self.v.append(wide[1])
            if int8:
                self.v_scale.append(f.double())

    def dev(self):
        place = lambda x: None if x is None else _like(x)  # noqa: E731
        return dict(past=torch.tensor(self.past, dtype=torch.int32, device=DEV), cu=self.cu.to(DEV), table=self.table.to(DEV),
                    k_cache=place(self.kc), v_cache=place(self.vc)), dict(k_scale=place(self.ks), v_scale=place(self.vs))


def _like(x):
    """x on the GPU with its strides."""
    base = torch.empty(max(1, 1 + sum((n - 1) * s for n, s in zip(x.shape, x.stride()))), dtype=x.dtype, device=DEV)
    y = base.as_strided(x.shape, x.stride())
    y.copy_(x)
    return y


def reference(c, Q, Hq, window, scale, see=lambda s, j: True):
    """o, lse, and the bounds of their errors."""
    D, G = c.D, Hq // c.Hkv
    o = torch.zeros(c.T, Hq, D, dtype=torch.float64)
    lse = torch.full((c.T, Hq), -math.inf, dtype=torch.float64)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    u_w = 0.0 if c.t == F32 else 2.0 ** -11 if c.int8 and 8 <= c.D <= 256 else 2.0 ** -8
    q = Q.double().view(c.T, Hq, D)
    for s in range(len(c.lens)):
        for i in range(c.lens[s]):
            t, p = int(c.cu[s]) + i, c.past[s] + i
            lo = max(0, p - window + 1) if window else 0
            js = [j for j in range(lo, p + 1) if see(s, j)]
            if not js:
                continue
            k, v = (x[s][js].repeat_interleave(G, 1) for x in (c.k, c.v))          # [n, Hq, D]
            x = (q[t] * k).sum(-1) * scale
            mag = (q[t] * k).abs().sum(-1) * scale
            m = x.max(0).values
            w = (x - m).exp()
            l = w.sum(0)
            o[t] = (w[..., None] * v).sum(0) / l[:, None]
            lse[t] = m + l.log()
            A = (w[..., None] * v.abs()).sum(0) / l[:, None]
            delta = ((D + 4) * U * mag + 4 * U * (x - m).abs()).max(0).values + (len(js) + 20) * U
            if c.int8 and c.t == BF:
                sc = c.v_scale[s][js].repeat_interleave(G, 1)                      # [n, Hq]
                eo[t] = 1.02 * 2.0 ** -29 * ((w * sc).max(0).values / l)[:, None] * (v / sc[..., None]).abs().sum(0)
            eo[t] += 1.02 * A * (u_w + 2 * delta[:, None]) + torch.finfo(c.t).eps / 2 * o[t].abs()
            el[t] = 1.02 * delta + 4 * U * lse[t].abs()
    return o, lse, eo, el


def rows(c):
    """Which rows a sequence owns."""
    m = torch.zeros(c.T, dtype=torch.bool)
    m[int(c.cu[0]):int(c.cu[-1])] = True
    return m


def check(c, Hq, window=0, scale=None, extra=0, shift=0, see=lambda s, j: True, bad=0, lse=True, q_scale=2.0, ws=None):
    print("attention", c.lens, c.past, Hq, c.Hkv, c.D, c.page, c.t, c.int8, window, flush=True)
    g = torch.Generator().manual_seed(7)
    Q = (torch.randn((c.T, Hq * c.D), generator=g) * q_scale).to(c.t)
    n = Hq * c.D
    Qb = torch.full((c.T, n + extra + shift), 50.0, dtype=c.t, device=DEV)
    Ob = torch.full((c.T, n + extra + shift), 9.0, dtype=c.t, device=DEV)
    Lb = torch.full((c.T, Hq + extra), 9.0, device=DEV)
    Qd, O, L = Qb[:, shift:shift + n], Ob[:, shift:shift + n], Lb[:, :Hq]
    Qd.copy_(Q)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    args, scales = c.dev()
    if ws is None:
        ws = workspace(c.T, len(c.lens), Hq, c.Hkv, c.D)
    tl.tp_kv_attention(Qd, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], O, ws, **scales, scale=scale, window=window,
                       lse=L if lse else None, bad=flag)
    torch.cuda.synchronize()
    assert flag.item() == bad
    want, wl, eo, el = reference(c, Q, Hq, window, c.D ** -0.5 if scale is None else scale, see)
    own = rows(c)
    got, gl = O.cpu().double().view(c.T, Hq, c.D), L.cpu().double()
    assert (got[~own] == 9.0).all() and (not lse or (gl[~own] == 9.0).all())
    assert (Ob[:, :shift] == 9.0).all() and (Ob[:, shift + n:] == 9.0).all() and (Lb[:, Hq:] == 9.0).all()
    off = (got - want).abs()[own]
    assert torch.isfinite(got[own]).all()
    assert (off <= eo[own] + 1e-30).all(), (off - eo[own]).max()
    if lse:
        same = (gl == wl) | ((gl - wl).abs() <= el)
        assert same[own].all(), (gl - wl)[own][~same[own]][:5]
    return O, L


SHAPES = [  # Hq, Hkv, D, page
    (1, 1, 128, 16), (8, 1, 128, 16), (8, 8, 64, 16), (6, 2, 80, 16), (12, 4, 96, 5), (4, 4, 256, 32), (32, 2, 128, 64), (33, 1, 64, 1),
    (3, 1, 7, 16), (4, 2, 40, 48), (2, 1, 72, 16), (5, 5, 100, 16), (4, 2, 192, 16), (2, 2, 300, 16), (64, 1, 128, 256), (20, 2, 120, 16),
    (2, 1, 600, 16), (4, 2, 33, 16), (6, 3, 127, 16), (2, 1, 250, 8), (3, 1, 9, 4), (8, 2, 204, 16), (16, 4, 12, 16), (10, 2, 16, 16), (7, 7, 8, 3), (80, 1, 32, 16)]
TYPES = [(BF, False), (F32, False), (BF, True), (F32, True)]


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_decode(shape, t, int8):
    """One token a sequence: nothing before it, a few keys, tiles' ends, several tiles."""
    Hq, Hkv, D, page = shape
    check(Cached([1] * 9, [0, 1, 15, 31, 32, 63, 64, 130, 517], Hkv, D, page, t, int8), Hq)


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_chunks(shape, t, int8):
    """Ragged chunks, sequences without tokens among them, rows before the first and behind the last."""
    Hq, Hkv, D, page = shape
    check(Cached([3, 0, 17, 1, 40, 0], [0, 4, 60, 100, 9, 2], Hkv, D, page, t, int8, lead=2, tail=3), Hq)


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("window", [1, 7, 64, 100, 10 ** 6, 2 ** 62 + 5])
def test_window(window, t, int8):
    check(Cached([5, 1, 70, 1], [0, 130, 75, 31], 2, 64, 16, t, int8, seed=3), 6, window=window)


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("order,pad,extra,shift", [("head", 0, 0, 0), ("slot", 8, 8, 0), ("slot", 3, 1, 1), ("head", 16, 16, 8), ("head", 1, 5, 3)])
def test_strides(order, pad, extra, shift, t, int8):
    check(Cached([1, 33, 2], [200, 11, 64], 2, 128, 16, t, int8, order=order, pad=pad), 8, extra=extra, shift=shift)
    check(Cached([1, 33, 2], [200, 11, 64], 3, 88, 16, t, int8, order=order, pad=pad), 3, extra=extra, shift=shift, window=50)


@pytest.mark.parametrize("t,int8", [(BF, False), (F32, False), (BF, True)])
@pytest.mark.parametrize("lens,past,shape", [
    ([1], [6000], (8, 1, 128, 16)), ([1, 1], [3000, 10], (16, 2, 128, 32)), ([2, 1], [2500, 0], (4, 4, 64, 16)), ([1] * 40, [37 * i for i in range(40)], (8, 4, 64, 16)),
    ([9], [4000], (32, 4, 128, 16)), ([300], [0], (8, 2, 128, 16)), ([130, 260], [500, 0], (4, 1, 96, 64)), ([200], [900], (4, 4, 256, 16)),
    ([1], [2000], (40, 1, 256, 16)), ([65], [700], (2, 2, 128, 16)), ([1, 700], [900, 0], (2, 1, 128, 16)),
    ([1100, 20], [3, 200], (16, 2, 64, 16)), ([0, 5, 0, 1600, 0], [9, 9, 9, 100, 9], (8, 1, 32, 16)), ([1] * 70, [30 * i % 97 for i in range(70)], (2, 1, 64, 16)),
    ([1 + 40 * (i % 7 == 3) for i in range(300)], [i % 50 for i in range(300)], (4, 1, 32, 16)),
    ([11 + i % 5 - 11 * (i % 9 == 4) for i in range(300)], [i % 70 for i in range(300)], (4, 1, 32, 16)), ([1] * 700, [i % 40 for i in range(700)], (2, 1, 32, 16))])
def test_long(lens, past, shape, t, int8):
    """Keys enough that several workgroups share a row, and rows enough that they do not."""
    Hq, Hkv, D, page = shape
    check(Cached(lens, past, Hkv, D, page, t, int8, seed=11), Hq)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("v_scales", [(-90, -90), (-60, -50), (60, 60), (-40, 40), (-12, 3)])
@pytest.mark.parametrize("lens,past,shape", [([1, 1], [700, 5], (8, 2, 128, 16)), ([40, 3], [100, 0], (4, 2, 64, 16)), ([1], [3000], (4, 1, 96, 16))])
def test_scales_of_any_size(lens, past, shape, v_scales, t):
    """8-bit values whose scales are tiny or huge, or both in one row."""
    Hq, Hkv, D, page = shape
    check(Cached(lens, past, Hkv, D, page, t, True, seed=4, v_scales=v_scales), Hq)


@pytest.mark.parametrize("t,int8", TYPES)
def test_scale(t, int8):
    check(Cached([1, 20], [90, 30], 2, 64, 16, t, int8), 4, scale=0.02)
    check(Cached([1, 20], [90, 30], 2, 64, 16, t, int8), 4, scale=1.0, q_scale=0.5)


def test_no_lse():
    check(Cached([1, 20], [90, 30], 2, 64, 16, BF), 4, lse=False)


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (8, 1, 128), (3, 3, 50)])
def test_pages_outside(Hq, Hkv, D, t, int8):
    """Pages that are not in the cache, and positions past the table: left out; rows left with nothing are zeros."""
    c = Cached([1, 30, 1, 4], [40, 50, 20, 0], Hkv, D, 16, t, int8, seed=5)
    c.table[0, 1] = -1
    c.table[1, 3] = c.n_pages
    c.table[2, :] = 2 ** 31 - 1
    c.table[3, :] = -2 ** 31
    gone = {0: {1}, 1: {3}, 2: {0, 1}, 3: {0}}
    check(c, Hq, see=lambda s, j: j // 16 not in gone[s], bad=1)
    check(c, Hq, window=9, see=lambda s, j: j // 16 not in gone[s], bad=1)
    c = Cached([1, 40], [80, 30], Hkv, D, 16, t, int8)
    c.table = c.table[:, :3].contiguous()
    check(c, Hq, see=lambda s, j: j < 48, bad=1)


@pytest.mark.parametrize("t,int8", TYPES)
def test_positions_before_the_first(t, int8):
    c = Cached([5, 1], [-3, -1], 2, 64, 16, t, int8)
    check(c, 4, bad=1)


def test_nothing_to_do():
    c = Cached([0, 0], [5, 0], 2, 64, 16, BF, tail=3)
    check(c, 4)
    args, _ = c.dev()
    none = torch.empty((0, 256), dtype=BF, device=DEV)
    tl.tp_kv_attention(none, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], none)
    O = torch.full((3, 256), 4.0, dtype=BF, device=DEV)
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    tl.tp_kv_attention(O.clone(), empty, torch.zeros(1, dtype=torch.int32, device=DEV), torch.empty((0, 4), dtype=torch.int32, device=DEV),
                       args["k_cache"], args["v_cache"], O)
    assert (O == 4.0).all()


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (8, 1, 128), (3, 3, 50), (2, 2, 256)])
def test_later_tokens_have_no_effect(Hq, Hkv, D, t, int8):
    """A row is the same whatever the tokens behind it hold, in keys, values and queries."""
    lens, past = [37, 70, 1], [30, 0, 64]
    c = Cached(lens, past, Hkv, D, 16, t, int8, seed=2)
    O, L = check(c, Hq)
    for poison in (NAN, math.inf, -math.inf):
        d = Cached(lens, past, Hkv, D, 16, t, int8, seed=2)
        cut = [20, 33, 1]
        for s in range(3):
            for i in range(cut[s], lens[s]):
                j = past[s] + i
                page, slot = int(d.table[s, j // 16]), j % 16
                if int8:
                    d.ks[page, slot], d.vs[page, slot] = poison, poison
                else:
                    d.kc[page, slot], d.vc[page, slot] = poison, poison
        args, scales = d.dev()
        g = torch.Generator().manual_seed(7)
        Q = (torch.randn((d.T, Hq * D), generator=g) * 2).to(t)
        keep = torch.zeros(d.T, dtype=torch.bool)
        for s in range(3):
            a = int(d.cu[s])
            keep[a:a + cut[s]] = True
        Q[~keep] = poison
        P, M = torch.empty_like(O).contiguous(), torch.empty_like(L).contiguous()
        tl.tp_kv_attention(Q.to(DEV), args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], P, workspace(d.T, 3, Hq, Hkv, D),
                           **scales, lse=M)
        assert torch.equal(P[keep.to(DEV)], O[keep.to(DEV)]) and torch.equal(M[keep.to(DEV)], L[keep.to(DEV)])
        # the rows that see them show it
        assert not torch.isfinite(P[~keep.to(DEV)]).any()


@pytest.mark.parametrize("t,int8", TYPES)
def test_what_a_row_sees_shows(t, int8):
    """An infinity or NaN among the values that a row sees is in its output, in that feature."""
    for poison in (math.inf, -math.inf, NAN):
        c = Cached([6], [70], 2, 64, 16, t, int8, seed=2)
        j = 72                                     # seen from the third new token on
        page, slot = int(c.table[0, j // 16]), j % 16
        if int8:
            c.vs[page, slot, 1] = poison
        else:
            c.vc[page, slot, 1, 5] = poison
        args, scales = c.dev()
        Q = torch.randn((6, 4 * 64), generator=torch.Generator().manual_seed(1)).to(t).to(DEV)
        O = torch.empty_like(Q)
        tl.tp_kv_attention(Q, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], O, workspace(6, 1, 4, 2, 64), **scales)
        x = O.cpu().float().view(6, 4, 64)
        assert torch.isfinite(x[:2]).all() and torch.isfinite(x[:, :2]).all()
        if int8:
            assert not torch.isfinite(x[2:, 2:]).any()
        else:
            assert torch.equal(x[2:, 2:, 5].isnan(), torch.full((4, 2), math.isnan(poison)))
            assert math.isnan(poison) or (x[2:, 2:, 5] == poison).all()
            x[2:, 2:, 5] = 0
            assert torch.isfinite(x).all()


def test_one_workspace_in_order_and_again():
    """Calls of different sizes one after another in one workspace, and the same call again, bit for bit."""
    a, b = Cached([1] * 7, [900, 3, 40, 0, 2000, 77, 1], 2, 128, 16, BF), Cached([90, 1], [300, 2500], 2, 128, 16, BF)
    n = max(tl.tp_kv_attention_workspace_bytes(c.T, len(c.lens), 8, 2, 128) for c in (a, b))
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device=DEV)
    first = [check(c, 8, ws=ws) for c in (a, b)]
    again = [check(c, 8, ws=ws) for c in (a, b)]
    for x, y in zip(first, again):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_graph_with_growing_sequences():
    """A captured call replayed while its lengths and pages change in place."""
    c = Cached([1] * 5, [800, 3, 64, 1200, 130], 2, 128, 16, BF)
    args, _ = c.dev()
    Q = torch.randn((5, 8 * 128), generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    O, L = torch.empty_like(Q), torch.empty((5, 8), device=DEV)
    ws = workspace(5, 5, 8, 2, 128)
    call = lambda: tl.tp_kv_attention(Q, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], O, ws, lse=L)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step, past in enumerate(([800, 3, 64, 1200, 130], [100, 0, 30, 1100, 7], [0, 2, 63, 64, 65], [799, 1, 5, 1199, 129])):
        args["past"].copy_(torch.tensor(past, dtype=torch.int32))
        O.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got, gl = O.clone(), L.clone()
        O.fill_(3.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, O) and torch.equal(gl, L)
        d = Cached([1] * 5, past, 2, 128, 16, BF)
        d.k, d.v = c.k, c.v
        want, _, eo, _ = reference(d, Q.cpu(), 8, 0, 128 ** -0.5)
        assert ((got.cpu().double().view(5, 8, 128) - want).abs() <= eo).all(), step


def test_two_streams():
    c = [Cached([1] * 6, [700, 3, 900, 41, 0, 300], 2, 128, 16, BF, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in c]
    outs = []
    Q = torch.randn((6, 8 * 128), generator=torch.Generator().manual_seed(1)).to(BF)
    keep = []
    for x, st in zip(c, streams):
        args, _ = x.dev()
        q, o, ws = Q.to(DEV), torch.empty((6, 8 * 128), dtype=BF, device=DEV), workspace(6, 6, 8, 2, 128)
        keep.append((args, q, ws))
        outs.append(o)
    torch.cuda.synchronize()
    for _ in range(5):
        for (args, q, ws), o, st in zip(keep, outs, streams):
            tl.tp_kv_attention(q, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], o, ws, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for x, o in zip(c, outs):
        want, _, eo, _ = reference(x, Q, 8, 0, 128 ** -0.5)
        assert ((o.cpu().double().view(6, 8, 128) - want).abs() <= eo).all()


def test_long_cache_offsets():
    """A cache whose rows lie past 2^32 bytes and 2^31 elements."""
    page, Hkv, D = 16, 1, 128
    n_pages = (1 << 31) // (page * D) + 40
    kc, vc = (torch.empty((n_pages, page, Hkv, D), dtype=BF, device=DEV) for _ in "kv")
    c = Cached([1, 5], [70, 30], Hkv, D, page, BF)
    args, _ = c.dev()
    at = torch.tensor([n_pages - 1 - i for i in range(c.n_pages)], device=DEV)
    kc[at], vc[at] = args["k_cache"], args["v_cache"]
    table = (n_pages - 1 - args["table"]).to(torch.int32)
    Q = torch.randn((6, 4 * D), generator=torch.Generator().manual_seed(1)).to(BF)
    O = torch.empty((6, 4 * D), dtype=BF, device=DEV)
    tl.tp_kv_attention(Q.to(DEV), args["past"], args["cu"], table, kc, vc, O, workspace(6, 2, 4, 1, D))
    want, _, eo, _ = reference(c, Q, 4, 0, D ** -0.5)
    assert ((O.cpu().double().view(6, 4, D) - want).abs() <= eo).all()


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (3, 1, 50)])
@pytest.mark.parametrize("T", [9, 300])
def test_lengths_that_are_none(T, Hq, Hkv, D, t, int8):
    """Row offsets out of order or outside the call and any past: nothing outside the call's rows is touched."""
    big = 2 ** 31 - 1
    c = Cached([T // 3] * 3, [40, 50, 20], Hkv, D, 16, t, int8, seed=5)
    args, scales = c.dev()
    ws = workspace(c.T, 3, Hq, Hkv, D)
    Q = torch.randn((c.T, Hq * D), generator=torch.Generator().manual_seed(1)).to(t).to(DEV)
    for cu in ([0, T, 0, T], [T, 5, 3, 0], [-7, 4, big, -big - 1], [5, 5, 5, big], [-big, -5, -3, -1], [big] * 4, [-big - 1, big, -big - 1, big]):
        for past in ([0, 9, 30], [big, -big - 1, big], [-big - 1] * 3, [-5, big, 0]):
            O, L = torch.full((c.T + 8, Hq * D), 9.0, dtype=t, device=DEV), torch.full((c.T + 8, Hq), 9.0, device=DEV)
            print("lengths", T, Hq, Hkv, D, t, int8, cu, past, flush=True)
            tl.tp_kv_attention(Q, torch.tensor(past, dtype=torch.int32, device=DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), args["table"],
                               args["k_cache"], args["v_cache"], O[4:-4], ws, **scales, lse=L[4:-4])
            torch.cuda.synchronize()
            assert (O[:4] == 9.0).all() and (O[-4:] == 9.0).all() and (L[:4] == 9.0).all() and (L[-4:] == 9.0).all()


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (3, 1, 50)])
@pytest.mark.parametrize("n", [1, 50])
def test_positions_past_the_table(n, Hq, Hkv, D, t, int8):
    """A past far beyond the table sees all that the table holds, or with a window nothing, as one just beyond it does."""
    c = Cached([n, n], [200, 90], Hkv, D, 16, t, int8, seed=5)
    c.table %= c.n_pages
    c.ks, c.vs = (None if x is None else torch.where(x.isnan(), torch.ones_like(x), x) for x in (c.ks, c.vs))
    c.kc, c.vc = (x if int8 else torch.where(x.isnan(), torch.ones_like(x), x) for x in (c.kc, c.vc))
    args, scales = c.dev()
    ws = workspace(c.T, 2, Hq, Hkv, D)
    Q = torch.randn((c.T, Hq * D), generator=torch.Generator().manual_seed(1)).to(t).to(DEV)
    end = c.max_pages * c.page

    def call(past, window):
        O, L, flag = torch.empty_like(Q), torch.empty((c.T, Hq), device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        args["past"].fill_(past)
        tl.tp_kv_attention(Q, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], O, ws, **scales, window=window, lse=L, bad=flag)
        assert flag.item() == 1
        return O, L
    want, wl = call(end, 0)
    assert torch.isfinite(want).all() and torch.isfinite(wl).all()
    for past in (2 ** 29 + 5, 2 ** 31 - 1 - n):
        O, L = call(past, 0)
        assert torch.equal(O, want) and torch.equal(L, wl)
        O, L = call(past, 77)
        assert (O == 0).all() and (L == -math.inf).all()


def test_rows_of_many_tokens_again():
    """Calls whose items fill the GPU by themselves, bit for bit the same again."""
    c = Cached([500, 3, 257, 128], [100, 900, 0, 64], 2, 128, 16, BF, seed=9)
    args, _ = c.dev()
    Q = torch.randn((c.T, 16 * 128), generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    ws = workspace(c.T, 4, 16, 2, 128)

    def call():
        O = torch.empty_like(Q)
        tl.tp_kv_attention(Q, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], O, ws)
        return O
    first = call()
    for _ in range(5):
        assert torch.equal(call(), first)


def test_two_graphs_in_one_workspace():
    """Two captured calls of different sizes that share a workspace, replayed in turn with eager calls between them."""
    cs = [Cached([1] * 7, [900, 3, 40, 0, 2000, 77, 1], 2, 128, 16, BF), Cached([90, 1], [300, 2500], 2, 128, 16, BF)]
    n = max(tl.tp_kv_attention_workspace_bytes(c.T, len(c.lens), 8, 2, 128) for c in cs)
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device=DEV)
    calls, outs, graphs = [], [], []
    for c in cs:
        args, _ = c.dev()
        Q = torch.randn((c.T, 8 * 128), generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
        O = torch.empty_like(Q)
        calls.append(lambda a=args, q=Q, o=O: tl.tp_kv_attention(q, a["past"], a["cu"], a["table"], a["k_cache"], a["v_cache"], o, ws))
        outs.append(O)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        graphs.append(graph)
    for call in calls:
        call()
    want = [o.clone() for o in outs]
    for k in (0, 1, 1, 0, 1, 0):
        outs[k].zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[k], want[k])
        calls[1 - k]()
        assert torch.equal(outs[1 - k], want[1 - k])
