"""Attention over 8-bit values whose scales lie anywhere between the smallest and the largest fp32 numbers.

Tolerances: those of test_gpu_attention.py.  Scales near the smallest normal number add roundings to 2^-150 (half of
fp32's smallest step): one of each weight times its scale, one of that times the shift where it is at its largest (2^125
times, to half of fp16's smallest step 2^-24), and one of the sums, all of which a value's code multiplies: with c the
codes |o - o*| gains 3 2^-150 sum |c| / sum w.  Results under bf16's (fp32's) smallest normal number round to half of its
smallest step, 2^-134 (2^-150), at best, after a rounding to 2^-150."""
import math

import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV
from test_gpu_attention import BF, F32, Cached, reference, workspace

pytestmark = pytest.mark.gpu


def run(c, Hq, Q=None, window=0):
    if Q is None:
        Q = (torch.randn((c.T, Hq * c.D), generator=torch.Generator().manual_seed(7)) * 2).to(c.t)
    args, scales = c.dev()
    Qd = Q.to(DEV)
    O, L = torch.empty_like(Qd), torch.empty((c.T, Hq), device=DEV)
    tl.tp_kv_attention(Qd, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], O, workspace(c.T, len(c.lens), Hq, c.Hkv, c.D),
                       **scales, lse=L, window=window)
    return Q, O, L


def check(c, Hq, window=0):
    print("scales", c.lens, c.past, Hq, c.Hkv, c.D, c.t, window, flush=True)
    Q, O, L = run(c, Hq, window=window)
    o, lse, eo, el = reference(c, Q, Hq, window, c.D ** -0.5)
    own = torch.zeros(c.T, dtype=torch.bool)
    own[int(c.cu[0]):int(c.cu[-1])] = True
    q = Q.double().view(c.T, Hq, c.D)
    for s in range(len(c.lens)):
        for i in range(c.lens[s]):
            t, p = int(c.cu[s]) + i, c.past[s] + i
            lo = max(0, p - window + 1) if window else 0
            k, v, f = (x[s][lo:p + 1].repeat_interleave(Hq // c.Hkv, 1) for x in (c.k, c.v, c.v_scale))
            x = (q[t] * k).sum(-1) * c.D ** -0.5
            w = (x - x.max(0).values).exp().sum(0)
            codes = torch.where(f[..., None] > 0, (v / f[..., None]).abs(), 0.0).sum(0)
            eo[t] += 3 * 2.0 ** -150 * codes / w[:, None]
    eo = eo.nan_to_num(0.0) + (2.0 ** -134 if c.t == BF else 2.0 ** -150) + 2.0 ** -150
    got = O.cpu().double().view(c.T, Hq, c.D)
    assert torch.isfinite(got[own]).all()
    off = (got - o).abs()[own]
    assert (off <= eo[own]).all(), ((off - eo[own]).max(), off.max())
    gl = L.cpu().double()
    assert ((gl - lse).abs() <= el)[own].all()


SHAPES = [([1, 1], [700, 5], (8, 2, 128, 16)), ([40, 3], [100, 0], (4, 2, 64, 16)), ([1], [3000], (4, 1, 96, 16)), ([70], [200], (3, 1, 100, 16)),
          ([1, 9], [300, 40], (2, 1, 256, 16)), ([1], [90], (2, 2, 72, 16))]


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("e", [(100, 100), (112, 112), (119, 119), (115, 119), (-100, 112), (-105, -105), (-119, -119), (-119, -100), (-131, -131), (-140, -131), (-119, 119)])
@pytest.mark.parametrize("lens,past,shape", SHAPES)
def test_scales(lens, past, shape, e, t):
    """One exponent, or any between two in one row (further factors of scales between 2^-7 and 2^-5)."""
    Hq, Hkv, D, page = shape
    check(Cached(lens, past, Hkv, D, page, t, True, seed=4, v_scales=e), Hq)


@pytest.mark.parametrize("lens,past,shape", SHAPES)
def test_window_of_scales(lens, past, shape):
    Hq, Hkv, D, page = shape
    check(Cached(lens, past, Hkv, D, page, BF, True, seed=6, v_scales=(-110, 119)), Hq, window=33)


def staged(order, lens=(1,), past=(199,), shape=(4, 2, 64, 16)):
    """Keys whose values' scales go through the exponents of `order`, a fifth of the positions each."""
    Hq, Hkv, D, page = shape
    c = Cached(list(lens), list(past), Hkv, D, page, BF, True, seed=8)
    for s in range(len(lens)):
        n = lens[s] + past[s]
        for j in range(n):
            f = 2.0 ** order[j * len(order) // n]
            page_, slot = int(c.table[s, j // page]), j % page
            c.vs[page_, slot] *= f
            c.v[s][j] *= f
            c.v_scale[s][j] *= f
    return c


@pytest.mark.parametrize("lens,past", [((1,), (199,)), ((60,), (140,)), ((1, 60), (399, 500))])
@pytest.mark.parametrize("order", [(-112, 119, -112, 0, 119), (119, -112, 0, 119, -112), (0, -112, 119, 0, 0), (-112, -112, -112, -112, 119), (119, -112, -112, -112, -112)])
def test_scales_that_change_along_a_row(order, lens, past):
    """From the smallest to the largest and back: the weights' sum stays what it is."""
    check(staged(order, lens, past), 4)


@pytest.mark.parametrize("lens,past", [([40, 3], [100, 0]), ([1, 30], [90, 64])])
@pytest.mark.parametrize("f", [2.0 ** 120, 3e38, 2.0 ** -140, math.inf, math.nan])
def test_scales_behind_a_row_have_no_effect(f, lens, past):
    """The bits of a row do not depend on the scales of later tokens, however large."""
    a, b = (Cached(lens, past, 2, 64, 16, BF, True, seed=4) for _ in "ab")
    for s in range(len(lens)):
        for i in range(lens[s] // 2 + 1, lens[s]):
            j = past[s] + i
            b.vs[int(b.table[s, j // 16]), j % 16] = f
    Q, O, L = run(a, 4)
    _, P, M = run(b, 4, Q)
    for s in range(len(lens)):
        at = int(a.cu[s])
        keep = slice(at, at + lens[s] // 2 + 1)
        assert torch.equal(O[keep], P[keep]) and torch.equal(L[keep], M[keep])


@pytest.mark.parametrize("f", [2.0 ** 121, 2.0 ** 112, 2.0 ** -120, 2.0 ** -125])
def test_what_the_append_writes(f):
    """Values up to bf16's largest: the append's scales to 2^121, and attention of one token to one key is that value."""
    D, page = 64, 16
    X = torch.zeros((2, 3 * D), dtype=BF)
    X[:, 2 * D:] = torch.linspace(-127, 127, D).round() * f
    X[1, 2 * D:] *= 2.0 ** -4
    X = X.to(DEV)
    kc, vc = (torch.zeros((3, page, 1, D), dtype=torch.int8, device=DEV) for _ in "kv")
    ks, vs = (torch.zeros((3, page, 1), device=DEV) for _ in "kv")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cu, past, table = i32([0, 1, 2]), i32([0, 0]), i32([[2], [0]])
    Q = torch.empty((2, D), dtype=BF, device=DEV)
    tl.tp_kv_append_quant(X, None, None, past, cu, table, kc, vc, ks, vs, 1, 1, 1, Q=Q)
    O = torch.empty((2, D), dtype=BF, device=DEV)
    tl.tp_kv_attention(Q, past, cu, table, kc, vc, O, workspace(2, 2, 1, 1, D), k_scale=ks, v_scale=vs)
    # codes times a scale that is f or a fraction of it: whole numbers of at most 127
    assert torch.equal(O, X[:, 2 * D:])
