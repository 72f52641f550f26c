"""Attention with windows and pasts near the ends of 32 bits: as the same call with small ones."""
import copy
import math

import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV
from test_gpu_attention import BF, TYPES, Cached, reference, workspace

pytestmark = pytest.mark.gpu

FAR = 2 ** 29


def filled(lens, past, Hkv, D, t, int8, seed=5):
    """A cache whose whole table holds finite values, as 64-bit rows in c.k, c.v, c.v_scale."""
    c = Cached(lens, past, Hkv, D, 16, t, int8, seed=seed)
    c.table %= c.n_pages
    c.ks, c.vs = (None if x is None else torch.where(x.isnan(), torch.full_like(x, 2.0 ** -6), x) for x in (c.ks, c.vs))
    c.kc, c.vc = (x if int8 else torch.where(x.isnan(), torch.ones_like(x), x) for x in (c.kc, c.vc))
    rows = lambda x, s: x[c.table[s].long()].flatten(0, 1).double()  # noqa: E731
    n = range(len(lens))
    if int8:
        c.k, c.v = ([rows(x, s) * rows(f, s)[..., None] for s in n] for x, f in ((c.kc, c.ks), (c.vc, c.vs)))
        c.v_scale = [rows(c.vs, s) for s in n]
    else:
        c.k, c.v = ([rows(x, s) for s in n] for x in (c.kc, c.vc))
    return c


def call(c, Q, past, window, Hq):
    args, scales = c.dev()
    args["past"].fill_(past)
    O, L = torch.empty_like(Q), torch.empty((c.T, Hq), device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = workspace(c.T, len(c.lens), Hq, c.Hkv, c.D)
    tl.tp_kv_attention(Q, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], O, ws, **scales, window=window, lse=L, bad=flag)
    return O, L, flag.item()


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (3, 1, 50)])
@pytest.mark.parametrize("n", [1, 50])
@pytest.mark.parametrize("low", [51, -30])
def test_far_windows_of_far_positions(low, n, Hq, Hkv, D, t, int8):
    """Rows beyond the table whose first visible position is `low`, the position and the window as far as 32 bits go."""
    c = filled([n, n], [200, 90], Hkv, D, t, int8)
    end = c.max_pages * c.page
    Q = torch.randn((c.T, Hq * D), generator=torch.Generator().manual_seed(1)).to(t)
    Qd = Q.to(DEV)
    near = end + 40
    want, wl, bad = call(c, Qd, near, near - low + 1, Hq)
    assert bad == 1
    d = copy.copy(c)
    d.past = [near, near]
    o, lse, eo, el = reference(d, Q, Hq, near - low + 1, D ** -0.5, see=lambda s, j: j < end)
    assert ((want.cpu().double().view(c.T, Hq, D) - o).abs() <= eo + 1e-30).all() and ((wl.cpu().double() - lse).abs() <= el).all()
    for window in (near + 1000, FAR - 5000, FAR + 1, 10 ** 9, 2 * FAR - 1, 2 * FAR, 2 * FAR + 1, 3 * FAR, 2 ** 31 - 5000):
        past = window + low - 1
        assert end < past < 2 ** 31 - n
        O, L, bad = call(c, Qd, past, window, Hq)
        assert bad == 1 and torch.equal(O, want) and torch.equal(L, wl), window


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("n", [1, 50])
def test_far_positions_that_see_nothing(n, t, int8):
    c = filled([n, n], [200, 90], 2, 64, t, int8)
    Q = torch.randn((c.T, 4 * 64), generator=torch.Generator().manual_seed(1)).to(t).to(DEV)
    end = c.max_pages * c.page
    for past in (FAR + end, 2 * FAR, 3 * FAR - 1, 3 * FAR, 2 ** 31 - 1 - n):
        for window in (1, 77, FAR + 1, 2 * FAR, 2 * FAR + 5, past - end, past - end + 1, past + 1, past + n + 100, 2 ** 31 - 1, 2 ** 31 + 7, 2 ** 40, 2 ** 63 - 1):
            low = past - window + 1            # of the first row, the later ones' one more each
            O, L, bad = call(c, Q, past, window, 4)
            assert bad == 1
            nothing = [low + i >= end for i in range(n)] * 2
            for i, none in enumerate(nothing):
                assert ((O[i] == 0).all() and (L[i] == -math.inf).all()) if none else torch.isfinite(L[i]).all(), (past, window, i)


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("lens,past", [([1, 1, 1], [200, 0, 90]), ([40, 3, 0, 90], [0, 200, 5, 31])])
def test_windows_wider_than_any_sequence(lens, past, t, int8):
    """"None" written as a large number: the bits of no window."""
    c = Cached(lens, past, 2, 64, 16, t, int8, seed=3)
    args, scales = c.dev()
    Q = torch.randn((c.T, 6 * 64), generator=torch.Generator().manual_seed(1)).to(t).to(DEV)
    ws = workspace(c.T, len(lens), 6, 2, 64)

    def run(window):
        O, L = torch.empty_like(Q), torch.empty((c.T, 6), device=DEV)
        tl.tp_kv_attention(Q, args["past"], args["cu"], args["table"], args["k_cache"], args["v_cache"], O, ws, **scales, window=window, lse=L)
        return O, L
    want, wl = run(0)
    for window in (2 ** 20, FAR + 1, 10 ** 9, 2 * FAR - 1, 2 * FAR, 2 ** 31 - 1, 2 ** 63 - 1):
        O, L = run(window)
        assert torch.equal(O, want) and torch.equal(L, wl), window


def test_rows_before_the_call_count():
    """A sequence that begins before the call's first row, its past near the end of 32 bits."""
    c = filled([30, 30], [100, 100], 2, 64, BF, False)
    Q = torch.randn((c.T, 4 * 64), generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    args, _ = c.dev()
    ws = workspace(c.T, 2, 4, 2, 64)

    def run(cu, past, window):
        O, L = torch.full_like(Q, 9.0), torch.empty((c.T, 4), device=DEV)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        tl.tp_kv_attention(Q, i32(past), i32(cu), args["table"], args["k_cache"], args["v_cache"], O, ws, window=window, lse=L)
        return O, L
    end = c.max_pages * c.page
    want = run([0, 30, 60], [end + 4, 20], 50)
    for before in (1, 1000, 2 ** 30, 2 ** 31):
        got = run([-before, 30, 60], [end + 4 - before, 20], 50)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), before
    want = run([0, 30, 60], [20, 20], 0)
    for before in (7, 2 ** 20, 2 ** 31):
        got = run([-before, 30, 60], [20 - before, 20], 0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), before
    # positions past 32 bits: beyond the table, all of which a row sees without a window
    want = run([0, 30, 60], [end + 4, 20], 0)
    got = run([-2 ** 31, 30, 60], [2 ** 31 - 1, 20], 0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = run([-2 ** 31, 30, 60], [2 ** 31 - 1, 20], 2 ** 31)
    assert (got[0][:30] == 0).all() and (got[1][:30] == -math.inf).all()
