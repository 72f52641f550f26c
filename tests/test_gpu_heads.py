"""Norm and rotation of query and key heads, their gradients, and the append to
a paged cache against plain computations in 64 bits on the CPU.

Tolerances.  u = 2^-24, u_out = finfo(type).eps / 2.  A norm: the sum of D squares
has D + 6 roundings before the reciprocal root halves them, the root itself 2 u
(the hardware's), then two products; a rotation adds two products and a sum, each
relative to |a cos| + |b sin|: (D / 2 + 12) u of that magnitude, and u_out of the
result.  Gradients: the mean of the h n adds D + 6 roundings of the sum of |h n|;
weight gradients one rounding for each of the T * heads terms at most.  The factor
1.01 covers the second order."""
import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]


def half_step(t):
    return torch.finfo(t).eps / 2


def values(seed, shape, t):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(t)


def tables(n, R):
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def split(x, P, Hq, Hkv, shards):
    """q, k, v [T, heads, D] in 64 bits of a QKV matrix."""
    x = x.double().transpose(0, 1) if shards else x.double()
    hq, hk = Hq // P, Hkv // P
    x = x.reshape(x.shape[0], P, hq + 2 * hk, -1)
    return x[:, :, :hq].flatten(1, 2), x[:, :, hq:hq + hk].flatten(1, 2), x[:, :, hq + hk:].flatten(1, 2)


def rotate(x, c, s, R, pairs):
    y = x.clone()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])
    p, q = a * c - b * s, b * c + a * s
    if pairs:
        y[..., 0:R:2], y[..., 1:R:2] = p, q
    else:
        y[..., :R // 2], y[..., R // 2:R] = p, q
    return y


def forward(x, w, c, s, R, pairs, ok, eps):
    """Values and the magnitude that rounding is relative to."""
    y = x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    mag = rotate(y.abs(), c.abs(), -s.abs(), R, pairs)
    # both elements of a pair: |a| |c| + |b| |s|
    a = rotate(y.abs(), c.abs(), s.abs(), R, pairs)
    return torch.where(ok, rotate(y, c, s, R, pairs), 0.0), torch.maximum(mag.abs(), a.abs())


CASES = [  # T, Hq, Hkv, D, R, P, pairs, norms, shards, extra
    (1, 1, 1, 16, 16, 1, False, "qk", False, 0), (3, 8, 2, 128, 128, 2, False, "qk", False, 0),
    (5, 8, 2, 128, 128, 2, True, "qk", True, 8), (4, 6, 3, 64, 32, 3, False, "", False, 0),
    (7, 4, 4, 80, 80, 2, True, "q", True, 0), (2, 12, 4, 96, 32, 4, False, "k", False, 16),
    (3, 16, 8, 256, 256, 8, False, "qk", False, 0), (9, 4, 2, 40, 20, 2, False, "qk", True, 0),
    (6, 3, 1, 7, 6, 1, True, "qk", False, 1), (5, 4, 2, 128, 128, 2, False, "qk", True, 1),
    (2, 2, 2, 512, 64, 1, False, "qk", False, 0), (3, 2, 1, 600, 600, 1, True, "qk", False, 0),
    (4, 8, 8, 32, 0, 8, False, "qk", False, 0), (300, 8, 1, 128, 128, 1, False, "qk", False, 0),
    (2, 5, 0, 48, 48, 1, False, "q", False, 0), (9001, 2, 1, 32, 32, 1, False, "qk", False, 0),
    (5, 4, 2, 80, 40, 2, False, "qk", True, 0), (6, 6, 3, 80, 40, 3, True, "qk", False, 1), (3, 2, 1, 16, 8, 1, False, "q", False, 0),
    (4, 4, 2, 48, 24, 2, True, "k", False, 0), (5, 3, 1, 512, 504, 1, False, "qk", False, 3), (200, 4, 4, 128, 120, 4, False, "", True, 0)]


def make(case, t):
    T, Hq, Hkv, D, R, P, pairs, norms, shards, extra = case
    N = (Hq + 2 * Hkv) * D
    x = values(T + D, (P, T, N // P) if shards else (T, N), t)
    buf = torch.full((P, T, N // P + extra) if shards else (T, N + extra), 50.0, dtype=t, device=DEV)
    X = buf[..., :x.shape[-1]]
    X.copy_(x)
    n = 2 * T + 5
    cos, sin = tables(n, R)
    pos = torch.randint(0, n, (T,), generator=torch.Generator().manual_seed(T))
    if T > 2:
        pos[1], pos[2] = -1, n
    if T > 4:
        pos[3], pos[4] = n - 1, 2 ** 40
    wq = (1 + 0.2 * values(1, (D,), torch.float32)).to(t) if "q" in norms else None
    wk = (1 + 0.2 * values(2, (D,), torch.float32)).to(t) if "k" in norms else None
    return x, X, buf, cos, sin, pos, wq, wk


def dev(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("case", CASES)
def test_qk_norm_rope(case, t):
    print("qk", case, t, flush=True)
    T, Hq, Hkv, D, R, P, pairs, norms, shards, extra = case
    x, X, _, cos, sin, pos, wq, wk = make(case, t)
    ok = ((pos >= 0) & (pos < cos.shape[0])) if R else torch.ones(T, dtype=torch.bool)
    at = torch.where(ok, pos, 0)
    c, s = cos.double()[at][:, None], sin.double()[at][:, None]
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    Qb = torch.full((T, Hq * D + extra), 9.0, dtype=t, device=DEV)
    Kb = torch.full((T, Hkv * D + extra), 9.0, dtype=t, device=DEV)
    Q, K = Qb[:, :Hq * D], Kb[:, :Hkv * D]
    args = dict(q_weight=dev(wq), k_weight=dev(wk), style=tl.TP_ROPE_PAIRS if pairs else tl.TP_ROPE_HALVES,
                x_mode=tl.TP_Y_SHARDS if shards else tl.TP_Y_CONCAT, eps=1e-5)
    rot = (dev(pos), dev(cos), dev(sin)) if R else (None, None, None)
    tl.tp_qk_norm_rope(X, *rot, Q, K if Hkv else None, P, Hq, Hkv, bad=bad, **args)
    q, k, _ = split(x, P, Hq, Hkv, shards)
    for got, src, w, H in ((Q, q, wq, Hq), (K, k, wk, Hkv)):
        want, mag = forward(src, w, c, s, R, pairs, ok[:, None, None], 1e-5)
        n = (D / 2 + 12) if w is not None else 4
        err = 1.01 * (n * U * mag + half_step(t) * want.abs())
        off = (got.cpu().double().view(T, H, D) - want).abs() - err
        assert H == 0 or float(off.max()) <= 0, float(off.max())
    assert bool(bad.item()) == (not bool(ok.all()))
    if extra:
        assert torch.all(Qb[:, Hq * D:] == 9.0) and torch.all(Kb[:, Hkv * D:] == 9.0)
    if Hkv:   # each output alone is the same
        Q2, K2 = torch.empty_like(Q), torch.empty_like(K)
        tl.tp_qk_norm_rope(X, *rot, Q2, None, P, Hq, Hkv, **args)
        tl.tp_qk_norm_rope(X, *rot, None, K2, P, Hq, Hkv, **args)
        assert torch.equal(Q2, Q) and torch.equal(K2, K)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("case", CASES)
def test_qk_norm_rope_backward(case, t):
    print("qk backward", case, t, flush=True)
    T, Hq, Hkv, D, R, P, pairs, norms, shards, extra = case
    x, X, _, cos, sin, pos, wq, wk = make(case, t)
    ok = ((pos >= 0) & (pos < cos.shape[0])) if R else torch.ones(T, dtype=torch.bool)
    at = torch.where(ok, pos, 0)
    c, s = cos.double()[at][:, None], sin.double()[at][:, None]
    dq, dk, dv = (values(20 + i, (T, H * D), t) for i, H in enumerate((Hq, Hkv, Hkv)))
    dXb = torch.full((*x.shape[:-1], x.shape[-1] + extra), 9.0, dtype=t, device=DEV)
    dX = dXb[..., :x.shape[-1]]
    dwq, dwk = (torch.full((D,), 9.0, device=DEV) if w is not None else None for w in (wq, wk))
    ws = torch.empty(tl.tp_qk_norm_rope_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
    args = dict(q_weight=dev(wq), k_weight=dev(wk), style=tl.TP_ROPE_PAIRS if pairs else tl.TP_ROPE_HALVES,
                x_mode=tl.TP_Y_SHARDS if shards else tl.TP_Y_CONCAT, eps=1e-5)
    rot = (dev(pos), dev(cos), dev(sin)) if R else (None, None, None)

    def run(out, dwq, dwk):
        tl.tp_qk_norm_rope_backward(X if wq is not None or wk is not None else None, *rot, dev(dq), dev(dk) if Hkv else None, out, P,
                                    Hq, Hkv, dV=dev(dv) if Hkv else None, dq_weight=dwq, dk_weight=dwk, workspace=ws, **args)
    run(dX, dwq, dwk)
    q, k, _ = split(x, P, Hq, Hkv, shards)
    gq, gk, gv = split(dX.cpu(), P, Hq, Hkv, shards)
    if Hkv:
        assert torch.equal(gv.flatten(1), dv.double())
    for got, src, dy, w, dw in ((gq, q, dq, wq, dwq), (gk, k, dk, wk, dwk)):
        if src.shape[1] == 0:
            continue
        dy = dy.double().view(src.shape)
        g = torch.where(ok[:, None, None], rotate(dy, c, -s, R, pairs), 0.0)
        gm = rotate(dy.abs(), c.abs(), s.abs(), R, pairs).abs().maximum(rotate(dy.abs(), c.abs(), -s.abs(), R, pairs).abs())
        gm = torch.where(ok[:, None, None], gm, 0.0)
        if w is None:
            want, err = g, 4 * U * gm
        else:
            r = torch.rsqrt(src.square().mean(-1, keepdim=True) + 1e-5)
            n, h = src * r, g * w.double()
            m = (h * n).mean(-1, keepdim=True)
            want = r * (h - n * m)
            hm = gm * w.double().abs()
            err = (D / 2 + 16) * U * r * (hm + n.abs() * m.abs()) + (1.5 * D + 20) * U * r * n.abs() * (hm * n.abs()).mean(-1, keepdim=True)
            dwant = (g * n).sum((0, 1))
            dwm = (gm * n.abs()).sum((0, 1))
            off = (dw.cpu().double() - dwant).abs() - 1.01 * (T * src.shape[1] + D / 2 + 16) * U * dwm
            assert float(off.max()) <= 0, float(off.max())
        off = (got - want).abs() - 1.01 * (err + half_step(t) * want.abs())
        assert float(off.max()) <= 0, float(off.max())
    if extra:
        assert torch.all(dXb[..., x.shape[-1]:] == 9.0)
    again = [torch.empty_like(dX)] + [None if d is None else torch.empty_like(d) for d in (dwq, dwk)]
    run(*again)
    assert all(a is None or torch.equal(a, b) for a, b in zip(again, (dX, dwq, dwk))), "the sums have a fixed order"


def test_backward_against_differences():
    """The gradient of a fixed weighting of the outputs against central
    differences of the kernel's own forward pass in fp32."""
    T, Hq, Hkv, D, R, P = 2, 2, 1, 16, 8, 1
    x = values(5, (T, (Hq + 2 * Hkv) * D), torch.float32)
    cos, sin = (dev(a) for a in tables(9, R))
    pos = torch.tensor([3, 7], device=DEV)
    w = dev(1 + 0.2 * values(6, (D,), torch.float32))
    aq, ak = values(7, (T, Hq * D), torch.float32), values(8, (T, Hkv * D), torch.float32)

    def f(xs, ws):
        Q, K = torch.empty((T, Hq * D), device=DEV), torch.empty((T, Hkv * D), device=DEV)
        tl.tp_qk_norm_rope(xs, pos, cos, sin, Q, K, P, Hq, Hkv, q_weight=ws, k_weight=ws)
        return float((Q.cpu().double() * aq.double()).sum() + (K.cpu().double() * ak.double()).sum())

    X = dev(x)
    dX, dwq, dwk = torch.zeros_like(X), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    ws = torch.empty(tl.tp_qk_norm_rope_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
    tl.tp_qk_norm_rope_backward(X, pos, cos, sin, dev(aq), dev(ak), dX, P, Hq, Hkv, q_weight=w, k_weight=w, dq_weight=dwq,
                                dk_weight=dwk, workspace=ws)
    # step h: the difference's own error is h^2 |f'''| / 6 (values of order 10) and
    # 128 fp32 roundings of values up to 4 over 2 h
    h = 2.0 ** -8
    tol = h * h * 10 + 128 * 4 * 24 * U / (2 * h)
    for i in range(0, x.numel(), 5):
        e = torch.zeros_like(X).view(-1)
        e[i] = h
        e = e.view_as(X)
        assert abs((f(X + e, w) - f(X - e, w)) / (2 * h) - float(dX.view(-1)[i])) <= tol, i
    for i in range(0, D, 3):
        e = torch.zeros_like(w)
        e[i] = h
        assert abs((f(X, w + e) - f(X, w - e)) / (2 * h) - float((dwq + dwk)[i])) <= tol, i


# ---- append --------------------------------------------------------------------

APPEND = [  # lens, past, Hq, Hkv, D, R, P, page, pairs, norm, shards, order, tail
    ([1], [0], 1, 1, 16, 16, 1, 4, False, True, False, "nhd", 0),
    ([1, 1, 1], [0, 15, 16], 8, 2, 128, 128, 2, 16, False, True, False, "nhd", 0),
    ([3, 0, 17, 1], [2, 5, 30, 63], 4, 2, 64, 32, 2, 16, True, False, True, "hnd", 3),
    ([5, 40], [11, 0], 4, 2, 80, 80, 1, 8, False, True, False, "nhd", 0),
    ([2, 9], [1, 6], 3, 1, 10, 6, 1, 3, True, True, False, "hnd", 2),
    ([33, 1], [100, 7], 8, 8, 128, 0, 8, 32, False, True, True, "nhd", 1),
    ([1] * 70, list(range(0, 140, 2)), 2, 1, 32, 32, 1, 16, False, True, False, "nhd", 0),
    ([0, 0, 1] * 60, [3] * 180, 2, 1, 32, 32, 1, 16, False, False, False, "nhd", 1),
    ([7, 1], [2, 90], 4, 2, 80, 40, 2, 16, False, True, True, "hnd", 1), ([3, 20], [0, 5], 2, 2, 48, 8, 1, 4, True, True, False, "nhd", 0)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("case", APPEND)
def test_kv_append(case, t):
    print("append", [len(case[0])] + list(case[2:]), t, flush=True)
    lens, past, Hq, Hkv, D, R, P, page, pairs, norm, shards, order, tail = case
    B, n_own = len(lens), sum(lens)
    T, lead = n_own + tail, 2 if tail else 0
    T += lead                                     # rows before the first and behind the last sequence
    cu = torch.tensor([lead] + [lead + sum(lens[:i + 1]) for i in range(B)], dtype=torch.int32)
    need = [(p + n + page - 1) // page for p, n in zip(past, lens)]
    most, pages = max(need) + 1, sum(need) + 2
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(B)).to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32)
    k0 = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[k0:k0 + n]
        k0 += n
    N = (Hq + 2 * Hkv) * D
    x = values(T, (P, T, N // P) if shards else (T, N), t)
    cos, sin = tables(max(p + n for p, n in zip(past, lens)) + 1, R)
    w = (1 + 0.2 * values(1, (D,), torch.float32)).to(t) if norm else None
    shape = (pages, page, Hkv, D) if order == "nhd" else (pages, Hkv, page, D)
    kc, vc = (values(i, shape, t) for i in (30, 31))
    kd, vd = dev(kc), dev(vc)
    view = (lambda c: c) if order == "nhd" else (lambda c: c.transpose(1, 2))
    Q = torch.full((T, Hq * D), 9.0, dtype=t, device=DEV)
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = dict(q_weight=dev(w), k_weight=dev(w), style=tl.TP_ROPE_PAIRS if pairs else tl.TP_ROPE_HALVES,
                x_mode=tl.TP_Y_SHARDS if shards else tl.TP_Y_CONCAT)
    rot = (dev(cos), dev(sin)) if R else (None, None)
    pd = dev(torch.tensor(past, dtype=torch.int32))
    tl.tp_kv_append(dev(x), *rot, pd, dev(cu), dev(table), view(kd), view(vd), P, Hq, Hkv, Q=Q, bad=bad, **args)
    assert int(bad) == 0
    q, k, v = split(x, P, Hq, Hkv, shards)
    kw, vw, ke = view(kc).double().clone(), view(vc).double().clone(), torch.zeros(pages, page, Hkv, D, dtype=torch.float64)
    qw, qe = torch.full((T, Hq, D), 9.0, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    n = (D / 2 + 12) if norm else 4
    for i in range(B):
        for j in range(lens[i]):
            row, p = int(cu[i]) + j, past[i] + j
            pg, sl = int(table[i, p // page]), p % page
            c, s = cos.double()[p] if R else cos.double()[0], sin.double()[p] if R else sin.double()[0]
            yes = torch.tensor(True)
            kw[pg, sl], m = forward(k[row], w, c, s, R, pairs, yes, 1e-6)
            ke[pg, sl] = n * U * m + half_step(t) * kw[pg, sl].abs()
            qw[row], m = forward(q[row], w, c, s, R, pairs, yes, 1e-6)
            qe[row] = n * U * m + half_step(t) * qw[row].abs()
            vw[pg, sl] = v[row]
    assert torch.equal(view(vd).cpu().double(), vw)
    assert float(((view(kd).cpu().double() - kw).abs() - 1.01 * ke).max()) <= 0     # untouched slots exactly
    assert float(((Q.cpu().double().view(T, Hq, D) - qw).abs() - 1.01 * qe).max()) <= 0
    # without the queries the caches are the same
    k2, v2 = dev(kc), dev(vc)
    tl.tp_kv_append(dev(x), *rot, pd, dev(cu), dev(table), view(k2), view(v2), P, Hq, Hkv, **args)
    assert torch.equal(k2, kd) and torch.equal(v2, vd)


def test_append_leaves_out_what_has_no_place():
    """Positions past the tables or the page list, and pages that are not in
    the cache: nothing is written, the query rows are zero, the flag is set."""
    H, D, page = 2, 32, 4
    x = values(1, (6, 3 * H * D), torch.float32)
    cu = torch.tensor([0, 1, 2, 3, 4, 5, 6], dtype=torch.int32)
    past = torch.tensor([3, 8, 5, 7, -1, 2], dtype=torch.int32)     # 8: past the page list; 7: past the tables; -1
    table = torch.tensor([[2, 0], [1, 1], [0, 9], [3, 4], [5, 5], [-3, 5]], dtype=torch.int32)   # 9, -3: not in the cache
    cos, sin = tables(7, D)
    kc, vc = values(2, (6, page, H, D), torch.float32), values(3, (6, page, H, D), torch.float32)
    kd, vd, Q = dev(kc), dev(vc), torch.full((6, H * D), 9.0, device=DEV)
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    tl.tp_kv_append(dev(x), dev(cos), dev(sin), dev(past), dev(cu), dev(table), kd, vd, 1, H, H, Q=Q, bad=bad)
    assert int(bad) == 1
    assert torch.all(Q[1:] == 0) and not torch.any(Q[0] == 9.0)
    kd[2, 3], vd[2, 3] = dev(kc[2, 3]), dev(vc[2, 3])                # the one row that has a place
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)


def test_append_far_into_a_large_cache():
    """Row offsets past 32 bits: a cache of over 2^32 elements."""
    H, D, page, pages = 8, 128, 64, 66000
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of free GPU memory")
    kc = torch.empty((pages, page, H, D), dtype=torch.bfloat16, device=DEV)
    assert kc.numel() > 2 ** 32
    vc = torch.empty_like(kc)
    x = values(1, (2, 3 * H * D), torch.bfloat16)
    table = torch.tensor([[pages - 1], [0]], dtype=torch.int32, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    tl.tp_kv_append(dev(x), None, None, i32(page - 1, 5), i32(0, 1, 2), table, kc, vc, 1, H, H)
    _, k, v = split(x, 1, H, H, False)
    assert torch.equal(kc[-1, -1].cpu().double(), k[0]) and torch.equal(vc[-1, -1].cpu().double(), v[0])
    assert torch.equal(kc[0, 5].cpu().double(), k[1]) and torch.equal(vc[0, 5].cpu().double(), v[1])


@pytest.mark.parametrize("T", [3, 200])
def test_attention_projections_together(T):
    """A decode step of the attention block's projections in 8 bits: quantize,
    QKV column layer into shard blocks, append with the queries; captured in a
    graph and replayed with new inputs and growing sequences."""
    Hq, Hkv, D, P, H, page = 8, 4, 64, 4, 256, 16
    t = torch.bfloat16
    N = (Hq + 2 * Hkv) * D
    w = values(1, (N, H), t)
    wq, ws = torch.empty((N, H), dtype=torch.int8, device=DEV), torch.empty(N, device=DEV)
    tl.tp_quantize_rows(dev(w), wq, ws)
    X, xq, xs = torch.empty((T, H), dtype=t, device=DEV), torch.empty((T, H), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    qkv = torch.empty((P, T, N // P), dtype=t, device=DEV)
    cos, sin = (dev(a) for a in tables(64, D))
    nw = dev((1 + 0.1 * values(2, (D,), torch.float32)).to(t))
    cu = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    past = torch.zeros(T, dtype=torch.int32, device=DEV)
    table = torch.arange(2 * T, dtype=torch.int32, device=DEV).view(T, 2)
    kc, vc = (torch.zeros((2 * T, page, Hkv, D), dtype=t, device=DEV) for _ in "kv")
    Q = torch.empty((T, Hq * D), dtype=t, device=DEV)

    def step(q, k, v):
        tl.tp_quantize_rows(X, xq, xs)
        tl.tp_linear_column_quant(xq, xs, wq, ws, qkv, P, tl.TP_Y_SHARDS)
        tl.tp_kv_append(qkv, cos, sin, past, cu, table, k, v, P, Hq, Hkv, Q=q, q_weight=nw, k_weight=nw, x_mode=tl.TP_Y_SHARDS)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(Q, kc, vc)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(Q, kc, vc)
    k2, v2, Q2 = torch.zeros_like(kc), torch.zeros_like(vc), torch.empty_like(Q)
    kc.zero_()
    vc.zero_()
    for r in range(4):
        X.copy_(dev(values(50 + r, (T, H), t)))
        past.fill_(14 + r)                             # across the end of the first page
        graph.replay()
        torch.cuda.synchronize()
        step(Q2, k2, v2)
        torch.cuda.synchronize()
        assert torch.equal(Q, Q2) and torch.equal(kc, k2) and torch.equal(vc, v2), f"replay {r}"
    # the cache holds what the cacheless pass gives
    K = torch.empty((T, Hkv * D), dtype=t, device=DEV)
    tl.tp_qk_norm_rope(qkv, past.long(), cos, sin, Q2, K, P, Hq, Hkv, q_weight=nw, k_weight=nw, x_mode=tl.TP_Y_SHARDS)
    assert torch.equal(Q2, Q) and torch.equal(kc[table[:, 1].long(), 1].view(T, -1), K)


def test_backward_in_a_graph():
    T, Hq, Hkv, D, P = 40, 4, 2, 64, 2
    t = torch.bfloat16
    N = (Hq + 2 * Hkv) * D
    X, dq, dk = (dev(values(i, s, t)) for i, s in enumerate(((T, N), (T, Hq * D), (T, Hkv * D))))
    pos = torch.arange(T, device=DEV)
    cos, sin = (dev(a) for a in tables(T, D))
    w = dev((1 + 0.1 * values(9, (D,), torch.float32)).to(t))
    ws = torch.empty(tl.tp_qk_norm_rope_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)

    def step():
        out = torch.zeros_like(X), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
        tl.tp_qk_norm_rope_backward(X, pos, cos, sin, dq, dk, out[0], P, Hq, Hkv, dV=dk, q_weight=w, k_weight=w, dq_weight=out[1],
                                    dk_weight=out[2], workspace=ws)
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for r in range(3):
        X.copy_(dev(values(70 + r, (T, N), t)))
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), f"replay {r}"


def test_no_tokens_give_zero_weight_gradients():
    D, z = 64, lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    cos, sin = (dev(a) for a in tables(4, D))
    dwq, dwk = torch.full((D,), 3.0, device=DEV), torch.full((D,), 3.0, device=DEV)
    ws = torch.empty(tl.tp_qk_norm_rope_workspace_bytes(0, D), dtype=torch.uint8, device=DEV)
    tl.tp_qk_norm_rope_backward(z(0, 4 * D), torch.zeros(0, dtype=torch.int64, device=DEV), cos, sin, z(0, 2 * D), z(0, D), z(0, 4 * D), 1, 2, 1,
                                q_weight=z(D), k_weight=z(D), dq_weight=dwq, dk_weight=dwk, workspace=ws)
    assert torch.all(dwq == 0) and torch.all(dwk == 0)
    # a kind without an output gradient has none of the weight either, and its part of dX is left
    X, dX = dev(values(1, (3, 4 * D), torch.bfloat16)), torch.full((3, 4 * D), 9.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(tl.tp_qk_norm_rope_workspace_bytes(3, D), dtype=torch.uint8, device=DEV)
    dwq.fill_(3.0)
    tl.tp_qk_norm_rope_backward(X, torch.arange(3, device=DEV), cos, sin, None, dev(values(2, (3, D), torch.bfloat16)), dX, 1, 2, 1, q_weight=z(D) + 1,
                                k_weight=z(D) + 1, dq_weight=dwq, dk_weight=dwk, workspace=ws)
    assert torch.all(dwq == 0) and float(dwk.abs().sum()) > 0
    assert torch.all(dX[:, :2 * D] == 9.0) and torch.all(dX[:, 3 * D:] == 9.0) and not torch.any(dX[:, 2 * D:3 * D] == 9.0)


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    x, q, s = torch.zeros((2, 8), device=DEV), torch.zeros((2, 8), dtype=torch.int8, device=DEV), torch.zeros(2, device=DEV)
    tl.tp_quantize_rows(x, q, s)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        tl.tp_quantize_rows(x, q, s)
    with pytest.raises(ValueError, match="current device"):
        tl.tp_qk_norm_rope(torch.zeros((2, 24), device=DEV), None, None, None, torch.zeros((2, 8), device=DEV), None, 1, 1, 1)


def test_two_streams_at_once():
    """Calls on two streams with their own buffers and workspaces."""
    T, Hq, Hkv, D = 600, 8, 2, 128
    t = torch.bfloat16
    N = (Hq + 2 * Hkv) * D
    cos, sin = (dev(a) for a in tables(T, D))
    pos, w = torch.arange(T, device=DEV), dev((1 + 0.1 * values(9, (D,), torch.float32)).to(t))
    args = [[dev(values(10 * k + i, s, t)) for i, s in enumerate(((T, N), (T, Hq * D), (T, Hkv * D)))] for k in range(2)]

    def run(k, stream=None):
        X, dq, dk = args[k]
        out = torch.zeros_like(X), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
        ws = torch.empty(tl.tp_qk_norm_rope_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
        torch.cuda.current_stream().synchronize()
        tl.tp_qk_norm_rope_backward(X, pos, cos, sin, dq, dk, out[0], 2, Hq, Hkv, dV=dk, q_weight=w, k_weight=w, dq_weight=out[1],
                                    dk_weight=out[2], workspace=ws, stream=stream)
        return out, ws

    want = [run(k)[0] for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [run(k, streams[k].cuda_stream) for k in range(2)]
    torch.cuda.synchronize()
    for (g, _), w_ in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w_))


def test_more_wavefronts_than_one_launch_holds():
    # a * 1/2 - b * 2 of small whole numbers: exact in bf16
    T, H, D = 300001, 160, 3
    x = torch.randint(-8, 9, (T, H * D), device=DEV).to(torch.bfloat16)
    cos, sin = torch.full((4, 1), 0.5, device=DEV), torch.full((4, 1), 2.0, device=DEV)
    out = torch.empty_like(x)
    tl.tp_qk_norm_rope(x, torch.full((T,), 2, device=DEV), cos, sin, out, None, 1, H, 0)
    v = x.view(T, H, D)
    a, b = v[..., 0], v[..., 1]
    want = torch.stack([a * 0.5 - b * 2, b * 0.5 + a * 2, v[..., 2]], -1)
    assert torch.equal(out.view(T, H, D), want)


def test_append_of_more_tokens_than_one_launch_holds():
    T, D, page = 2 ** 25 + 77, 16, 65536
    n = (T + page - 1) // page
    x = torch.randint(-99, 99, (T, 2 * D), dtype=torch.int8, device=DEV).to(torch.bfloat16)
    table = torch.randperm(n, device=DEV)[None].to(torch.int32)
    kc, vc = (torch.zeros(n, page, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    tl.tp_kv_append(x, None, None, zero, cu, table, kc, vc, 1, 0, 1, bad=bad)
    for c, part in ((kc, x[:, :D]), (vc, x[:, D:])):
        assert torch.equal(c.view(n, page, D)[table[0].long()].view(-1, D)[:T], part)
    assert not bad.item()
