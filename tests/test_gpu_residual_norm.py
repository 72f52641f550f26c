"""The step between two blocks (norm, gate, residual, norm) and its gradients against
the definition in 64 bits on the CPU, the gradients also against differences.

Tolerances.  u = 2^-24, u_out = finfo(type).eps / 2.  A norm's sum of F squares is off by
at most (F + 6) u relative, halved by the root, which is off by 2 u itself; in the order
of these sums (strands, then trees) far less, but the bound is kept: f = (F / 2 + 12) u.
So u = f |u|; h is off by e_h = f beta |g u| + 4 u (alpha |R| + beta |g u|); n by its own
f |n|, by e_h r |pre| and by the root's change |n| sum(|h| e_h) / sum(h^2); each output by
u_out of itself.  Gradients: products and sums of terms that are off by these, bounded by
running the formulas on magnitudes: K f times the sum of the terms' magnitudes, with K = 8
for the chain of two norms, and one rounding u for each of the T rows in sums over them.
The factor 1.02 covers the second order."""
import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]


def rnd(seed, *shape, t=torch.float32, s=1.0, mean=0.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * s + mean).to(t)


def norm(x, w, eps):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def forward(Y, R, gate, post, pre, alpha, beta, eps):
    u = norm(Y, post, eps)
    h = beta * (u if gate is None else gate * u) + (0 if R is None else alpha * R)
    return u, h, norm(h, pre, eps)


def bounds(Y, R, gate, post, pre, alpha, beta, eps):
    """Bounds of the errors of h and n before their last rounding."""
    F = Y.shape[1]
    f = (F / 2 + 12) * U
    u, h, n = forward(Y, R, gate, post, pre, alpha, beta, eps)
    b = abs(beta) * (u if gate is None else gate * u).abs()
    r = 0 if R is None else abs(alpha) * R.abs()
    eh = (f if post is not None else 0) * b + 4 * U * (b + r)
    if pre is None:
        return u, h, n, eh, eh
    rr = torch.rsqrt(h.square().mean(-1, keepdim=True) + eps)
    shift = (h.abs() * eh).sum(-1, keepdim=True) / h.square().sum(-1, keepdim=True).clamp(min=1e-300)
    return u, h, n, eh, f * n.abs() + eh * rr * pre.abs() + n.abs() * shift


def buffer(x, extra, shift=0):
    """x on the GPU as columns of a wider matrix."""
    if x is None:
        return None
    b = torch.full((x.shape[0], x.shape[1] + extra + shift), 50.0 if x.dtype != torch.int8 else 50, dtype=x.dtype, device=DEV)
    v = b[:, shift:shift + x.shape[1]]
    v.copy_(x)
    return v


def dev(x):
    return None if x is None else x.to(DEV)


PARTS = [  # residual, gate, post, pre
    (True, "none", False, True), (True, "feature", True, True), (False, "none", False, True), (True, "token", True, False), (True, "feature", False, True),
    (False, "token", True, True), (True, "none", True, True), (True, "token", False, True)]
SIZES = [(1, 1), (3, 7), (5, 64), (2, 100), (4, 128), (3, 1000), (7, 1024), (2, 2000), (6, 4096), (1, 5000), (3, 8192), (2, 8200), (2, 16384), (1, 16385), (2, 20001),
         (700, 72), (1, 2), (9, 515)]


def inputs(T, F, parts, t):
    residual, gate, post, pre = parts
    return dict(Y=rnd(1, T, F, t=t), R=rnd(2, T, F, t=t, s=2.0) if residual else None,
                gate=None if gate == "none" else rnd(3, F, t=t, s=0.5) if gate == "feature" else rnd(3, T, F, t=t, s=0.5),
                post=rnd(4, F, t=t, s=0.1, mean=1.0) if post else None, pre=rnd(5, F, t=t, s=0.1, mean=1.0) if pre else None)


def wide(x):
    return {k: None if v is None else v.double() for k, v in x.items()}


def placed(x, extra, shift):
    y = {k: buffer(v, extra, shift) if v is not None and v.dim() == 2 else dev(v) for k, v in x.items()}
    return y["Y"], dict(residual=y["R"], gate=y["gate"], post_weight=y["post"], pre_weight=y["pre"])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("T,F", SIZES)
def test_forward(T, F, parts, t):
    print("norm", T, F, parts, t, flush=True)
    extra, shift = ((0, 0), (8, 8), (3, 1))[(T + F) % 3]
    x = inputs(T, F, parts, t)
    Y, kw = placed(x, extra, shift)
    Hb, Nb = (torch.full((T + 1, F + extra), 9.0, dtype=t, device=DEV) for _ in "hn")
    H, N = Hb[:T, :F], Nb[:T, :F]
    sc = dict(residual_scale=0.75, branch_scale=-1.5, eps=1e-5)
    tl.tp_residual_norm(Y, H, N, **kw, **sc)
    _, h, n, eh, en = bounds(**wide(x), alpha=0.75, beta=-1.5, eps=1e-5)
    half = torch.finfo(t).eps / 2
    tiny = 2.0 ** -126
    for got, want, e in ((H, h, eh), (N, n, en)):
        off = (got.cpu().double() - want).abs()
        assert (off <= 1.02 * e + half * want.abs() + tiny).all(), (off - e - half * want.abs()).max()
    assert (Hb[T] == 9.0).all() and (Nb[T] == 9.0).all() and (Hb[:, F:] == 9.0).all() and (Nb[:, F:] == 9.0).all()
    # either output alone, and the 8-bit form: the same values through the quantizer's rule
    only = torch.empty_like(Hb)[:T, :F]
    tl.tp_residual_norm(Y, only, None, **kw, **sc)
    assert torch.equal(only, H)
    tl.tp_residual_norm(Y, None, only, **kw, **sc)
    assert torch.equal(only, N)
    qb = torch.full((T, F + extra), 77, dtype=torch.int8, device=DEV)
    q, s = qb[:, :F], torch.empty(T, device=DEV)
    only.fill_(3.0)
    tl.tp_residual_norm(Y, only, q, scale=s, **kw, **sc)
    assert torch.equal(only, H)
    big, gs, gq = n.abs().amax(1), s.cpu().double(), q.cpu().double()
    es = en.amax(1) * 1.02 / 127 + 2 * U * big / 127 + 2.0 ** -149
    assert ((gs - big / 127).abs() <= es).all()
    off = (gq * gs[:, None] - n).abs()
    assert (off <= (gs / 2 + 127 * es)[:, None] + 1.02 * en).all()
    assert (gq.abs().amax(1) == 127).all() and (qb[:, F:] == 77).all()
    if t == torch.float32:      # the fp32 norm itself, quantized
        q2, s2 = torch.empty((T, F), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
        tl.tp_quantize_rows(N, q2, s2)
        assert torch.equal(q, q2) and torch.equal(s, s2)


def gradients(Y, R, gate, post, pre, alpha, beta, eps, dH, dN):
    """The gradients from the formulas, and the sums of their terms' magnitudes."""
    F = Y.shape[1]
    u, h, n = forward(Y, R, gate, post, pre, alpha, beta, eps)
    zero = torch.zeros_like(Y)
    dh = zero if dH is None else dH
    mh = dh.abs()
    out, mag = {}, {}
    if dN is not None:
        if pre is None:
            dh, mh = dh + dN, mh + dN.abs()
        else:
            r = torch.rsqrt(h.square().mean(-1, keepdim=True) + eps)
            m, z = h * r, dN * pre
            dh = dh + r * (z - m * (z * m).mean(-1, keepdim=True))
            mh = mh + r * (z.abs() + m.abs() * (z * m).abs().mean(-1, keepdim=True))
            # a change of h through the products of the norm's gradient
            _, _, _, eh, _ = bounds(Y, R, gate, post, pre, alpha, beta, eps)
            em = eh * r / ((F / 2 + 12) * U)
            mh = mh + r * (em * (z * m).abs().mean(-1, keepdim=True) + m.abs() * (z.abs() * em).mean(-1, keepdim=True) +
                           (z.abs() + m.abs() * (z * m).abs().mean(-1, keepdim=True)) * (m.abs() * em).mean(-1, keepdim=True))
            out["pre"], mag["pre"] = (dN * m).sum(0), (dN.abs() * (m.abs() + em + m.abs() * (m.abs() * em).mean(-1, keepdim=True))).sum(0)
    g = 1.0 if gate is None else gate
    ag = 1.0 if gate is None else gate.abs()
    out["R"], mag["R"] = alpha * dh, abs(alpha) * mh
    if gate is not None:
        out["gate"], mag["gate"] = beta * dh * u, abs(beta) * mh * u.abs()
        if gate.dim() == 1:
            out["gate"], mag["gate"] = out["gate"].sum(0), mag["gate"].sum(0)
    du, mu = beta * g * dh, abs(beta) * ag * mh
    if post is not None:
        r1 = torch.rsqrt(Y.square().mean(-1, keepdim=True) + eps)
        v = Y * r1
        out["post"], mag["post"] = (du * v).sum(0), (mu * v.abs()).sum(0)
        w, mw = du * post, mu * post.abs()
        du, mu = r1 * (w - v * (w * v).mean(-1, keepdim=True)), r1 * (mw + v.abs() * (mw * v.abs()).mean(-1, keepdim=True))
    out["Y"], mag["Y"] = du, mu
    return out, mag


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("T,F", SIZES + [(3000, 64), (1500, 520)])
def test_backward(T, F, parts, t):
    print("norm backward", T, F, parts, t, flush=True)
    extra, shift = ((0, 0), (8, 8), (3, 1))[(T + F) % 3]
    x = inputs(T, F, parts, t)
    Y, kw = placed(x, extra, shift)
    dH, dN = rnd(6, T, F, t=t), rnd(7, T, F, t=t)
    sc = dict(residual_scale=0.75, branch_scale=-1.5, eps=1e-5)
    ws = torch.full((max(256, tl.tp_residual_norm_workspace_bytes(T, F)),), 255, dtype=torch.uint8, device=DEV)
    half, f = torch.finfo(t).eps / 2, (F / 2 + 12) * U
    for with_h, with_n in ((True, True), (False, True), (True, False)):
        if not (with_h and with_n) and T * F > 40000:
            continue
        a, b = (dH if with_h else None), (dN if with_n else None)
        want, mag = gradients(**wide(x), alpha=0.75, beta=-1.5, eps=1e-5, dH=None if a is None else a.double(), dN=None if b is None else b.double())
        dYb, dRb, dGb = (torch.full((T + 1, F + extra), 9.0, dtype=t, device=DEV) for _ in range(3))
        out = dict(dY=dYb[:T, :F], dR=dRb[:T, :F] if parts[0] else None,
                   dgate=None if parts[1] == "none" else torch.full((F,), 9.0, device=DEV) if parts[1] == "feature" else dGb[:T, :F],
                   dpost_weight=torch.full((F,), 9.0, device=DEV) if parts[2] else None, dpre_weight=torch.full((F,), 9.0, device=DEV) if parts[3] else None)
        tl.tp_residual_norm_backward(Y, buffer(a, extra, shift), buffer(b, extra, shift), workspace=ws, **kw, **sc, **out)
        for name, key in (("dY", "Y"), ("dR", "R"), ("dgate", "gate"), ("dpost_weight", "post"), ("dpre_weight", "pre")):
            if out[name] is None:
                continue
            got = out[name].cpu().double()
            if key == "pre" and not with_n:
                assert (got == 0).all()
                continue
            last = half if got.dim() == 2 else U * (T + 64)
            e = 1.02 * (8 * f + (U * (T + 64) if got.dim() == 1 else 0)) * mag[key] + last * want[key].abs() + 2.0 ** -126
            off = (got - want[key]).abs()
            assert (off <= e).all(), (name, (off - e).max())
        for buf in (dYb, dRb, dGb):
            assert (buf[T] == 9.0).all() and (buf[:, F:] == 9.0).all()
    # the sums again, bit for bit, and each output without the others
    first = {k: v.clone() for k, v in out.items() if v is not None}
    for k, v in first.items():
        out[k].fill_(4.0)
        tl.tp_residual_norm_backward(Y, buffer(a, extra, shift), buffer(b, extra, shift), workspace=ws, **kw, **sc, **{k: out[k]})
        assert torch.equal(out[k], v), k


@pytest.mark.parametrize("parts", PARTS)
def test_backward_is_the_slope(parts):
    """Differences of the fp32 kernel's outputs in 64-bit sums against its gradients."""
    T, F, d = 3, 96, 2.0 ** -7
    x = inputs(T, F, parts, torch.float32)
    dH, dN = rnd(6, T, F), rnd(7, T, F)
    sc = dict(residual_scale=0.75, branch_scale=-1.5, eps=1e-5)

    def loss(x):
        Y, kw = placed(x, 0, 0)
        H, N = torch.empty_like(Y), torch.empty_like(Y)
        tl.tp_residual_norm(Y, H, N, **kw, **sc)
        return float((H.cpu().double() * dH).sum() + (N.cpu().double() * dN).sum())

    Y, kw = placed(x, 0, 0)
    ws = torch.empty(max(256, tl.tp_residual_norm_workspace_bytes(T, F)), dtype=torch.uint8, device=DEV)
    out = dict(dY=torch.empty_like(Y), dR=torch.empty_like(Y) if parts[0] else None, dgate=None if x["gate"] is None else torch.empty_like(kw["gate"]),
               dpost_weight=torch.empty(F, device=DEV) if parts[2] else None, dpre_weight=torch.empty(F, device=DEV) if parts[3] else None)
    tl.tp_residual_norm_backward(Y, dev(dH), dev(dN), workspace=ws, **kw, **sc, **out)
    for key, name in (("Y", "dY"), ("R", "dR"), ("gate", "dgate"), ("post", "dpost_weight"), ("pre", "dpre_weight")):
        if out[name] is None:
            continue
        way = rnd(9, *x[key].shape)
        hi, lo = ({**x, key: x[key] + s * d * way} for s in (1, -1))
        slope = (loss(hi) - loss(lo)) / (2 * d)
        want = float((out[name].cpu().double() * way).sum())
        # the third derivative's part is of the order d^2; rounding of the outputs over 2 d
        scale = float((out[name].cpu().double() * way).abs().sum()) + 1.0
        assert abs(slope - want) <= scale * (20 * d * d + 100 * U / d), (key, slope, want)


@pytest.mark.parametrize("t", TYPES)
def test_rows_that_are_not_finite(t):
    """A NaN or infinity stays in its row; in 8 bits the row's scale is NaN and its numbers zeros."""
    T, F = 6, 200
    x = inputs(T, F, (True, "feature", True, True), t)
    Y, kw = placed(x, 0, 0)
    H, N = torch.empty_like(Y), torch.empty_like(Y)
    tl.tp_residual_norm(Y, H, N, **kw)
    x["Y"][2, 5], x["R"][4, 9] = float("nan"), float("inf")
    Y2, kw2 = placed(x, 0, 0)
    H2, N2 = torch.empty_like(Y), torch.empty_like(Y)
    tl.tp_residual_norm(Y2, H2, N2, **kw2)
    fine = [0, 1, 3, 5]
    assert torch.equal(H2[fine], H[fine]) and torch.equal(N2[fine], N[fine])
    assert H2[2].isnan().all() and N2[2].isnan().all() and N2[4, 9].isnan()
    q, s = torch.empty((T, F), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    tl.tp_residual_norm(Y2, None, q, scale=s, **kw2)
    assert s.isnan().tolist() == [False, False, True, False, True, False] and (q[2] == 0).all() and (q[4] == 0).all()


def test_zero_rows_and_no_tokens():
    for t in TYPES:
        Y = torch.zeros((3, 64), dtype=t, device=DEV)
        w = torch.ones(64, dtype=t, device=DEV)
        H, N, q, s = torch.empty_like(Y), torch.empty_like(Y), torch.empty((3, 64), dtype=torch.int8, device=DEV), torch.empty(3, device=DEV)
        tl.tp_residual_norm(Y, H, N, post_weight=w, pre_weight=w)
        assert (H == 0).all() and (N == 0).all()
        tl.tp_residual_norm(Y, None, q, post_weight=w, pre_weight=w, scale=s)
        assert (q == 0).all() and (s == 0).all()
        none = Y[:0]
        tl.tp_residual_norm(none, none, none, pre_weight=w)
        ws = torch.empty(max(256, tl.tp_residual_norm_workspace_bytes(0, 64)), dtype=torch.uint8, device=DEV)
        dw = torch.full((64,), 3.0, device=DEV)
        tl.tp_residual_norm_backward(none, none, none, none, pre_weight=w, dpre_weight=dw, workspace=ws)
        assert (dw == 0).all()


def test_graph():
    T, F, t = 33, 512, torch.bfloat16
    x = inputs(T, F, (True, "feature", True, True), t)
    Y, kw = placed(x, 0, 0)
    H, N, q, s = torch.empty_like(Y), torch.empty_like(Y), torch.empty((T, F), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    dY, dR, dg, dp, dq = torch.empty_like(Y), torch.empty_like(Y), *(torch.empty(F, device=DEV) for _ in range(3))
    ws = torch.empty(tl.tp_residual_norm_workspace_bytes(T, F), dtype=torch.uint8, device=DEV)

    def step():
        tl.tp_residual_norm(Y, H, N, **kw)
        tl.tp_residual_norm(Y, None, q, scale=s, **kw)
        tl.tp_residual_norm_backward(Y, H, N, dY, dR, dgate=dg, dpost_weight=dp, dpre_weight=dq, workspace=ws, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (H, N, q, s, dY, dR, dg, dp, dq)
    for i in range(4):
        Y.copy_(rnd(20 + i, T, F, t=t))
        step()
        torch.cuda.synchronize()
        eager = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, outs):
            assert torch.equal(a, b)


def test_more_rows_than_a_launch_holds():
    T, F = (1 << 21) + 5, 8
    Y = torch.randn((T, F), device=DEV).bfloat16()
    w = torch.ones(F, dtype=torch.bfloat16, device=DEV)
    N = torch.empty_like(Y)
    tl.tp_residual_norm(Y, None, N, pre_weight=w)
    want = Y.float() * torch.rsqrt(Y.float().square().mean(1, keepdim=True) + 1e-6)
    assert ((N.float() - want).abs() <= 2.0 ** -8 * want.abs() * 1.02 + 1e-6).all()
