"""The 8-bit integer Linear (tp_quantize_rows, tp_linear_column_quant,
tp_linear_row_quant) against plain computations in 64 bits on the CPU.

Tolerances.  u = 2^-24 is half a step of fp32, half a step of the output type is
u_out = finfo(type).eps / 2.  An output before the activation is fma(fl(fl(acc)
sx), sw, b) with acc exact: the conversion, the product and the multiply-add
round once each, so |error| <= 2 u |acc sx sw| + u |v| to first order, and u_out
|v| for the output.  A fold over P scaled sums adds one rounding a shard, each
at most u times the sum of the |acc_i sx_i|.  The factor 1.01 covers the second
order.  Powers of two as scales make every step exact: those cases are compared
bit for bit."""
import numpy as np
import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV, FOLD_POLICIES, row_fold, workspace

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]


def half_step(t):
    return torch.finfo(t).eps / 2


def ints(seed, shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)


def scales(seed, shape, pow2=False):
    g = torch.Generator().manual_seed(seed)
    if pow2:
        return torch.pow(2.0, torch.randint(-9, -3, shape, generator=g).float())
    return torch.rand(shape, generator=g) * 0.02 + 0.001


def values(seed, shape, t):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(t)


def strided(t, extra, offset=0):
    """t on the GPU as a view of a wider buffer (row stride + extra, first
    element at `offset`), guard values around it."""
    flat = torch.full((t.shape[0] * (t.shape[1] + extra) + offset + 64,), 77, dtype=t.dtype, device=DEV)
    v = flat[offset:offset + t.shape[0] * (t.shape[1] + extra)].view(t.shape[0], -1)[:, :t.shape[1]]
    v.copy_(t)
    return v


# ---- quantize ----------------------------------------------------------------

def quantize_plain(x, G):
    """Whole numbers and scales of x (any float type) from the definition."""
    M, K = x.shape
    x = x.double().view(M, G, K // G)
    a = x.abs().amax(2) if K else torch.zeros(M, G, dtype=torch.float64)
    s = (a / 127).float()
    s[~torch.isfinite(x).all(2)] = float("nan")
    d = s.double()[:, :, None]
    q = torch.where(d > 0, x / torch.where(d > 0, d, 1.0), 0.0).round().clamp(-127, 127)
    return torch.nan_to_num(q, 0.0).to(torch.int8).view(M, K), s


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K,G,extra,offset", [
    (1, 1, 1, 0, 0), (3, 8, 1, 0, 0), (5, 24, 3, 0, 0), (2, 30, 2, 1, 1), (7, 512, 1, 8, 0), (9, 1024, 8, 0, 0),
    (4, 4096, 4, 0, 0), (3, 1800, 1, 8, 8), (6, 2056, 1, 0, 0), (2, 8192, 1, 0, 0), (2, 8200, 1, 0, 0),
    (3, 3000, 3, 3, 0), (2, 40000, 1, 0, 0), (1, 24576, 3, 0, 0), (5, 1023, 1, 0, 1), (2, 2051, 1, 0, 0),
    (3, 6003, 3, 2, 1), (2, 12290, 1, 1, 3), (2, 16392, 1, 0, 0), (3, 16001, 1, 3, 1), (2, 40003, 1, 1, 1), (9, 7, 7, 0, 0),
    (300, 2056, 1, 0, 0), (270, 4091, 1, 2, 1), (130, 32768, 4, 0, 0), (520, 8001, 1, 0, 0), (520, 8200, 1, 0, 0), (515, 16381, 1, 0, 3)])
def test_quantize_matches_definition(M, K, G, extra, offset, t):
    print("quantize", M, K, G, extra, offset, t, flush=True)
    x = values(M * 1000 + K, (M, K), t)
    x[0, 0] = 0.0
    want, ws = quantize_plain(x, G)
    X = strided(x, extra, offset)
    Q = strided(torch.zeros(M, K, dtype=torch.int8), extra, offset)
    sc = torch.full((M, G + 1), -5.0, device=DEV)
    tl.tp_quantize_rows(X, Q, sc[:, :G])
    assert torch.equal(sc[:, :G].cpu(), ws)          # fp32 division, one rounding
    assert torch.equal(Q.cpu(), want)
    assert torch.all(sc[:, G] == -5.0)
    assert torch.all(Q.as_strided((M, extra), (K + extra, 1), Q.storage_offset() + K) == 77) if extra else True


@pytest.mark.parametrize("t", TYPES)
def test_quantize_halves_go_to_even(t):
    # amax 127 * 2^e: the scale is a power of two and halves are exact
    k = torch.arange(-126, 127, dtype=torch.float32)
    x = torch.cat([k + 0.5, torch.tensor([127.0])])[None]
    x = x[:, (x.to(t).float() == x)[0]].repeat(3, 1)        # what the type holds
    x = x * torch.tensor([1.0, 2.0 ** -70, 2.0 ** 80])[:, None]
    want, ws = quantize_plain(x.to(t), 1)
    X = x.to(t).to(DEV)
    Q, s = torch.zeros(x.shape, dtype=torch.int8, device=DEV), torch.zeros(3, device=DEV)
    tl.tp_quantize_rows(X, Q, s)
    assert torch.equal(s.cpu(), ws[:, 0]) and torch.equal(Q.cpu(), want)
    assert torch.equal(want[0], want[1]) and int(want[0].max()) == 127


@pytest.mark.parametrize("K", [40, 4104])
def test_quantize_special_values(K):
    x = values(3, (8, K), torch.float32)
    x[0] = 0.0
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3, 1] = float("-inf")
    x[4] *= 1e-38                                     # subnormal scale
    x[5] = torch.where(torch.arange(K) % 3 == 0, 2.0 ** -149, 0.0)   # smallest value: scale rounds to 0
    x[6] = 3.0e38 * torch.sign(x[6])
    x[7] = x[7] * 2.0 ** -149 * 100                   # a few steps of the smallest value
    want, ws = quantize_plain(x, 1)
    Q, s = torch.zeros((8, K), dtype=torch.int8, device=DEV), torch.zeros(8, device=DEV)
    tl.tp_quantize_rows(x.to(DEV), Q, s)
    assert torch.equal(torch.nan_to_num(s.cpu(), -1.0), torch.nan_to_num(ws[:, 0], -1.0))
    assert torch.isnan(s[1:4]).all() and float(s[0]) == 0.0 and float(s[5]) == 0.0
    assert torch.equal(Q.cpu(), want)


def test_quantize_more_groups_than_one_launch_holds():
    x = torch.randint(-126, 127, (2 ** 23 + 5, 3), device=DEV).float()
    x[:, 1] = 127.0
    q = torch.empty(x.shape, dtype=torch.int8, device=DEV)
    s = torch.empty(len(x), 1, device=DEV)
    tl.tp_quantize_rows(x, q, s)
    assert torch.equal(q.float(), x) and bool((s == 1).all())


# ---- column ------------------------------------------------------------------

COLUMN = [  # M, K, N/P (outputs and, gated, up features), P
    (1, 16, 1, 1), (3, 128, 17, 3), (16, 256, 64, 2), (17, 144, 33, 8), (5, 100, 20, 2), (33, 2048, 96, 1),
    (48, 4352, 160, 2), (64, 640, 130, 4), (100, 1376, 264, 8), (130, 512, 1000, 2), (257, 1024, 2100, 8),
    (300, 384, 520, 3), (700, 272, 1288, 8), (40, 33, 70, 2), (260, 129, 66, 1), (1025, 128, 4104, 8), (20, 0, 24, 2),
    (70, 2064, 200, 2), (200, 2176, 130, 3), (1, 4112, 40, 1), (129, 4000, 68, 1)]


def column_plain(x, sx, w, sw, b, P, act):
    """Outputs [M, P, outputs] and their error bounds before the output's rounding."""
    M, N = x.shape[0], w.shape[0]
    acc = x.double() @ w.double().t()
    v = acc * sx.double()[:, None] * sw.double()
    err = 2 * U * v.abs()
    if b is not None:
        v = v + b.double()
    err = err + U * v.abs()
    v, err = v.view(M, P, N // P), err.view(M, P, N // P)
    if not act:
        return v, err
    h = N // P // 2
    g, u, eg, eu = v[..., :h], v[..., h:], err[..., :h], err[..., h:]
    s = torch.sigmoid(g)
    y = g * s * u
    slope = (s * (1 + g * (1 - s))).abs()
    # the fast exponential: its argument rounds at u |g| log2(e), its result at 2 u; then
    # a sum, a quotient and a product
    # from 1 + e^-g >= 2^126, that is g <= -87.33, on the hardware's reciprocal is subnormal
    # and comes out 0, as does the unit: off by |g| e^g, which falls with -g, so by at most
    # 87.34 * 2^-126 < 1.04e-36
    gone = torch.where(g < -87.3, 1.04e-36, 0.0) * u.abs()
    return y, slope * eg * u.abs() + (g * s).abs() * eu + y.abs() * (1.5 * g.abs() + 8) * U + gone


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("act", [tl.TP_ACT_NONE, tl.TP_ACT_SWIGLU])
@pytest.mark.parametrize("M,K,n,P", COLUMN)
def test_column_quant(M, K, n, P, act, t):
    print("column quant", M, K, n, P, act, t, flush=True)
    N = n * P * (2 if act else 1)
    x, w = ints(M + K, (M, K)), ints(N + K, (N, K))
    sx, sw = scales(1, (M,)), scales(2, (N,)) * 0.1
    for shards, bias in ((False, False), (True, True)):
        b = values(3, (N,), t) if bias else None
        want, err = column_plain(x, sx, w, sw, b, P, act)
        buf = torch.full((P, M, n + 3) if shards else (M, P * n + 3), -7.0, dtype=t, device=DEV)
        Y = buf[..., :n] if shards else buf[:, :P * n]
        tl.tp_linear_column_quant(x.to(DEV), sx.to(DEV), w.to(DEV), sw.to(DEV), Y, P,
                                  tl.TP_Y_SHARDS if shards else tl.TP_Y_CONCAT, bias=None if b is None else b.to(DEV), act=act)
        got = (Y.transpose(0, 1) if shards else Y.reshape(M, P, n)).cpu().double()
        bad = (got - want).abs() - 1.01 * (err + half_step(t) * want.abs() + 2.0 ** -133)
        assert float(bad.max()) <= 0, (shards, float(bad.max()))
        assert torch.all(buf[..., -3:] == -7.0)


@pytest.mark.parametrize("M,K,N,P", [(16, 512, 256, 2), (64, 1024, 512, 4), (300, 256, 768, 3), (512, 640, 2048, 8),
                                     (7, 75, 30, 3), (33, 8192, 64, 2)])
@pytest.mark.parametrize("t", TYPES)
def test_column_quant_exact_with_power_of_two_scales(M, K, N, P, t):
    x, w = ints(5, (M, K)), ints(6, (N, K))
    x[0], w[0] = -128, -128                          # the largest sums
    sx, sw = scales(7, (M,), True), scales(8, (N,), True)
    want = ((x.double() @ w.double().t()).float() * sx[:, None] * sw).to(t)
    Y = torch.empty((M, N), dtype=t, device=DEV)
    tl.tp_linear_column_quant(x.to(DEV), sx.to(DEV), w.to(DEV), sw.to(DEV), Y, P)
    assert torch.equal(Y.cpu(), want)


@pytest.mark.parametrize("M", [4, 40, 300])
def test_quant_operands_of_any_stride_and_start(M):
    K, N, P = 272, 144, 2
    x, w = ints(1, (M, K)), ints(2, (N, K))
    sx, sw = scales(3, (M,), True), scales(4, (N,), True)
    want = (x.double() @ w.double().t()).float() * sx[:, None] * sw
    for ex, ox, ew, ow in ((16, 16, 32, 0), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 5, 3), (7, 2, 16, 16)):
        Y = torch.empty((M, N), device=DEV)
        sxd = torch.zeros((M, 3), device=DEV)
        sxd[:, 1] = sx.to(DEV)
        tl.tp_linear_column_quant(strided(x, ex, ox), sxd[:, 1:2], strided(w, ew, ow), sw.to(DEV), Y, P)
        assert torch.equal(Y.cpu(), want), (ex, ox, ew, ow)


@pytest.mark.parametrize("M,K", [(2, 131071), (40, 131056), (130, 131056)])
def test_longest_sum_does_not_overflow(M, K):
    x = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((8, K), -128, dtype=torch.int8, device=DEV)
    Y = torch.empty((M, 8), device=DEV)
    one = torch.ones(M, device=DEV)
    tl.tp_linear_column_quant(x, one, w, one.new_ones(8), Y, 1)
    assert torch.all(Y == float(np.float32(16384 * K)))


def test_nan_scale_marks_its_row():
    M, K, N = 20, 256, 64
    x, w = values(1, (M, K), torch.bfloat16), ints(2, (N, K))
    x[3, 9] = float("inf")
    Q, s = torch.zeros((M, K), dtype=torch.int8, device=DEV), torch.zeros((M, 2), device=DEV)
    tl.tp_quantize_rows(x.to(DEV), Q, s)
    Y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    tl.tp_linear_row_quant(Q, s, w.to(DEV), torch.ones(N, device=DEV), Y, 2, tl.TP_ROW_FUSED, workspace(tl.TP_ROW_FUSED, M, N, 2))
    assert torch.isnan(Y[3]).all() and torch.isfinite(Y[[i for i in range(M) if i != 3]]).all()


# ---- row ---------------------------------------------------------------------

ROW = [  # M, K/P, N, P
    (1, 16, 1, 1), (3, 128, 20, 3), (16, 1024, 64, 8), (16, 512, 8200, 2), (17, 144, 33, 8), (6, 100, 24, 2), (33, 2048, 96, 2),
    (64, 256, 136, 4), (128, 1376, 264, 2), (512, 256, 264, 2), (768, 144, 200, 3), (2048, 48, 136, 8), (48, 1040, 520, 2), (300, 1376, 2056, 3), (520, 256, 1160, 8), (300, 384, 520, 3), (260, 33, 72, 2), (1024, 128, 8200, 4),
    (40, 2064, 136, 3), (100, 2304, 72, 2), (48, 2176, 100, 1), (12, 0, 24, 2)]


def row_plain(x, sx, w, sw, b, P):
    """Y and its error bound: x_scale [M, G]."""
    M, K = x.shape
    G = sx.shape[1]
    Kg = K // G
    parts = torch.stack([(x[:, i * Kg:(i + 1) * Kg].double() @ w[:, i * Kg:(i + 1) * Kg].double().t()) * sx[:, i:i + 1].double()
                         for i in range(G)])
    mag = parts.abs().sum(0) * sw.double()
    y = parts.sum(0) * sw.double()
    y = y if b is None else y + b.double()
    return y, (G + 1) * U * mag + U * y.abs()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("per_shard", [False, True])
@pytest.mark.parametrize("M,Ks,N,P", ROW)
def test_row_quant(M, Ks, N, P, per_shard, t):
    print("row quant", M, Ks, N, P, per_shard, t, flush=True)
    K, G = Ks * P, P if per_shard else 1
    x, w = ints(M + K, (M, K)), ints(N + K, (N, K))
    sx, sw = scales(1, (M, G)), scales(2, (N,)) * 0.1
    xd, wd, sxd, swd = x.to(DEV), w.to(DEV), sx.to(DEV), sw.to(DEV)
    outs = {}
    for bias in (False, True):
        b = values(3, (N,), t) if bias else None
        bd = None if b is None else b.to(DEV)
        want, err = row_plain(x, sx, w, sw, b, P)
        for mode in (tl.TP_ROW_SUM, tl.TP_ROW_FUSED) + ((tl.TP_ROW_SCATTER,) if M % P == 0 else ()):
            buf = torch.full((M, N + 3), -7.0, dtype=t, device=DEV)
            tl.tp_linear_row_quant(xd, sxd, wd, swd, buf[:, :N], P, mode, workspace(mode, M, N, P), bias=bd)
            got = buf[:, :N].cpu()
            for policy in FOLD_POLICIES[1:]:          # the other kernels that take the shape
                other = torch.full((M, N + 3), -7.0, dtype=t, device=DEV)
                with row_fold(policy):
                    tl.tp_linear_row_quant(xd, sxd, wd, swd, other[:, :N], P, mode, workspace(mode, M, N, P), bias=bd)
                assert torch.equal(other[:, :N].cpu(), got) and torch.all(other[:, N:] == -7.0)
            bad = (got.double() - want).abs() - 1.01 * (err + half_step(t) * want.abs() + 2.0 ** -133)
            assert float(bad.max()) <= 0, (mode, bias, float(bad.max()))
            assert torch.all(buf[:, N:] == -7.0)
            assert torch.equal(outs.setdefault(bias, got), got), "the modes give the same bits"
        if M % P == 0:
            ys = [torch.full((M // P, N), -7.0, dtype=t, device=DEV) for _ in range(P)]
            tl.tp_linear_row_quant(xd, sxd, wd, swd, None, P, tl.TP_ROW_SCATTER, workspace(tl.TP_ROW_SCATTER, M, N, P), bias=bd, y_slices=ys)
            assert torch.equal(torch.cat(ys).cpu(), outs[bias])
            with row_fold("gemm"):
                ys = [torch.full((M // P, N), -7.0, dtype=t, device=DEV) for _ in range(P)]
                tl.tp_linear_row_quant(xd, sxd, wd, swd, None, P, tl.TP_ROW_SCATTER, workspace(tl.TP_ROW_SCATTER, M, N, P), bias=bd, y_slices=ys)
                assert torch.equal(torch.cat(ys).cpu(), outs[bias])
            gap = torch.full((P * (M // P * N + 40),), -7.0, dtype=t, device=DEV)
            tl.tp_linear_row_quant(xd, sxd, wd, swd, gap[:M // P * N].view(M // P, N), P, tl.TP_ROW_SCATTER,
                                   workspace(tl.TP_ROW_SCATTER, M, N, P), bias=bd, y_slice_stride=M // P * N + 40)
            gap = gap.view(P, -1)
            assert torch.equal(gap[:, :M // P * N].reshape(M, N).cpu(), outs[bias]) and torch.all(gap[:, M // P * N:] == -7.0)
    parts = torch.full((P, M, N), -7.0, device=DEV)
    tl.tp_linear_row_quant(xd, sxd, wd, swd, parts, P, tl.TP_ROW_PARTIAL)
    for i in range(P):
        p = (x[:, i * Ks:(i + 1) * Ks].double() @ w[:, i * Ks:(i + 1) * Ks].double().t()) * sx[:, i * (G > 1)][:, None].double() * sw.double()
        assert float(((parts[i].cpu().double() - p).abs() - 1.01 * 3 * U * p.abs()).max()) <= 0


def test_row_with_one_scale_does_not_depend_on_the_split():
    M, K, N = 96, 1920, 200
    x, w, sx, sw = ints(1, (M, K)).to(DEV), ints(2, (N, K)).to(DEV), scales(3, (M,)).to(DEV), scales(4, (N,)).to(DEV)
    outs = []
    for P in (1, 2, 3, 5, 8, 15):
        Y = torch.empty((M, N), device=DEV)
        tl.tp_linear_row_quant(x, sx, w, sw, Y, P, tl.TP_ROW_SUM, workspace(tl.TP_ROW_SUM, M, N, P))
        outs.append(Y)
    assert all(torch.equal(o, outs[0]) for o in outs)


# ---- used together -------------------------------------------------------------

@pytest.mark.parametrize("M", [5, 72, 300])
def test_gated_layer_in_8_bits_follows_the_16_bit_layer(M):
    """quantize -> gate+up -> quantize per shard -> down, against the same
    steps in 64 bits; and captured in a graph, replayed on new inputs."""
    H, I, P = 512, 1024, 4
    t = torch.bfloat16
    wgu, wd = values(1, (2 * I, H), t), values(2, (H, I), t) * 0.1
    q1, s1 = torch.empty((2 * I, H), dtype=torch.int8, device=DEV), torch.empty(2 * I, device=DEV)
    q2, s2 = torch.empty((H, I), dtype=torch.int8, device=DEV), torch.empty(H, device=DEV)
    tl.tp_quantize_rows(wgu.to(DEV), q1, s1)
    tl.tp_quantize_rows(wd.to(DEV), q2, s2)
    X = values(3, (M, H), t).to(DEV)
    xq, xs = torch.empty((M, H), dtype=torch.int8, device=DEV), torch.empty((M, 1), device=DEV)
    Hh, hq, hs = (torch.empty((M, I), dtype=t, device=DEV), torch.empty((M, I), dtype=torch.int8, device=DEV),
                  torch.empty((M, P), device=DEV))
    Y, ws = torch.empty((M, H), dtype=t, device=DEV), workspace(tl.TP_ROW_FUSED, M, H, P)

    def layer():
        tl.tp_quantize_rows(X, xq, xs)
        tl.tp_linear_column_quant(xq, xs, q1, s1, Hh, P, act=tl.TP_ACT_SWIGLU)
        tl.tp_quantize_rows(Hh, hq, hs)
        tl.tp_linear_row_quant(hq, hs, q2, s2, Y, P, tl.TP_ROW_FUSED, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for r in range(3):
        X.copy_(values(10 + r, (M, H), t).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = Y.clone()
        layer()
        torch.cuda.synchronize()
        assert torch.equal(got, Y), f"replay {r}"
        # each step against 64 bits on the step's own inputs
        xw, xsw = quantize_plain(X.cpu(), 1)
        assert torch.equal(xw, xq.cpu()) and torch.equal(xsw, xs.cpu())
        want, err = column_plain(xq.cpu(), xs[:, 0].cpu(), q1.cpu(), s1.cpu(), None, P, 1)
        assert float(((Hh.cpu().double() - want.reshape(M, I)).abs() - 1.01 * (err.reshape(M, I) + half_step(t) * want.reshape(M, I).abs())).max()) <= 0
        hw, hsw = quantize_plain(Hh.cpu(), P)
        assert torch.equal(hw, hq.cpu()) and torch.equal(hsw, hs.cpu())
        want, err = row_plain(hq.cpu(), hs.cpu(), q2.cpu(), s2.cpu(), None, P)
        assert float(((Y.cpu().double() - want).abs() - 1.01 * (err + half_step(t) * want.abs())).max()) <= 0


def test_quant_on_another_stream_and_repeated():
    M, K, N, P = 300, 1024, 1000, 4
    x, w, sx, sw = ints(1, (M, K)).to(DEV), ints(2, (N, K)).to(DEV), scales(3, (M, P)).to(DEV), scales(4, (N,)).to(DEV)
    Y0 = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    tl.tp_linear_row_quant(x, sx, w, sw, Y0, P, tl.TP_ROW_FUSED, workspace(tl.TP_ROW_FUSED, M, N, P))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        Y = torch.empty_like(Y0)
        ws = workspace(tl.TP_ROW_FUSED, M, N, P)
        side.wait_stream(torch.cuda.current_stream())
        tl.tp_linear_row_quant(x, sx, w, sw, Y, P, tl.TP_ROW_FUSED, ws, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(Y, Y0)
