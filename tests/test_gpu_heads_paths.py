"""The head steps where a wavefront takes several groups of heads, or several
tokens: prompts and training steps.  With T tokens the forward and the append
split a token's groups of heads over 8192 / T wavefronts, and the backward has 768
workgroups of four for both kinds of heads; the sizes here leave each wavefront
more than one group, the last one ragged.  Compared as in test_gpu_heads.py, with
its tolerances.  And values that are not finite where nothing reads them."""
import pytest
import torch

import tensor_linear_amd as tl
import test_gpu_heads as base
from gpu_util import DEV
from test_gpu_heads import dev, tables, values

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

LONG = [  # T, Hq, Hkv, D, R, P, pairs, norms, shards, extra; type
    ((4100, 20, 4, 128, 128, 2, False, "qk", False, 8), BF),     # 3 groups in 2 parts; gradients: 2 and 6 tokens a wavefront
    ((4100, 20, 4, 128, 128, 2, False, "qk", False, 8), F32),
    ((3500, 20, 9, 128, 120, 1, False, "qk", False, 0), BF),     # R / 2 pairs end inside a lane; 4 groups in 3 parts
    ((3300, 20, 10, 80, 40, 2, True, "qk", True, 1), BF),
    ((3300, 20, 10, 80, 40, 2, False, "qk", False, 0), F32),
    ((2100, 8, 3, 512, 512, 1, False, "qk", False, 0), BF),      # 32 lanes a head: 6 groups in 4 parts
    ((700, 32, 20, 128, 64, 4, False, "qk", False, 0), BF),      # gradients: 4 and 6 groups in 2 parts
    ((700, 32, 20, 128, 64, 4, True, "qk", True, 3), F32),
    ((8200, 96, 16, 16, 16, 8, False, "k", False, 0), BF),       # a lane a head: 2 groups of 64, one part
    ((4200, 40, 8, 64, 32, 4, False, "", True, 0), BF),
    ((2500, 24, 6, 256, 8, 1, True, "q", False, 0), BF)]


@pytest.fixture
def padded(monkeypatch):
    """Padding tokens all over the rows, not only among the first."""
    make = base.make

    def more(case, t):
        out = make(case, t)
        pos = out[5]
        pos[7::61] = -1
        pos[11::97] = out[3].shape[0] + 3
        return out

    monkeypatch.setattr(base, "make", more)


@pytest.mark.parametrize("case,t", LONG)
def test_forward(case, t, padded):
    base.test_qk_norm_rope(case, t)


@pytest.mark.parametrize("case,t", LONG)
def test_backward(case, t, padded):
    base.test_qk_norm_rope_backward(case, t)


@pytest.mark.parametrize("case,t", [
    (([1900, 1, 0, 2195], [5, 0, 3, 60], 16, 4, 128, 128, 2, 16, False, True, False, "nhd", 2), BF),   # 3 groups in 2 parts
    (([2500, 300], [1, 700], 20, 8, 80, 40, 2, 64, True, True, True, "hnd", 0), F32),                   # 5 groups in 3 parts
    (([4100], [0], 36, 6, 64, 16, 6, 32, False, False, False, "nhd", 1), BF)])
def test_append(case, t):
    base.test_kv_append(case, t)


SIZES = [  # T, Hq, Hkv, D, R, P: 16 values a lane (R a multiple of 16, of 8), a value a lane
    (9, 4, 2, 128, 128, 2), (9, 4, 2, 80, 40, 2), (9, 4, 2, 40, 20, 2), (2100, 12, 6, 512, 64, 1)]


def not_finite(t, rows):
    """Those rows of t without a finite value."""
    t = t.clone()
    t[rows] = torch.tensor([float("nan"), float("inf"), float("-inf")], dtype=t.dtype, device=t.device)[
        torch.arange(t.shape[1], device=t.device) % 3]
    return t


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,P", SIZES)
def test_padding_tokens_that_are_not_finite(T, Hq, Hkv, D, R, P, t):
    """A token without a position has zero rows and no gradient, whatever its
    values; nothing of it reaches another token or a weight's gradient."""
    print("padding", T, Hq, Hkv, D, R, P, t, flush=True)
    N, per = (Hq + 2 * Hkv) * D, (Hq + 2 * Hkv) // P * D
    pos = torch.arange(T) % 50
    pad = torch.zeros(T, dtype=torch.bool)
    pad[2::5] = True
    pos[2::10], pos[7::10] = -1, 50
    cos, sin = (dev(a) for a in tables(50, R))
    w = dev((1 + 0.2 * values(9, (D,), F32)).to(t))
    x, dq, dk, dv = (dev(values(i, (T, n), t)) for i, n in enumerate((N, Hq * D, Hkv * D, Hkv * D)))
    pos, pad = dev(pos), dev(pad)
    fwd, bwd = [], []
    for x_, dq_, dk_ in ((x, dq, dk), (not_finite(x, pad), not_finite(dq, pad), not_finite(dk, pad))):
        Q, K = torch.empty_like(dq), torch.empty_like(dk)
        bad = torch.zeros(1, dtype=torch.int32, device=DEV)
        tl.tp_qk_norm_rope(x_, pos, cos, sin, Q, K, P, Hq, Hkv, q_weight=w, k_weight=w, bad=bad)
        assert int(bad) == 1 and torch.all(Q[pad] == 0) and torch.all(K[pad] == 0)
        fwd.append((Q, K))
        dX, dwq, dwk = torch.empty_like(x), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
        ws = torch.empty(tl.tp_qk_norm_rope_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
        tl.tp_qk_norm_rope_backward(x_, pos, cos, sin, dq_, dk_, dX, P, Hq, Hkv, dV=dv, q_weight=w, k_weight=w, dq_weight=dwq,
                                    dk_weight=dwk, workspace=ws)
        g = dX[pad].view(-1, P, per)
        assert torch.all(g[:, :, :per - Hkv // P * D] == 0)
        assert torch.equal(g[:, :, per - Hkv // P * D:].reshape(-1, Hkv * D), dv[pad])
        bwd.append((dX, dwq, dwk))
    for a, b in zip(fwd[0] + bwd[0], fwd[1] + bwd[1]):
        assert torch.isfinite(b).all() and torch.equal(a, b)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,P", SIZES)
def test_rows_of_an_append_that_are_not_finite(T, Hq, Hkv, D, R, P, t):
    """Rows no sequence owns, and rows whose page is not in the cache."""
    print("append padding", T, Hq, Hkv, D, R, P, t, flush=True)
    N, page = (Hq + 2 * Hkv) * D, 4
    B = T // 3                                    # sequences of two tokens from row 2 on; the rest is owned by none
    cu = (2 + 2 * torch.arange(B + 1)).int()
    past = (torch.arange(B) % 7).int()
    table = torch.arange(B * 2).view(B, 2).int()
    lost = torch.arange(B) % 3 == 1
    table[lost] = 2 * B                           # one past the cache
    rows = torch.ones(T, dtype=torch.bool)        # those without a place
    for i in range(B):
        rows[2 + 2 * i:4 + 2 * i] = bool(lost[i])
    cos, sin = (dev(a) for a in tables(9, R))
    w = dev((1 + 0.2 * values(9, (D,), F32)).to(t))
    x = dev(values(1, (T, N), t))
    cu, past, table, rows = dev(cu), dev(past), dev(table), dev(rows)
    owned = torch.zeros(T, dtype=torch.bool, device=DEV)
    owned[2:2 + 2 * B] = True
    outs = []
    for x_ in (x, not_finite(x, rows)):
        kc, vc = (dev(values(i, (2 * B, page, Hkv, D), t)) for i in (30, 31))
        Q = torch.full((T, Hq * D), 9.0, dtype=t, device=DEV)
        bad = torch.zeros(1, dtype=torch.int32, device=DEV)
        tl.tp_kv_append(x_, cos, sin, past, cu, table, kc, vc, P, Hq, Hkv, Q=Q, q_weight=w, k_weight=w, bad=bad)
        assert int(bad) == 1 and torch.all(Q[rows & owned] == 0) and torch.all(Q[~owned] == 9.0)
        outs.append((Q, kc, vc))
    for a, b in zip(*outs):
        assert torch.isfinite(b).all() and torch.equal(a, b)


@pytest.mark.parametrize("D,R", [(128, 128), (80, 40), (40, 20)])
def test_a_head_that_is_not_finite_stays_alone(D, R):
    """The heads beside it, in the same wavefront, and the gradients of the
    other kind are as without it."""
    T, Hq, Hkv, t = 6, 8, 4, BF
    N = (Hq + 2 * Hkv) * D
    cos, sin = (dev(a) for a in tables(9, R))
    pos = torch.arange(T, device=DEV)
    w = dev((1 + 0.2 * values(9, (D,), F32)).to(t))
    x, dq, dk = (dev(values(i, (T, n), t)) for i, n in enumerate((N, Hq * D, Hkv * D)))
    y = x.clone()
    y[3, 5 * D + 1] = float("nan")                       # a query head,
    y[4, (Hq + Hkv + 2) * D] = float("inf")              # a value head
    outs = []
    for x_ in (x, y):
        Q, K, dX, dwk = torch.empty_like(dq), torch.empty_like(dk), torch.zeros_like(x), torch.empty(D, device=DEV)
        tl.tp_qk_norm_rope(x_, pos, cos, sin, Q, K, 1, Hq, Hkv, q_weight=w, k_weight=w)
        ws = torch.empty(tl.tp_qk_norm_rope_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
        tl.tp_qk_norm_rope_backward(x_, pos, cos, sin, dq, dk, dX, 1, Hq, Hkv, q_weight=w, k_weight=w, dk_weight=dwk, workspace=ws)
        outs.append((Q, K, dX, dwk))
    (Q, K, dX, dwk), (Q2, K2, dX2, dwk2) = outs
    for a in (Q2, dX2):
        assert torch.isnan(a[3, 5 * D:6 * D]).all()
        a[3, 5 * D:6 * D] = 0
    for a in (Q, dX):
        a[3, 5 * D:6 * D] = 0
    assert torch.equal(Q, Q2) and torch.equal(K, K2) and torch.equal(dX, dX2) and torch.equal(dwk, dwk2)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("D,R", [(128, 128), (80, 40), (40, 20)])
def test_a_sum_of_squares_past_fp32_is_normed_to_zeros(D, R, t):
    T, Hq, Hkv = 3, 4, 2
    cos, sin = (dev(a) for a in tables(9, R))
    x = dev(values(1, (T, (Hq + 2 * Hkv) * D), t))
    y = x.clone()
    y[1, 2 * D] = 2.0 ** 65                              # its square is past the largest fp32 value
    outs = []
    for x_ in (x, y):
        Q, K = torch.empty((T, Hq * D), dtype=t, device=DEV), torch.empty((T, Hkv * D), dtype=t, device=DEV)
        w = torch.ones(D, dtype=t, device=DEV)
        tl.tp_qk_norm_rope(x_, torch.arange(T, device=DEV), cos, sin, Q, K, 1, Hq, Hkv, q_weight=w, k_weight=w)
        outs.append((Q, K))
    assert torch.all(outs[1][0][1, 2 * D:3 * D] == 0)
    outs[0][0][1, 2 * D:3 * D] = 0
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
