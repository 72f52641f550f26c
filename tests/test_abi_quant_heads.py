"""CPU tests of the argument checks of the 8-bit Linear and the per-head steps.
Every call is refused, or is an empty problem, before anything is queued: fake
non-null addresses are never dereferenced and no kernel runs."""
import ctypes

import pytest
import torch

import tensor_linear_amd as tl

A = [0x100000 * i for i in range(1, 16)]     # fake device addresses, 256-byte aligned


def quantize(**kw):
    a = dict(X=A[0], ldx=8, Q=A[1], ldq=8, s=A[2], lds=2, M=4, K=8, G=2, dtype=tl.TP_BF16)
    a.update(kw)
    return tl.lib.tp_quantize_rows(*a.values(), None)


def column(**kw):
    a = dict(X=A[0], ldx=8, xs=A[1], ldxs=1, W=A[2], ldw=8, ws=A[3], b=None, Y=A[4], ldy=12, y_mode=tl.TP_Y_CONCAT,
             act=tl.TP_ACT_NONE, M=4, N=12, K=8, P=4, dtype=tl.TP_BF16)
    a.update(kw)
    return tl.lib.tp_linear_column_quant(*a.values(), None)


def row(**kw):
    a = dict(X=A[0], ldx=8, xs=A[1], ldxs=4, G=4, W=A[2], ldw=8, ws=A[3], b=None, Y=A[4], ys=None, ldy=12, ss=0,
             mode=tl.TP_ROW_SUM, wk=A[5], wkb=1 << 20, M=4, N=12, K=8, P=4, dtype=tl.TP_BF16)
    a.update(kw)
    return tl.lib.tp_linear_row_quant(*a.values(), None)


ROT = dict(cos=A[6], sin=A[7], n_pos=16, R=8, style=tl.TP_ROPE_HALVES, wq=A[8], wk=A[9], eps=1e-6)
HEADS = dict(T=3, Hq=4, Hkv=2, D=8, P=2, dtype=tl.TP_BF16, bad=None)


def qk(**kw):
    a = dict(X=A[0], ldx=64, x_mode=tl.TP_Y_CONCAT, pos=A[1], **ROT, Q=A[2], ldq=32, K=A[3], ldk=16, **HEADS)
    a.update(kw)
    return tl.lib.tp_qk_norm_rope(*a.values(), None)


def backward(**kw):
    a = dict(X=A[0], ldx=64, x_mode=tl.TP_Y_CONCAT, pos=A[1], **ROT, dQ=A[2], lddq=32, dK=A[3], lddk=16, dV=A[4], lddv=16,
             dX=A[5], lddx=64, dwq=A[10], dwk=A[11], ws=A[12], wsb=1 << 20, **HEADS)
    a.update(kw)
    return tl.lib.tp_qk_norm_rope_backward(*a.values(), None)


def append(**kw):
    a = dict(X=A[0], ldx=64, x_mode=tl.TP_Y_CONCAT, **ROT, cu=A[1], past=A[2], B=2, table=A[3], ldt=4, max_pages=4, kc=A[4],
             vc=A[5], n_pages=6, page=16, sp=256, ss=16, sh=8, Q=A[10], ldq=32, **HEADS)
    a.update(kw)
    return tl.lib.tp_kv_append(*a.values(), None)


def test_quantize_refusals():
    assert quantize(M=0) == tl.TP_OK
    for bad in (dict(M=-1), dict(K=-2), dict(ldx=7), dict(ldq=7), dict(lds=1), dict(G=0), dict(G=65), dict(M=1 << 58)):
        assert quantize(**bad) == tl.TP_ERR_SHAPE, bad
    assert quantize(K=7) == tl.TP_ERR_INDIVISIBLE
    assert quantize(dtype=2) == tl.TP_ERR_DTYPE
    for p in "XQs":
        assert quantize(**{p: None}) == tl.TP_ERR_NULL


def test_column_refusals():
    assert column(M=0) == tl.TP_OK and column(N=0, ldy=1) == tl.TP_OK
    for bad in (dict(M=-1), dict(ldx=7), dict(ldw=7), dict(ldxs=0), dict(ldy=11), dict(P=0), dict(P=65, N=65), dict(ldx=131072, ldw=131072, K=131072),
                dict(M=1 << 58)):
        assert column(**bad) == tl.TP_ERR_SHAPE, bad
    assert column(N=13, ldy=13) == tl.TP_ERR_INDIVISIBLE and column(act=tl.TP_ACT_SWIGLU) == tl.TP_ERR_INDIVISIBLE
    assert column(dtype=7) == tl.TP_ERR_DTYPE and column(act=9) == tl.TP_ERR_MODE and column(y_mode=2) == tl.TP_ERR_MODE
    for p in ("X", "xs", "W", "ws", "Y"):
        assert column(**{p: None}) == tl.TP_ERR_NULL, p


def test_row_refusals():
    assert row(M=0) == tl.TP_OK
    for bad in (dict(G=2), dict(G=0), dict(ldxs=3), dict(ldy=11), dict(ss=-1), dict(K=-8), dict(mode=tl.TP_ROW_SCATTER, ss=3),
                dict(K=4 * 131072, ldx=1 << 20, ldw=1 << 20), dict(G=1, K=131072, ldx=1 << 20, ldw=1 << 20)):
        assert row(**bad) == tl.TP_ERR_SHAPE, bad
    assert row(K=7) == tl.TP_ERR_INDIVISIBLE and row(mode=tl.TP_ROW_SCATTER, M=5) == tl.TP_ERR_INDIVISIBLE
    assert row(mode=4) == tl.TP_ERR_MODE and row(mode=tl.TP_ROW_PARTIAL, b=A[7]) == tl.TP_ERR_MODE
    assert row(ys=(ctypes.c_void_p * 4)(*A[:4])) == tl.TP_ERR_MODE
    assert row(mode=tl.TP_ROW_SCATTER, Y=None, ys=(ctypes.c_void_p * 4)(A[0], None, A[1], A[2])) == tl.TP_ERR_NULL
    for p in ("X", "xs", "W", "ws", "Y"):
        assert row(**{p: None}) == tl.TP_ERR_NULL, p
    for bad in (dict(wk=None), dict(wkb=4), dict(wk=A[5] + 8)):
        assert row(**bad) == tl.TP_ERR_WORKSPACE, bad


@pytest.mark.parametrize("call", [qk, backward, append])
def test_head_refusals(call):
    for bad in (dict(T=-1), dict(Hq=-2), dict(Hkv=-2), dict(D=0), dict(D=1025, ldx=1 << 20), dict(R=7), dict(R=10), dict(R=-2),
                dict(n_pos=-1), dict(ldx=63), dict(P=0), dict(P=65), dict(eps=-1.0), dict(eps=float("nan")), dict(Hq=1 << 20),
                dict(T=1 << 58)):
        assert call(**bad) == tl.TP_ERR_SHAPE, bad
    assert call(Hq=5) == tl.TP_ERR_INDIVISIBLE and call(Hkv=3) == tl.TP_ERR_INDIVISIBLE
    assert call(dtype=3) == tl.TP_ERR_DTYPE
    assert call(x_mode=2) == tl.TP_ERR_MODE and call(style=2) == tl.TP_ERR_MODE
    assert call(cos=None) == tl.TP_ERR_NULL and call(sin=None) == tl.TP_ERR_NULL and call(X=None) == tl.TP_ERR_NULL


def test_qk_refusals():
    assert qk(T=0) == tl.TP_OK
    assert qk(ldq=31) == tl.TP_ERR_SHAPE and qk(ldk=15) == tl.TP_ERR_SHAPE
    assert qk(pos=None) == tl.TP_ERR_NULL and qk(Q=None, K=None) == tl.TP_ERR_NULL


def test_backward_refusals():
    assert backward(T=0, dwq=None, dwk=None) == tl.TP_OK
    for bad in (dict(lddq=31), dict(lddk=15), dict(lddv=15), dict(lddx=63)):
        assert backward(**bad) == tl.TP_ERR_SHAPE, bad
    assert backward(pos=None) == tl.TP_ERR_NULL and backward(dX=None) == tl.TP_ERR_NULL
    assert backward(wq=None) == tl.TP_ERR_NULL and backward(dQ=None, dK=None, dV=None) == tl.TP_ERR_NULL
    for bad in (dict(ws=None), dict(wsb=16), dict(ws=A[12] + 4)):
        assert backward(**bad) == tl.TP_ERR_WORKSPACE, bad
    assert tl.tp_qk_norm_rope_workspace_bytes(-1, 8) == 0 and tl.tp_qk_norm_rope_workspace_bytes(5, 128) >= 2 * 2 * 128 * 4


def test_append_refusals():
    assert append(T=0) == tl.TP_OK and append(B=0) == tl.TP_OK
    for bad in (dict(B=-1), dict(max_pages=5), dict(page=0), dict(n_pages=-1), dict(ldq=31), dict(ss=15), dict(sp=255), dict(sh=7),
                dict(sp=-256), dict(ldt=0), dict(max_pages=1 << 59, ldt=1 << 59)):
        assert append(**bad) == tl.TP_ERR_SHAPE, bad
    for p in ("cu", "past", "table", "kc", "vc"):
        assert append(**{p: None}) == tl.TP_ERR_NULL, p


def test_binding_refusals():
    i8, f32 = torch.zeros((4, 8), dtype=torch.int8), torch.zeros((4, 8))
    with pytest.raises(TypeError):
        tl.tp_quantize_rows(f32, f32, torch.zeros(4))
    with pytest.raises(ValueError):
        tl.tp_quantize_rows(f32, i8, torch.zeros(5))
    with pytest.raises(ValueError, match="GPU"):
        tl.tp_quantize_rows(f32, i8, torch.zeros(4))
    with pytest.raises(TypeError):
        tl.tp_linear_column_quant(f32, torch.zeros(4), i8, torch.zeros(4), f32, 1)
    with pytest.raises(ValueError):
        tl.tp_linear_column_quant(i8, torch.zeros((4, 2)), i8, torch.zeros(4), torch.zeros((4, 4)), 1)
    with pytest.raises(ValueError):
        tl.tp_linear_row_quant(i8, torch.zeros((4, 3)), i8, torch.zeros(4), torch.zeros((4, 4)), 2)
    with pytest.raises(TypeError):
        tl.tp_linear_row_quant(i8, torch.zeros(4, dtype=torch.float64), i8, torch.zeros(4), torch.zeros((4, 4)), 2)
    x, pos, c = torch.zeros((3, 64)), torch.zeros(3, dtype=torch.int64), torch.zeros((9, 4))
    Q, K = torch.zeros((3, 32)), torch.zeros((3, 16))
    for bad in (dict(X=torch.zeros((3, 63))), dict(pos=pos.int()), dict(pos=None), dict(sin=None), dict(sin=torch.zeros((9, 3))), dict(Q=K),
                dict(cos=c.double()), dict(P=3), dict(Hq=0, Hkv=0)):
        a = dict(X=x, pos=pos, cos=c, sin=c, Q=Q, K=K, P=2, Hq=4, Hkv=2)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            tl.tp_qk_norm_rope(**a)
    with pytest.raises(ValueError, match="GPU"):
        tl.tp_qk_norm_rope(x, pos, c, c, Q, K, 2, 4, 2)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kc = torch.zeros((5, 16, 2, 8))
    for bad in (dict(cu=i32(2)), dict(past=pos), dict(table=i32(3, 4)), dict(k_cache=kc.bfloat16()), dict(v_cache=kc.transpose(1, 2)),
                dict(v_cache=kc.transpose(1, 2).contiguous().transpose(1, 2)), dict(q_weight=torch.zeros(7)),
                dict(k_weight=torch.zeros(8, dtype=torch.bfloat16))):
        a = dict(X=x, cos=c, sin=c, past=i32(2), cu=i32(3), table=i32(2, 4), k_cache=kc, v_cache=kc.clone(), P=2, Hq=4, Hkv=2)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            tl.tp_kv_append(**a)


def test_expanded_rows_are_refused():
    """A view whose rows share memory has no leading dimension; taken as one it
    would be read or written past its end."""
    row = torch.zeros((1, 8))
    i8 = torch.zeros((4, 8), dtype=torch.int8)
    with pytest.raises(ValueError, match="row stride"):
        tl.tp_quantize_rows(row.expand(4, 8), i8, torch.zeros(4))
    with pytest.raises(ValueError, match="row stride"):
        tl.tp_linear_column_quant(i8[:1].expand(4, 8), torch.zeros(4), i8, torch.zeros(4), torch.zeros((4, 4)), 1)
    with pytest.raises(ValueError, match="row stride"):
        tl.tp_linear_column_quant(i8, torch.zeros(4), i8, torch.zeros(4), torch.zeros((2, 1, 2)).expand(2, 4, 2), 2, tl.TP_Y_SHARDS)
    with pytest.raises(ValueError, match="row stride"):
        tl.tp_quantize_rows(torch.zeros((4, 8)), i8, torch.zeros(1).expand(4))
    c = torch.zeros((9, 4))
    with pytest.raises(ValueError, match="row stride"):
        tl.tp_qk_norm_rope(torch.zeros((1, 64)).expand(3, 64), torch.zeros(3, dtype=torch.int64), c, c, torch.zeros((3, 32)), None, 2, 4, 2)
