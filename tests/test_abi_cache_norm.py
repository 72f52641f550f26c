"""CPU tests of the argument checks of the calls on a cache in 8 bits, of attention
over a paged cache, and of the step between two blocks.  Every call is refused, or is
an empty problem, before anything is queued: fake non-null addresses are never
dereferenced and no kernel runs."""
import pytest
import torch

import tensor_linear_amd as tl

A = [0x100000 * i for i in range(1, 24)]     # fake device addresses, 256-byte aligned
ROT = dict(cos=A[6], sin=A[7], n_pos=16, R=8, style=tl.TP_ROPE_HALVES, wq=A[8], wk=A[9], eps=1e-6)
SEQ = dict(cu=A[1], past=A[2], B=2, table=A[3], ldt=4, max_pages=4, kc=A[4], vc=A[5], n_pages=6, page=16, sp=256, ss=16, sh=8)
SCALES = dict(ks=A[11], vs=A[12], ssp=32, sss=2, ssh=1)


def append(**kw):
    a = dict(X=A[0], ldx=64, x_mode=tl.TP_Y_CONCAT, **ROT, **SEQ, **SCALES, Q=A[10], ldq=32, T=3, Hq=4, Hkv=2, D=8, P=2, dtype=tl.TP_BF16, bad=None)
    a.update(kw)
    return tl.lib.tp_kv_append_quant(*a.values(), None)


def read(**kw):
    a = dict(**SEQ, **SCALES, K=A[13], ldk=16, V=A[14], ldv=16, T=3, Hkv=2, D=8, dtype=tl.TP_BF16, bad=None)
    a.update(kw)
    return tl.lib.tp_kv_read(*a.values(), None)


def attention(**kw):
    a = dict(Q=A[0], ldq=32, **SEQ, **SCALES, scale=1.0, window=0, O=A[10], ldo=32, lse=A[13], ldl=4, ws=A[14], wsb=1 << 30, T=3, Hq=4, Hkv=2, D=8,
             dtype=tl.TP_BF16, bad=None)
    a.update(kw)
    return tl.lib.tp_kv_attention(*a.values(), None)


def norm(**kw):
    a = dict(Y=A[0], ldy=8, R=A[1], ldr=8, gate=A[2], ldg=8, post=A[3], pre=A[4], alpha=1.0, beta=1.0, eps=1e-6, H=A[5], ldh=8, N=A[6], ldn=8, s=A[7],
             T=3, F=8, dtype=tl.TP_BF16)
    a.update(kw)
    return tl.lib.tp_residual_norm(*a.values(), None)


def backward(**kw):
    a = dict(Y=A[0], ldy=8, R=A[1], ldr=8, gate=A[2], ldg=8, post=A[3], pre=A[4], alpha=1.0, beta=1.0, eps=1e-6, dH=A[5], lddh=8, dN=A[6], lddn=8,
             dY=A[7], lddy=8, dR=A[8], lddr=8, dg=A[9], lddg=8, dpost=A[10], dpre=A[11], ws=A[12], wsb=1 << 30, T=3, F=8, dtype=tl.TP_BF16)
    a.update(kw)
    return tl.lib.tp_residual_norm_backward(*a.values(), None)


def test_append_refusals():
    assert append(T=0) == tl.TP_OK and append(B=0) == tl.TP_OK
    for bad in (dict(T=-1), dict(B=-1), dict(D=0), dict(R=7), dict(ldx=63), dict(ldq=31), dict(page=0), dict(ldt=3), dict(n_pages=-1), dict(max_pages=-1),
                dict(sh=7), dict(ss=15), dict(sp=255), dict(sp=-256), dict(ssh=0), dict(sss=1), dict(ssp=31), dict(ssp=-32), dict(eps=float("nan")),
                dict(sp=1 << 59), dict(ssp=1 << 59), dict(max_pages=1 << 50, ldt=1 << 50, page=1 << 20)):
        assert append(**bad) == tl.TP_ERR_SHAPE, bad
    assert append(Hq=5) == tl.TP_ERR_INDIVISIBLE and append(dtype=5) == tl.TP_ERR_DTYPE and append(style=3) == tl.TP_ERR_MODE and append(x_mode=7) == tl.TP_ERR_MODE
    for p in ("X", "cos", "sin", "cu", "past", "table", "kc", "vc", "ks", "vs"):
        assert append(**{p: None}) == tl.TP_ERR_NULL, p


@pytest.mark.parametrize("call", [read, attention])
def test_cache_refusals(call):
    assert call(T=0) == tl.TP_OK and call(B=0) == tl.TP_OK
    for bad in (dict(T=-1), dict(B=-1), dict(Hkv=-2), dict(Hkv=1 << 17, Hq=1 << 17) if call is attention else dict(Hkv=1 << 17), dict(D=0), dict(D=1025),
                dict(page=0), dict(ldt=3), dict(ldt=0, max_pages=0), dict(n_pages=-1), dict(max_pages=-1), dict(sp=-1), dict(ss=-1), dict(sh=-1), dict(ssp=-1),
                dict(sss=-1), dict(ssh=-1), dict(sp=1 << 60), dict(ssp=1 << 60), dict(B=1 << 59)):
        assert call(**bad) == tl.TP_ERR_SHAPE, bad
    assert call(dtype=2) == tl.TP_ERR_DTYPE
    for p in ("cu", "past", "table", "kc", "vc"):
        assert call(**{p: None}) == tl.TP_ERR_NULL, p
    assert call(ks=None) == tl.TP_ERR_NULL and call(vs=None) == tl.TP_ERR_NULL


def test_read_refusals():
    assert read(Hkv=0) == tl.TP_OK
    for bad in (dict(ldk=15), dict(ldv=15), dict(ldk=1 << 60)):
        assert read(**bad) == tl.TP_ERR_SHAPE, bad
    assert read(K=None, V=None) == tl.TP_ERR_NULL


def test_attention_refusals():
    assert attention(Hq=0) == tl.TP_OK
    for bad in (dict(ldq=31), dict(ldo=31), dict(ldl=3), dict(Hkv=0), dict(Hq=-4), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(window=-1), dict(T=1 << 31), dict(B=1 << 31), dict(ldq=1 << 60)):
        assert attention(**bad) == tl.TP_ERR_SHAPE, bad
    assert attention(Hq=5, ldq=40, ldo=40, ldl=5) == tl.TP_ERR_INDIVISIBLE
    assert attention(Q=None) == tl.TP_ERR_NULL and attention(O=None) == tl.TP_ERR_NULL
    need = tl.tp_kv_attention_workspace_bytes(3, 2, 4, 2, 8)
    if need:
        for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=A[14] + 64)):
            assert attention(**bad) == tl.TP_ERR_WORKSPACE, bad
    for sizes in ((-1, 2, 4, 2, 8), (3, -1, 4, 2, 8), (3, 2, 5, 2, 8), (3, 2, 4, 0, 8), (3, 2, 4, 2, 0), (3, 2, 4, 2, 1025), (1 << 31, 2, 4, 2, 8)):
        assert tl.tp_kv_attention_workspace_bytes(*sizes) == 0, sizes
    for sizes in ((1, 1, 1, 1, 1), (1 << 20, 1, 64, 8, 128), (64, 64, 64, 1, 256), (1 << 30, 1 << 30, 1 << 16, 1 << 16, 256), (4096, 1, 80, 1, 256), (7, 7, 33, 1, 64)):
        assert tl.tp_kv_attention_workspace_bytes(*sizes) <= 256 << 20, sizes


def test_norm_refusals():
    assert norm(T=0) == tl.TP_OK and norm(F=0, s=None, ldg=0) == tl.TP_OK
    for bad in (dict(T=-1), dict(F=-1), dict(F=(1 << 20) + 1, ldy=1 << 21), dict(ldy=7), dict(ldr=7), dict(ldg=7), dict(ldg=-8), dict(ldh=7), dict(ldn=7),
                dict(eps=-1.0), dict(eps=float("nan")), dict(ldy=1 << 60)):
        assert norm(**bad) == tl.TP_ERR_SHAPE, bad
    assert norm(dtype=2) == tl.TP_ERR_DTYPE
    assert norm(Y=None) == tl.TP_ERR_NULL and norm(H=None, N=None, s=None) == tl.TP_ERR_NULL and norm(N=None) == tl.TP_ERR_NULL


def test_backward_refusals():
    assert backward(T=0, dg=None, dpost=None, dpre=None) == tl.TP_OK
    for bad in (dict(T=-1), dict(ldy=7), dict(ldr=7), dict(ldg=7), dict(lddh=7), dict(lddn=7), dict(lddy=7), dict(lddr=7), dict(lddg=7), dict(eps=-1.0)):
        assert backward(**bad) == tl.TP_ERR_SHAPE, bad
    assert backward(dtype=-1) == tl.TP_ERR_DTYPE
    for bad in (dict(gate=None), dict(post=None), dict(pre=None), dict(R=None), dict(Y=None), dict(dH=None, dN=None), dict(dY=None, dR=None, dg=None, dpost=None, dpre=None)):
        assert backward(**bad) == tl.TP_ERR_NULL, bad
    need = tl.tp_residual_norm_workspace_bytes(3, 8)
    assert need >= 3 * 8 * 4
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=A[12] + 4)):
        assert backward(**bad) == tl.TP_ERR_WORKSPACE, bad
    assert tl.tp_residual_norm_workspace_bytes(-1, 8) == 0 and tl.tp_residual_norm_workspace_bytes(3, (1 << 20) + 1) == 0
    # room for 1024 workgroups' sums at most
    assert tl.tp_residual_norm_workspace_bytes(1 << 30, 4096) <= 3 * 1024 * 4096 * 4


def test_binding_refusals():
    """What the binding itself refuses, before the library sees it (host tensors: nothing could run)."""
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    seq = (z(2, t=torch.int32), z(3, t=torch.int32), z(2, 4, t=torch.int32))
    kc, k8, ks = z(6, 16, 2, 8), z(6, 16, 2, 8, t=torch.int8), z(6, 16, 2, t=torch.float32)
    q = z(3, 32)
    for bad, err in ((lambda: tl.tp_kv_attention(q, *seq, kc, kc, q), ValueError),                          # not on a GPU
                     (lambda: tl.tp_kv_attention(q, *seq, k8, k8, q), TypeError),                           # int8 without scales
                     (lambda: tl.tp_kv_attention(q, *seq, kc, kc, q, k_scale=ks, v_scale=ks), TypeError),
                     (lambda: tl.tp_kv_attention(q, *seq, k8, k8, q, k_scale=ks), ValueError),
                     (lambda: tl.tp_kv_attention(q, *seq, k8, k8, q, k_scale=ks[:5], v_scale=ks[:5]), ValueError),
                     (lambda: tl.tp_kv_attention(z(3, 31), *seq, kc, kc, q), ValueError),
                     (lambda: tl.tp_kv_attention(q, *seq, kc, kc, z(3, 33)), ValueError),
                     (lambda: tl.tp_kv_attention(q, *seq, kc, kc, z(3, 32, t=torch.float32)), TypeError),
                     (lambda: tl.tp_kv_attention(q, *seq, kc, kc[..., :4], q), ValueError),
                     (lambda: tl.tp_kv_attention(q, *seq, kc[0], kc[0], q), ValueError),
                     (lambda: tl.tp_kv_attention(q, seq[0], seq[1][:2], seq[2], kc, kc, q), ValueError),
                     (lambda: tl.tp_kv_attention(q, seq[0].long(), seq[1], seq[2], kc, kc, q), ValueError),
                     (lambda: tl.tp_kv_attention(q, *seq, kc, kc, q, lse=z(3, 4)), TypeError),
                     (lambda: tl.tp_kv_attention(q, *seq, kc, kc, q, lse=z(3, 5, t=torch.float32)), ValueError),
                     (lambda: tl.tp_kv_attention(q, *seq, kc, kc, None), ValueError),
                     (lambda: tl.tp_kv_read(*seq, kc, kc, None, None), ValueError),
                     (lambda: tl.tp_kv_read(*seq, kc, kc, z(3, 15), None), ValueError),
                     (lambda: tl.tp_kv_read(*seq, k8, k8, z(3, 16), z(4, 16), k_scale=ks, v_scale=ks), ValueError),
                     (lambda: tl.tp_kv_read(*seq, kc, kc, z(3, 16), z(3, 16)), ValueError),
                     (lambda: tl.tp_kv_append_quant(z(3, 64), None, None, *seq, kc, kc, ks, ks, 1, 4, 2), TypeError),
                     (lambda: tl.tp_kv_append_quant(z(3, 64), None, None, *seq, k8, k8, ks, None, 1, 4, 2), ValueError),
                     (lambda: tl.tp_kv_append_quant(z(3, 64), None, None, *seq, k8, k8, ks, ks.transpose(0, 1).contiguous().transpose(0, 1), 1, 4, 2), ValueError),
                     (lambda: tl.tp_kv_append_quant(z(3, 64), None, None, *seq, k8, k8, ks, ks, 1, 4, 2), ValueError),
                     (lambda: tl.tp_residual_norm(q, q, z(3, 31)), ValueError),
                     (lambda: tl.tp_residual_norm(q, q, q, gate=z(4, 32)), ValueError),
                     (lambda: tl.tp_residual_norm(q, q, q, gate=z(31)), ValueError),
                     (lambda: tl.tp_residual_norm(q, q, q, pre_weight=z(32, t=torch.float32)), TypeError),
                     (lambda: tl.tp_residual_norm(q, q, q, scale=z(3, t=torch.float32)), TypeError),
                     (lambda: tl.tp_residual_norm(q, q, None, scale=z(3, t=torch.float32)), ValueError),
                     (lambda: tl.tp_residual_norm(q, q, z(3, 32, t=torch.int8), scale=z(2, t=torch.float32)), ValueError),
                     (lambda: tl.tp_residual_norm(q, z(3, 32, t=torch.float32), q), TypeError),
                     (lambda: tl.tp_residual_norm(q, q, q), ValueError),
                     (lambda: tl.tp_residual_norm_backward(q, q, q, q, pre_weight=z(32), dpre_weight=z(32)), TypeError),
                     (lambda: tl.tp_residual_norm_backward(q, q, q, q, gate=z(3, 32), dgate=z(32, t=torch.float32)), ValueError),
                     (lambda: tl.tp_residual_norm_backward(q, q, q, q), ValueError)):
        with pytest.raises(err):
            bad()
