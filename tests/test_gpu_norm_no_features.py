"""Rows of no features between two blocks: into 8 bits they have the scale 0, as tp_quantize_rows gives it."""
import ctypes

import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 5, 300])
def test_scales_of_rows_without_features(T, t):
    x = torch.randn((T, 8), device=DEV).to(t)
    w, q = torch.ones(8, dtype=t, device=DEV), torch.full((T, 8), 7, dtype=torch.int8, device=DEV)
    want = torch.full((T,), 9.0, device=DEV)
    tl.tp_quantize_rows(x[:, :0], q[:, :0], want)
    assert (want == 0).all()
    dt = tl.TP_BF16 if t == torch.bfloat16 else tl.TP_F32
    p = lambda y: None if y is None else y.data_ptr()  # noqa: E731
    # (from C: the addresses of no features need not be NULL)
    for post, pre in ((None, None), (w, None), (None, w), (w, w)):
        for alpha, beta, eps in ((1.0, 1.0, 1e-6), (0.5, float("inf"), 0.0)):
            for H in (None, x):
                for N in (q, None):
                    s = torch.full((T,), 9.0, device=DEV)
                    stream = torch.cuda.current_stream().cuda_stream
                    st = tl.lib.tp_residual_norm(p(x), 8, p(x), 8, p(w), 0, p(post), p(pre), alpha, beta, eps, p(H), 8, p(N), 8, p(s), T, 0, dt, ctypes.c_void_p(stream))
                    assert st == tl.TP_OK
                    torch.cuda.synchronize()
                    assert torch.equal(s, want), (post is None, pre is None, alpha, beta, eps)
    assert (q == 7).all()
    # from Python: views and tensors of no columns
    for Y, N in ((x[:, :0], q[:, :0]), (torch.empty((T, 0), dtype=t, device=DEV), torch.empty((T, 0), dtype=torch.int8, device=DEV))):
        s = torch.full((T,), 9.0, device=DEV)
        tl.tp_residual_norm(Y, None, N, pre_weight=w[:0], scale=s)
        assert torch.equal(s, want)
