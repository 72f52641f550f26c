"""The 8-bit layers where one launch (fewer than 2^32 threads) does not hold the
work.  Small whole numbers and powers of two as scales: every step is exact, in
bfloat16 too, and the expected values are computed on the GPU piece by piece."""
import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV, workspace

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def small(seed, shape, most):
    """Whole numbers of -most .. most as int8, drawn on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, dtype=torch.int8, device=DEV)


def powers(n):
    """n scales of 1/2, 1, 2 in turn."""
    return torch.tensor([0.5, 1.0, 2.0], device=DEV).repeat(n // 3 + 1)[:n]


def need(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free GPU memory")


def rows_product(x, w):
    """x w^T, a row of x at a time."""
    return torch.stack([(w.float() * row).sum(1) for row in x.float()])


def pieces(n, step):
    return [slice(i, min(i + step, n)) for i in range(0, n, step)]


@pytest.mark.parametrize("M,N", [(4097, 2 ** 20 + 3), (2 ** 26 + 5, 4)])
def test_fold_of_more_outputs_than_one_launch_holds(M, N):
    """A value a thread (N odd) and 16 bytes a lane (a wavefront a row)."""
    print("fold", M, N, flush=True)
    need(60)
    P = 2
    x, w = small(1, (M, P), 2), small(2, (N, P), 3)
    sx, sw = powers(M * P).view(M, P), powers(N)
    bias = small(3, (N,), 5).to(BF)
    Y = torch.full((M, N), 99.0, dtype=BF, device=DEV)
    tl.tp_linear_row_quant(x, sx, w, sw, Y, P, tl.TP_ROW_SUM, workspace(tl.TP_ROW_SUM, M, N, P, zero=False), bias=bias)
    xs, ws = x.float() * sx, w.float() * sw[:, None]
    for r in pieces(M, max(1, 2 ** 28 // N)):
        want = xs[r, :1] * ws[:, 0] + xs[r, 1:] * ws[:, 1] + bias.float()
        assert torch.equal(Y[r], want.to(BF)), r


@pytest.mark.parametrize("M,n,P", [(2 ** 25 + 200, 1, 64), (2 ** 31 + 100, 1, 1)])
def test_generic_column_of_more_tiles_than_one_launch_holds(M, n, P):
    """An odd K: many shards, and many tokens of one."""
    print("generic", M, n, P, flush=True)
    need(60)
    N = n * P
    x, w = small(1, (M, 1), 2), small(2, (N, 1), 3)
    sx, sw = powers(M), powers(N)
    bias = small(3, (N,), 5).to(BF)
    for shards in (False, True) if P > 1 else (False,):
        Y = torch.full((P, M, n) if shards else (M, N), 99.0, dtype=BF, device=DEV)
        tl.tp_linear_column_quant(x, sx, w, sw, Y, P, tl.TP_Y_SHARDS if shards else tl.TP_Y_CONCAT, bias=bias)
        for r in pieces(M, 2 ** 28 // N):
            want = (x[r].float() * sx[r, None] * (w[:, 0].float() * sw) + bias.float()).to(BF)
            assert torch.equal(Y[:, r, 0].t() if shards else Y[r], want), r
        del Y


def test_generic_gated_column_of_more_tiles_than_one_launch_holds():
    """Many hidden units of one shard: gate rows, then up rows."""
    print("generic gated", flush=True)
    need(60)
    n = 2 ** 30 + 100
    x = torch.tensor([[1]], dtype=torch.int8, device=DEV)
    w = small(2, (2 * n, 1), 3)
    w[:n] = 100                              # silu(100) is 100 in fp32
    sw = torch.ones(2 * n, device=DEV)
    sw[n:] = powers(n)
    Y = torch.full((1, n), 99.0, device=DEV)
    tl.tp_linear_column_quant(x, torch.ones(1, device=DEV), w, sw, Y, 1, act=tl.TP_ACT_SWIGLU)
    for r in pieces(n, 2 ** 28):
        up = slice(n + r.start, n + r.stop)
        assert torch.equal(Y[0, r], 100.0 * w[up, 0].float() * sw[up]), r


@pytest.mark.parametrize("M", [1, 3])
def test_skinny_column_of_more_workgroups_than_one_launch_holds(M):
    print("skinny", M, flush=True)
    need(60)
    N, K, P = 2 ** 28 + 64, 16, 2
    x, w = small(1, (M, K), 1), small(2, (N, K), 3)
    sx, sw = powers(M), powers(N)
    bias = small(3, (N,), 5).to(BF)
    Y = torch.full((M, N), 99.0, dtype=BF, device=DEV)
    tl.tp_linear_column_quant(x, sx, w, sw, Y, P, bias=bias)
    for r in pieces(N, 2 ** 26):
        want = rows_product(x, w[r]) * sx[:, None] * sw[r] + bias[r].float()
        assert torch.equal(Y[:, r], want.to(BF)), r


def test_skinny_fold_of_more_workgroups_than_one_launch_holds():
    print("skinny fold", flush=True)
    need(90)
    M, N, K, P = 1, 2 ** 29 + 64, 32, 2
    x, w = small(1, (M, K), 1), small(2, (N, K), 2)
    sx, sw = powers(M * P).view(M, P), powers(N)
    bias = small(3, (N,), 5).to(BF)
    Y = torch.full((M, N), 99.0, dtype=BF, device=DEV)
    tl.tp_linear_row_quant(x, sx, w, sw, Y, P, tl.TP_ROW_FUSED, workspace(tl.TP_ROW_FUSED, M, N, P, zero=False), bias=bias)
    xs = x.float() * sx.repeat_interleave(K // P, 1)
    for r in pieces(N, 2 ** 26):
        want = rows_product(xs, w[r]) * sw[r] + bias[r].float()
        assert torch.equal(Y[:, r], want.to(BF)), r


def test_quantize_more_long_groups_than_one_launch_holds():
    """2^21 groups, and a few, of a workgroup of 1024 threads each."""
    print("quantize", flush=True)
    need(130)
    M, K = 2 ** 21 + 5, 16392
    x = torch.empty((M, K), dtype=BF, device=DEV)
    row = small(1, (K,), 100)
    x[:] = row.to(BF)
    last = (torch.arange(M, device=DEV) % 255 - 127).to(torch.int8)     # a value of its own for each row
    x[:, 0], x[:, K - 1] = 127.0, last.to(BF)
    q, s = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    tl.tp_quantize_rows(x, q, s)
    assert torch.all(s == 1.0) and torch.all(q[:, 0] == 127) and torch.equal(q[:, K - 1], last)
    for r in pieces(M, 2 ** 17):
        assert torch.all(q[r, 1:K - 1] == row[1:K - 1]), r
