"""Int8 products on the tile shapes that only larger products take (256 CUs),
compared as in test_gpu_quant.py, with its tolerances."""
import pytest
import torch

import test_gpu_quant as base

pytestmark = pytest.mark.gpu

ACTS = [base.tl.TP_ACT_NONE, base.tl.TP_ACT_SWIGLU]


@pytest.mark.parametrize("t", base.TYPES)
@pytest.mark.parametrize("M,K,n,P,act", [
    (200, 272, 2100, 8, ACTS[0]), (256, 512, 3584, 8, ACTS[0]),       # 256 x 128 narrow tiles, with and without a K tail
    (200, 272, 1800, 8, ACTS[1]), (256, 512, 1792, 8, ACTS[1]),       # and with the gated unit
    (1025, 400, 2056, 8, ACTS[0]), (1025, 400, 2056, 8, ACTS[1])])    # 256 x 256, several tiles a workgroup, 4 K steps
def test_column(M, K, n, P, act, t):
    base.test_column_quant(M, K, n, P, act, t)


@pytest.mark.parametrize("t", base.TYPES)
@pytest.mark.parametrize("M,Ks,N,P", [(1024, 272, 8200, 2), (1024, 384, 8200, 2)])   # 260 tiles of 256 x 128, 3 K steps a shard
def test_row_with_the_fold_in_registers(M, Ks, N, P, t):
    base.test_row_quant(M, Ks, N, P, True, t)
