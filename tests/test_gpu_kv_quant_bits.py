"""Keys and values that no norm and no rotation touches, appended in 8 bits: scales and whole numbers bit for bit, from
any number of shards, in either layout of the QKV matrix and either order of the cache in memory."""
import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV
from test_gpu_heads import TYPES, make, split
from test_gpu_kv_quant import Pages, lengths

pytestmark = pytest.mark.gpu

CASES = [  # T, Hq, Hkv, D, R, P, pairs, norms, shards, extra: no rotation (R 0)
    (9, 8, 2, 128, 0, 2, False, "", False, 0), (9, 8, 4, 64, 0, 4, False, "", True, 8), (6, 6, 3, 80, 0, 3, False, "", False, 1),
    (7, 4, 2, 40, 0, 2, False, "", True, 0), (5, 4, 4, 16, 0, 1, False, "", False, 0), (300, 4, 2, 128, 0, 2, False, "q", True, 0),
    (5, 2, 1, 7, 0, 1, False, "", False, 3), (4, 2, 2, 600, 0, 2, False, "q", True, 0), (5, 16, 8, 256, 0, 8, False, "", False, 0)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("order,pad", [("slot", 0), ("head", 5)])
def test_bits(case, order, pad, t):
    print("append bits", case, order, t, flush=True)
    T, Hq, Hkv, D, _, P, _, _, shards, _ = case
    x, X, _, _, _, _, wq, _ = make(case, t)
    lens = lengths(T)
    past = [(7 * s + 3) % 40 for s in range(len(lens))]
    pg = Pages(lens, past, Hkv, D, 16, order, pad, lead=1)
    tl.tp_kv_append_quant(X, None, None, pg.past, pg.cu, pg.table, pg.kc, pg.vc, pg.ks, pg.vs, P, Hq, Hkv, q_weight=None if wq is None else wq.to(DEV),
                          x_mode=tl.TP_Y_SHARDS if shards else tl.TP_Y_CONCAT)
    torch.cuda.synchronize()
    _, k, v = split(x, P, Hq, Hkv, shards)
    rows = [r for _, r, _ in pg.rows]
    pi, si = (torch.tensor(z) for z in zip(*[pg.place(s, p) for s, _, p in pg.rows]))
    for cache, scale, want in ((pg.kc, pg.ks, k), (pg.vc, pg.vs, v)):
        want = want[rows].double()
        s = (want.abs().amax(-1).float() / 127.0)
        q = torch.where(s[..., None] > 0, want / s.double()[..., None], 0.0).round().clamp(-127, 127)
        assert torch.equal(scale.cpu()[pi, si], s)
        assert torch.equal(cache.cpu()[pi, si].double(), q)
