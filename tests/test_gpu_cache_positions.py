"""Positions that a sequence's offsets and past give beyond 32 bits: none of the table's."""
import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("int8", [False, True])
def test_read_past_32_bits(int8, t):
    """A past of 2^31 - 1 and a sequence that begins 2^31 rows before the call: row t's position is 2^32 - 1 + t."""
    T, Hkv, D, page = 5, 2, 16, 4
    g = torch.Generator().manual_seed(1)
    if int8:
        kc, vc = (torch.randint(1, 128, (6, page, Hkv, D), generator=g).to(torch.int8).to(DEV) for _ in "kv")
        scales = dict(k_scale=torch.ones((6, page, Hkv), device=DEV), v_scale=torch.ones((6, page, Hkv), device=DEV))
    else:
        kc, vc = (torch.rand((6, page, Hkv, D), generator=g).add_(1.0).to(t).to(DEV) for _ in "kv")
        scales = {}
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table = i32([[3, 1, 0, 5]])
    for cu, past, ok in (([-2 ** 31, T], [2 ** 31 - 1], False), ([-2 ** 31 + 6, T], [2 ** 31 - 1], False), ([-4, T], [0], True), ([-4, T], [12], False)):
        K, V = (torch.full((T, Hkv * D), 9.0, dtype=t, device=DEV) for _ in "kv")
        bad = torch.zeros(1, dtype=torch.int32, device=DEV)
        tl.tp_kv_read(i32(past), i32(cu), table, kc, vc, K, V, bad=bad, **scales)
        assert bad.item() == (0 if ok else 1)
        for got, cache in ((K, kc), (V, vc)):
            if ok:
                want = cache[table[0].long()].view(4 * page, Hkv * D)[4:4 + T].to(t)
                assert torch.equal(got, want)
            else:
                assert (got == 0).all()
