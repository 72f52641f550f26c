"""Workspaces whose elements do not lie one behind the other: an expanded one
names more bytes than it has, a strided one would have the bytes between its
elements overwritten.  Refused before anything is queued (CPU only)."""
import pytest
import torch

import tensor_linear_amd as tl

BAD = {"expanded": lambda: torch.empty(1, dtype=torch.uint8).expand(1 << 20),
       "strided": lambda: torch.empty((1 << 10, 1 << 10), dtype=torch.uint8)[:, ::2]}


@pytest.mark.parametrize("kind", BAD)
def test_row_quant(kind):
    i8 = lambda *n: torch.zeros(n, dtype=torch.int8)  # noqa: E731
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        tl.tp_linear_row_quant(i8(4, 8), torch.zeros(4, 2), i8(6, 8), torch.zeros(6), torch.zeros(4, 6), 2, tl.TP_ROW_SUM, BAD[kind]())


@pytest.mark.parametrize("kind", BAD)
def test_qk_norm_rope_backward(kind):
    D, z = 8, torch.zeros
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        tl.tp_qk_norm_rope_backward(z(3, 4 * D), None, None, None, z(3, 2 * D), z(3, D), z(3, 4 * D), 1, 2, 1, q_weight=z(D),
                                    dq_weight=z(D), workspace=BAD[kind]())
