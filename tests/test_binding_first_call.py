"""The binding's first call made from two threads at once (CPU only)."""
import sys
import threading
import types

import torch

import tensor_linear_amd as tl


def test_a_second_thread_in_the_middle_of_the_first_call(monkeypatch):
    """While the first call is filling the table of types, another thread asks
    for a type: it must get the type's code, not an empty table's refusal."""
    found = []

    def other():
        try:
            found.append(tl._dtype_code(torch.zeros(1)))
        except Exception as e:
            found.append(e)

    class Slow(types.ModuleType):
        entered = False

        @property
        def bfloat16(self):
            if not Slow.entered:              # the first thread is held here until the second is done
                Slow.entered = True
                t = threading.Thread(target=other)
                t.start()
                t.join()
            return torch.bfloat16

        float32 = torch.float32

    monkeypatch.setattr(tl, "_torch_module", None)
    monkeypatch.setattr(tl, "_DTYPES", {})
    monkeypatch.setitem(sys.modules, "torch", Slow("torch"))
    assert tl._dtype_code(torch.zeros(1, dtype=torch.bfloat16)) == tl.TP_BF16
    assert found == [tl.TP_F32]


def test_a_second_thread_between_the_table_and_the_module(monkeypatch):
    """The table is filled, the module not yet published: what the checks of the
    head steps read must not depend on the module being there."""
    monkeypatch.setattr(tl, "_DTYPES", {torch.bfloat16: tl.TP_BF16, torch.float32: tl.TP_F32})
    T, R, D = 3, 4, 8
    cos = torch.zeros(5, R // 2)
    for call in (lambda: tl._rotation(cos, cos, None, torch.zeros(D), D, tl.TP_F32, 1e-6, tl.TP_ROPE_HALVES),
                 lambda: tl._positions(torch.zeros(T, dtype=torch.int64), T, R),
                 lambda: tl._flag(torch.zeros(1, dtype=torch.int32))):
        monkeypatch.setattr(tl, "_torch_module", None)
        assert call() is not None
