"""Attention calls whose items (a sequence's rows, a key head) take a workgroup each: many sequences of single tokens or
of ragged chunks, prompts from their first tokens on.  tests/host/attention_form_driver.cpp has the same sizes and shows
that they take that form; calls that need no workspace take no other."""
import pytest
import torch

import tensor_linear_amd as tl
from test_gpu_attention import BF, TYPES, Cached, check

pytestmark = pytest.mark.gpu


def singles(B):
    """One token each, now and then none or a few."""
    return [(1, 1, 1, 0, 1, 3, 1, 1, 20, 1)[i % 10] for i in range(B)], [(7 * i) % 71 for i in range(B)]


def chunks(B):
    """Nothing, single tokens and chunks of several row tiles, behind pasts of any length."""
    return [(1, 0, 37, 9, 60, 5, 0)[i % 7] for i in range(B)], [(13 * i) % 90 if i % 5 else 0 for i in range(B)]


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("shape,pad,window", [((2, 1, 32, 16), 0, 0), ((4, 2, 64, 8), 0, 33), ((3, 1, 50, 16), 0, 0), ((2, 1, 128, 16), 3, 0), ((2, 1, 256, 16), 0, 40)])
def test_items_of_single_tokens(shape, pad, window, t, int8):
    Hq, Hkv, D, page = shape
    lens, past = singles(2100)
    c = Cached(lens, past, Hkv, D, page, t, int8, seed=21, pad=pad, lead=3, tail=5)
    assert c.T * (Hq // Hkv) <= 32 * len(lens) and tl.tp_kv_attention_workspace_bytes(c.T, len(lens), Hq, Hkv, D) == 0
    check(c, Hq, window=window)


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("shape,pad,window", [((8, 1, 64, 16), 0, 0), ((16, 2, 32, 16), 0, 50), ((8, 1, 36, 5), 0, 0), ((8, 1, 128, 16), 1, 0)])
def test_items_of_chunks(shape, pad, window, t, int8):
    Hq, Hkv, D, page = shape
    lens, past = chunks(540)
    c = Cached(lens, past, Hkv, D, page, t, int8, seed=22, pad=pad, lead=3, tail=5)
    assert c.T * (Hq // Hkv) > 32 * len(lens) and tl.tp_kv_attention_workspace_bytes(c.T, len(lens), Hq, Hkv, D) == 0
    check(c, Hq, window=window)


@pytest.mark.parametrize("t,int8", TYPES)
def test_items_of_many_heads(t, int8):
    """Few row tiles, each of 8 key heads."""
    lens, past = [(33, 0, 70, 34, 31)[i % 5] for i in range(300)], [(3 * i) % 40 for i in range(300)]
    c = Cached(lens, past, 8, 32, 16, t, int8, seed=23, tail=1)
    assert tl.tp_kv_attention_workspace_bytes(c.T, 300, 8, 8, 32) == 0
    check(c, 8)


@pytest.mark.parametrize("t,int8", TYPES)
@pytest.mark.parametrize("shape", [(8, 2, 128, 16), (4, 4, 80, 16), (8, 1, 100, 16)])
def test_prompts_from_their_first_tokens(shape, t, int8):
    """A table no wider than the longest prompt, and prompts that fill half of it or more on average."""
    Hq, Hkv, D, page = shape
    check(Cached([200, 0, 150, 90], [0, 0, 0, 0], Hkv, D, page, t, int8, seed=24), Hq)
    check(Cached([129, 208, 200], [0, 0, 8], Hkv, D, page, t, int8, seed=25, lead=2), Hq)


def test_what_the_wider_table_changes():
    """The same prompts with a table for many more positions: cut otherwise, the same rows within the same bounds."""
    c = Cached([200, 0, 150, 90], [0, 0, 0, 0], 2, 128, 16, BF, seed=24)
    check(c, 8)
    c.table = torch.cat([c.table, torch.full((4, 3000), c.n_pages, dtype=torch.int32)], 1)
    c.max_pages += 3000
    check(c, 8)
