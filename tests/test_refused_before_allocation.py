"""Sizes that the plan and mask calls do not take are refused before outputs of that size are made."""

import gc
import os
import re

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
from attention_fa2_attn_gb300 import _lib, api

DEV = "cuda:0"


def test_limits_are_those_of_the_header():
    text = open(os.path.join(os.path.dirname(_lib._HEADER), "fa_gb300.h")).read()
    for name in ("FA_PLAN_MAX_T", "FA_TREE_MASK_MAX_T", "FA_TREE_MASK_MAX_B"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(_lib, name)


@pytest.fixture(params=["extension", "python"])
def way(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(api, "fast", lambda: _lib._NoFastCalls())
    return request.param


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


class _Nothing:
    """Within it, memory in use does not rise by a megabyte."""

    def __enter__(self):
        gc.collect()
        torch.cuda.synchronize()
        self.was = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()

    def __exit__(self, *exc):
        if exc[0] is None:
            assert torch.cuda.max_memory_allocated() - self.was < 1 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(1, 8193), (65536, 32)])
def test_masks(way, B, T):
    # 8193 nodes of 257 words each would be 8 MB, 65536 trees of 32 nodes 16 MB
    parents, seqlens = torch.full((B, T), -1, dtype=torch.int32, device=DEV), _i32(np.full(B, T))
    with _Nothing():
        with pytest.raises(fa.FAError) as e:
            fa.fa_tree_mask(parents, seqlens)
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(1, 65535 * 128 + 1), (1, 2**31 - 1), (1 << 10, 1 << 21)])
def test_plans(way, B, T):
    # 8 million rows and more: 64 MB of slots and positions at least
    one, table = _i32(np.ones(B)), _i32(np.zeros((B, 1)))
    with _Nothing():
        with pytest.raises(fa.FAError) as e:
            fa.fa_paged_plan(one, one, one, table, T)
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED


@pytest.mark.gpu
def test_the_largest_that_are_taken(way):
    T = 65535 * 128
    one, table = _i32([1]), _i32([[3]])
    seqlens, slots, positions, used = fa.fa_paged_plan(one, one, one, table, T, align_end=True)
    assert seqlens.tolist() == [2] and used.tolist() == [0]
    assert slots[0, -2:].tolist() == [-1, 3 * 16 + 1] and positions[0, -2:].tolist() == [0, 1]
    assert int((slots != -1).sum()) == 1 and int((positions != 0).sum()) == 1
    mask, pos = fa.fa_tree_mask(_i32(np.full((65535, 1), -1)), _i32(np.full(65535, 9)))
    assert (mask == 1).all() and (pos == 8).all()
