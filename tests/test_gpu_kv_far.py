"""Append and eviction where their tables and pools are much larger than their sequences: bytes past 2^32, tables as wide as
a model's context."""
import pytest
import torch

import expert_offloaded_serving_b200 as ft
from _kv import Cache
from test_gpu_kv_append import Step
from test_gpu_kv_evict import check, same

pytestmark = pytest.mark.gpu

KV_HEADS, PAGE, DIM = 2, 64, 128
FAR = (5 << 30) // (KV_HEADS * PAGE * DIM * 2)  # pages of a pool of 5 GiB


def far_away(c):
    """The same cache with its pages at both ends of pools of 5 GiB; returns the pages' numbers there, by their old ones."""
    where = torch.tensor([(p // 2 if p % 2 else FAR - 1 - p // 2) for p in range(c.n_pages)], device="cuda")
    for name in ("k", "v", "mass", "pos"):
        small = getattr(c, name)
        big = torch.empty(FAR, *small.shape[1:], dtype=small.dtype, device="cuda")
        big[where] = small
        setattr(c, name, big)
    c.table = torch.where(c.table < c.n_pages, where[c.table.long().clamp(max=c.n_pages - 1)].int(), FAR + 7)
    c.n_pages = FAR
    return where


def test_append_past_32_bits():
    small, c = (Cache([300, 70], 4, KV_HEADS, DIM, PAGE, seed=41) for _ in range(2))
    where = far_away(c)
    assert c.k.numel() * 2 > 1 << 32
    steps = [Step(x, [40, 70], 2, seed=2) for x in (small, c)]
    for step in steps:
        step.run()
    torch.cuda.synchronize()
    assert torch.equal(steps[0].q_out, steps[1].q_out)
    for name in ("k", "v", "mass", "pos"):
        assert same(getattr(small, name), getattr(c, name)[where]), name
    assert c.status.item() == 0 and small.status.item() == 0


def test_eviction_past_32_bits():
    small, c = (Cache([500, 333], KV_HEADS, KV_HEADS, DIM, PAGE, seed=42) for _ in range(2))
    where = far_away(c)
    budgets = torch.tensor([210, 100], dtype=torch.int32, device="cuda")
    check(small, budgets.tolist(), 30)
    kv = c.kv()
    ft.ft_kv_evict(kv, budgets, 30, c.workspace(kv))
    for name in ("k", "v", "mass", "pos"):
        assert same(getattr(small, name), getattr(c, name)[where]), name
    assert torch.equal(c.lengths, budgets) and c.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lengths,budgets,kv_heads", [([2112] * 8, [2048] * 8, 8), ([17000, 40, 0, 5000], [16000, 1, 3, 0], 2),
                                                      ([i * 13 % 700 for i in range(90)], [100] * 90, 1)])
def test_eviction_in_tables_as_wide_as_a_context(lengths, budgets, kv_heads, e4m3):
    """Room for 131,072 entries a sequence: what is kept does not depend on it."""
    c = Cache(lengths, kv_heads, kv_heads, 64, 16, e4m3, seed=len(lengths))
    c.table = torch.nn.functional.pad(c.table, (0, 131072 // 16 - c.table.shape[1]), value=c.n_pages + 7)
    check(c, budgets, 100)
