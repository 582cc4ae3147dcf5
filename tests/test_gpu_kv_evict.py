"""ft_kv_evict against a plain selection on the host, entry by entry: every byte of the pools has to be the same."""
import math

import pytest
import torch

import expert_offloaded_serving_b200 as ft
from _kv import Cache, evict

pytestmark = pytest.mark.gpu


def same(x, y):
    x, y = x.cpu(), y.cpu()
    if x.dtype == torch.bfloat16:
        x, y = x.view(torch.int16), y.view(torch.int16)
    if x.dtype == torch.float32:
        x, y = x.view(torch.int32), y.view(torch.int32)
    return torch.equal(x, y)


def check(c, budgets, recent):
    want = evict(c, budgets, recent)
    kv = c.kv()
    ft.ft_kv_evict(kv, torch.tensor(budgets, dtype=torch.int32, device="cuda"), recent, c.workspace(kv))
    assert c.status.item() == 0
    for name, got, w in zip(("lengths", "pos", "mass", "k", "v"), (c.lengths, c.pos, c.mass, c.k, c.v),
                            (want[4], want[3], want[2], want[0], want[1])):
        assert same(got, w), name


@pytest.mark.parametrize("dim,kv_heads,page,e4m3", [
    (64, 1, 16, False), (64, 3, 8, True), (96, 2, 32, False), (96, 1, 8, True), (128, 4, 16, False), (128, 2, 64, True),
    (192, 1, 8, False), (192, 2, 128, True), (256, 2, 16, False), (256, 1, 1024, True)])
def test_ragged_batches(dim, kv_heads, page, e4m3):
    lengths = [100, 0, 1, 33, 600, 64, 31]
    c = Cache(lengths, kv_heads, kv_heads, dim, page, e4m3, seed=dim + kv_heads)
    check(c, [50, 3, 0, 33, 64, 63, 40], 10)
    check(c, [10, 0, 0, 32, 64, 1, 31], 0)   # and again, from what is left


@pytest.mark.parametrize("n,keep,recent", [
    (2, 1, 0), (1, 0, 0), (32, 31, 1), (33, 1, 5), (4097, 2048, 100), (5000, 4999, 0), (9000, 10, 10), (20000, 12345, 20000),
    (20000, 500, 2 ** 31 - 1), (70001, 35000, 64)])
def test_one_sequence(n, keep, recent):
    c = Cache([n], 2, 2, 64, 16, seed=n)
    check(c, [keep], recent)


def test_ties_zeros_and_what_is_no_mass():
    c = Cache([3000, 200], 1, 1, 64, 16, seed=2)
    at = c.place(0, torch.arange(3000, device="cuda"))
    c.mass[at] = (torch.arange(3000, device="cuda") % 3)[:, None].float()     # a thousand of each
    at = c.place(1, torch.arange(200, device="cuda"))
    c.mass[at] = 0.0
    some = c.place(1, torch.arange(0, 200, 7, device="cuda"))
    c.mass[some] = torch.tensor([math.nan, -1.0, -0.0, math.inf, 1e-45, -math.inf, 3.0], device="cuda").repeat(5)[:29, None]
    check(c, [1500, 100], 0)


def test_recent_entries_that_share_positions():
    """Image tokens share a position: more of them are recent than the budget holds; the newest stay, the lower slots first."""
    c = Cache([500, 500], 2, 2, 64, 16, seed=3)
    for b in range(2):
        at = c.place(b, torch.arange(500, device="cuda"))
        c.pos[at] = (torch.arange(500, device="cuda") // (60 if b else 200))[:, None].int()
    check(c, [90, 250], 2)


def test_positions_out_of_order_and_near_the_top():
    c = Cache([800], 2, 2, 64, 16, seed=4)
    at = c.place(0, torch.arange(800, device="cuda"))
    for h in range(2):
        c.pos[at[0][:, 0], h, at[2][:, 0]] = (2 ** 31 - 1 - torch.randperm(800, device="cuda")).int()
    check(c, [300], 120)


def test_many_items_and_one_that_is_too_long_for_shared_memory():
    lengths = [60000] + [(i * 37) % 90 for i in range(159)]
    c = Cache(lengths, 1, 1, 64, 64, seed=5)
    check(c, [20000] + [30] * 159, 16)


def test_no_sequence_over_its_budget_changes_nothing():
    c = Cache([10, 0, 30], 2, 2, 64, 16, seed=6)
    before = [x.clone() for x in (c.k, c.v, c.mass, c.pos, c.lengths)]
    kv = c.kv()
    ft.ft_kv_evict(kv, torch.tensor([10, 0, 99], dtype=torch.int32, device="cuda"), 5, c.workspace(kv))
    assert all(same(x, y) for x, y in zip((c.k, c.v, c.mass, c.pos, c.lengths), before))


def test_bad_contents():
    c = Cache([100, 100, 100], 2, 2, 64, 16, seed=7)
    want = evict(c, [100, 40, 100], 3)
    c.lengths[2] = 5000
    kv = c.kv()
    ft.ft_kv_evict(kv, torch.tensor([-1, 40, 10], dtype=torch.int32, device="cuda"), 3, c.workspace(kv))
    assert c.status.item() == 2
    assert c.lengths.tolist() == [100, 40, 5000]
    assert same(c.k, want[0]) and same(c.pos, want[3])
    # a page that is missing: its entries go first, nothing out of bounds is touched
    c = Cache([64], 1, 1, 64, 16, seed=8)
    c.table[0, 1] = -1
    kv = c.kv()
    ft.ft_kv_evict(kv, torch.tensor([48], dtype=torch.int32, device="cuda"), 0, c.workspace(kv))
    assert c.status.item() == 2 and c.lengths.item() == 48


def test_a_page_listed_twice_stays_in_bounds():
    """Two sequences over the same pages: what they hold after that is open, the status says so or it fits."""
    c = Cache([64, 64], 1, 1, 64, 16, seed=9, spare=0)
    c.table[1] = c.table[0]
    c.k, c.v, c.mass, c.pos = c.k[:4].contiguous(), c.v[:4].contiguous(), c.mass[:4].contiguous(), c.pos[:4].contiguous()
    c.n_pages = 4
    c.table %= 4
    kv = c.kv()
    ft.ft_kv_evict(kv, torch.tensor([10, 10], dtype=torch.int32, device="cuda"), 0, c.workspace(kv))
    torch.cuda.synchronize()
    assert c.status.item() == 2  # 128 entries listed, the pool holds 64


def test_captured_eviction_follows_lengths_and_budgets():
    c = Cache([300, 200], 2, 2, 64, 16, seed=10)
    d = Cache([300, 200], 2, 2, 64, 16, seed=10)
    budgets = torch.tensor([300, 200], dtype=torch.int32, device="cuda")
    kv = c.kv()
    work = c.workspace(kv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ft.ft_kv_evict(kv, budgets, 8, work)
    for b in ([250, 200], [100, 77], [100, 3]):
        budgets.copy_(torch.tensor(b, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check(d, b, 8)
        assert all(same(x, y) for x, y in zip((c.k, c.v, c.mass, c.pos, c.lengths), (d.k, d.v, d.mass, d.pos, d.lengths)))
