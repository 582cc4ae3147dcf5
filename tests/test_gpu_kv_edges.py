"""The key-value cache calls where their inputs end: infinite keys under weights, weights that are far apart, long rows
tile by tile, tables much wider than their sequences, pools past 32 bits."""
import math

import pytest
import torch

import expert_offloaded_serving_b200 as ft
from _kv import Cache
from test_gpu_kv_attention import call, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [40, 5000])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 12, 16, 20, 33])
def test_an_entry_whose_scores_are_all_minus_infinity_weighs_nothing(G, n):
    """Its own mass stays as it was, the others' grow as without it."""
    c = Cache([n, 9], 2 * G, 2, 64, 16, seed=G)
    q = queries(c, 2)
    q[:, :, 7] = q[:, :, 7].abs() + 1  # every head turns the infinity below into a score of -inf
    gone = n // 3
    at = c.place(0, torch.tensor([gone], device="cuda"))
    c.k[at[0], 0, at[2], 7] = -math.inf  # KV head 0 alone
    before = c.mass.double()
    out, _ = call(c, q, 0.125, ft.FT_KV_MASS)
    assert torch.isfinite(out).all() and c.status.item() == 0
    for b, m in ((0, n), (1, 9)):
        k = c.values(c.k, b, m)
        score = 0.125 * torch.einsum("hgd,nhd->hgn", q[b].double().view(2, G, 64), k)
        add = torch.softmax(score, -1).sum(1).T  # [n][kv heads]
        place = c.place(b, torch.arange(m, device="cuda"))
        got, old = c.mass[place].double(), before[place]
        if b == 0:
            assert add[gone, 0] == 0 and got[gone, 0] == old[gone, 0]
        # a score is off by 68 x 2^-23 of at most 0.125 x 64 x 5 x 5 = 200 in size: weights by 2 x 200 x 68 x 2^-23 at most
        assert ((got - old - add).abs() <= add * 0.0035 + (old + add) * 2.0 ** -23).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("gap", [10.0, 17.3, 23.6, 25.1, 28.0])
def test_one_entry_over_a_long_tail(gap, e4m3):
    """The tail's weights are 2^-gap of the first entry's; 600 sequences share the pages, so that parts are long.

    In the dims where the first entry's value is 0, out is the tail's share alone: each weight of it may be off by
    2^-32 of the largest.  Sums: 600 rows of 4,096 tiles of 32 over 592 warps (BF16; E4M3 has twice as many) are 4,152 tiles a part at most,
    2 steps and 2 parts of p each: 16,608 products added to O, each cutting off up to 2^-23 of it, 2^-8.98; a lane's
    share of l is 4,152 x 4 additions that round by 2^-24, 2^-9.98.  Together 2^-8.4 < 2^-8; l alone 2^-9.98 < 2^-9."""
    n, B, D, sums = 131072, 600, 128, 2.0 ** -8
    c = Cache([n], 2, 1, D, 64, e4m3, seed=1, k_scale=1.0, v_scale=1.0625)
    v = 1.875 if e4m3 else 1.9921875  # 1.9921875 each way, a value of bf16
    at = c.place(0, torch.arange(n, device="cuda"))
    x = torch.zeros(n, 1, D, device="cuda")
    x[0, 0, 0] = 1.0
    c.k[at] = c.stored(x, 1.0)
    x = torch.full((n, 1, D), v, device="cuda")
    x[0, 0, :32] = 0.0
    c.v[at] = c.stored(x, 1.0)
    c.table = c.table.expand(B, -1).contiguous()
    c.lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, 2, D, dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = 1.0  # head 1 sees all entries alike
    out, lse = call(c, q, gap * math.log(2))
    tail = (n - 1) * 2.0 ** -gap
    want = 1.9921875 * tail / (1 + tail)
    off = (out[:, 0, :32].double() - want).abs().max().item()
    assert off <= want * (2.0 ** -8 + sums) + n * 2.0 ** -32 * 1.9921875, off / want
    assert (out[:, 0, 32:].double() - 1.9921875).abs().max() <= 1.9921875 * (2.0 ** -8 + sums)
    assert (lse[:, 0].double() - gap * math.log(2) - math.log1p(tail)).abs().max() <= 2.0 ** -9
    want = 1.9921875 * (n - 1) / n
    assert (out[:, 1, :32].double() - want).abs().max() <= want * (2.0 ** -8 + sums)
    assert (lse[:, 1].double() - math.log(n)).abs().max() <= 2.0 ** -9


@pytest.mark.parametrize("e4m3", [False, True])
def test_an_infinite_query_beside_a_large_one(e4m3):
    """Every key is positive: an element of -inf makes every score -inf whatever the finite others are, one of +inf NaN."""
    c = Cache([60], 8, 2, 64, 16, e4m3, seed=6)
    at = c.place(0, torch.arange(60, device="cuda"))
    c.k[at] = c.stored(torch.rand(60, 2, 64, device="cuda") + 0.5, c.k_scale)
    q = queries(c, 1)
    clean, _ = call(c, q, 0.125)
    q[0, 1, 5], q[0, 1, 9] = -math.inf, 1e30
    q[0, 2, 5], q[0, 2, 9] = math.inf, 1e30
    q[0, 6, 5], q[0, 6, 9] = -math.inf, -3e38
    out, lse = call(c, q, 0.125)
    assert (out[0, [1, 6]] == 0).all() and (lse[0, [1, 6]] == -math.inf).all()
    assert torch.isnan(out[0, 2]).all()
    rest = [0, 3, 4, 5, 7]
    assert torch.equal(out[0, rest], clean[0, rest])
