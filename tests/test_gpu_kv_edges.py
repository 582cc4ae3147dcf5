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
