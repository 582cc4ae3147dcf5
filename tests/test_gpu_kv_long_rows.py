"""Rows in many parts, entry by entry: with a query of zero every entry weighs 1/n, so that sums of weights are whole numbers,
exact in fp32 up to 2^24, in every part and in their join.  Each dim then counts the entries of its own few
tiles: one tile that is lost, read twice or given to the wrong row changes its dim by far more than the bound."""
import math

import pytest
import torch

import expert_offloaded_serving_b200 as ft
from _kv import Cache
from test_gpu_kv_attention import call

pytestmark = pytest.mark.gpu

RAGGED = [(i * 7919) % 9001 if i % 9 else 0 for i in range(1, 70)]


def check(lengths, heads, kv_heads, dim, e4m3, run, weigh, page=64):
    """v is 1 in dim (i / run) % (dim - 1) of entry i and in the last dim, 0 elsewhere."""
    c = Cache(lengths, heads, kv_heads, dim, page, e4m3, seed=dim + run, v_scale=0.5)
    for b, n in enumerate(lengths):
        if n:
            i = torch.arange(n, device="cuda")
            x = torch.zeros(n, kv_heads, dim, device="cuda")
            x[i, :, (i // run) % (dim - 1)] = 1.0
            x[:, :, dim - 1] = 1.0
            c.v[c.place(b, i)] = c.stored(x, 1.0)
    v = c.v_scale
    q = torch.zeros(len(lengths), heads, dim, dtype=torch.bfloat16, device="cuda")
    before = c.mass.double()
    out, lse = call(c, q, 0.125, ft.FT_KV_MASS if weigh else 0)
    assert c.status.item() == 0
    for b, n in enumerate(lengths):
        if not n:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        count = torch.bincount((torch.arange(n, device="cuda") // run) % (dim - 1), minlength=dim).double()
        count[dim - 1] = n
        want = v * count / n
        # one fp32 quotient and product, then bf16: 2^-8 of the value together with 2^-22; a missing tile is 16 entries at least
        bound = want * (2.0 ** -8 + 2.0 ** -22)
        if run > 1:
            assert (v * 16 / n >= 2 * bound[:dim - 1][count[:dim - 1] > 0]).all()
        off = (out[b].double() - want).abs()
        assert (off <= bound).all(), (b, n, off.argmax().item())
        assert (out[b, :, dim - 1] == v).all()
        # log2 of a whole number to an ulp or two, times ln 2: 2^-21 of itself; a missing tile is 16 / n
        assert ((lse[b].double() - math.log(n)).abs() <= math.log(n) * 2.0 ** -21 + 1e-7).all()
        if weigh:
            at = c.place(b, torch.arange(n, device="cuda"))
            add = heads / kv_heads / n
            # __log2f may be 2 units in the last place off: 2^-18 for a sum of up to 2^31 (an E4M3 row's are 2^7 n); the
            # two differences that use it round by 2^-21 each and ex2 by 2^-22: a weight is off by
            # ln 2 (2^-18 + 2^-20) + 2^-22 < 2^-18 of itself; a missing tile is 16 / n.  The sum of G weights rounds G - 1
            # times; every 16 query heads of a KV head are one addition to the mass, which rounds.
            G = heads // kv_heads
            bound = add * (2.0 ** -18 + G * 2.0 ** -24) + (before[at] + add) * -(-G // 16) * 2.0 ** -24
            assert ((c.mass[at].double() - before[at] - add).abs() <= bound).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 1, 1), (64, 8, 2), (96, 5, 1), (128, 8, 1), (128, 20, 1), (192, 12, 1),
                                                (256, 2, 1), (256, 32, 2)])
@pytest.mark.parametrize("lengths", [[4097], [20011], [9001, 9000, 5, 8000], [5001, 1, 1, 29], RAGGED])
def test_every_tile_counts_once(lengths, dim, heads, kv_heads, e4m3):
    run = 16  # half a tile, or a whole one of wide rows
    # so few tiles a dim that each shows: 2^-7 of a dim's entries stay below 16
    n = max(lengths)
    while n > (dim - 1) * 2000:
        run *= 2
        n //= 2
    check(lengths, heads, kv_heads, dim, e4m3, run, weigh=True)
    check(lengths, heads, kv_heads, dim, e4m3, 1, weigh=False)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim,heads", [(128, 16), (256, 8)])
def test_every_tile_of_a_long_row_counts_once(dim, heads, e4m3):
    check([131071, 40001], heads, 1, dim, e4m3, 16, weigh=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("dim,heads,lengths", [(64, 4, [20011]), (128, 8, [40001, 300]), (128, 20, [9001, 9000, 5, 8000]), (256, 16, [20011, 7]),
                                               (96, 3, [2000] * 40)])
def test_parts_with_references_far_apart(dim, heads, lengths, order, e4m3):
    """Scores are whole numbers of log2 from -8 to 8, alike over stretches of entries: weights 2^0 to 2^16 of the least, so that
    parts join under other references.

    A score is off by 2^-23 of 8 (scale times log2(e) is 1 to 2^-23), twice (it and the reference): a weight by 2^-19.  A part has at
    most 80,000 / 592 = 136 entries of one row (137 with the tile's rest) and a row at most 1,184 parts: fewer than 2,048 additions
    in a row, 2^-12 of a sum of one sign at 2^-23 each.  Twice that for the quotient."""
    c = Cache(lengths, heads, 1, dim, 32, e4m3, seed=dim, k_scale=1.0, v_scale=0.5)
    q = torch.zeros(len(lengths), heads, dim, dtype=torch.bfloat16, device="cuda")
    q[:, :, 3] = 1.0
    q[:, 1::2, 3] = -1.0  # the order turns around for every second head
    levels = []
    for b, n in enumerate(lengths):
        i = torch.arange(n, device="cuda")
        if order == "mixed":
            level = (i // 41 * 7919) % 17 - 8
        else:
            level = i * 17 // n - 8
            level = level if order == "rising" else -level
        levels.append(level.double())
        at = c.place(b, i)
        x = torch.zeros(n, 1, dim, device="cuda")
        x[:, 0, 3] = level.float()
        c.k[at] = c.stored(x, 1.0)
        x.zero_()
        x[i, 0, (i // 16) % (dim - 1)] = 1.0
        x[:, 0, dim - 1] = 1.0
        c.v[at] = c.stored(x, 1.0)
    out, lse = call(c, q, math.log(2))
    v = c.v_scale
    for b, n in enumerate(lengths):
        where = (torch.arange(n, device="cuda") // 16) % (dim - 1)
        for h in range(heads):
            p = torch.exp2(levels[b] * (1 if h % 2 == 0 else -1))
            share = torch.zeros(dim, dtype=torch.float64, device="cuda").index_add_(0, where, p) / p.sum()
            share[dim - 1] = 1.0
            bound = v * share * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18)
            assert ((out[b, h].double() - v * share).abs() <= bound).all(), (b, h)
            want = math.log(p.sum().item())
            assert abs(lse[b, h].item() - want) <= 2.0 ** -12 + 2.0 ** -19 + abs(want) * 2.0 ** -21
