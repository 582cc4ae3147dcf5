"""ft_kv_attention against its definition in 64 bits: every head size and format, head layouts, lengths from none to
long ones, pages smaller than a tile, split rows, accumulated weights, streams and graphs."""
import math

import pytest
import torch

import expert_offloaded_serving_b200 as ft
from _kv import Cache, attention, attention_bounds

pytestmark = pytest.mark.gpu


def queries(c, B, seed=5, magnitude=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (magnitude * torch.randn(B, c.heads, c.dim, generator=g, device="cuda")).to(torch.bfloat16)


def call(c, q, scale, flags=0, kv=None, stream=None):
    kv = kv or c.kv()
    out = torch.full((q.shape[0], c.heads, c.dim), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], c.heads), math.nan, device="cuda")
    ft.ft_kv_attention(kv, q, scale, out, lse, c.workspace(kv), flags, stream)
    return out, lse


def check(c, lengths, q, scale, mass=False):
    before = c.mass.clone() if mass else None
    out, lse = call(c, q, scale, ft.FT_KV_MASS if mass else 0)
    want, want_lse, size, reach, weights = attention(c, q, scale, lengths)
    b_out, b_lse, b_weight = attention_bounds(c, want, size, reach, lengths)
    assert torch.isfinite(out).all()
    err = (out.double() - want).abs()
    assert (err <= b_out).all(), f"out off by {(err / b_out).max():.3f} of its bound"
    live = torch.isfinite(want_lse)
    assert torch.equal(live, torch.isfinite(lse)) and (lse[~live] == -math.inf).all()
    err = (lse.double() - want_lse).abs()[live]
    assert (err <= b_lse[live]).all()
    if mass:
        after = before.double()
        slack = torch.zeros_like(after)
        G = c.heads // c.kv_heads
        for b, n in enumerate(lengths):
            if n:
                at = c.place(b, torch.arange(n, device="cuda"))
                add = weights[b]  # [kv heads][G][n]
                after[at] += add.sum(1).T
                w = b_weight[b].view(c.kv_heads, G)[:, :, None]
                # the sum of G weights and the mass round once more each: 2^-24 relative
                slack[at] = (add * (w + G * 2.0 ** -24)).sum(1).T + after[at].abs() * 2.0 ** -24 + 1e-30
        off = (c.mass.double() - after).abs()
        assert torch.equal(torch.isnan(off), torch.isnan(before))  # entries of no sequence stay as they were
        assert (torch.nan_to_num(off) <= slack * 1.01).all()
    assert c.status.item() == 0


MIXED = [0, 1, 2, 15, 16, 17, 0, 33, 100, 257, 1000, 0]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads,page", [
    (64, 4, 4, 16), (64, 24, 1, 64), (96, 6, 2, 32), (96, 33, 3, 8), (128, 16, 2, 16), (128, 15, 3, 8),
    (128, 40, 1, 128), (192, 9, 1, 16), (192, 32, 2, 8), (256, 16, 2, 64), (256, 12, 1, 16), (256, 64, 4, 1024),
    (64, 12, 3, 16), (128, 6, 3, 32), (256, 3, 3, 16), (96, 9, 3, 16)])
def test_mixed_lengths(dim, heads, kv_heads, page, e4m3):
    c = Cache(MIXED, heads, kv_heads, dim, page, e4m3, seed=dim + heads)
    check(c, MIXED, queries(c, len(MIXED)), dim ** -0.5, mass=True)
    check(c, MIXED, queries(c, len(MIXED), 6), dim ** -0.5)


@pytest.mark.parametrize("lengths", [[1], [16], [17], [4000], [20011], [0], [0, 0, 3], [30001, 1, 1, 29]])
@pytest.mark.parametrize("e4m3", [False, True])
def test_few_rows_split_over_the_gpu(lengths, e4m3):
    c = Cache(lengths, 8, 1, 128, 16, e4m3, seed=3)
    check(c, lengths, queries(c, len(lengths)), 128 ** -0.5, mass=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,kv_heads,lengths", [(17, 1, [5000, 3, 0, 700]), (96, 3, [4001, 1, 2222]), (128, 2, [9000]),
                                                    (1024, 1, [1, 40, 333]), (1000, 2, [129])])
def test_groups_of_heads_over_rows_in_many_parts(heads, kv_heads, lengths, e4m3):
    c = Cache(lengths, heads, kv_heads, 64, 16, e4m3, seed=heads)
    check(c, lengths, queries(c, len(lengths)), 0.125, mass=True)


@pytest.mark.parametrize("n_seqs", [32, 33, 128, 129, 257])
def test_counts_of_sequences_around_the_ways_to_find_a_place(n_seqs):
    lengths = [0 if i % 5 == 3 else (i * 977) % 301 for i in range(n_seqs)]
    c = Cache(lengths, 6, 2, 64, 16, seed=n_seqs)
    check(c, lengths, queries(c, n_seqs), 0.125, mass=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim,heads", [(128, 1), (128, 2), (64, 3), (64, 12), (256, 20)])
@pytest.mark.parametrize("lengths", [[40001], [9001, 9000, 5, 8000]])
def test_weights_of_rows_in_many_parts(lengths, dim, heads, e4m3):
    c = Cache(lengths, heads, 1, dim, 32, e4m3, seed=heads)
    check(c, lengths, queries(c, len(lengths)), dim ** -0.5, mass=True)


@pytest.mark.parametrize("heads", [2, 12])
@pytest.mark.parametrize("n_seqs", [128, 129, 513, 1100])
def test_counts_of_sequences_with_rows_of_64_bytes(n_seqs, heads):
    lengths = [0 if i % 7 == 2 else (i * 977) % 97 for i in range(n_seqs)]
    c = Cache(lengths, heads, 1, 64, 16, True, seed=n_seqs)
    check(c, lengths, queries(c, n_seqs), 0.125, mass=True)


@pytest.mark.parametrize("e4m3", [False, True])
def test_scores_of_a_hundred_million(e4m3):
    """Neighbouring fp32 scores are 16 apart there: a weight of 2^16 would not fit f16."""
    c = Cache([200], 8, 1, 64, 16, e4m3, seed=21)
    q = torch.zeros(1, 8, 64, device="cuda")
    q[:, :, 0] = 2.0 ** 20
    q = q.to(torch.bfloat16)
    at = c.place(0, torch.arange(200, device="cuda"))
    x = torch.zeros(200, 1, 64, device="cuda")
    x[:, 0, 0] = torch.randint(90, 129, (200,), device="cuda").float()
    c.k[at] = c.stored(x * c.k_scale, c.k_scale)  # whole numbers in steps of 8 in E4M3, exact in bf16 (up to 128)
    out, lse = call(c, q, 1.0 / c.k_scale)
    k = c.values(c.k, 0, 200)[:, 0, 0] * (1.0 if e4m3 else c.k_scale)
    best = k == k.max()
    want = (c.values(c.v, 0, 200)[best, 0] * c.v_scale).mean(0)  # the others weigh nothing: e^-1000000
    bound = want.abs() * 2.0 ** -8 + 2.0 ** -10 * (c.values(c.v, 0, 200)[:, 0] * c.v_scale).abs().amax(0)
    assert torch.isfinite(out).all() and ((out[0].double() - want).abs() <= bound).all()
    top = k.max() * 2.0 ** 20 * (c.k_scale if e4m3 else 1.0) / c.k_scale
    assert ((lse.double() - top).abs() <= top * 2.0 ** -20).all()


def test_without_pools_of_weights_and_without_lse():
    c = Cache([40, 3], 4, 2, 128, 16, seed=22, meta=False)
    q, kv = queries(c, 2), c.kv()
    out = torch.empty_like(q)
    ft.ft_kv_attention(kv, q, 0.1, out, None, c.workspace(kv))
    assert torch.equal(out, call(c, q, 0.1)[0])
    with pytest.raises(ft.FtError, match="mass"):
        ft.ft_kv_attention(kv, q, 0.1, out, None, c.workspace(kv), ft.FT_KV_MASS)


def test_thousands_of_sequences():
    lengths = [(i * 7919) % 41 for i in range(3001)]
    c = Cache(lengths, 4, 2, 64, 16, seed=4)
    check(c, lengths, queries(c, len(lengths)), 0.125, mass=True)


@pytest.mark.parametrize("e4m3", [False, True])
def test_wide_ranges(e4m3):
    """Scores in the hundreds (one entry takes all the weight), queries that f16 alone would not hold, and a zero query."""
    lengths = [700, 64, 5]
    c = Cache(lengths, 8, 2, 128, 16, e4m3, seed=9)
    q = queries(c, 3)
    q[0] *= 300
    q[1] *= 2.0 ** 60
    q[2, :4] = 0
    q[2, 4:] *= 2.0 ** -40
    out, lse = call(c, q, 0.1 * 2.0 ** -60)
    want, want_lse, size, reach, _ = attention(c, q, 0.1 * 2.0 ** -60, lengths)
    b_out, b_lse, _ = attention_bounds(c, want, size, reach, lengths)
    assert ((out.double() - want).abs() <= b_out).all() and ((lse.double() - want_lse).abs() <= b_lse).all()
    q = q[[0, 2, 2]].clone()
    check(c, lengths, q, 0.1)
    check(c, lengths, q, -0.1)
    check(c, lengths, q, 0.0)


def test_strided_and_repeated_queries():
    lengths = [50, 0, 333]
    c = Cache(lengths, 8, 2, 64, seed=11)
    fused = queries(c, 3).reshape(3, -1)
    wide = torch.randn(3, 8 * 64 + 2 * 2 * 64, device="cuda").to(torch.bfloat16)
    wide[:, :512] = fused
    q = wide[:, :512].unflatten(1, (8, 64))
    assert not q.is_contiguous()
    check(c, lengths, q, 0.125)
    check(c, lengths, q[:1].expand(3, 8, 64), 0.125)  # row stride 0


def test_nan_and_infinite_entries_reach_their_own_head_only():
    lengths = [100, 40, 7]
    c = Cache(lengths, 4, 2, 64, seed=12)
    q = queries(c, 3)
    clean, clean_lse = call(c, q, 0.125)
    c.k[c.table[0, 5 // 16].long(), 0, 5] = math.nan            # sequence 0, KV head 0
    p, s = c.table[1, 33 // 16].long(), 33 % 16
    c.v[p, 1, s, 3] = math.inf                                  # sequence 1, KV head 1, one dim
    at = c.place(2, torch.arange(7, device="cuda"))
    c.k[at[0], 0, at[2]] = 0
    c.k[at[0], 0, at[2], 0] = -math.inf                         # sequence 2, KV head 0: every score -inf or +inf
    q[2, 0, 0], q[2, 1, 0] = 1.0, -1.0
    out, lse = call(c, q, 0.125)
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert torch.equal(out[0, 2:], clean[0, 2:]) and torch.equal(out[1, :2], clean[1, :2])
    assert not torch.isfinite(out[1, 2:, 3]).any() and torch.isfinite(out[1, 2:, 4:]).all()
    assert torch.equal(out[1, 2:, 4:], clean[1, 2:, 4:])
    assert (out[2, 0] == 0).all() and lse[2, 0] == -math.inf    # all -inf: like no entries
    assert torch.isnan(out[2, 1]).all()                         # +inf: NaN
    assert torch.equal(out[2, 2:], clean[2, 2:]) and torch.equal(lse[2, 2:], clean_lse[2, 2:])


def test_same_bits_every_time_and_whatever_the_workspace_held():
    lengths = [5000, 0, 77, 1200]
    c = Cache(lengths, 16, 2, 128, seed=13)
    q, kv = queries(c, 4), c.kv()
    work = c.workspace(kv)
    outs = []
    for fill in (0, 0xFF, 0x3C):
        work.fill_(fill)
        out, lse = torch.empty_like(q), torch.empty(4, 16, device="cuda")
        ft.ft_kv_attention(kv, q, 0.09, out, lse, work)
        outs.append((out, lse))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_shared_prefix_pages():
    """Sequences may read the same pages: here the same 64 entries begin both."""
    c = Cache([90, 64], 4, 2, 64, 16, seed=14)
    c.table[1, :4] = c.table[0, :4]
    check(c, [90, 64], queries(c, 2), 0.125)


def test_bad_contents_set_the_status_and_touch_nothing_else():
    lengths = [100, 50, 60, 70]
    c = Cache(lengths, 4, 2, 64, 16, seed=15)
    q = queries(c, 4)
    clean, clean_lse = call(c, q, 0.125)
    c.lengths[1] = -3
    c.lengths[2] = c.table.shape[1] * 16 + 1
    page = int(c.table[0, 1])
    c.table[0, 1] = c.n_pages
    out, lse = call(c, q, 0.125, ft.FT_KV_MASS)
    assert c.status.item() == 2
    with pytest.raises(ft.FtError) as e:
        ft.ft_kv_sync_status(c.kv())
    assert e.value.status == ft.FT_ERR_INVALID
    ft.ft_kv_sync_status(c.kv())  # cleared
    assert (out[1:3] == 0).all() and (lse[1:3] == -math.inf).all()
    assert torch.equal(out[3], clean[3]) and torch.equal(lse[3], clean_lse[3])
    # sequence 0: its other entries alone
    keep = [i for i in range(100) if i // 16 != 1]
    c.table[0, 1] = page
    qq = q[0].double().view(2, 2, 64)
    k = c.values(c.k, 0, 100)[keep]
    want = torch.logsumexp(0.125 * torch.einsum("hgd,nhd->hgn", qq, k), -1).reshape(4)
    assert ((lse[0].double() - want).abs() < 1e-4).all()


def test_side_stream_and_graph_replay_with_grown_lengths():
    lengths = [40, 0, 700]
    c = Cache([200, 30, 1500], 8, 2, 128, seed=16)
    full = c.lengths.clone()
    c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
    q, kv = queries(c, 3), c.kv()
    work, out, lse = c.workspace(kv), torch.empty_like(q), torch.empty(3, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ft.ft_kv_attention(kv, q, 0.1, out, lse, work)
    side.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ft.ft_kv_attention(kv, q, 0.1, out, lse, work, ft.FT_KV_MASS)
    out.fill_(math.nan)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    c.lengths.copy_(full)
    q.copy_(queries(c, 3, 99))
    graph.replay()
    torch.cuda.synchronize()
    again, lse2 = call(c, q, 0.1)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    check(c, full.tolist(), q, 0.1)


def test_two_graphs_in_turn_on_one_workspace():
    c, d = Cache([300, 9], 8, 2, 64, seed=17), Cache([5, 2000], 8, 2, 64, seed=18)
    kvs, qs = [c.kv(), d.kv()], [queries(c, 2, 1), queries(d, 2, 2)]
    work = max((x.workspace(kv) for x, kv in zip((c, d), kvs)), key=torch.numel)
    outs = [torch.empty_like(q) for q in qs]
    alone = [call(x, q, 0.125)[0] for x, q in zip((c, d), qs)]
    graphs = []
    for kv, q, out in zip(kvs, qs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ft.ft_kv_attention(kv, q, 0.125, out, None, work)
    for i in (0, 1, 1, 0, 1):
        outs[i].fill_(math.nan)
        graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])


def test_long_cache_past_32_bit_offsets():
    """A pool of more than 2^32 bytes: the sequence's pages lie at both ends of it."""
    kv_heads, page, dim = 2, 64, 128
    pages = (5 << 30) // (kv_heads * page * dim * 2)
    n = 64 * 8 - 5
    k = torch.empty(pages, kv_heads, page, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Cache([n], 4, kv_heads, dim, page, seed=19, spare=0, meta=False)
    table = torch.tensor([[0, pages - 1, 1, pages - 2, pages // 2, pages - 3, 7, pages - 9, 5]], dtype=torch.int32, device="cuda")
    for i in range(8):
        k[table[0, i].long()], v[table[0, i].long()] = c.k[c.table[0, i].long()], c.v[c.table[0, i].long()]
    q = queries(c, 1)
    want, want_lse = call(c, q, 0.1)
    c.k, c.v, c.table, c.n_pages = k, v, table, pages
    out, lse = call(c, q, 0.1)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
