"""Decode steps of a whole layer with the key-value cache: append, attention, the MoE layer on what it gives, eviction,
one after another as a serving loop runs them, eager and captured."""
import math

import numpy as np
import pytest
import torch

import expert_offloaded_serving_b200 as ft
import synth
import synth.gpu
from _gpu import Ctx, assert_close, bf16_bits
from _kv import Cache, attention, attention_bounds, evict
from oracle import layer as olayer

pytestmark = pytest.mark.gpu

HEADS, KV_HEADS, DIM, EXPERTS, TOP_K, INTER = 4, 2, 64, 16, 2, 128
HIDDEN = HEADS * DIM
FLAGS = ft.FT_ROUTE_RENORM | ft.FT_ACT_BF16


class Loop:
    """One layer's decode loop over four sequences, one of them idle."""

    def __init__(self, ctx, wr, e4m3, seed=1):
        self.ctx, self.wr = ctx, wr
        self.c = Cache([40, 0, 7, 90], HEADS, KV_HEADS, DIM, 16, e4m3, seed=seed, room=48)
        self.kv = self.c.kv()
        self.work = self.c.workspace(self.kv)
        self.live = (self.c.lengths > 0).int()
        self.qkv = torch.zeros(4, (HEADS + 2 * KV_HEADS) * DIM, dtype=torch.bfloat16, device="cuda")
        self.positions = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
        self.inv_freq = 10000.0 ** (-torch.arange(DIM // 2, dtype=torch.float64, device="cuda") / (DIM // 2))
        self.axis = torch.zeros(DIM // 2, dtype=torch.int32, device="cuda")
        self.q = torch.zeros(4, HEADS, DIM, dtype=torch.bfloat16, device="cuda")
        self.attn, self.out = torch.zeros_like(self.q), torch.zeros(4, HIDDEN, dtype=torch.bfloat16, device="cuda")
        self.budgets = torch.tensor([40, 5, 5, 64], dtype=torch.int32, device="cuda")

    def parts(self):
        return [x.unflatten(1, (-1, DIM)) for x in self.qkv.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1)]

    def read(self):
        """The scheduler counts the new tokens, then the step appends and attends."""
        self.c.lengths.add_(self.live)
        ft.ft_kv_append(self.kv, *self.parts(), None, self.positions, self.inv_freq, self.axis, self.q)
        ft.ft_kv_attention(self.kv, self.q, DIM ** -0.5, self.attn, None, self.work, ft.FT_KV_MASS)

    def layer(self):
        ft.ft_moe_layer_forward(self.ctx, 0, self.attn.view(4, HIDDEN), 4, self.wr, None, self.out, FLAGS)

    def shrink(self):
        ft.ft_kv_evict(self.kv, self.budgets, 8, self.work)

    def step(self):
        self.read()
        self.layer()
        self.shrink()

    def next_token(self, t):
        g = torch.Generator("cuda").manual_seed(100 + t)
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g, device="cuda"))
        self.positions.fill_(200 + t)


@pytest.fixture(scope="module")
def moe():
    seed = 77
    pool = synth.gpu.layer_pool(HIDDEN, INTER, EXPERTS, seed, 0)
    wr = synth.router_weights(seed, 0, EXPERTS, HIDDEN)
    with Ctx(ft.make_desc(HIDDEN, INTER, EXPERTS, TOP_K, 1, 0, 0, 16), None, [pool]) as ctx:
        yield ctx.h, torch.from_numpy(wr).cuda(), wr, seed


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_loop_step_by_step(moe, e4m3):
    handle, wr, wr_host, seed = moe
    loop = Loop(handle, wr, e4m3)
    c = loop.c
    blobs = {e: synth.expert_blob(seed, 0, e, HIDDEN, INTER) for e in range(EXPERTS)}
    for t in range(12):
        loop.next_token(t)
        lengths = (c.lengths + loop.live).tolist()
        before = c.mass.clone()
        loop.read()
        want, _, size, reach, weights = attention(c, loop.q, DIM ** -0.5, lengths)
        bound, _, _ = attention_bounds(c, want, size, reach, lengths)
        assert ((loop.attn.double() - want).abs() <= bound).all()
        for b, n in enumerate(lengths):
            if n:
                at = c.place(b, torch.arange(n, device="cuda"))
                old = before[at].double()
                old[n - 1] = 0.0  # the new entry
                add = weights[b].sum(1).T
                assert ((c.mass[at].double() - old - add).abs() <= 1e-5 * (old + add)).all()
                assert (c.pos[at][n - 1] == 200 + t).all()
        loop.layer()
        r = olayer.moe_layer(bf16_bits(loop.attn).reshape(4, HIDDEN), blobs.__getitem__, HIDDEN, INTER, EXPERTS, TOP_K,
                             router_w=wr_host)
        assert_close(bf16_bits(loop.out), np.asarray(r["out_f64"]))
        k, v, mass, pos, after = evict(c, loop.budgets.tolist(), 8)
        loop.shrink()
        ft.ft_kv_sync_status(loop.kv)
        ft.ft_sync_status(handle)
        assert torch.equal(c.lengths.cpu(), after) and torch.equal(c.pos.cpu(), pos)
        assert torch.equal(c.mass.cpu().view(torch.int32), mass.view(torch.int32))
        for got, w in ((c.k, k), (c.v, v)):
            assert torch.equal(got.cpu().view(torch.uint8), w.view(torch.uint8))
        assert c.lengths.tolist()[1] == 0 and c.lengths.tolist()[2] <= 5


def test_decode_loop_captured_gives_the_same_bits(moe):
    handle, wr, _, _ = moe
    eager, replay = Loop(handle, wr, False, seed=2), Loop(handle, wr, False, seed=2)
    outs = []
    for t in range(8):
        eager.next_token(t)
        eager.step()
        outs.append((eager.attn.clone(), eager.out.clone()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replay.step()
    for t in range(8):
        replay.next_token(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(replay.attn, outs[t][0]) and torch.equal(replay.out, outs[t][1])
    for x, y in ((eager.c.k, replay.c.k), (eager.c.v, replay.c.v), (eager.c.mass, replay.c.mass)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(eager.c.pos, replay.c.pos) and torch.equal(eager.c.lengths, replay.c.lengths)


def test_calls_refuse_memory_that_is_not_the_gpus():
    c = Cache([10], 4, 2, 64, seed=3)
    kv = c.kv()
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    work = c.workspace(kv)
    host = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for args in ((host, torch.empty_like(q), None, work), (q, host, None, work), (q, torch.empty_like(q), torch.zeros(1, 4), work),
                 (q, torch.empty_like(q), None, work.cpu())):
        with pytest.raises(ft.FtError, match="device memory") as e:
            ft.ft_kv_attention(kv, args[0], 0.1, *args[1:])
        assert e.value.status == ft.FT_ERR_INVALID
    with pytest.raises(ft.FtError, match="device memory"):
        ft.ft_kv_evict(kv, torch.zeros(1, dtype=torch.int32), 0, work)
    kn = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ft.FtError, match="device memory"):
        ft.ft_kv_append(kv, None, kn, kn, None, pos, None, None, None)
    table = c.table.cpu()
    k, v = c.pools()
    bad = ft.make_kv(4, k, v, table, c.lengths, mass=c.mass, pos=c.pos)
    with pytest.raises(ft.FtError, match="block_table is not device memory"):
        ft.ft_kv_attention(bad, q, 0.1, torch.empty_like(q), None, work)
    assert math.isfinite(c.mass[c.place(0, torch.arange(10, device="cuda"))].sum().item())
