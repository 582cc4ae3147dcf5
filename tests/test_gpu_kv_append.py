"""ft_kv_append against its definition in 64 bits: rotary layouts and axes, far positions, both cache formats, decode
rows and ragged prompts, padding, strides, bad contents."""
import math

import pytest
import torch

import expert_offloaded_serving_b200 as ft
from _kv import Cache

pytestmark = pytest.mark.gpu


class Step:
    """New tokens for the last slots of each sequence."""

    def __init__(self, c, new, axes=1, rot=None, adjacent=False, decode=False, pad=0, seed=1, top=5000, queries=True):
        g = torch.Generator("cuda").manual_seed(seed)
        self.c, self.new, self.adjacent, self.pad = c, new, adjacent, pad
        T = self.T = (len(new) if decode else sum(new)) + pad
        qkv = torch.randn(T, (c.heads + 2 * c.kv_heads) * c.dim, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = qkv.split([c.heads * c.dim, c.kv_heads * c.dim, c.kv_heads * c.dim], 1)
        self.q = q.unflatten(1, (-1, c.dim)) if queries else None
        self.k, self.v = k.unflatten(1, (-1, c.dim)), v.unflatten(1, (-1, c.dim))
        self.cu = None if decode else torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        self.positions = torch.randint(0, top, (axes, T), generator=g, device="cuda", dtype=torch.int64).int()
        rot = c.dim if rot is None else rot
        half = rot // 2
        self.rot = rot
        i = torch.arange(half, dtype=torch.float64, device="cuda")
        self.inv_freq = 10000.0 ** (-i / max(half, 1)) if rot else None
        self.axis = (i % axes).int() if rot else None
        self.q_out = torch.full((T, c.heads, c.dim), 7.0, dtype=torch.bfloat16, device="cuda") if queries else None

    def run(self, kv=None):
        ft.ft_kv_append(kv or self.c.kv(), self.q, self.k, self.v, self.cu, self.positions, self.inv_freq, self.axis,
                        self.q_out, ft.FT_ROPE_ADJACENT if self.adjacent else 0)

    def turned(self, x):
        """[T][heads][dim] in 64 bits, and the size |x1| + |x2| of each element's pair (0 where nothing turns)."""
        x = x.double()
        size = torch.zeros_like(x)
        if not self.rot:
            return x, size
        angle = self.positions.double()[self.axis.long()].T * self.inv_freq  # exact to 2^-53 of itself
        cos, sin = angle.cos()[:, None], angle.sin()[:, None]
        y = x.clone()
        half = self.rot // 2
        a, b = (slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.adjacent else (slice(0, half), slice(half, self.rot))
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
        return y, size

    def slots(self):
        """(token, sequence, slot) of every token that is not padding or idle."""
        out, t = [], 0
        for b, w in enumerate(self.new):
            n = int(self.c.lengths[b])
            rows = [b] if self.cu is None and w else range(t, t + w)
            out += [(r, b, n - w + i) for i, r in enumerate(rows)]
            t += w
        return out


def check(step):
    c = step.c
    k0, v0, mass0, pos0 = (None if x is None else x.clone() for x in (c.k, c.v, c.mass, c.pos))
    step.run()
    assert c.status.item() == 0
    where = step.slots()
    used = torch.tensor([t for t, _, _ in where], device="cuda", dtype=torch.long)
    kk, k_size = step.turned(step.k)
    # sine and cosine: the angle within 2^-24 (rounded to fp32 below pi, 2^-53 of up to 2^31 before),
    # 2^-23 of the function: 2^-21 of the pair together with the rotation's three roundings
    if step.q is not None:
        want, size = step.turned(step.q)
        err = (step.q_out.double() - want).abs()[used]
        assert (err <= (want.abs() * 2.0 ** -8 + size * 2.0 ** -21 + 1e-38)[used]).all(), err.max()
        rest = torch.ones(step.T, dtype=torch.bool, device="cuda")
        rest[used] = False
        assert (step.q_out[rest] == 7.0).all()  # padding and idle rows stay as they were
    touched = torch.zeros(c.n_pages, c.page, dtype=torch.bool, device="cuda")
    for name, pool, pool0, new, size, scale in (("k", c.k, k0, kk, k_size, c.k_scale),
                                                ("v", c.v, v0, step.v.double(), torch.zeros_like(kk), c.v_scale)):
        for t, b, slot in where:
            p, s = int(c.table[b, slot // c.page]), slot % c.page
            touched[p, s] = True
            got = pool[p, :, s]
            got = got.view(torch.float8_e4m3fn).double() if c.e4m3 else got.double()
            w = new[t] / scale
            slack = size[t] / scale * 2.0 ** -21
            if c.e4m3:  # half a step of E4M3, of its smallest exponent below 2^-6; one fp32 rounding of the quotient
                w = w.clamp(-448, 448)
                bound = torch.maximum(w.abs() * 2.0 ** -4, torch.full_like(w, 2.0 ** -10)) + slack + w.abs() * 2.0 ** -23
            else:
                bound = w.abs() * 2.0 ** -8 + slack + 1e-38
            assert ((got - w).abs() <= bound).all(), (name, t, ((got - w).abs() / bound).max())
        same = (pool.view(torch.uint8) if c.e4m3 else pool.view(torch.int16)) == (pool0.view(torch.uint8) if c.e4m3 else pool0.view(torch.int16))
        assert same.permute(0, 2, 1, 3)[~touched].all()
    if c.mass is not None:
        for t, b, slot in where:
            p, s = int(c.table[b, slot // c.page]), slot % c.page
            assert (c.mass[p, :, s] == 0).all() and (c.pos[p, :, s] == step.positions[0, t]).all()
        keep = ~touched[:, None].expand_as(c.pos)
        assert torch.equal(c.pos[keep], pos0[keep]) and torch.equal(c.mass[keep].nan_to_num(-1), mass0[keep].nan_to_num(-1))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads,rot,axes,adjacent", [
    (64, 4, 2, 64, 1, False), (64, 3, 1, 32, 2, True), (96, 6, 6, 96, 3, False), (128, 8, 2, 128, 3, False),
    (128, 8, 2, 128, 1, True), (128, 7, 7, 16, 4, False), (192, 2, 1, 64, 1, False), (256, 16, 2, 64, 1, False),
    (256, 4, 4, 256, 3, True), (128, 4, 2, 0, 1, False)])
def test_decode_and_prompts(dim, heads, kv_heads, rot, axes, adjacent, e4m3):
    c = Cache([1, 0, 17, 64, 300], heads, kv_heads, dim, 16, e4m3, seed=dim)
    check(Step(c, [1, 0, 1, 1, 1], axes, rot, adjacent, decode=True))
    c = Cache([33, 5, 0, 64, 300], heads, kv_heads, dim, 32, e4m3, seed=dim + 1)
    check(Step(c, [33, 0, 0, 20, 57], axes, rot, adjacent, pad=3))


@pytest.mark.parametrize("T", [1, 1183, 1185, 2500, 10007])
def test_blocks_of_several_tokens(T):
    c = Cache([T + 3, 7], 2, 1, 64, 64, seed=T)
    step = Step(c, [T - min(T - 1, 5), min(T - 1, 5)], 2)
    step.run()
    want, size = step.turned(step.q)
    assert ((step.q_out.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2.0 ** -21).all()
    want, size = step.turned(step.k)
    first = step.new[0]
    got = c.values(c.k, 0, T + 3)[T + 3 - first:]
    assert ((got - want[:first]).abs() <= want[:first].abs() * 2.0 ** -8 + size[:first] * 2.0 ** -21).all()
    assert torch.equal(c.values(c.v, 0, T + 3)[T + 3 - first:], step.v[:first].double())
    assert c.status.item() == 0


def test_thousands_of_sequences():
    """Decode rows and ragged prompts of 3,001 sequences, most of them without new tokens."""
    lengths = [(i * 31) % 7 for i in range(3001)]
    c = Cache(lengths, 2, 1, 64, 8, seed=31)
    step = Step(c, [1 if n else 0 for n in lengths], decode=True)
    step.run()
    live = [(i, n) for i, n in enumerate(lengths) if n]
    rows = torch.tensor([i for i, _ in live], device="cuda")
    last = torch.tensor([n - 1 for _, n in live], device="cuda")
    page = c.table.long()[rows, last // 8]
    assert torch.equal(c.v[page, 0, last % 8], step.v[rows, 0])
    assert torch.equal(c.pos[page, 0, last % 8], step.positions[0, rows])
    assert (step.q_out[torch.tensor([i for i, n in enumerate(lengths) if not n], device="cuda")] == 7).all()
    new = [n if i % 97 == 5 else 0 for i, n in enumerate(lengths)]
    step = Step(c, new, 2, pad=11, seed=5)
    step.run()
    assert c.status.item() == 0
    for t, b, slot in step.slots():
        p = int(c.table[b, slot // 8])
        assert torch.equal(c.v[p, 0, slot % 8], step.v[t, 0]) and int(c.pos[p, 0, slot % 8]) == int(step.positions[0, t])
    assert (step.q_out[sum(new):] == 7).all() and (step.q_out[:sum(new)] != 7).any()


def test_weights_without_positions_and_no_rotation():
    c = Cache([20, 0, 7], 4, 2, 96, 16, seed=32)
    c.pos = None
    step = Step(c, [3, 0, 2], rot=0)
    step.positions = None
    k = step.k.clone()
    step.run()
    at = c.place(0, torch.arange(17, 20, device="cuda"))
    assert (c.mass[at] == 0).all() and torch.equal(c.k[at], k[:3]) and torch.equal(step.q_out, step.q)
    assert c.status.item() == 0


def test_far_positions():
    """Positions up to 2^31 - 1: an angle of 2 x 10^9 radians still has its 20 bits behind the point."""
    c = Cache([64], 4, 4, 64, seed=3)
    step = Step(c, [64], 1, top=2 ** 31 - 1)
    step.positions[0, :4] = torch.tensor([0, 1, 2 ** 31 - 1, 2 ** 31 - 2], dtype=torch.int32)
    angle = step.positions[0].double()[:, None] * step.inv_freq
    c2 = 2.0 ** -53 * angle.max()  # what fp64 leaves of the angle, on both sides
    assert c2 < 2.0 ** -21
    step.run()
    want, size = step.turned(step.q)
    assert ((step.q_out.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * (2.0 ** -20 + 4 * c2)).all()


def test_keys_and_values_alone_and_dense_rows():
    c = Cache([20, 9], 6, 2, 128, 16, meta=False, seed=5)
    check(Step(c, [20, 3], 2, queries=False))
    c = Cache([20, 9], 6, 2, 128, 16, seed=6)
    step = Step(c, [5, 9], 1)
    step.q, step.k, step.v = step.q.contiguous(), step.k.contiguous(), step.v.contiguous()
    check(step)


def test_saturation_nan_and_ties_of_the_stored_format():
    c = Cache([1], 1, 1, 64, 16, e4m3=True, k_scale=1.0, v_scale=0.5, seed=7)
    step = Step(c, [1], rot=0, decode=True)
    x = torch.tensor([448.0, 464, 480, 1e30, -math.inf, math.nan, 17, 19, 21, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10,
                      3 * 2.0 ** -10, -0.0, 0.0], device="cuda")
    step.k[0, 0, :16], step.v[0, 0, :16] = x, x / 2
    step.run()
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    p = c.table[0, 0].long()
    assert torch.equal(c.k[p, 0, 0, :16], want) and torch.equal(c.v[p, 0, 0, :16], want)
    assert want[5].item() & 0x7F == 0x7F


def test_bad_contents_are_skipped_and_reported():
    def fresh():
        c = Cache([20, 30, 40], 4, 2, 64, 16, seed=8)
        return c, Step(c, [2, 2, 2], 2)

    def skipped(c, step, tokens):
        before = c.k.clone(), c.v.clone(), c.pos.clone()
        step.run()
        assert c.status.item() == 2
        bad = set(tokens)
        assert all((step.q_out[t] == 7).all() == (t in bad) for t in range(step.T))
        for t, b, slot in step.slots():
            at = c.place(b, torch.tensor([slot], device="cuda"))
            same = torch.equal(c.v[at].view(torch.int16), before[1][at].view(torch.int16))
            assert same == (t in bad)

    c, step = fresh()
    step.positions[0, 3] = -1
    skipped(c, step, [3])
    c, step = fresh()
    step.positions[1, 0] = -(2 ** 31)
    skipped(c, step, [0])
    c, step = fresh()
    step.axis[5] = 2
    skipped(c, step, range(6))
    c, step = fresh()
    slots = step.slots()
    c.table[1, slots[2][2] // 16] = -1
    step.slots = lambda: [s for s in slots if s[1] != 1]
    skipped(c, step, [2, 3])
    c, step = fresh()
    step.slots = lambda s=step.slots(): [x for x in s if x[1] != 2]
    c.lengths[2] = -1
    skipped(c, step, [4, 5])
    c, step = fresh()
    step.slots = lambda s=step.slots(): [x for x in s if x[1] != 0]
    c.lengths[0] = 1  # two new tokens in a sequence of one: the first has no slot
    skipped(c, step, [0])


def test_captured_step():
    c = Cache([50, 0, 80], 4, 2, 64, 16, seed=9)
    step = Step(c, [1, 0, 1], 3, decode=True)
    kv = c.kv()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(kv)
    k0 = c.k.clone()
    c.lengths.copy_(torch.tensor([49, 0, 33], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got, want = c.k.clone(), c.k.copy_(k0)
    step.run()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    check(step)
