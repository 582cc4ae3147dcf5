"""Paged key-value caches for the tests, and the operators' definitions in 64 bits (not collected by pytest)."""
from __future__ import annotations

import math

import torch

import expert_offloaded_serving_b200 as ft


class Cache:
    """A cache with shuffled pages.  What no sequence wrote holds NaN, unused table entries a page out of range."""

    def __init__(self, lengths, heads, kv_heads, dim, page=16, e4m3=False, seed=0, spare=2, k_scale=None, v_scale=None,
                 meta=True, room=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.page, self.e4m3 = heads, kv_heads, dim, page, e4m3
        self.k_scale = (k_scale or 0.0173) if e4m3 else 1.0
        self.v_scale = (v_scale or 0.0091) if e4m3 else 1.0
        need = [-(-(n + room) // page) for n in lengths]
        self.n_pages = sum(need) + spare
        width = max(need + [1]) + 1
        ids = torch.randperm(self.n_pages, generator=g, device="cuda").tolist()
        rows = [[ids.pop() for _ in range(p)] + [self.n_pages + 7] * (width - p) for p in need]
        self.table = torch.tensor(rows, dtype=torch.int32, device="cuda").reshape(len(lengths), width)
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        shape = (self.n_pages, kv_heads, page, dim)
        self.k = self.stored(torch.full(shape, math.nan, device="cuda"), 1.0)
        self.v = self.k.clone()
        self.mass = torch.full(shape[:3], math.nan, device="cuda") if meta else None
        self.pos = torch.full(shape[:3], -5, dtype=torch.int32, device="cuda") if meta else None
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lengths):
            if n:
                at = self.place(b, torch.arange(n, device="cuda"))
                self.k[at] = self.stored(torch.randn(n, kv_heads, dim, generator=g, device="cuda"), self.k_scale)
                self.v[at] = self.stored(torch.randn(n, kv_heads, dim, generator=g, device="cuda"), self.v_scale)
                if meta:
                    self.mass[at] = torch.rand(n, kv_heads, generator=g, device="cuda") ** 4
                    self.pos[at] = torch.arange(n, dtype=torch.int32, device="cuda")[:, None] * 2

    def stored(self, x, scale):
        if not self.e4m3:
            return x.to(torch.bfloat16)
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def place(self, b, slots):
        """Index of the entries `slots` of sequence b: pool[place] is [slots][kv heads] (...)"""
        slots = slots.long()
        return (self.table[b].long()[slots // self.page][:, None], torch.arange(self.kv_heads, device="cuda")[None],
                (slots % self.page)[:, None])

    def pools(self):
        t = torch.float8_e4m3fn if self.e4m3 else torch.bfloat16
        return self.k.view(t), self.v.view(t)

    def kv(self, **more):
        k, v = self.pools()
        return ft.make_kv(self.heads, k, v, self.table, self.lengths, mass=self.mass, pos=self.pos, k_scale=self.k_scale,
                          v_scale=self.v_scale, status=self.status, **more)

    def values(self, pool, b, n):
        x = pool[self.place(b, torch.arange(n, device="cuda"))]
        x = x.view(torch.float8_e4m3fn).double() if self.e4m3 else x.double()
        return x  # [n][kv heads][dim], what the bytes stand for, without the scale

    def workspace(self, kv):
        return torch.full((ft.ft_kv_workspace_bytes(kv),), 0xA5, dtype=torch.uint8, device="cuda")


def attention(c: Cache, q, scale, lengths):
    """out, lse, sum_i p_i |v_i| and the largest sum |q||k| of a head, in 64 bits; p per (sequence, query head)."""
    B, H, D = q.shape
    G = H // c.kv_heads
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    size, reach = out.clone(), torch.zeros(B, H, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    weights = {}
    for b, n in enumerate(lengths):
        if n == 0:
            continue
        k, v = c.values(c.k, b, n) * c.k_scale, c.values(c.v, b, n) * c.v_scale
        qq = q[b].double().view(c.kv_heads, G, D)
        s = scale * torch.einsum("hgd,nhd->hgn", qq, k)
        reach[b] = (abs(scale) * torch.einsum("hgd,nhd->hgn", qq.abs(), k.abs())).amax(-1).reshape(H)
        lse[b] = torch.logsumexp(s, -1).reshape(H)
        p = torch.softmax(s, -1)
        out[b] = torch.einsum("hgn,nhd->hgd", p, v).reshape(H, D)
        size[b] = torch.einsum("hgn,nhd->hgd", p, v.abs()).reshape(H, D)
        weights[b] = p
    return out, lse, size, reach, weights


def attention_bounds(c: Cache, out, size, reach, lengths):
    """How far out, lse and a weight (relative) may be off.

    A score is a sum of D exact products in fp32: off by at most (D + 4) 2^-23 reach (the tensor core may cut a
    bit off each addition); a weight by twice that relative, plus 2^-21 of the exponential and the statistics.  Sums over n
    entries add n 2^-23.  p meets v with 2^-16 (two bf16 parts), or in f16 with 2^-11 and 2^-24 absolute
    (below 2^-14 f16 has no more bits), of the sum of p |v|.  The result is rounded to bf16: 2^-8 relative."""
    n = torch.tensor(lengths, dtype=torch.float64, device=out.device)[:, None]
    ds = (c.dim + 4) * 2.0 ** -23 * reach
    weight = 2 * ds + 2.0 ** -21 + n * 2.0 ** -23
    p = 2.0 ** -11 if c.e4m3 else 2.0 ** -16
    more = size * (weight + p)[..., None]
    if c.e4m3:
        more = more + (n * 2.0 ** -24 * 448 * c.v_scale)[..., None]
    return out.abs() * 2.0 ** -8 + more * 1.01 + 1e-30, ds + 2.0 ** -21 + n * 2.0 ** -23 + reach * 2.0 ** -22, weight


def evict(c: Cache, budgets, recent):
    """The cache after eviction, computed on the host entry by entry: new k, v, mass, pos, lengths."""
    k, v, mass, pos = (x.clone().cpu() for x in (c.k, c.v, c.mass, c.pos))
    table, lengths = c.table.cpu(), c.lengths.cpu().clone()
    for b, keep in enumerate(budgets):
        n = int(lengths[b])
        if n <= keep:
            continue
        at = [(int(table[b, i // c.page]), i % c.page) for i in range(n)]
        for h in range(c.kv_heads):
            m = [float(mass[p, h, s]) for p, s in at]
            x = [int(pos[p, h, s]) for p, s in at]
            newest = max(x)
            order = sorted(range(n), key=lambda i: (0, -x[i], i) if x[i] > newest - recent and x[i] >= 0
                           else (1, -m[i] if m[i] > 0 else 0.0, i))
            kept = set(order[:keep])
            freed = [i for i in range(keep) if i not in kept]
            movers = [i for i in range(keep, n) if i in kept]
            assert len(freed) == len(movers)
            for to, frm in zip(freed, movers):
                (pt, st), (pf, sf) = at[to], at[frm]
                for pool in (k, v, mass, pos):
                    pool[pt, h, st] = pool[pf, h, sf]
        lengths[b] = keep
    return k, v, mass, pos, lengths
