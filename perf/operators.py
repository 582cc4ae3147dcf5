"""The key-value cache operators, case by case: inputs, a plain form in elementary torch operations, and the call a
user makes of this library.

Three operators over one paged cache (pools [pages][kv heads][page size][head dim], a block table, lengths):

  append   rotary positions (one to three axes) on the new tokens' q and k, k and v written into the cache
  attend   attention of one new token a sequence over the cache, optionally adding each entry's weight to its mass
  evict    the entries with the least accumulated weight leave, survivors move into the freed slots

A case is real work of a serving step: latency-bound single sequences, ragged batches with idle rows, long caches,
bf16 and E4M3 caches, the head layouts of grouped-query and multi-head models.
"""
import math
import random

import torch

own = False

NAN = float("nan")


def listed():
    return [
        # one chat: the step's single token, two KV heads of 256 with rotary on their first 64 dims
        dict(name="append_one", op="append", batch=1, lo=700, hi=700, idle=0, heads=16, kv_heads=2, dim=256, page=64,
             e4m3=False, rot=64, axes=1, adjacent=False, tokens=0, pick=1),
        # a full decode batch of a served model with image and video positions, E4M3 cache, some rows idle
        dict(name="append_step_e4m3", op="append", batch=96, lo=40, hi=3000, idle=7, heads=64, kv_heads=8, dim=128,
             page=16, e4m3=True, rot=128, axes=3, adjacent=False, tokens=0, pick=2),
        # five prompts of different lengths in one prefill chunk
        dict(name="append_prompts", op="append", batch=5, lo=900, hi=9000, idle=0, heads=32, kv_heads=8, dim=128,
             page=32, e4m3=False, rot=128, axes=3, adjacent=False, tokens=8191, pick=3),
        # the first tokens of one chat: latency alone counts
        dict(name="attend_one_short", op="attend", batch=1, lo=37, hi=37, idle=0, heads=16, kv_heads=2, dim=256,
             page=64, e4m3=False, weigh=False, pick=4),
        # one agent with a long history
        dict(name="attend_one_long", op="attend", batch=1, lo=131071, hi=131071, idle=0, heads=64, kv_heads=8,
             dim=128, page=64, e4m3=False, weigh=False, pick=5),
        # a decode batch of mixed lengths, some rows idle
        dict(name="attend_batch", op="attend", batch=64, lo=300, hi=16000, idle=5, heads=32, kv_heads=8, dim=128,
             page=16, e4m3=False, weigh=False, pick=6),
        # the same over an E4M3 cache whose entries are weighed for eviction, sixteen query heads a KV head
        dict(name="attend_batch_e4m3", op="attend", batch=48, lo=500, hi=12000, idle=3, heads=64, kv_heads=4, dim=128,
             page=64, e4m3=True, weigh=True, pick=7),
        # multi-head attention, small heads
        dict(name="attend_multi_head", op="attend", batch=24, lo=100, hi=5000, idle=0, heads=16, kv_heads=16, dim=64,
             page=32, e4m3=False, weigh=True, pick=8),
        # heads of 256, eight query heads a KV head, entries weighed
        dict(name="attend_wide", op="attend", batch=12, lo=1000, hi=24000, idle=0, heads=16, kv_heads=2, dim=256,
             page=64, e4m3=False, weigh=True, pick=9),
        # steady state: every sequence is 64 entries over its budget
        dict(name="evict_step", op="evict", batch=8, lo=2112, hi=2112, idle=0, heads=32, kv_heads=8, dim=128, page=16,
             e4m3=False, keep=2048, share=0.0, recent=128, pick=10),
        # memory is short: a ragged batch gives up half of its entries
        dict(name="evict_half", op="evict", batch=32, lo=500, hi=8000, idle=3, heads=32, kv_heads=8, dim=128, page=32,
             e4m3=False, keep=0, share=0.5, recent=256, pick=11),
        # two long histories cut to 32k entries, E4M3 cache
        dict(name="evict_long_e4m3", op="evict", batch=2, lo=131000, hi=131071, idle=0, heads=16, kv_heads=2, dim=256,
             page=64, e4m3=True, keep=32768, share=0.0, recent=1024, pick=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict"])
    dim = rng.choice([64, 64, 96, 128, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    group = rng.choice([1, 2, 4, 5, 7, 8, 12, 16] if kv_heads > 2 else [1, 4, 8, 16, 24, 32])
    c = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
             e4m3=rng.random() < 0.4, pick=rng.randrange(1 << 20))
    entry = 2 * kv_heads * dim  # values of one cached token; the largest cache here holds 450 M values
    c["batch"] = _log(rng, 1, 96)
    top = max(64, min(131071, 450_000_000 // (entry * c["batch"])))
    c["hi"] = _log(rng, 17, top)
    c["lo"] = max(1, min(c["hi"], _log(rng, 1, c["hi"])))
    c["idle"] = rng.randrange(0, 1 + c["batch"] // 8)
    if op == "append":
        c["axes"] = rng.choice([1, 2, 3])
        c["rot"] = rng.choice([r for r in (32, 64, 96, 128, 192, 256) if r <= dim])
        c["adjacent"] = rng.random() < 0.3
        c["tokens"] = 0 if rng.random() < 0.5 else min(_log(rng, 1, 8191), c["lo"] * (c["batch"] - c["idle"]))
    elif op == "attend":
        c["weigh"] = rng.random() < 0.5
    else:
        c["keep"], c["share"] = (0, rng.uniform(0.1, 0.95)) if rng.random() < 0.5 else (_log(rng, 1, c["hi"]), 0.0)
        c["recent"] = rng.choice([0, 1, 17, 128, 1000])
    return c


def _lengths(c):
    """Cached entries of each sequence, the new tokens among them: spread over their logarithm, idle rows (0) among them."""
    r = random.Random(c["pick"])
    n = [c["hi"]] + [_log(r, c["lo"], c["hi"]) for _ in range(c["batch"] - 1)]
    for b in r.sample(range(1, c["batch"]), c["idle"]) if c["idle"] else []:
        n[b] = 0
    return n


def _new(c, n):
    """New tokens of each sequence: one each (tokens=0), or `tokens` in all, shared out by length."""
    if not c["tokens"]:
        return [1 if x else 0 for x in n]
    total, left, out = sum(n), c["tokens"], []
    for x in n:
        out.append(min(x, c["tokens"] * x // total))
        left -= out[-1]
    for b, x in enumerate(n):
        more = min(left, x - out[b])
        out[b] += more
        left -= more
    return out


def _budgets(c, n):
    return [int(x * c["share"]) if c["share"] else c["keep"] for x in n]


def prepare(c, seed):
    g = torch.Generator("cuda").manual_seed(seed * 1000003 + c["pick"])
    host = random.Random(seed * 7919 + c["pick"])
    d, hk, hq, page = c["dim"], c["kv_heads"], c["heads"], c["page"]
    n = _lengths(c)
    pages = [-(-x // page) for x in n]
    n_pages, width = sum(pages) + 3, max(pages) + 1
    ids = list(range(n_pages))
    host.shuffle(ids)
    table, rows = ids[:], []
    for p in pages:  # an unused entry of the table is -1
        rows.append([table.pop() for _ in range(p)] + [-1] * (width - p))
    table = torch.tensor(rows, dtype=torch.int32, device="cuda")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    slot = torch.arange(width * page, device="cuda")
    valid = slot[None, :] < lengths[:, None]
    used = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
    at = (table.long().clamp(min=0)[:, slot // page] * page + slot % page)[valid]
    used.view(-1)[at] = True
    s = dict(c, table=table, lengths=lengths, k_scale=0.0123 if c["e4m3"] else 1.0, v_scale=0.0091 if c["e4m3"] else 1.0)
    for name in ("k", "v"):
        pool = normal(n_pages, hk, page, d)
        pool = pool.masked_fill_(~used[:, None, :, None], NAN)  # what no sequence wrote is whatever memory held
        s[name] = (pool.float() / s[name + "_scale"]).clamp_(-448, 448).to(torch.float8_e4m3fn) if c["e4m3"] else pool
    # accumulated weights and positions of the entries, and the lengths, in one buffer with a copy of its first state:
    # a pass that changes them starts with that state again
    size = n_pages * hk * page
    meta = torch.empty(2 * size + len(n), dtype=torch.int32, device="cuda")
    s["mass"], s["pos"] = meta[:size].view(torch.float32).view(n_pages, hk, page), meta[size:2 * size].view(n_pages, hk, page)
    weights = torch.exp(2 * torch.randn(n_pages, hk, page, generator=g, device="cuda") - 3)
    fresh = torch.rand(n_pages, hk, page, generator=g, device="cuda") < 0.02
    s["mass"].copy_(weights.masked_fill_(fresh, 0.0))  # equal ones among them: entries nothing has attended to yet
    # positions grow along a sequence with gaps (evicted tokens), out of order here and there (survivors that moved)
    wide = torch.arange(width * page, device="cuda", dtype=torch.int64)
    order = (wide + 40 * torch.rand(len(n), hk, width * page, generator=g, device="cuda")).argsort(-1)
    where = (table.long().clamp(min=0)[:, None, slot // page] * hk + torch.arange(hk, device="cuda")[:, None]) * page + slot % page
    keep = valid[:, None, :].expand_as(where)
    s["pos"].zero_()
    s["pos"].view(-1)[where[keep]] = (3 * order + order % 3)[keep].int()
    s["lengths"] = meta[2 * size:]
    s["lengths"].copy_(lengths)
    s["meta"], s["meta0"] = meta, meta.clone()
    if c["op"] == "append":
        new = _new(c, n)
        t = sum(new) if c["tokens"] else len(n)
        qkv = normal(t, (hq + 2 * hk) * d)  # one projection's output: q, k and v are views of it
        s["q"], s["k_new"], s["v_new"] = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], 1))
        s["cu"] = torch.tensor([sum(new[:b]) for b in range(len(n) + 1)], dtype=torch.int32, device="cuda") if c["tokens"] else None
        first = [3 * (x - w) + i for x, w in zip(n, new) for i in range(w)] if c["tokens"] else [3 * x for x in n]
        first = torch.tensor([first], dtype=torch.int32, device="cuda")
        more = torch.randint(0, 128, (c["axes"] - 1, t), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = torch.cat([first, first + more])  # rows and columns of an image begin where its time stands
        half = c["rot"] // 2
        i = torch.arange(half, dtype=torch.float64, device="cuda")
        s["inv_freq"] = 1e6 ** (-i / half)
        s["axis"] = (i % c["axes"]).int() if c["pick"] % 2 else (i * c["axes"] / half).int()  # interleaved, or in sections
        s["q_out"] = torch.zeros(t, hq, d, dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "attend":
        s["q"] = normal(len(n), hq, d)
        s["out"] = torch.zeros(len(n), hq, d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(len(n), hq, device="cuda")
        s["scale"] = d ** -0.5
    else:
        s["budgets"] = torch.tensor(_budgets(c, n), dtype=torch.int32, device="cuda")
    if own:  # the cache's description and the workspace that a serving program keeps
        import expert_offloaded_serving_b200 as ft
        s["kv"] = ft.make_kv(hq, s["k"], s["v"], table, s["lengths"], mass=s["mass"], pos=s["pos"], k_scale=s["k_scale"],
                             v_scale=s["v_scale"])
        s["work"] = torch.empty(ft.ft_kv_workspace_bytes(s["kv"]), dtype=torch.uint8, device="cuda")
    return s


def _entries(s):
    """[batch][width * page]: which slots a sequence has, and the flat (page, 0, slot) place of each."""
    page, hk = s["page"], s["kv_heads"]
    slot = torch.arange(s["table"].shape[1] * page, device="cuda")
    valid = slot[None, :] < s["lengths"][:, None]
    return valid, s["table"].long().clamp(min=0)[:, slot // page] * hk * page + slot % page


def _rotate(x, cos, sin, rot, adjacent):
    x = x.float()
    if adjacent:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if adjacent else -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    hk, page, rot = s["kv_heads"], s["page"], s["rot"]
    angle = s["positions"].double()[s["axis"].long()].T * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    t = torch.arange(s["q"].shape[0], device="cuda")
    if s["cu"] is None:
        seq, slot = t, s["lengths"].long() - 1
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu, t, right=True) - 1
        slot = s["lengths"].long()[seq] - (cu[seq + 1] - t)
    some = (slot >= 0)[:, None, None]
    s["q_out"].copy_(torch.where(some, _rotate(s["q"], cos, sin, rot, s["adjacent"]), s["q_out"].float()))
    live = slot.clamp(min=0)
    at = (s["table"].long()[seq, live // page].clamp(min=0) * hk)[:, None] + torch.arange(hk, device="cuda")
    at = (at * page + (live % page)[:, None])[slot >= 0]
    for name, new in (("k", _rotate(s["k_new"], cos, sin, rot, s["adjacent"])), ("v", s["v_new"].float())):
        new = new[slot >= 0]
        new = (new / s[name + "_scale"]).clamp(-448, 448) if s["e4m3"] else new
        rows = s[name].view(-1, s["dim"])
        rows.view(torch.uint8 if s["e4m3"] else rows.dtype)[at] = (
            new.to(torch.float8_e4m3fn).view(torch.uint8) if s["e4m3"] else new.to(rows.dtype))
    s["mass"].view(-1)[at] = 0.0
    s["pos"].view(-1)[at] = s["positions"][0][slot >= 0][:, None].expand_as(at)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "mass": s["mass"], "pos": s["pos"]}


def _plain_attend(s):
    hk, hq, page, d = s["kv_heads"], s["heads"], s["page"], s["dim"]
    valid, _ = _entries(s)
    b, n = valid.shape
    pages = s["table"].long().clamp(min=0)

    def gathered(pool, scale):  # [batch][kv heads][slots][dim], zero where no sequence wrote
        x = pool.view(torch.uint8)[pages].view(torch.float8_e4m3fn) if s["e4m3"] else pool[pages]
        x = x.float().transpose(1, 2).reshape(b, hk, n, d) * scale
        return x.masked_fill_(~valid[:, None, :, None], 0.0)

    q = s["q"].float().view(b, hk, hq // hk, d)
    score = (q @ gathered(s["k"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    score = score.masked_fill_(~valid[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    p = p / total.clamp(min=1e-38)  # a row without entries is zero
    out = {"out": (p @ gathered(s["v"], s["v_scale"])).view(b, hq, d).to(torch.bfloat16),
           "lse": torch.where(total > 0, top + total.log(), -math.inf).view(b, hq)}
    if s["weigh"]:
        s["meta"].copy_(s["meta0"])
        _, at = _entries(s)
        at = at[:, None] + page * torch.arange(hk, device="cuda")[:, None]
        keep = valid[:, None].expand_as(at)
        s["mass"].view(-1)[at[keep]] += p.sum(2)[keep]
        out["mass"] = s["mass"]
    return out


def _plain_evict(s):
    s["meta"].copy_(s["meta0"])
    hk, page = s["kv_heads"], s["page"]
    valid, at = _entries(s)
    at = at[:, None] + page * torch.arange(hk, device="cuda")[:, None]  # [batch][kv heads][slots]
    valid = valid[:, None].expand_as(at)
    budget = torch.minimum(s["budgets"], s["lengths"]).long()[:, None, None]
    pos = torch.where(valid, s["pos"].view(-1)[at].long(), -1)
    mass = s["mass"].view(-1)[at]
    recent = pos > pos.amax(-1, keepdim=True) - s["recent"]
    # an order of whole numbers: recent ones first, the newest before the others, then by weight, then the lowest slot
    key = torch.where(recent, (1 << 31) + pos, mass.view(torch.int32).long())
    key = torch.where(valid, key, -1)
    rank = key.argsort(stable=True, dim=-1, descending=True).argsort(dim=-1)
    kept = valid & (rank < budget)
    slot = torch.arange(at.shape[-1], device="cuda")
    hole, mover = valid & ~kept & (slot < budget), kept & (slot >= budget)
    to, frm = at[hole], at[mover]  # as many of each in a (sequence, head), both in the order of their slots
    for name in ("k", "v"):
        rows = s[name].view(torch.uint8 if s["e4m3"] else torch.bfloat16).view(-1, s["dim"])
        rows[to] = rows[frm]
    s["mass"].view(-1)[to] = s["mass"].view(-1)[frm]
    s["pos"].view(-1)[to] = s["pos"].view(-1)[frm]
    s["lengths"].copy_(budget[:, 0, 0])
    return {"k": s["k"], "v": s["v"], "mass": s["mass"], "pos": s["pos"], "lengths": s["lengths"]}


def _own_append(s):
    import expert_offloaded_serving_b200 as ft
    ft.ft_kv_append(s["kv"], s["q"], s["k_new"], s["v_new"], s["cu"], s["positions"], s["inv_freq"], s["axis"], s["q_out"],
                    ft.FT_ROPE_ADJACENT if s["adjacent"] else 0)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "mass": s["mass"], "pos": s["pos"]}


def _own_attend(s):
    import expert_offloaded_serving_b200 as ft
    if s["weigh"]:
        s["meta"].copy_(s["meta0"])
    ft.ft_kv_attention(s["kv"], s["q"], s["scale"], s["out"], s["lse"], s["work"], ft.FT_KV_MASS if s["weigh"] else 0)
    out = {"out": s["out"], "lse": s["lse"]}
    if s["weigh"]:
        out["mass"] = s["mass"]
    return out


def _own_evict(s):
    import expert_offloaded_serving_b200 as ft
    s["meta"].copy_(s["meta0"])
    ft.ft_kv_evict(s["kv"], s["budgets"], s["recent"], s["work"])
    return {"k": s["k"], "v": s["v"], "mass": s["mass"], "pos": s["pos"], "lengths": s["lengths"]}


def run(s):
    if own:
        return {"append": _own_append, "attend": _own_attend, "evict": _own_evict}[s["op"]](s)
    return {"append": _plain_append, "attend": _plain_attend, "evict": _plain_evict}[s["op"]](s)


def work(c):
    d, hk, hq = c["dim"], c["kv_heads"], c["heads"]
    n = _lengths(c)
    es = 1 if c["e4m3"] else 2
    live = sum(x > 0 for x in n)
    if c["op"] == "append":
        t = sum(_new(c, n))
        # q in and out, k and v in, both into the cache with their weight and position, the positions
        return {"bytes": t * (4 * hq * d + 4 * hk * d + 2 * hk * d * es + 8 * hk + 4 * c["axes"]),
                "flops": t * (hq + hk) * c["rot"] * 3}
    if c["op"] == "attend":
        # the cached keys and values once, q, out and lse; each entry's weight read and written
        return {"bytes": sum(n) * hk * (2 * d * es + 8 * c["weigh"]) + live * hq * (4 * d + 4), "flops": 4 * sum(n) * hq * d}
    # every over-full sequence's weights and positions; the survivors above the budget (about their share of it) are moved
    size, moved = 0, 0
    for x, b in zip(n, _budgets(c, n)):
        if x > b:
            size += x
            moved += b * (x - b) // x
    return {"bytes": hk * (8 * size + 2 * moved * (2 * d * es + 8)) + 8 * len(n), "flops": hk * size}


def exact(c, seed):
    """From the definitions, in 64 bits, one sequence after another."""
    if c["op"] == "evict":
        return None  # entries move, nothing is computed
    s = prepare(c, seed)
    n, page, hk, d = _lengths(c), c["page"], c["kv_heads"], c["dim"]
    group = c["heads"] // hk
    if c["op"] == "append":
        q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
        new, row, half = _new(c, n), 0, c["rot"] // 2
        left = torch.arange(half, device="cuda") * (2 if c["adjacent"] else 1)
        right = left + (1 if c["adjacent"] else half)
        for b, w in enumerate(new):
            if not c["tokens"]:
                row = b
            if w:
                phase = s["positions"][:, row:row + w].double()[s["axis"].long()] * s["inv_freq"][:, None]
                turn = torch.polar(torch.ones_like(phase), phase).T[:, None]  # a pair is a complex number

                def turned(x):
                    x = x.double().clone()
                    z = torch.complex(x[..., left], x[..., right]) * turn
                    x[..., left], x[..., right] = z.real, z.imag
                    return x

                q[row:row + w] = turned(s["q"][row:row + w])
                slots = torch.arange(n[b] - w, n[b], device="cuda")
                pages = s["table"][b].long()[slots // page]
                limit = 448.0 if c["e4m3"] else math.inf
                k[pages, :, slots % page] = (turned(s["k_new"][row:row + w]) / s["k_scale"]).clamp(-limit, limit)
                v[pages, :, slots % page] = (s["v_new"][row:row + w].double() / s["v_scale"]).clamp(-limit, limit)
            row += w
        return {"q": q, "k": k, "v": v, "mass": None, "pos": None}
    out = torch.zeros(len(n), c["heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((len(n), c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    mass = s["mass"].double()
    for b, x in enumerate(n):
        pages = s["table"][b, :-(-x // page)].long()
        for h in range(hk if x else 0):
            k = s["k"][pages, h].double().reshape(-1, d)[:x] * s["k_scale"]
            v = s["v"][pages, h].double().reshape(-1, d)[:x] * s["v_scale"]
            heads = slice(h * group, (h + 1) * group)
            score = s["scale"] * (s["q"][b, heads].double() @ k.T)
            lse[b, heads] = torch.logsumexp(score, -1)
            p = torch.exp(score - lse[b, heads, None])
            out[b, heads] = p @ v
            place = torch.zeros(len(pages) * page, dtype=torch.float64, device="cuda")
            place[:x] = p.sum(0)
            mass[pages, h] += place.view(len(pages), page)
    return {"out": out, "lse": lse, "mass": mass} if c["weigh"] else {"out": out, "lse": lse}
