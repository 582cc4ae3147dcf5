"""Argument checks of the key-value cache calls: every refusal comes before any CUDA call, so it is tested without a GPU
(fake pointers stand in for device buffers and are never dereferenced), and the binding's own checks of tensors."""
import ctypes as C
import math

import pytest
import torch

import expert_offloaded_serving_b200 as ft

K, V, MASS, POS, TABLE, LEN, STATUS = (0x10000 * i for i in range(1, 8))
Q, KN, VN, CU, PP, INV, AXIS, QO, OUT, LSE, WORK, BUD = (0x1000000 * i for i in range(1, 13))
BIG = 1 << 40


def cache(**kw):
    a = dict(head_dim=128, n_heads=8, n_kv_heads=2, page_size=16, n_seqs=4, max_pages=8, n_pages=32, format=ft.FT_KV_BF16,
             k_scale=1.0, v_scale=1.0, k=K, v=V, mass=MASS, pos=POS, block_table=TABLE, lengths=LEN, status=STATUS)
    a.update(kw)
    return ft.KvCache(**a)


def refused(st, what):
    assert st == ft.FT_ERR_INVALID, st
    assert what in ft.lib().ft_last_error().decode(), ft.lib().ft_last_error()


def append(kv=None, **kw):
    a = dict(T=4, q=Q, qs=1024, k=KN, ks=256, v=VN, vs=256, cu=None, pos=PP, axes=1, inv=INV, axis=AXIS, rot=128, q_out=QO, flags=0)
    a.update(kw)
    return ft.lib().ft_kv_append(C.byref(kv or cache()), a["T"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["cu"],
                                 a["pos"], a["axes"], a["inv"], a["axis"], a["rot"], a["q_out"], a["flags"], None)


def attend(kv=None, **kw):
    a = dict(q=Q, qs=1024, scale=0.1, out=OUT, lse=LSE, work=WORK, bytes=BIG, flags=0)
    a.update(kw)
    return ft.lib().ft_kv_attention(C.byref(kv or cache()), a["q"], a["qs"], a["scale"], a["out"], a["lse"], a["work"],
                                    a["bytes"], a["flags"], None)


def evict(kv=None, **kw):
    a = dict(budgets=BUD, recent=4, work=WORK, bytes=BIG)
    a.update(kw)
    return ft.lib().ft_kv_evict(C.byref(kv or cache()), a["budgets"], a["recent"], a["work"], a["bytes"], None)


SHAPES = [
    (dict(head_dim=80), "head_dim"), (dict(head_dim=0), "head_dim"), (dict(n_kv_heads=0), "n_heads"),
    (dict(n_heads=0), "n_heads"), (dict(n_heads=9), "n_heads"), (dict(n_heads=131072), "n_heads"),
    (dict(page_size=0), "page_size"), (dict(page_size=4), "page_size"), (dict(page_size=24), "page_size"), (dict(page_size=2048), "page_size"),
    (dict(n_seqs=-1), "n_seqs"), (dict(n_seqs=65537), "n_seqs"), (dict(max_pages=0), "max_pages"),
    (dict(max_pages=1 << 27), "max_pages"), (dict(n_pages=0), "n_pages"), (dict(n_pages=1 << 26), "n_pages"),
    (dict(n_seqs=65536, max_pages=1 << 14), "too large"), (dict(format=2), "format"), (dict(format=-1), "format"),
    (dict(format=ft.FT_KV_E4M3, k_scale=0.0), "k_scale"), (dict(format=ft.FT_KV_E4M3, v_scale=-1.0), "v_scale"),
    (dict(format=ft.FT_KV_E4M3, v_scale=math.inf), "finite"), (dict(format=ft.FT_KV_E4M3, k_scale=math.nan), "finite"),
    (dict(k_scale=0.5), "BF16"),
]


@pytest.mark.parametrize("kw,what", SHAPES)
def test_every_call_refuses_a_bad_shape(kw, what):
    kv = cache(**kw)
    for call in (append, attend, evict):
        refused(call(kv), what)
    n = ft.I64(-7)
    refused(ft.lib().ft_kv_workspace_bytes(C.byref(kv), C.byref(n)), what)
    assert n.value == -7


def test_every_call_refuses_more_than_1024_query_heads_a_kv_head():
    kv = cache(n_heads=1025, n_kv_heads=1)
    for call in (append, attend, evict):
        refused(call(kv), "above 1024")
    refused(ft.lib().ft_kv_workspace_bytes(C.byref(kv), C.byref(ft.I64())), "above 1024")
    assert ft.ft_kv_workspace_bytes(cache(n_heads=1024, n_kv_heads=1)) > 0


@pytest.mark.parametrize("kw,what", [
    (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(block_table=None), "NULL"), (dict(lengths=None), "NULL"),
    (dict(k=K + 8), "16-byte"), (dict(v=V + 2), "16-byte"), (dict(mass=MASS + 2), "4-byte"), (dict(pos=POS + 1), "4-byte"),
    (dict(block_table=TABLE + 2), "4-byte"), (dict(lengths=LEN + 3), "4-byte"), (dict(status=STATUS + 2), "4-byte")])
def test_every_call_refuses_bad_buffers(kw, what):
    for call in (append, attend, evict):
        refused(call(cache(**kw)), what)


@pytest.mark.parametrize("kw,what", [
    (dict(T=-1), "T -1"), (dict(T=1 << 31, cu=CU), "T "), (dict(T=5), "without cu_new"), (dict(T=3), "without cu_new"),
    (dict(flags=2), "flags"), (dict(rot=-16), "rot_dim"), (dict(rot=8), "rot_dim"), (dict(rot=144), "rot_dim"),
    (dict(axes=0), "n_axes"), (dict(axes=5), "n_axes"), (dict(axes=-1), "n_axes"), (dict(k=None), "NULL"),
    (dict(v=None), "NULL"), (dict(q=None), "q_out"), (dict(q_out=None), "q_out"), (dict(pos=None), "positions"),
    (dict(inv=None), "inv_freq"), (dict(axis=None), "axis"), (dict(q=Q + 8), "16-byte"), (dict(k=KN + 2), "16-byte"),
    (dict(v=VN + 8), "16-byte"), (dict(q_out=QO + 8), "16-byte"), (dict(qs=1020), "multiple of 8"), (dict(ks=252), "multiple of 8"),
    (dict(qs=1016), "stride"), (dict(ks=248), "stride"), (dict(vs=-256), "stride"), (dict(vs=1 << 33), "stride"),
    (dict(cu=CU + 2), "aligned"), (dict(pos=PP + 2), "aligned"), (dict(inv=INV + 4), "aligned"), (dict(axis=AXIS + 1), "aligned"),
    (dict(q_out=Q), "overlap"), (dict(q_out=Q + 1024 * 8 - 16), "overlap"), (dict(q_out=KN - 16), "overlap"),
    (dict(q_out=VN + 256 * 8 - 16), "overlap")])
def test_append_refuses(kw, what):
    refused(append(**kw), what)


@pytest.mark.parametrize("kw,what", [
    (dict(flags=2), "flags"), (dict(scale=math.nan), "scale"), (dict(scale=math.inf), "scale"), (dict(q=None), "NULL"),
    (dict(out=None), "NULL"), (dict(q=Q + 8), "16-byte"), (dict(out=OUT + 8), "16-byte"), (dict(lse=LSE + 2), "4-byte"),
    (dict(qs=1028), "multiple of 8"), (dict(qs=512), "stride"), (dict(out=Q), "overlap"), (dict(out=Q + 16), "overlap"),
    (dict(out=Q - 16), "overlap"), (dict(work=None), "workspace"), (dict(bytes=1000), "workspace"), (dict(work=WORK + 8), "16-byte")])
def test_attention_refuses(kw, what):
    refused(attend(**kw), what)


def test_attention_needs_mass_to_weigh():
    refused(attend(cache(mass=None), flags=ft.FT_KV_MASS), "mass")


@pytest.mark.parametrize("kw,what", [
    (dict(recent=-1), "recent"), (dict(budgets=None), "budgets"), (dict(budgets=BUD + 2), "budgets"), (dict(work=None), "workspace"),
    (dict(bytes=8), "workspace"), (dict(work=WORK + 4), "16-byte")])
def test_evict_refuses(kw, what):
    refused(evict(**kw), what)


def test_evict_needs_mass_and_positions():
    refused(evict(cache(mass=None)), "mass and pos")
    refused(evict(cache(pos=None)), "mass and pos")


def test_null_caches_and_results():
    L = ft.lib()
    refused(L.ft_kv_workspace_bytes(None, C.byref(ft.I64())), "NULL")
    refused(L.ft_kv_workspace_bytes(C.byref(cache()), None), "NULL")
    refused(L.ft_kv_append(None, 0, None, 0, None, 0, None, 0, None, None, 0, None, None, 0, None, 0, None), "NULL")
    refused(L.ft_kv_attention(None, None, 0, 1.0, None, None, None, 0, 0, None), "NULL")
    refused(L.ft_kv_evict(None, None, 0, None, 0, None), "NULL")
    refused(L.ft_kv_sync_status(None, None), "NULL")


def test_no_sequences_or_tokens_is_a_no_op():
    none = cache(n_seqs=0, k=None, v=None, block_table=None, lengths=None, mass=None, pos=None)
    assert append(none, T=0, q=None, k=None, v=None, pos=None, inv=None, axis=None, rot=0, q_out=None) == ft.FT_OK
    assert attend(none, q=None, out=None, work=None, bytes=0) == ft.FT_OK
    assert evict(none, budgets=None, work=None, bytes=0) == ft.FT_OK
    assert append(T=0, cu=CU, q=None, k=None, v=None, q_out=None) == ft.FT_OK


def test_workspace_grows_with_the_pool_only_where_it_is_weighed():
    small, large = cache(mass=None, pos=None), cache(mass=None, pos=None, n_pages=100000)
    assert ft.ft_kv_workspace_bytes(small) == ft.ft_kv_workspace_bytes(large)
    rows = 100000 * 2 * 16
    assert ft.ft_kv_workspace_bytes(cache(n_pages=100000)) >= rows * 4 * 4  # four query heads' scores an entry


def tensors(**kw):
    a = dict(k=torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16), block_table=torch.zeros(3, 5, dtype=torch.int32),
             lengths=torch.zeros(3, dtype=torch.int32), mass=torch.zeros(6, 2, 16), pos=torch.zeros(6, 2, 16, dtype=torch.int32))
    a.update(kw)
    a.setdefault("v", torch.zeros_like(a["k"]))
    return a


def test_make_kv_describes_the_tensors_and_holds_them():
    import gc
    import weakref
    t = tensors()
    kv = ft.make_kv(8, **t)
    assert (kv.head_dim, kv.n_heads, kv.n_kv_heads, kv.page_size, kv.n_seqs, kv.max_pages, kv.n_pages, kv.format) == \
        (64, 8, 2, 16, 3, 5, 6, ft.FT_KV_BF16)
    assert kv.k == t["k"].data_ptr() and kv.pos == t["pos"].data_ptr() and not kv.status
    ref = weakref.ref(t["k"])
    del t
    gc.collect()
    assert ref() is not None
    del kv
    gc.collect()
    assert ref() is None
    f = ft.make_kv(8, **tensors(k=torch.zeros(6, 2, 16, 64).to(torch.float8_e4m3fn)), k_scale=0.5)
    assert f.format == ft.FT_KV_E4M3 and f.k_scale == 0.5 and f.v_scale == 1.0


@pytest.mark.parametrize("kw,what", [
    (dict(k=torch.zeros(6, 2, 16, 64)), "dtype"), (dict(k=torch.zeros(6, 2, 16, 64, dtype=torch.float16)), "dtype"),
    (dict(k=torch.zeros(6, 2, 1024, dtype=torch.bfloat16)), "two pools"),
    (dict(v=torch.zeros(6, 2, 16, 128, dtype=torch.bfloat16)), "two pools"),
    (dict(v=torch.zeros(6, 2, 16, 64).to(torch.float8_e4m3fn)), "two pools"), (dict(mass=torch.zeros(6, 2, 8)), "mass"),
    (dict(mass=torch.zeros(6, 2, 16, dtype=torch.float64)), "mass"), (dict(pos=torch.zeros(6, 2, 16)), "pos"),
    (dict(block_table=torch.zeros(15, dtype=torch.int32)), "block_table"), (dict(block_table=torch.zeros(3, 5)), "block_table"),
    (dict(lengths=torch.zeros(4, dtype=torch.int32)), "lengths"), (dict(lengths=torch.zeros(3, dtype=torch.int64)), "lengths"),
    (dict(status=torch.zeros(2, dtype=torch.int32)), "status"),
    (dict(k=torch.zeros(6, 2, 64, 16, dtype=torch.bfloat16).transpose(2, 3)), "contiguous"),
    (dict(block_table=torch.zeros(5, 3, dtype=torch.int32).t()), "contiguous")])
def test_make_kv_refuses(kw, what):
    with pytest.raises(ValueError, match=what):
        ft.make_kv(8, **tensors(**kw))


def test_binding_refuses_rows_of_another_shape():
    kv = ft.make_kv(8, **tensors())
    new = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    q, pos = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 3, dtype=torch.int32)
    inv, axis, work = torch.zeros(32, dtype=torch.float64), torch.zeros(32, dtype=torch.int32), torch.zeros(8, dtype=torch.uint8)

    def append(q=q, k=new, v=new, cu=None, pos=pos, inv=inv, axis=axis, q_out=q):
        ft.ft_kv_append(kv, q, k, v, cu, pos, inv, axis, q_out, 0, 0)

    for kw in (dict(k=new[:, :1]), dict(k=new[:, :, :32]), dict(v=new[:2]), dict(q=q[:2]), dict(q_out=q[:2]), dict(k=new.float()),
               dict(k=torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), dict(pos=pos[:, :2]), dict(pos=pos[0]),
               dict(cu=torch.zeros(3, dtype=torch.int32)), dict(axis=axis[:31]), dict(axis=None), dict(inv=inv.float()),
               dict(axis=axis.long()), dict(q_out=q.float())):
        with pytest.raises(ValueError):
            append(**kw)
    for args in ((q[:2], q[:2]), (q, q[:2]), (q[:, :4], q[:, :4]), (q.float(), q)):
        with pytest.raises(ValueError):
            ft.ft_kv_attention(kv, args[0], 0.1, args[1], None, work, 0, 0)
    with pytest.raises(ValueError):
        ft.ft_kv_attention(kv, q, 0.1, torch.zeros_like(q), torch.zeros(3, 7), work, 0, 0)
    with pytest.raises(ValueError):
        ft.ft_kv_evict(kv, torch.zeros(4, dtype=torch.int32), 0, work, 0)
