"""More argument checks of the key-value cache calls at the edges of what they take, without a GPU."""
import ctypes as C

import pytest
import torch

import expert_offloaded_serving_b200 as ft
from test_kv_host import OUT, append, attend, cache, evict, refused, tensors


@pytest.mark.parametrize("args,what", [((0, 10, 10, OUT), "blocks"), ((1025, 10, 10, OUT), "blocks"), ((4, 0, 10, OUT), "limit_us"),
                                       ((4, 1000001, 10, OUT), "limit_us"), ((4, 10, 1000001, OUT), "arrive_us"),
                                       ((4, 10, 10, None), "lanes"), ((4, 10, 10, OUT + 2), "lanes")])
def test_the_wait_hook_refuses(args, what):
    refused(ft.lib().ft_debug_kv_wait(*args, None), what)


@pytest.mark.parametrize("shape", [
    dict(head_dim=256, n_heads=1024, n_kv_heads=1), dict(head_dim=64, n_heads=1024, n_kv_heads=1),
    dict(head_dim=64, n_heads=1000, n_kv_heads=2, format=ft.FT_KV_E4M3), dict(head_dim=128, n_heads=32, n_kv_heads=8),
    dict(head_dim=96, n_heads=33, n_kv_heads=3, format=ft.FT_KV_E4M3)])
@pytest.mark.parametrize("sms", [16, 108, 148, 160, 200])
def test_the_split_covers_every_tile(shape, sms):
    """All tiles lie on the chunks there are, up to the 2^30 the shapes allow; none is larger than an equal share
    needs, but for the 4 tiles that a short row's chunks may have."""
    kv = cache(n_seqs=1, **shape)
    for tiles in [*range(0, 700, 13), 4735, 4736, 4737, 99999, (1 << 24) + 1, 268485103, 268485104, 536970461, (1 << 30) - 1,
                  *range(1 << 28, 1 << 30, 9999991)]:
        tile, chunk, used, there = ft.ft_kv_geometry(kv, tiles, sms)
        assert tile in (16, 32) and chunk >= 1 and used <= there
        assert used * chunk >= tiles > (used - 1) * chunk or tiles == used == 0
        assert chunk <= max(4, -(-tiles // there))


@pytest.mark.parametrize("tiles,sms,what", [(-1, 148, "tiles"), (1 << 30, 148, "tiles"), (5, 15, "sms"), (5, 1025, "sms")])
def test_the_split_refuses(tiles, sms, what):
    refused(ft.lib().ft_kv_geometry(C.byref(cache()), tiles, sms, (ft.I64 * 4)()), what)
    refused(ft.lib().ft_kv_geometry(C.byref(cache()), 5, 148, None), "NULL")
    refused(ft.lib().ft_kv_geometry(C.byref(cache(n_seqs=0)), 5, 148, (ft.I64 * 4)()), "n_seqs")
    refused(ft.lib().ft_kv_geometry(C.byref(cache(head_dim=7)), 5, 148, (ft.I64 * 4)()), "head_dim")


def test_positions_without_an_axis_are_refused():
    """Nothing turns and nothing is stored, so no axis is needed; but positions of none of them hold no token's."""
    refused(append(cache(pos=None), rot=0, inv=None, axis=None, axes=0), "n_axes")
    assert append(cache(pos=None), T=0, cu=OUT, rot=0, inv=None, axis=None, axes=0, pos=None) == ft.FT_OK


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_a_scale_without_a_finite_reciprocal_is_refused(which):
    """What is stored is the value times 1 / scale: infinity would make NaN of a zero."""
    for scale in (2.0 ** -149, 2.0 ** -129, 2.0 ** -128):  # 2^128 is past fp32
        for call in (append, attend, evict):
            refused(call(cache(format=ft.FT_KV_E4M3, **{which: scale})), "reciprocal")
    for scale in (2.0 ** -127, 2.0 ** 127):
        assert append(cache(format=ft.FT_KV_E4M3, **{which: scale}), T=0, cu=OUT) == ft.FT_OK


def test_a_scale_that_leaves_fp32_is_refused():
    """Scores are taken in units of log2(e) and of k_scale: scale times both has to be finite, or a score of 0 is NaN."""
    refused(attend(scale=3e38), "scale")
    refused(attend(cache(format=ft.FT_KV_E4M3, k_scale=2.0 ** 100), scale=-2.0 ** 28), "scale")
    refused(attend(scale=2e38, work=None), "workspace")  # 2.9e38 fits, the next check speaks


def test_binding_refuses_other_types_of_the_same_size():
    """fp16 bits read as bf16, or float32 ones as int32, would give wrong numbers without a word."""
    kv = ft.make_kv(8, **tensors())
    bf, half, i32, f32 = torch.bfloat16, torch.float16, torch.int32, torch.float32
    work = torch.zeros(8, dtype=torch.uint8)

    def rows(heads, dtype):
        return torch.zeros(3, heads, 64, dtype=dtype)

    def append(q=bf, k=bf, v=bf, cu=i32, pos=i32, inv=torch.float64, axis=i32, q_out=bf):
        ft.ft_kv_append(kv, rows(8, q), rows(2, k), rows(2, v), torch.zeros(4, dtype=cu), torch.zeros(1, 3, dtype=pos),
                        torch.zeros(32, dtype=inv), torch.zeros(32, dtype=axis), rows(8, q_out), 0, 0)

    for kw in (dict(q=half), dict(k=half), dict(v=torch.int16), dict(q_out=half), dict(cu=f32), dict(pos=f32),
               dict(inv=torch.int64), dict(axis=f32)):
        with pytest.raises(ValueError, match=str(*kw.values())):
            append(**kw)
    for q, out, lse in ((half, bf, f32), (bf, half, f32), (bf, bf, i32)):
        with pytest.raises(ValueError, match="float16" if half in (q, out) else "int32"):
            ft.ft_kv_attention(kv, rows(8, q), 0.1, rows(8, out), torch.zeros(3, 8, dtype=lse), work, 0, 0)
    with pytest.raises(ValueError, match="float32"):
        ft.ft_kv_evict(kv, torch.zeros(3), 0, work, 0)
    with pytest.raises(ValueError, match="float32"):
        ft.ft_debug_kv_wait(torch.zeros(3), 10, 10, 0)
    with pytest.raises(ft.FtError, match="workspace"):  # the right types pass to the library's own checks
        ft.ft_kv_attention(kv, rows(8, bf), 0.1, rows(8, bf), torch.zeros(3, 8), work, 0, 0)
