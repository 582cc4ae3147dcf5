"""More argument checks of the key-value cache calls at the edges of what they take, without a GPU."""
import ctypes as C

import pytest

import expert_offloaded_serving_b200 as ft
from test_kv_host import OUT, append, attend, cache, evict, refused


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
