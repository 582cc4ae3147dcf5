"""The bounded wait of the cache attention for its copies: one that runs out, one that does not, and arrivals around
the limit, where all lanes of a warp have to go the same way (they meet in votes and products afterwards)."""
import pytest
import torch

import expert_offloaded_serving_b200 as ft

pytestmark = pytest.mark.gpu


def wait(blocks, limit_us, arrive_us):
    lanes = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
    ft.ft_debug_kv_wait(lanes, limit_us, arrive_us)
    return lanes


def test_a_wait_that_nothing_ends_runs_out_for_every_lane():
    assert (wait(40, 2000, -1) == 0).all()
    torch.cuda.synchronize()
    assert (wait(40, 500000, 50) == 32).all()  # and the next one ends as it should


@pytest.mark.parametrize("arrive_us", [0, 200, 990, 998, 1000, 1002, 1004, 1010, 1030, 1060, 1100, 1500])
def test_lanes_go_the_same_way_around_the_limit(arrive_us):
    for _ in range(4):
        lanes = wait(1024, 1000, arrive_us)
        assert ((lanes == 0) | (lanes == 32)).all(), lanes.unique().tolist()
