"""More argument checks of the key-value cache calls at the edges of what they take, without a GPU."""
import pytest

import expert_offloaded_serving_b200 as ft
from test_kv_host import OUT, refused


@pytest.mark.parametrize("args,what", [((0, 10, 10, OUT), "blocks"), ((1025, 10, 10, OUT), "blocks"), ((4, 0, 10, OUT), "limit_us"),
                                       ((4, 1000001, 10, OUT), "limit_us"), ((4, 10, 1000001, OUT), "arrive_us"),
                                       ((4, 10, 10, None), "lanes"), ((4, 10, 10, OUT + 2), "lanes")])
def test_the_wait_hook_refuses(args, what):
    refused(ft.lib().ft_debug_kv_wait(*args, None), what)
