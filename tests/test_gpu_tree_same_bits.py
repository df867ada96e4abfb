"""The drafted-tree attention gives the same bits whatever ran on the GPU before."""
import pytest

from test_gpu_tree import call, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,T,Hq,H,d,kb,dtype", [(40, 3, 8, 8, 64, 6, "bf16"), (1, 1, 8, 8, 128, 128, "bf16"), (20, 5, 8, 1, 128, 24, "bf16"),
                                                (3, 43, 18, 3, 128, 19, "bf16"), (2, 7, 4, 2, 256, 30, "bf16"), (9, 11, 6, 2, 96, 40, "bf16"),
                                                (5, 3, 6, 2, 64, 20, "f32"), (2, 5, 8, 2, 128, 60, "f32")])
def test_what_shared_memory_held_before_has_no_part(R, T, Hq, H, d, kb, dtype):
    """Behind calls whose queries, keys and values are large, small, and of other shapes and types; the tiles of a
    group's rows are not full, and what lies behind them is what the last kernel left."""
    import torch
    x = make(R, T, Hq, H, d, 16, kb, dtype, seed=80)
    want = call(x)
    for i, (s, size) in enumerate([((40, 16, 32, 8, 128, 16, 16, "bf16"), 30.0), ((30, 64, 16, 2, 128, 16, 20, "bf16"), 1e4),
                                   ((20, 32, 16, 4, 256, 16, 12, "bf16"), 0.0), ((40, 8, 16, 4, 64, 16, 8, "f32"), 1e3),
                                   ((40, 64, 16, 8, 64, 16, 16, "bf16"), 3e2)]):
        y = make(*s, seed=81 + i, stale=0.0)
        y["q"] *= size
        y["pool"] *= 10
        for _ in range(3):
            call(y)
            assert torch.equal(call(x), want), s
