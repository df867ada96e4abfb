"""Calls without a context from several host threads at once."""
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_gpu_tree import call, make

pytestmark = pytest.mark.gpu


def test_every_call_of_every_thread_gives_its_result():
    """Of different shapes, types and streams; a refusal or an error in a thread fails the test."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    shapes = [(1, 8, 32, 8, 128, 16, 40, "bf16"), (2, 64, 16, 2, 128, 16, 20, "bf16"), (3, 5, 8, 2, 64, 32, 9, "f32"),
              (2, 9, 4, 2, 256, 16, 30, "bf16"), (2, 20, 8, 2, 96, 16, 12, "f32"), (40, 3, 8, 8, 64, 16, 6, "bf16")]
    xs = [make(*s[:-1], s[-1], seed=70 + i) for i, s in enumerate(shapes)]
    want = [call(x) for x in xs]
    rows = torch.randn(50, 12 * 64, device="cuda")
    pos, rot = torch.arange(50, dtype=torch.int32, device="cuda"), Rotary(torch.rand(32, device="cuda"))
    row_want = torch.empty(50, 8, 64, device="cuda")
    norm_rope(rows, pos, row_want, q_heads=8, kv_heads=2, head_dim=64, rotary=rot)
    torch.cuda.synchronize()

    def work(i):
        st, same = torch.cuda.Stream(), 0
        with torch.cuda.stream(st):
            for _ in range(25):
                got, row = call(xs[i]), torch.empty_like(row_want)
                norm_rope(rows, pos, row, q_heads=8, kv_heads=2, head_dim=64, rotary=rot)
                st.synchronize()
                same += torch.equal(got, want[i]) and torch.equal(row, row_want)
        return same

    with ThreadPoolExecutor(len(xs)) as ex:
        assert list(ex.map(work, range(len(xs)))) == [25] * len(xs)
