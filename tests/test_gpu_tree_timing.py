"""The per-launch timing of a context whose calls are also captured into graphs."""
import pytest

from test_gpu_tree_context import R, Twin

pytestmark = pytest.mark.gpu


def test_captured_calls_are_counted_and_not_timed():
    import torch
    a = Twin("bf16", 8, 2, 128, stage=False)
    try:
        gen = torch.Generator().manual_seed(60)
        q, k, v = (torch.randn(R, 3, h, 128, generator=gen).to(torch.bfloat16).cuda() for h in (8, 2, 2))
        mask, outs = torch.full((R, 3), 7, dtype=torch.int64, device="cuda"), [torch.zeros_like(q) for _ in range(2)]
        a.ctx.set_timing(True)
        a.ctx.attend_tree(0, q, k, v, mask, outs[0])
        torch.cuda.synchronize()
        plain = a.ctx.read_timing()
        assert plain["launches"]["attend"] == 1 and plain["ms"]["attend"] > 0
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.ctx.attend_tree(0, q, k, v, mask, outs[1])
        g.replay()
        torch.cuda.synchronize()
        t = a.ctx.read_timing()
        assert t["launches"]["attend"] == 2 and t["ms"]["attend"] == plain["ms"]["attend"]
        assert torch.equal(*outs)
        a.ctx.attend_tree(0, q, k, v, mask, outs[1])
        torch.cuda.synchronize()
        t = a.ctx.read_timing()
        assert t["launches"]["attend"] == 3 and t["ms"]["attend"] > plain["ms"]["attend"]
    finally:
        a.close()
