"""The ends of the ranges that the drafted-tree attention takes."""
import pytest

from test_gpu_tree import call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs", [16, 12, 1, 64])
def test_the_last_block_of_the_longest_request(dtype, bs):
    """A request of 2^31 - 1 tokens: its last block, part-filled where bs does not divide that, holds valid tokens; the
    block behind it does not."""
    import torch
    n = 2 ** 31 - 1
    x = make(2, 5, 8, 2, 64, bs, 6, dtype, seed=41, lengths=[5 * bs, 4 * bs])
    last = (n - 1) // bs
    x["slot_block"][0, :, 1], x["slot_block"][0, :, 2] = last, min(last + 1, n)
    x["pool"][0, :, 1] = torch.randn(2, 2, bs, 64, generator=torch.Generator().manual_seed(bs)).to(x["pool"])
    x["pool"][0, :, 1, :, n - last * bs:] = float("nan")
    x["pool"][0, :, 2] = float("nan")
    x["lengths"][0] = n
    check(x, call(x))
    y = dict(x, slot_block=x["slot_block"].clone())
    y["slot_block"][0, :, 1] = -1
    assert not torch.equal(call(x)[0], call(y)[0])
