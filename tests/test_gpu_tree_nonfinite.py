"""NaN and infinite queries, keys and values of the drafted-tree attention: the result is the definition's however a
launch splits its items."""
import pytest

import tree_ref
from test_gpu_tree import call, check, make

pytestmark = pytest.mark.gpu

# one request over a long table is split over a cluster; a table of one tile never is
SPLIT, WHOLE = 128, 4
KINDS = [("bf16", 8, 128), ("bf16", 64, 128), ("bf16", 6, 256), ("f32", 8, 64), ("f32", 2, 128)]


@pytest.mark.parametrize("kb", [SPLIT, WHOLE])
@pytest.mark.parametrize("dtype,T,d", KINDS)
def test_nan_query_rows_are_nan(dtype, T, d, kb):
    """... and no other row is."""
    x = make(1, T, 8, 2, d, 16, kb, dtype, seed=31, lengths=[kb * 16 - 5])
    x["q"][0, 1, 2] = float("nan")
    x["q"][0, T - 1, 7, 3] = float("nan")
    out = call(x)
    assert bool(out[0, 1, 2].isnan().all()) and bool(out[0, T - 1, 7].isnan().all())
    check(x, out)


@pytest.mark.parametrize("dtype,T,d", KINDS)
def test_a_nan_key_alone_in_its_tile(dtype, T, d):
    """Every row of its KV head is NaN: the CTA that has this tile finds no maximum there, and is still heard."""
    x = make(1, T, 8, 2, d, 16, SPLIT, dtype, seed=32, lengths=[129])
    at = int((x["slot_block"][0, 1] == 8).nonzero()[0])  # the last block, of one token, goes to the last slot
    x["slot_block"][0, 1, at], x["slot_block"][0, 1, -1] = -1, 8
    x["pool"][0, 1, -1] = x["pool"][0, 1, at]
    x["pool"][0, 1, -1, 0, 0] = float("nan")
    out = call(x)
    assert bool(out[0, :, 4:].isnan().all())
    check(x, out)


@pytest.mark.parametrize("kb", [SPLIT, WHOLE])
@pytest.mark.parametrize("dtype,T,d", KINDS)
def test_rows_whose_scores_are_all_minus_infinity_are_zero(dtype, T, d, kb):
    """No token has a weight, as where a row sees none; infinite values are not reached then."""
    import torch
    x = make(1, T, 8, 2, d, 16, kb, dtype, seed=33, lengths=[kb * 16 - 5])
    x["q"][:] = x["q"].abs()
    x["pool"][0, 0, :, 0, :, 5] = float("-inf")
    x["pool"][0, 0, 0, 1, 2, 7] = float("inf")
    x["k"][0, :, 0, 5] = float("-inf")
    out = call(x)
    assert torch.equal(out[0, :, :4], torch.zeros_like(out[0, :, :4]))
    y = {n: t[:, 1:] if n in ("pool", "slot_block") else t[:, :, 4:] if n == "q" else t[:, :, 1:] if n in "kv" else t for n, t in x.items()}
    check(y, out[:, :, 4:].contiguous())


@pytest.mark.parametrize("kb", [SPLIT, WHOLE])
@pytest.mark.parametrize("dtype,T,d", KINDS)
def test_infinite_values_of_resident_tokens(dtype, T, d, kb):
    """Infinite in their own dimension for every row of their KV head, of their sign; NaN where both signs meet."""
    x = make(1, T, 8, 2, d, 16, kb, dtype, seed=34, lengths=[kb * 16 - 5])
    v = x["pool"][0, :, :, 1]
    v[0, 1, 3, 4], v[0, 2, 9, 6], v[1, 0, 0, d - 1] = float("inf"), float("-inf"), float("inf")
    v[1, 1, 5, 9], v[1, kb - 2, 1, 9] = float("inf"), float("-inf")
    out = call(x)
    assert bool((out[0, :, :4, 4] == float("inf")).all()) and bool((out[0, :, :4, 6] == float("-inf")).all())
    assert bool((out[0, :, 4:, d - 1] == float("inf")).all()) and bool(out[0, :, 4:, 9].isnan().all())
    check(x, out)


@pytest.mark.parametrize("kb", [SPLIT, WHOLE])
@pytest.mark.parametrize("dtype,T,d", KINDS)
def test_infinite_keys(dtype, T, d, kb):
    """A key with an infinite element has an infinite score, of the sign of the row's query there: rows where it is
    negative are those without the token, the others NaN. One resident token (alone in its block), one drafted."""
    import torch
    x = make(1, T, 8, 2, d, 16, kb, dtype, seed=35, lengths=[(kb - 1) * 16 + 1])
    last = (x["slot_block"][0, 0] == kb - 1).nonzero()[0]
    x["pool"][0, 0, int(last), 0, 0, 3] = float("inf")   # resident, of KV head 0
    x["k"][0, T - 1, 1, 5] = float("-inf")               # drafted, of KV head 1
    x["mask"][0, :] |= torch.tensor([-(1 << 63) if T == 64 else 1 << (T - 1)], device="cuda")
    out = call(x)
    lost = torch.cat((x["q"][0, :, :4, 3] > 0, x["q"][0, :, 4:, 5] < 0), 1)  # [T][Hq]: a score of +infinity
    y = dict(x, slot_block=x["slot_block"].clone(), mask=x["mask"] & ~torch.tensor([-(1 << 63) if T == 64 else 1 << (T - 1)], device="cuda"))
    y["slot_block"][0, 0, int(last)] = -1
    # KV head 0 sees the last drafted token still, head 1 the last block
    z0, z1 = dict(x, slot_block=y["slot_block"]), dict(x, mask=y["mask"])
    z0["k"], z1["k"] = x["k"].clone(), x["k"].clone()
    z0["k"][0, T - 1, 1] = z1["k"][0, T - 1, 1] = 0
    z1["pool"] = x["pool"].clone()
    z1["pool"][0, 0, int(last), 0, 0] = 0
    (w0, b0), (w1, b1) = tree_ref.attend(**z0), tree_ref.attend(**z1)
    want, bound = torch.cat((w0[0, :, :4], w1[0, :, 4:]), 1), torch.cat((b0[0, :, :4], b1[0, :, 4:]), 1)
    got = out[0].double()
    assert bool(got[lost].isnan().all()) and bool(lost.any()) and bool((~lost).any())
    assert float(((got - want).abs() - bound)[~lost].max()) <= 0


@pytest.mark.parametrize("kb", [SPLIT, WHOLE])
@pytest.mark.parametrize("T,d", [(8, 64), (2, 128), (20, 96)])
def test_binary32_up_to_its_largest_numbers(T, d, kb):
    """Finite keys, queries and values whose upper parts would round past the largest number: a resident and a drafted
    value (which some rows do not see), a key against a small query and a query against a small key."""
    import torch
    top = torch.finfo(torch.float32).max
    x = make(1, T, 8, 2, d, 16, kb, "f32", seed=36, lengths=[kb * 16 - 5])
    x["pool"][0, 0, 1, 1, 3, 4] = top
    x["v"][0, T - 1, 1, 6] = -top
    x["q"][..., 8:10] = 0
    x["q"][0, :, :, 8], x["q"][0, 0, :, 9] = 2e-38, top
    x["pool"][0, :, 2, 0, 5, 8] = -top
    x["pool"][0, :, :, 0, :, 9] = 0
    x["k"][0, :, :, 9] = 0
    x["pool"][0, 1, 3, 0, 7, 9] = 2e-38
    check(x, call(x))
