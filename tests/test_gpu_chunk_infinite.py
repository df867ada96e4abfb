"""Scores of infinity (okv_attend_chunk_static): the log sum of a row is infinite with its largest score, the weight of that score's
token is not a number, and every other token's is zero."""
import math

import pytest

from test_gpu_chunk import call, make
from tree_ref import U32, half_step

pytestmark = pytest.mark.gpu


def plain(x):
    """((out, lse, weight_out), bounds) in binary64, from the formulas alone: weights exp(score - lse). The bounds are chunk_ref's, with the
    largest of a unit's rows for each of them."""
    import torch
    q, pool, window, sinks = x["q"], x["pool"], x["window"], x["sinks"]
    R, T, Hq, d = q.shape
    H, kb, bs = pool.shape[1], pool.shape[2], pool.shape[4]
    g, bf16 = Hq // H, q.dtype == torch.bfloat16
    unit, rounded = (2.0 ** -23, half_step(q.dtype)) if bf16 else (U32, 0.0)
    out, lse = (torch.zeros(R, T, Hq, *s, dtype=torch.float64, device="cuda") for s in ((d,), ()))
    drawn = x["weight"].double().clone()
    out_b, lse_b, drawn_b = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(drawn)
    for r in range(R):
        p = x["lengths"][r].long() + torch.arange(T, device="cuda")[:, None]
        for h in range(H):
            b = x["slot_block"][r, h].long()[:, None]
            pos = b * bs + torch.arange(bs, device="cuda")
            keep = ((b >= 0) & (pos <= p[-1])).reshape(-1).nonzero()[:, 0]
            pos = pos.reshape(-1)[keep]
            sees = pos <= p
            if window:
                sees &= (p - pos < window) | (pos < sinks)
            k, v = (pool[r, h, :, i].reshape(-1, d)[keep].double() for i in (0, 1))
            total, total_b = (torch.zeros(kb * bs, dtype=torch.float64, device="cuda") for _ in range(2))
            for j in range(h * g, h * g + g):
                qi = q[r, :, j].double()
                z = (qi @ k.T / math.sqrt(d)).masked_fill(~sees, -math.inf)
                s = torch.logsumexp(z, -1, keepdim=True)
                none = s == -math.inf  # nothing seen, or nothing but scores of -infinity
                w = torch.where(sees & ~none, torch.exp(z - s), 0.0)
                out[r, :, j], lse[r, :, j] = w @ v, s[:, 0]
                size = (qi.abs() @ k.abs().nan_to_num(0.0, 0.0).T / math.sqrt(d)).max()
                err, big = float((d + 8) * unit * size), float(s[s.isfinite()].abs().max() + size) if s.isfinite().any() else 0.0
                out_b[r, :, j] = (math.expm1(2 * err) + 2.0 ** -21 + 2 * (len(keep) + 16) * unit + rounded) * (w.nan_to_num(0.0) @ v.abs()) * 1.01 + half_step(q.dtype) * out[r, :, j].abs()
                lse_b[r, :, j] = err + 2.0 ** -21 + (len(keep) + 16) * unit + 6 * U32 * big
                total.index_add_(0, keep, w.sum(0))
                total_b.index_add_(0, keep, w.nan_to_num(0.0).sum(0) * math.expm1(2 * err + 2.0 ** -20 + (len(keep) + 16) * unit + 10 * U32 * big))
            drawn[r, h] += total.view(kb, bs).sum(-1)
            drawn_b[r, h] = total_b.view(kb, bs).sum(-1) + (128 + T * g / 32 + bs + 8) * U32 * total.view(kb, bs).sum(-1) + U32 * drawn[r, h].abs()
    return (out, lse, drawn), (out_b, lse_b, drawn_b)


def check(x):
    import torch
    want, bound = plain(x)
    for name, g, w, b in zip(("out", "lse", "weight"), call(x), want, bound):
        g = g.double()
        assert torch.equal(torch.isnan(g), torch.isnan(w)), name
        assert torch.equal(g[torch.isinf(w)], w[torch.isinf(w)]), name
        finite = torch.isfinite(w)
        over = ((g - w).abs() - b)[finite]
        assert over.numel() == 0 or float(over.max()) <= 0, f"{name}: worst excess {float(over.max()):.3g}"
    return want


CASES = [("bf16", 128, 16, 12, 3), ("bf16", 128, 16, 120, 3), ("bf16", 128, 12, 20, 3), ("bf16", 64, 16, 12, 30), ("bf16", 128, 16, 40, 90), ("bf16", 96, 16, 40, 50),
         ("bf16", 256, 16, 30, 40), ("f32", 64, 16, 12, 20), ("f32", 128, 16, 40, 3), ("f32", 64, 16, 40, 70)]


@pytest.mark.parametrize("dtype,d,bs,kb,T", CASES)
@pytest.mark.parametrize("where", ["first", "middle", "last", "new"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 4)])
def test_an_infinite_score(dtype, d, bs, kb, T, where, window, sinks):
    """An infinite key: heads whose query has one sign there see +infinity, the others -infinity. In one unit of four."""
    import torch
    n = kb * bs - T
    x = make(2, T, 8, 2, d, bs, kb, dtype, seed=91, lengths=[n, n], holes=False)
    x.update(window=window, sinks=sinks)
    at = {"first": 1, "middle": n // 2, "last": n - 1, "new": n + T // 2}[where]
    x["pool"][0, 0, at // bs, 0, at % bs, 7] = math.inf
    q = x["q"][0, :, :, 7]
    q.copy_((q.abs() + 0.5) * torch.tensor([1, -1, 1, 1, 1, -1, 1, -1], device="cuda"))
    want = check(x)
    seen = not window or at < sinks or n + T - 1 - at < window  # by the last token
    assert bool((want[1][0, -1, [0, 2, 3]] == math.inf).all()) == seen and bool(torch.isfinite(want[1][0, -1, 1]))


@pytest.mark.parametrize("dtype,d,bs,kb,T", CASES)
def test_more_than_one_infinite_score(dtype, d, bs, kb, T):
    """+infinity from several tokens of several slots, and scores that are not a number beside them in another unit."""
    import torch
    n = kb * bs - T
    x = make(2, T, 8, 2, d, bs, kb, dtype, seed=92, lengths=[n, n], holes=False)
    for at in (0, 5, n // 2, n - 1, n + 1):
        x["pool"][0, 0, at // bs, 0, at % bs, 3] = math.inf
        x["pool"][1, 1, at // bs, 0, at % bs, 3] = math.inf
    x["pool"][1, 1, (n + 1) // bs, 0, (n + 1) % bs, 9] = math.nan
    q = x["q"][..., 3]
    q.copy_(q.abs() + 0.5)
    want = check(x)
    assert bool((want[1][0, :, :4] == math.inf).all()) and bool(torch.isnan(want[1][1, 1:, 4:]).all()) and bool(torch.isfinite(want[1][:, :, 4:][0]).all())


@pytest.mark.parametrize("dtype,d,bs,kb,T", CASES)
def test_scores_past_the_largest_number(dtype, d, bs, kb, T):
    """Finite operands whose product is past binary32 are a score of infinity, in every form of the call."""
    import torch
    n = kb * bs - T
    x = make(1, T, 4, 1, d, bs, kb, dtype, seed=93, lengths=[n], holes=False)
    at = n // 3
    x["pool"][0, 0, at // bs, 0, at % bs] = 0.0
    x["pool"][0, 0, at // bs, 0, at % bs, 2] = 2.0 ** 127
    x["q"][0, :, 1] = 0.0
    x["q"][0, :, 1, 2] = 16.0
    out, lse, drawn = call(x)
    assert bool((lse[0, :, 1] == math.inf).all()) and bool(torch.isnan(out[0, :, 1]).all())
    assert bool(torch.isnan(drawn[0, 0, at // bs])) and int(torch.isnan(drawn).sum()) == 1
