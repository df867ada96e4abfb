"""Attention of chunks of new tokens over a paged pool (okv_attend_chunk_static) against the plain binary64 form."""
import pytest

import chunk_ref

pytestmark = pytest.mark.gpu


def make(R, T, Hq, H, d, bs, kb, dtype, seed=0, lengths=None, counts=None, holes=True, stale=float("nan"), drawn=True):
    """Inputs with `stale` in every place of the pool that holds no token up to the last new one."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    dev = "cuda"
    if lengths is None:
        lengths = [int(x) for x in torch.randint(0, 2 * kb * bs, (R,), generator=gen)]
    cnt = [T] * R if counts is None else [min(max(c, 0), T) for c in counts]
    slot_block = torch.full((R, H, kb), -1, dtype=torch.int32)
    for r in range(R):
        nb = -(-(lengths[r] + cnt[r]) // bs)
        for h in range(H):
            n = min(kb, nb)
            if holes and n > 1:
                n -= int(torch.randint(0, n // 2 + 1, (1,), generator=gen))
            ids = torch.randperm(nb, generator=gen)[:n]
            last = min(n, nb - lengths[r] // bs)  # most new blocks are there
            if n:
                old = ids[ids < nb - last][:n - last]
                ids = torch.cat((old, torch.arange(nb - last, nb)))
                ids = ids[torch.randperm(len(ids), generator=gen)] if holes else ids.sort().values
            place = torch.randperm(kb, generator=gen)[:len(ids)] if holes else torch.arange(len(ids))
            slot_block[r, h, place] = ids.to(torch.int32)
    pool = torch.randn(R, H, kb, 2, bs, d, generator=gen).to(dt)
    pos = slot_block[..., None] * bs + torch.arange(bs)
    dead = (slot_block[..., None] < 0) | (pos >= (torch.tensor(lengths) + torch.tensor(cnt))[:, None, None, None])
    pool.permute(0, 1, 2, 4, 3, 5)[dead] = stale
    return dict(pool=pool.to(dev), slot_block=slot_block.to(dev), lengths=torch.tensor(lengths, dtype=torch.int32, device=dev),
                counts=None if counts is None else torch.tensor(counts, dtype=torch.int32, device=dev),
                q=(2 * torch.randn(R, T, Hq, d, generator=gen)).to(dt).to(dev), window=0, sinks=0,
                weight=torch.rand(R, H, kb, generator=gen).to(dev) if drawn else None)


def call(x, stream=None, weigh=True):
    """(out, lse, weight_out), rows that are not written at -7."""
    import torch
    from sparse_kv_cache_draft_gb300 import attend_chunk_static
    R, H, kb, _, bs, d = x["pool"].shape
    out = torch.full_like(x["q"], -7.0)
    lse = torch.full(x["q"].shape[:3], -7.0, device="cuda")
    drawn = torch.full((R, H, kb), -7.0, device="cuda") if weigh else None
    attend_chunk_static(x["pool"], x["slot_block"], x["lengths"], x["counts"], x["q"], out, lse, x["weight"] if weigh else None, drawn,
                        q_heads=x["q"].shape[2], kv_heads=H, head_dim=d, block_size=bs, slots=kb, window=x["window"], sinks=x["sinks"],
                        stream=stream)
    return out, lse, drawn


def check(x, got):
    import torch
    want, bound = chunk_ref.attend(**x)
    T = x["q"].shape[1]
    cnt = torch.tensor(chunk_ref.new_tokens(x["lengths"], x["counts"], T)[1], device="cuda")
    fresh = torch.arange(T, device="cuda") < cnt[:, None]
    for name, g, w, b in zip(("out", "lse", "weight"), got, want, bound):
        if g is None:
            continue
        g = g.double()
        if name != "weight":
            assert torch.equal(g[~fresh], torch.full_like(g[~fresh], -7.0)), f"{name}: rows past a request's count were written"
            g, w, b = g[fresh], w[fresh], b[fresh]
        finite = torch.isfinite(w)
        assert torch.equal(torch.isnan(g), torch.isnan(w)), name
        assert torch.equal(g[~finite & ~torch.isnan(w)], w[~finite & ~torch.isnan(w)]), name
        over = ((g - w).abs() - b)[finite]
        assert over.numel() == 0 or float(over.max()) <= 0, f"{name}: worst excess {float(over.max()):.3g}"


SHAPES = [  # R, T, Hq, Hkv, d, bs, kb, dtype
    (1, 1, 1, 1, 128, 16, 1, "bf16"),
    (1, 1, 32, 8, 128, 16, 128, "bf16"),
    (3, 5, 8, 2, 128, 16, 37, "bf16"),
    (2, 32, 8, 2, 128, 16, 33, "bf16"),         # 128 rows to a key head
    (2, 33, 8, 2, 128, 16, 20, "bf16"),         # 132
    (1, 300, 32, 8, 128, 16, 40, "bf16"),
    (2, 130, 8, 1, 128, 64, 9, "bf16"),         # 1040 rows
    (2, 77, 18, 3, 128, 16, 19, "bf16"),        # 6 heads: 126 rows to a warpgroup
    (2, 61, 24, 8, 64, 32, 33, "bf16"),
    (3, 9, 6, 2, 64, 16, 40, "bf16"),
    (2, 150, 8, 1, 64, 8, 65, "bf16"),
    (2, 70, 4, 2, 128, 1, 200, "bf16"),         # a token per block
    (2, 7, 4, 2, 128, 12, 21, "bf16"),          # blocks that do not divide a tile
    (2, 90, 8, 2, 128, 24, 21, "bf16"),
    (2, 60, 4, 4, 128, 33, 11, "bf16"),
    (2, 21, 10, 2, 96, 16, 19, "bf16"),
    (2, 100, 5, 1, 96, 7, 50, "bf16"),          # lines of 64 bytes and an odd block size
    (2, 9, 4, 2, 32, 16, 19, "bf16"),
    (2, 200, 4, 1, 32, 5, 90, "bf16"),
    (2, 9, 4, 2, 160, 16, 19, "bf16"),
    (1, 2, 1, 1, 160, 7, 30, "bf16"),
    (2, 17, 16, 2, 256, 16, 19, "bf16"),
    (1, 200, 8, 2, 256, 16, 30, "bf16"),
    (1, 40, 3, 1, 224, 16, 30, "bf16"),
    (1, 40, 14, 2, 192, 48, 12, "bf16"),
    (1, 4, 8, 2, 128, 64, 1024, "bf16"),        # the longest resident set
    (1, 150, 2, 1, 128, 64, 1024, "bf16"),
    (60, 3, 8, 8, 128, 16, 9, "bf16"),          # whole items and split ones
    (90, 33, 32, 4, 64, 16, 6, "bf16"),
    (1, 1, 1, 1, 32, 1, 1, "bf16"),             # the smallest
    (2, 100, 8, 2, 64, 16, 32, "f32"),
    (3, 1, 2, 1, 128, 16, 21, "f32"),
    (2, 64, 8, 1, 128, 16, 33, "f32"),
    (2, 5, 6, 2, 96, 5, 50, "f32"),
    (2, 29, 7, 1, 96, 24, 20, "f32"),
    (2, 9, 8, 8, 32, 64, 7, "f32"),
    (1, 3, 16, 2, 256, 16, 40, "f32"),
    (1, 30, 16, 2, 256, 16, 40, "f32"),
    (2, 2, 8, 1, 64, 16, 40, "f32"),            # 16 rows
    (2, 40, 8, 2, 192, 33, 9, "f32"),
    (2, 20, 4, 2, 224, 16, 9, "f32"),
    (1, 20, 4, 2, 160, 16, 9, "f32"),
    (70, 9, 8, 8, 32, 16, 5, "f32"),
    (1, 1, 1, 1, 32, 1, 1, "f32"),
]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 0), (100, 20)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(v) for v in s))
def test_against_plain(shape, window, sinks):
    R, T, Hq, H, d, bs, kb, dtype = shape
    x = make(*shape, seed=R * 1000 + T)
    x.update(window=window, sinks=sinks)
    check(x, call(x))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 96), ("bf16", 256), ("f32", 64)])
@pytest.mark.parametrize("T", [6, 90])
@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 3), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_lengths_and_counts(dtype, d, T, window, sinks):
    """Lengths of 0, 1, a block's edge and past the pool; counts of 0, 1, T, out of range; a negative length, and one
    that leaves no room for positions."""
    lengths = [0, 0, 1, 15, 16, 17, 160, 4000]
    x = make(8, T, 8, 2, d, 16, 10, dtype, seed=3, lengths=lengths, counts=[T, 3, 1, 0, T, 999, -4, T - 1])
    x.update(window=window, sinks=sinks)
    check(x, call(x))
    x["lengths"][2], x["lengths"][4] = -1, 2 ** 31 - T
    got = call(x)
    check(x, got)
    import torch
    assert torch.equal(got[2][[2, 4]], x["weight"][[2, 4]])


@pytest.mark.parametrize("dtype,d,kb,T", [("bf16", 128, 12, 40), ("bf16", 128, 12, 3), ("bf16", 64, 120, 100), ("f32", 64, 12, 20)])
def test_rows_that_see_nothing(dtype, d, kb, T):
    """No slot at all, and none of the blocks that a window leaves: zeros, -infinity and no weights."""
    import torch
    x = make(3, T, 8, 2, d, 16, kb, dtype, seed=4, lengths=[500, 640, 40])
    x["slot_block"][0] = -1
    x["slot_block"][1] = torch.where(x["slot_block"][1] >= 36, -1, x["slot_block"][1])  # positions from 576 on are gone
    x.update(window=30, sinks=0)
    got = call(x)
    check(x, got)
    assert not got[0][:2].any() and torch.isinf(got[1][:2]).all() and torch.equal(got[2][:2], x["weight"][:2])


@pytest.mark.parametrize("dtype,d,kb,T", [("bf16", 128, 12, 40), ("bf16", 128, 120, 9), ("bf16", 64, 12, 70), ("bf16", 96, 30, 50), ("f32", 64, 12, 30),
                                             ("f32", 64, 12, 9), ("f32", 128, 40, 9)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 4)])
def test_values_that_are_not_finite(dtype, d, kb, T, window, sinks):
    """Infinite and NaN keys and values of new tokens reach exactly the rows that see them."""
    import torch
    n = kb * 16 - T
    x = make(2, T, 8, 2, d, 16, kb, dtype, seed=5, lengths=[n, 0], holes=False)
    x.update(window=window, sinks=sinks)
    for r, at, what in ((0, n + 2, ("v", 3, "inf")), (0, n + 2, ("v", 5, "nan")), (0, n + 6, ("v", slice(None), "-inf")), (0, n + 7, ("v", 5, "inf")),
                        (0, n + T - 1, ("k", 0, "nan")), (1, 3, ("v", 1, "nan")), (1, 1, ("k", slice(None), "inf"))):
        slot = at // 16
        assert int(x["slot_block"][r, 0, slot]) == slot
        x["pool"][r, :, slot, 0 if what[0] == "k" else 1, at % 16, what[1]] = float(what[2])
    check(x, call(x))


@pytest.mark.parametrize("dtype,d,T", [("bf16", 128, 70), ("bf16", 128, 5), ("bf16", 256, 20), ("f32", 64, 20)])
def test_large_scores(dtype, d, T):
    """Scores far apart and a maximum that keeps growing along the tokens, in either order."""
    import torch
    x = make(2, T, 8, 2, d, 16, 40, dtype, seed=7, lengths=[640 - T, 640 - T], stale=0.0, holes=False)
    ramp = torch.linspace(0.1, 6.0, 640, device="cuda").reshape(40, 16)[..., None]
    x["pool"][0, :, :, 0] = ((1 + 0.1 * x["pool"][0, :, :, 0].float()) * ramp).to(x["pool"].dtype)
    x["pool"][1, :, :, 0] = ((1 + 0.1 * x["pool"][1, :, :, 0].float()) * ramp.flip(0)).to(x["pool"].dtype)
    x["q"][:] = (1 + 0.1 * x["q"].float()).to(x["q"].dtype)
    check(x, call(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs", [16, 12, 64])
def test_the_last_positions_there_are(dtype, bs):
    """Positions next to 2^31 - 1, blocks behind them, and the same block in two slots."""
    import torch
    T, n = 5, 2 ** 31 - 1 - 5
    x = make(2, T, 8, 2, 64, bs, 6, dtype, seed=41, lengths=[3 * bs, 2 * bs], holes=False)
    gen = torch.Generator().manual_seed(bs)
    x["pool"][0] = torch.randn(2, 6, 2, bs, 64, generator=gen).to(x["pool"])
    last = (n + T - 1) // bs
    x["slot_block"][0] = torch.tensor([0, last, last - 1, last, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    x["pool"][0, :, 4:] = float("nan")
    x["pool"][0, :, [1, 3], :, n + T - last * bs:] = float("nan")
    x["lengths"][0] = n
    for window, sinks in ((0, 0), (bs + 1, 3), (2 ** 31 - 1, 0)):
        x.update(window=window, sinks=sinks)
        check(x, call(x))


@pytest.mark.parametrize("R,T,kb", [(1, 1, 128), (1, 60, 128), (40, 16, 32), (3, 100, 64)])
def test_same_bits_every_time_and_from_a_graph(R, T, kb):
    """Two calls, calls on two streams beside it, and replays of captured calls (of new inputs in the same tensors) give the
    same bits as a plain call."""
    import torch
    from sparse_kv_cache_draft_gb300 import attend_chunk_static
    x, y = (make(R, T, 32, 8, 128, 16, kb, "bf16", seed=s) for s in (13, 14))
    a, b = call(x), call(y)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):  # side by side: nothing is shared between calls
        with torch.cuda.stream(s1):
            p = call(x)
        with torch.cuda.stream(s2):
            q = call(y)
        outs.append((p, q))
    torch.cuda.synchronize()
    for p, q in outs:
        assert all(torch.equal(u, v) for u, v in zip(p, a)) and all(torch.equal(u, v) for u, v in zip(q, b))

    def captured(z):
        got = [torch.full_like(t, -7.0) for t in a]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend_chunk_static(z["pool"], z["slot_block"], z["lengths"], None, z["q"], *got[:2], z["weight"], got[2], q_heads=32, kv_heads=8, head_dim=128,
                                block_size=16, slots=kb)
        return g, got

    z = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in x.items()}
    (g1, o1), (g2, o2) = captured(z), captured(y)
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(o1, a)) and all(torch.equal(u, v) for u, v in zip(o2, b))
    for n in ("pool", "slot_block", "lengths", "q", "weight"):
        z[n].copy_(y[n])
    g1.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(o1, b))


@pytest.mark.parametrize("T,dtype", [(1, "bf16"), (50, "bf16"), (9, "f32")])
def test_forms_of_the_call(T, dtype):
    """Without lse, without weights, weights from zero and in place: the same values."""
    import torch
    from sparse_kv_cache_draft_gb300 import attend_chunk_static
    x = make(3, T, 8, 2, 64, 16, 20, dtype, seed=21)
    out, lse, drawn = call(x)
    kw = dict(q_heads=8, kv_heads=2, head_dim=64, block_size=16, slots=20)
    args = (x["pool"], x["slot_block"], x["lengths"], None, x["q"])
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    attend_chunk_static(*args, o, **kw)
    assert torch.equal(o, out)
    w = x["weight"].clone()
    attend_chunk_static(*args, o.zero_(), l, w, **kw)
    assert torch.equal(o, out) and torch.equal(l, lse) and torch.equal(w, drawn)
    w.fill_(float("nan"))
    attend_chunk_static(*args, o, l, weight_out=w, **kw)
    zero = dict(x, weight=torch.zeros_like(w))
    assert torch.equal(w, call(zero)[2])
    with pytest.raises(ValueError, match="lse"):
        attend_chunk_static(*args, o, None, w, **kw)


def test_large_offsets():
    """A pool past 2^31 elements."""
    import torch
    x = make(2, 40, 2, 1, 256, 64, 8, "bf16", seed=9, lengths=[400, 300], holes=False)
    R = 132  # 132 x 1024 slots x 2 x 64 x 256 elements: 4.4e9
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    big = torch.full((R, 1, 1024, 2, 64, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    sb = torch.full((R, 1, 1024), -1, dtype=torch.int32, device="cuda")
    ln, q = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.randn(R, 40, 2, 256, device="cuda", dtype=torch.bfloat16)
    for r, at in ((0, 0), (R - 1, 1)):
        big[r, :, 1016:], sb[r, :, 1016:] = x["pool"][at], x["slot_block"][at]
        ln[r], q[r] = x["lengths"][at], x["q"][at]
    y = dict(pool=big, slot_block=sb, lengths=ln, counts=None, q=q, window=0, sinks=0, weight=torch.zeros(R, 1, 1024, device="cuda"))
    out, lse, drawn = call(y)
    part = dict(x, weight=torch.zeros_like(x["weight"]))
    check(part, (out[[0, R - 1]], lse[[0, R - 1]], drawn[[0, R - 1]][:, :, 1016:]))
    assert not out[1:R - 1].any() and not drawn[1:R - 1].any()
