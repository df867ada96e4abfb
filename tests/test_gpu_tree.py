"""Attention of drafted trees (okv_attend_tree_static) against the plain binary64 form."""
import pytest

import tree_ref

pytestmark = pytest.mark.gpu


def make(R, T, Hq, H, d, bs, kb, dtype, seed=0, lengths=None, holes=False, stale=float("nan")):
    """Inputs with `stale` in every place of the pool that holds no valid token."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    dev = "cuda"
    if lengths is None:
        lengths = [int(x) for x in torch.randint(0, 2 * kb * bs, (R,), generator=gen)]
    slot_block = torch.full((R, H, kb), -1, dtype=torch.int32)
    for r in range(R):
        nb = -(-lengths[r] // bs)
        for h in range(H):
            n = min(kb, nb)
            if holes and n > 1:
                n -= int(torch.randint(0, n // 2 + 1, (1,), generator=gen))
            ids = torch.randperm(nb, generator=gen)[:n]
            if n and nb - 1 not in ids.tolist():
                ids[0] = nb - 1  # the part-filled block is resident
            place = torch.randperm(kb, generator=gen)[:n] if holes else torch.arange(n)
            slot_block[r, h, place] = ids.to(torch.int32)
    pool = torch.randn(R, H, kb, 2, bs, d, generator=gen).to(dt)
    pos = slot_block[..., None] * bs + torch.arange(bs)
    dead = (slot_block[..., None] < 0) | (pos >= torch.tensor(lengths)[:, None, None, None])
    pool.permute(0, 1, 2, 4, 3, 5)[dead] = stale
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dt).to(dev)
    return dict(pool=pool.to(dev), slot_block=slot_block.to(dev), lengths=torch.tensor(lengths, dtype=torch.int32, device=dev),
                counts=None, q=(2 * torch.randn(R, T, Hq, d, generator=gen)).to(dt).to(dev), k=rnd(R, T, H, d), v=rnd(R, T, H, d),
                mask=tree_ref.random_trees(R, T, gen, dev))


def call(x, out=None, stream=None):
    import torch
    from sparse_kv_cache_draft_gb300 import attend_tree_static
    if out is None:
        out = torch.full_like(x["q"], -7.0)
    R, H, kb, _, bs, d = x["pool"].shape
    attend_tree_static(x["pool"], x["slot_block"], x["lengths"], x["counts"], x["q"], x["k"], x["v"], x["mask"], out,
                       q_heads=x["q"].shape[2], kv_heads=H, head_dim=d, block_size=bs, slots=kb, stream=stream)
    return out


def check(x, out):
    import torch
    want, bound = tree_ref.attend(**x)
    cnt = x["counts"] if x["counts"] is not None else torch.full_like(x["lengths"], x["q"].shape[1])
    fresh = torch.arange(x["q"].shape[1], device="cuda") < cnt.clamp(0, x["q"].shape[1])[:, None]
    got = out.double()
    assert torch.equal(got[~fresh], torch.full_like(got[~fresh], -7.0)), "rows past a request's count were written"
    got, want, bound = got[fresh], want[fresh], bound[fresh]
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~finite & ~torch.isnan(want)], want[~finite & ~torch.isnan(want)])
    over = ((got - want).abs() - bound)[finite]
    assert over.numel() == 0 or float(over.max()) <= 0, f"worst excess {float(over.max()):.3g}"


SHAPES = [  # R, T, Hq, Hkv, d, bs, kb, dtype, holes
    (1, 1, 1, 1, 128, 16, 1, "bf16", False),
    (1, 8, 32, 8, 128, 16, 128, "bf16", False),
    (3, 5, 8, 2, 128, 16, 37, "bf16", True),
    (2, 16, 32, 8, 128, 16, 33, "bf16", True),
    (2, 33, 8, 2, 128, 16, 20, "bf16", True),      # 132 rows: past one tile of 128
    (2, 64, 16, 2, 128, 16, 24, "bf16", True),     # 512 rows
    (3, 64, 7, 1, 128, 64, 9, "bf16", True),
    (2, 13, 24, 8, 64, 32, 33, "bf16", False),
    (3, 9, 6, 2, 64, 16, 40, "bf16", True),
    (2, 64, 8, 1, 64, 8, 65, "bf16", True),
    (2, 7, 4, 2, 128, 1, 200, "bf16", True),       # a token per block
    (2, 7, 4, 2, 128, 12, 21, "bf16", True),       # blocks that do not divide a tile
    (2, 6, 4, 4, 128, 33, 11, "bf16", True),
    (2, 21, 10, 2, 96, 16, 19, "bf16", True),
    (2, 9, 4, 2, 32, 16, 19, "bf16", True),
    (2, 9, 4, 2, 160, 16, 19, "bf16", True),
    (2, 17, 16, 2, 256, 16, 19, "bf16", True),
    (1, 4, 8, 2, 128, 64, 1024, "bf16", False),    # the longest resident set
    (2, 64, 16, 2, 256, 16, 21, "bf16", True),
    (2, 43, 18, 3, 128, 16, 19, "bf16", True),     # 6 heads: 126 rows to a warpgroup
    (2, 64, 5, 1, 96, 8, 50, "bf16", True),
    (3, 64, 8, 1, 32, 16, 30, "bf16", True),
    (2, 64, 8, 1, 64, 33, 20, "bf16", True),       # drafted tokens past a block's lines of a tile
    (2, 60, 8, 1, 128, 48, 20, "bf16", True),
    (1, 2, 1, 1, 160, 7, 30, "bf16", True),
    (60, 3, 8, 8, 128, 16, 9, "bf16", True),       # whole items and split ones
    (90, 33, 32, 4, 64, 16, 6, "bf16", True),
    (1, 1, 1, 1, 32, 1, 1, "bf16", False),         # the smallest
    (1, 64, 8, 1, 128, 64, 1024, "bf16", True),    # the longest tables beside the largest tiles
    (1, 20, 8, 1, 256, 64, 1024, "bf16", True),
    (1, 9, 8, 1, 64, 1, 1024, "bf16", True),
    (2, 12, 8, 2, 64, 16, 32, "f32", False),
    (3, 1, 2, 1, 128, 16, 21, "f32", True),
    (2, 64, 8, 1, 128, 16, 33, "f32", True),
    (2, 5, 6, 2, 96, 5, 50, "f32", True),
    (2, 9, 8, 8, 32, 64, 7, "f32", True),
    (1, 3, 16, 2, 256, 16, 40, "f32", True),
    (2, 2, 8, 1, 64, 16, 40, "f32", True),          # 16 rows
    (2, 5, 8, 2, 192, 33, 9, "f32", True),
    (70, 9, 8, 8, 32, 16, 5, "f32", True),
    (1, 1, 1, 1, 32, 1, 1, "f32", False),
    (1, 3, 8, 1, 256, 64, 1024, "f32", True),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(v) for v in s))
def test_against_plain(shape):
    R, T, Hq, H, d, bs, kb, dtype, holes = shape
    x = make(R, T, Hq, H, d, bs, kb, dtype, seed=R * 1000 + T, holes=holes)
    check(x, call(x))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 96), ("f32", 64)])
def test_lengths_counts_and_empty_rows(dtype, d):
    """Lengths of 0, 1, a block's edge and past the budget; counts of 0, 1, T, out of range; rows
    whose mask leaves nothing (zeros on a request without tokens)."""
    import torch
    lengths = [0, 0, 1, 15, 16, 17, 160, 4000]
    x = make(8, 6, 8, 2, d, 16, 10, dtype, seed=3, lengths=lengths)
    x["counts"] = torch.tensor([6, 3, 1, 0, 6, 99, -4, 5], dtype=torch.int32, device="cuda")
    x["mask"][:, 1] = 0
    x["mask"][:, 4] = -1 ^ 0b10000  # everything but itself, bits past the count among them
    out = call(x)
    check(x, out)
    assert float(out[0, 1].abs().max()) == 0.0 and float(out[1, 1].abs().max()) == 0.0


@pytest.mark.parametrize("dtype,d,kb", [("bf16", 128, 12), ("bf16", 128, 120), ("bf16", 64, 12), ("f32", 64, 12)])
def test_values_that_are_not_finite(dtype, d, kb):
    """Infinite and NaN keys and values of drafted tokens reach exactly the rows that see them."""
    import torch
    x = make(2, 9, 8, 2, d, 16, kb, dtype, seed=5, lengths=[kb * 16 - 3, 0])
    x["v"][:, 2, :, 3] = float("inf")
    x["v"][:, 2, :, 5] = float("nan")
    x["v"][:, 6] = float("-inf")
    x["v"][:, 7, 0, 3] = float("-inf")
    x["k"][:, 8] = float("nan")
    m = torch.tensor([1, 2, 0b101, 8, 0b10001, 0b100000, 0b1000001, 0b10000101, 0b100000001], dtype=torch.int64, device="cuda")
    x["mask"][:] = m
    check(x, call(x))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_large_scores(dtype, d):
    """Scores far apart and a maximum that keeps growing along the tokens (the running maximum's
    corrections), in either order."""
    import torch
    x = make(2, 5, 8, 2, d, 16, 40, dtype, seed=7, lengths=[640, 640], stale=0.0)
    ramp = torch.linspace(0.1, 6.0, 640, device="cuda").reshape(40, 16)[..., None]
    x["pool"][0, :, :, 0] = ((1 + 0.1 * x["pool"][0, :, :, 0].float()) * ramp).to(x["pool"].dtype)
    x["pool"][1, :, :, 0] = ((1 + 0.1 * x["pool"][1, :, :, 0].float()) * ramp.flip(0)).to(x["pool"].dtype)
    x["q"][:] = (1 + 0.1 * x["q"].float()).to(x["q"].dtype)
    check(x, call(x))


def test_block_ids_outside_the_request_are_empty_slots():
    import torch
    x = make(2, 4, 8, 2, 128, 16, 12, "bf16", seed=11, lengths=[150, 100])
    bad = x["slot_block"].clone()
    bad[0, 0, 3], bad[0, 1, 4], bad[1, 0, 0] = 10, 2 ** 31 - 1, -5  # 150 tokens: blocks 0..9
    x["slot_block"] = bad
    out = call(x)
    y = dict(x)
    y["slot_block"] = torch.where((bad < 0) | (bad.long() * 16 >= x["lengths"][:, None, None]), -1, bad).to(torch.int32)
    check(y, out)


@pytest.mark.parametrize("R,T,kb", [(1, 8, 128), (40, 16, 32), (3, 64, 64)])
def test_same_bits_every_time_and_from_a_graph(R, T, kb):
    """Two calls, a call on another stream beside it, and replays of a captured call (of new
    inputs in the same tensors) give the same bits as a plain call."""
    import torch
    x = make(R, T, 32, 8, 128, 16, kb, "bf16", seed=13)
    y = make(R, T, 32, 8, 128, 16, kb, "bf16", seed=14)
    a, b = call(x), call(y)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):  # side by side: nothing is shared between calls
        outs.append((call(x, stream=s1, out=torch.full_like(a, -7.0)), call(y, stream=s2, out=torch.full_like(b, -7.0))))
    torch.cuda.synchronize()
    for p, q in outs:
        assert torch.equal(p, a) and torch.equal(q, b)
    z = {n: (t.clone() if t is not None else None) for n, t in x.items()}
    out = torch.full_like(a, -7.0)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        call(z, out=out)
    out2 = torch.full_like(b, -7.0)
    with torch.cuda.graph(g2):
        call(y, out=out2)
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a) and torch.equal(out2, b)
    for n, t in z.items():
        if t is not None:
            t.copy_(y[n])
    g1.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, b)


def test_first_call_of_a_shape_in_a_capture():
    import torch
    x = make(3, 11, 10, 2, 128, 16, 27, "bf16", seed=19)
    out = torch.full_like(x["q"], -7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, out=out)
    g.replay()
    torch.cuda.synchronize()
    check(x, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pool_past_31_bits(dtype):
    """The last request of a pool of more than 2^31 elements."""
    import torch
    R, T, Hq, H, d, bs, kb = 70, 3, 8, 8, 128, 16, 1024
    x = make(1, T, Hq, H, d, bs, kb, dtype, seed=23, lengths=[kb * bs - 5], stale=0.0)
    assert R * x["pool"].numel() > 2 ** 31
    y = dict(counts=torch.zeros(R, dtype=torch.int32, device="cuda"))
    y["counts"][-1] = T
    for n in ("pool", "slot_block", "lengths", "q", "k", "v", "mask"):
        y[n] = torch.zeros((R,) + x[n].shape[1:], dtype=x[n].dtype, device="cuda")
        y[n][-1] = x[n][0]
    out = call(y)
    assert bool((out[:-1] == -7.0).all())
    check(x, out[-1:])


def test_calls_from_several_threads():
    """Calls of different shapes at once from several host threads, each on a stream of its own."""
    import threading
    import torch
    shapes = [(1, 8, 32, 8, 128, 16, 40), (2, 64, 16, 2, 128, 16, 20), (3, 5, 8, 2, 64, 32, 9), (2, 9, 4, 2, 256, 16, 30)]
    xs = [make(*sh, "bf16", seed=i) for i, sh in enumerate(shapes)]
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(20):
                got = call(xs[i])
                st.synchronize()
                if not torch.equal(got, want[i]):
                    wrong.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong


def test_mask_as_uint64_and_refusals():
    import torch
    from sparse_kv_cache_draft_gb300 import OkvError, binding
    x = make(1, 64, 4, 1, 128, 16, 5, "bf16", seed=17)
    a = call(x)
    assert torch.equal(call(dict(x, mask=x["mask"].view(torch.uint64))), a)
    with pytest.raises(ValueError):
        call(dict(x, q=x["q"].float()))
    with pytest.raises(ValueError):
        call(dict(x, k=x["k"].transpose(2, 3)))
    with pytest.raises(ValueError):
        call(dict(x, lengths=x["lengths"].long()))
    with pytest.raises(ValueError):
        call(dict(x, mask=x["mask"][:, :32]))
    with pytest.raises(ValueError):
        call(dict(x, counts=x["lengths"].cpu()))
    with pytest.raises(TypeError):
        call({n: (t.cpu() if t is not None else None) for n, t in x.items()}, out=a.cpu())
    big = make(1, 1, 4, 1, 128, 16, 5, "bf16", seed=17)
    wide = {n: (t.expand(1, 65, *t.shape[2:]).contiguous() if n in "qkv" or n == "mask" else t) for n, t in big.items()}
    with pytest.raises(OkvError) as e:
        call(wide)
    assert e.value.status == binding.EINVAL


@pytest.mark.parametrize("R,T,d,bs,kb,dtype", [(2, 8, 128, 16, 40, "bf16"), (150, 16, 64, 16, 24, "bf16"), (40, 64, 128, 16, 16, "bf16"),
                                               (3, 9, 192, 16, 30, "bf16"), (6, 7, 64, 8, 20, "f32")])
def test_calls_behind_one_another(R, T, d, bs, kb, dtype):
    """Launches overlap; each call's results and effects are those of calls that wait for one another."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static, norm_rope
    x = make(R, T, 8, 2, d, bs, kb, dtype, seed=23, stale=0.0)
    inv = 10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float32) / d)
    rot, kw = Rotary(inv, eps=1e-5), dict(q_heads=4, kv_heads=2, head_dim=d)
    pos = torch.arange(R * T, dtype=torch.int32, device="cuda")

    def chain(wait):
        pool, (y, z) = x["pool"].clone(), (x["q"].clone(), torch.zeros_like(x["q"]))
        q, (k, v) = torch.empty(R * T, 4, d, dtype=y.dtype, device="cuda"), (torch.empty_like(x["k"]) for _ in range(2))
        seen = []
        for i in range(30):
            norm_rope(y.view(R * T, 8 * d), pos, q, k.view(R * T, 2, d), v.view(R * T, 2, d), rotary=rot, **kw)
            wait()
            call(dict(x, pool=pool, q=y, k=k, v=v), out=z)
            wait()
            append_qkv_static(z.view(R, T, 8 * d), x["lengths"], None, pool, x["slot_block"], q.view(R, T, 4, d), block_size=bs,
                              slots=kb, rotary=rot, **kw)
            wait()
            if i % 7 == 3:  # a launch that does not overlap, in between
                z.add_(q.view(R, T, 4, d).repeat(1, 1, 2, 1))
                wait()
            y, z = z, y
            if i == 14:
                seen.append(y.clone())
        torch.cuda.synchronize()
        return seen + [y, z, pool, q, k, v]

    want = chain(torch.cuda.synchronize)
    assert all(bool(t.isfinite().all()) for t in want)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, chain(lambda: None)))
    with torch.cuda.stream(torch.cuda.Stream()):
        assert all(torch.equal(a, b) for a, b in zip(want, chain(lambda: None)))


def test_a_call_behind_an_event_of_another_stream():
    """A launch that would overlap the one before it still waits for an event that its stream waits for."""
    import torch
    x = make(2, 8, 8, 2, 128, 16, 24, "bf16", seed=29)
    other = torch.randn_like(x["q"])
    want = [call(dict(x, q=q)) for q in (x["q"], other)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    q, busy = x["q"].clone(), torch.randn(4096, 4096, device="cuda")
    outs = [torch.empty_like(q) for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(20):
        for k, source in enumerate((other, x["q"])):
            with torch.cuda.stream(a):
                a.wait_stream(b)
                y = busy @ busy  # some time before the queries are there
                q.copy_(source)
                ready = a.record_event()
            with torch.cuda.stream(b):
                if i % 2:
                    call(dict(x, q=other), out=outs[2])  # a launch of ours that the next one may overlap
                b.wait_event(ready)
                call(dict(x, q=q), out=outs[k])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[1]) and torch.equal(outs[1], want[0]), i
    del y
