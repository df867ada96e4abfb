"""Rows of a projection (okv_norm_rope) and their append to a pool (okv_append_qkv_static) against
the plain binary64 forms."""
import pytest

import tree_ref

pytestmark = pytest.mark.gpu


def dt_of(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def make_rotary(d, rot, dtype, gen, norm, interleaved, base=1e6, eps=1e-6):
    import torch
    inv = (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda() if rot else None
    w = [(1 + 0.3 * torch.randn(d, generator=gen)).to(dtype).cuda() if norm else None for _ in range(2)]
    return dict(inv_freq=inv, q_weight=w[0], k_weight=w[1], eps=eps, interleaved=interleaved)


def near(got, want, bound, what):
    over = (got.double() - want).abs() - bound
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: worst excess {float(over.max()):.3g}"


ROWS = [  # n, Hq, Hkv, d, rotary_dim, dtype, norm, interleaved, pad, first position
    (1, 32, 8, 128, 128, "bf16", True, False, 0, 0),
    (7, 32, 8, 128, 128, "bf16", True, False, 0, 16383),
    (300, 8, 2, 64, 64, "bf16", True, False, 8, 1000),
    (33, 3, 1, 96, 96, "bf16", True, False, 0, 5),
    (33, 5, 5, 32, 32, "bf16", True, True, 40, 5),
    (9, 4, 1, 256, 128, "bf16", True, False, 0, 77),
    (9, 7, 1, 160, 80, "bf16", False, False, 0, 77),
    (1, 2, 1, 64, 0, "bf16", True, False, 0, 3),
    (65, 8, 2, 64, 64, "f32", True, False, 4, 1 << 20),
    (65, 8, 2, 64, 32, "f32", False, True, 0, (1 << 31) - 100),   # the last positions
    (12, 16, 2, 128, 128, "f32", True, False, 0, 262143),
    (12, 3, 3, 96, 48, "f32", True, False, 12, 9),
    (12, 2, 1, 256, 256, "f32", True, True, 0, 9),
    (12, 2, 1, 224, 16, "f32", True, False, 0, 9),
    (1, 1, 1, 32, 32, "f32", False, False, 0, 0),
]


@pytest.mark.parametrize("shape", ROWS, ids=lambda s: "-".join(str(v) for v in s))
def test_rows_against_plain(shape):
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    n, Hq, H, d, rot, dtype, norm, inter, pad, first = shape
    gen = torch.Generator().manual_seed(n + d)
    dt = dt_of(dtype)
    W = (Hq + 2 * H) * d
    qkv = torch.randn(n, W + pad, generator=gen).to(dt).cuda()[:, :W]
    pos = (first + torch.randint(0, 100, (n,), generator=gen)).to(torch.int32).cuda()
    pos[0] = first
    rope = make_rotary(d, rot, dt, gen, norm, inter)
    out = [torch.full((n, h, d), -7.0, dtype=dt, device="cuda") for h in (Hq, H, H)]
    norm_rope(qkv, pos, *out, q_heads=Hq, kv_heads=H, head_dim=d, rotary=Rotary(**rope))
    q, k, v, bq, bk = tree_ref.rows(qkv, pos, Hq, H, d, **rope)
    near(out[0], q, bq, "q")
    near(out[1], k, bk, "k")
    assert torch.equal(out[2].double(), v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_left_out_and_outputs_left_out(dtype):
    """Rows with a negative position stay as they were; NaN there reaches nothing else; any output may
    be left out; no rows at all is no work."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    gen = torch.Generator().manual_seed(1)
    dt = dt_of(dtype)
    n, Hq, H, d = 23, 6, 2, 64
    kw = dict(q_heads=Hq, kv_heads=H, head_dim=d)
    qkv = torch.randn(n, (Hq + 2 * H) * d, generator=gen).to(dt).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    pos[::4] = -1
    qkv[::4] = float("nan")
    rope = make_rotary(d, d, dt, gen, True, False)
    rot = Rotary(**rope)
    out = [torch.full((n, h, d), -7.0, dtype=dt, device="cuda") for h in (Hq, H, H)]
    norm_rope(qkv, pos, *out, rotary=rot, **kw)
    keep = pos >= 0
    q, k, v, bq, bk = tree_ref.rows(qkv[keep], pos[keep], Hq, H, d, **rope)
    near(out[0][keep], q, bq, "q")
    near(out[1][keep], k, bk, "k")
    assert torch.equal(out[2][keep].double(), v)
    for o in out:
        assert bool((o[~keep] == -7.0).all())
    for i in range(3):
        one = [None, None, None]
        one[i] = torch.full_like(out[i], -7.0)
        norm_rope(qkv, pos, *one, rotary=rot, **kw)
        assert torch.equal(one[i], out[i])
    norm_rope(qkv[:0], pos[:0], *[o[:0] for o in out], rotary=rot, **kw)


def test_zero_rows_infinities_and_tiny_values():
    """A row of zeros is zero (eps holds the root up); an infinite element makes its own head NaN or
    infinite as the formula does, and no other head."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    gen = torch.Generator().manual_seed(2)
    Hq, H, d = 4, 2, 128
    qkv = torch.randn(3, (Hq + 2 * H) * d, generator=gen).to(torch.bfloat16).cuda()
    qkv[0] = 0
    qkv[1] *= 1e-15
    qkv[2, d:2 * d] = float("inf")
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    rope = make_rotary(d, d, torch.bfloat16, gen, True, False)
    out = [torch.empty(3, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H)]
    norm_rope(qkv, pos, *out, q_heads=Hq, kv_heads=H, head_dim=d, rotary=Rotary(**rope))
    q, k, v, bq, bk = tree_ref.rows(qkv, pos, Hq, H, d, **rope)
    assert float(out[0][0].abs().max()) == 0.0
    near(out[0][1], q[1], bq[1] + 1e-38, "tiny")
    assert bool(out[0][2, 1].isnan().all())
    rest = [0, 2, 3]
    near(out[0][2, rest], q[2, rest], bq[2, rest], "the heads beside it")


APPEND = [  # R, T, Hq, Hkv, d, bs, kb, dtype, ragged
    (1, 1, 32, 8, 128, 16, 128, "bf16", False),
    (5, 1, 32, 8, 128, 16, 40, "bf16", False),
    (3, 70, 8, 2, 128, 16, 12, "bf16", True),
    (4, 9, 6, 2, 64, 5, 9, "bf16", True),
    (3, 11, 4, 4, 96, 1, 30, "bf16", True),
    (2, 130, 64, 8, 128, 64, 4, "bf16", True),
    (3, 5, 8, 2, 64, 16, 32, "f32", True),
    (2, 33, 2, 1, 32, 8, 7, "f32", True),
    (2, 3, 2, 1, 256, 16, 1024, "f32", False),
]


@pytest.mark.parametrize("shape", APPEND, ids=lambda s: "-".join(str(v) for v in s))
def test_append_against_plain(shape):
    """Queries, keys and values within the rounding bounds in the slots that hold the tokens' blocks;
    every other place of the pool and every row past a count as they were."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static
    R, T, Hq, H, d, bs, kb, dtype, ragged = shape
    gen = torch.Generator().manual_seed(R * 100 + T)
    dt = dt_of(dtype)
    lengths = [int(x) for x in torch.randint(0, 3 * kb * bs, (R,), generator=gen)]
    lengths[0] = 0
    counts = [T] * R if not ragged else [int(x) for x in torch.randint(0, T + 3, (R,), generator=gen)]
    sb = torch.full((R, H, kb), -1, dtype=torch.int32)
    for r in range(R):
        first, last = lengths[r] // bs, (lengths[r] + T) // bs
        ids = [b for b in range(max(0, last - kb + 1), last + 1) if b % 5 != 3]  # one in five is not resident
        for h in range(H):
            place = torch.randperm(kb, generator=gen)[:len(ids)]
            sb[r, h, place] = torch.tensor(ids, dtype=torch.int32)
    pool = torch.randn(R, H, kb, 2, bs, d, generator=gen).to(dt).cuda()
    before = pool.clone()
    qkv = torch.randn(R, T, (Hq + 2 * H) * d, generator=gen).to(dt).cuda()
    rope = make_rotary(d, d, dt, gen, True, False)
    q = torch.full((R, T, Hq, d), -7.0, dtype=dt, device="cuda")
    append_qkv_static(qkv, torch.tensor(lengths, dtype=torch.int32).cuda(),
                      torch.tensor(counts, dtype=torch.int32).cuda() if ragged else None, pool, sb.cuda(), q, q_heads=Hq,
                      kv_heads=H, head_dim=d, block_size=bs, slots=kb, rotary=Rotary(**rope))
    touched = torch.zeros(R, H, kb, bs, dtype=torch.bool)
    for r in range(R):
        n = min(counts[r], T)
        assert bool((q[r, n:] == -7.0).all())
        if not n:
            continue
        pos = lengths[r] + torch.arange(n, device="cuda")
        wq, wk, wv, bq, bk = tree_ref.rows(qkv[r, :n], pos, Hq, H, d, **rope)
        near(q[r, :n], wq, bq, "q")
        for h in range(H):
            for t in range(n):
                hit = (sb[r, h] == (lengths[r] + t) // bs).nonzero()
                if not len(hit):
                    continue
                s, at = int(hit[0]), (lengths[r] + t) % bs
                touched[r, h, s, at] = True
                near(pool[r, h, s, 0, at], wk[t, h], bk[t, h], "key")
                assert torch.equal(pool[r, h, s, 1, at].double(), wv[t, h])
    same = ~touched.cuda()
    assert torch.equal(pool.permute(0, 1, 2, 4, 3, 5)[same], before.permute(0, 1, 2, 4, 3, 5)[same])
    assert touched.any()


def test_append_refuses_positions_past_31_bits_and_negative_lengths():
    """Such requests are left out whole; the others are appended."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static
    R, T, Hq, H, d, bs, kb = 4, 3, 4, 2, 64, 16, 6
    gen = torch.Generator().manual_seed(4)
    lengths = torch.tensor([-1, 2 ** 31 - 1, 2 ** 31 - 2, 40], dtype=torch.int32, device="cuda")
    sb = torch.arange(kb, dtype=torch.int32, device="cuda").expand(R, H, kb).contiguous()
    sb[1:3, :, 0] = (2 ** 31 - 1) // bs
    pool = torch.zeros(R, H, kb, 2, bs, d, dtype=torch.bfloat16, device="cuda")
    qkv = torch.randn(R, T, (Hq + 2 * H) * d, generator=gen).to(torch.bfloat16).cuda()
    q = torch.full((R, T, Hq, d), -7.0, dtype=torch.bfloat16, device="cuda")
    append_qkv_static(qkv, lengths, None, pool, sb, q, q_heads=Hq, kv_heads=H, head_dim=d, block_size=bs, slots=kb,
                      rotary=Rotary(**make_rotary(d, d, torch.bfloat16, gen, True, False)))
    assert bool((q[:3] == -7.0).all()) and float(pool[:3].abs().max()) == 0.0
    assert bool((q[3] != -7.0).any()) and float(pool[3, :, 2].abs().max()) > 0


def test_append_takes_the_lowest_of_equal_slots():
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static
    pool = torch.zeros(1, 1, 40, 2, 16, 64, device="cuda")
    sb = torch.full((1, 1, 40), 2, dtype=torch.int32, device="cuda")
    sb[0, 0, :7] = -1
    qkv = torch.ones(1, 1, 3 * 64, device="cuda")
    append_qkv_static(qkv, torch.tensor([33], dtype=torch.int32, device="cuda"), None, pool, sb, None, q_heads=1, kv_heads=1,
                      head_dim=64, block_size=16, slots=40, rotary=Rotary())
    want = torch.zeros_like(pool)
    want[0, 0, 7, :, 1] = 1.0
    assert torch.equal(pool, want)


def test_rows_and_pool_past_31_bits():
    """The last rows of more than 2^31 elements, and the last request of a pool as large."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static, norm_rope
    gen = torch.Generator().manual_seed(8)
    Hq, H, d = 32, 8, 128
    n = (1 << 31) // (48 * d) + 3
    rope = make_rotary(d, d, torch.bfloat16, gen, True, False)
    qkv = torch.zeros(n, 48 * d, dtype=torch.bfloat16, device="cuda")
    qkv[-5:] = torch.randn(5, 48 * d, generator=gen).to(torch.bfloat16).cuda()
    pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    pos[-5:] = torch.arange(5, dtype=torch.int32, device="cuda")
    k = torch.empty(n, H, d, dtype=torch.bfloat16, device="cuda")
    norm_rope(qkv, pos, None, k, None, q_heads=Hq, kv_heads=H, head_dim=d, rotary=Rotary(**rope))
    _, wk, _, _, bk = tree_ref.rows(qkv[-5:], pos[-5:], Hq, H, d, **rope)
    near(k[-5:], wk, bk, "k")
    rows = qkv[-5:].clone()
    del qkv, k
    R, bs, kb = 70, 16, 1024
    pool = torch.zeros(R, H, kb, 2, bs, d, dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 1 << 31
    sb = torch.full((R, H, kb), -1, dtype=torch.int32, device="cuda")
    sb[-1, :, -1] = 3
    counts = torch.zeros(R, dtype=torch.int32, device="cuda")
    counts[-1] = 5
    lengths = torch.full((R,), 50, dtype=torch.int32, device="cuda")
    x = torch.zeros(R, 5, 48 * d, dtype=torch.bfloat16, device="cuda")
    x[-1] = rows
    append_qkv_static(x, lengths, counts, pool, sb, None, q_heads=Hq, kv_heads=H, head_dim=d, block_size=bs, slots=kb,
                      rotary=Rotary(**rope))
    _, wk, wv, _, bk = tree_ref.rows(rows, 50 + torch.arange(5, device="cuda"), Hq, H, d, **rope)
    near(pool[-1, :, -1, 0, 2:7].transpose(0, 1), wk, bk, "key")
    assert torch.equal(pool[-1, :, -1, 1, 2:7].transpose(0, 1).double(), wv)
    pool[-1, :, -1, :, 2:7] = 0
    assert not bool(pool.any())


def test_rows_from_a_graph_and_another_stream():
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    gen = torch.Generator().manual_seed(6)
    n, Hq, H, d = 50, 8, 2, 128
    rot = Rotary(**make_rotary(d, d, torch.bfloat16, gen, True, False))
    x = [torch.randn(n, (Hq + 2 * H) * d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    kw = dict(q_heads=Hq, kv_heads=H, head_dim=d, rotary=rot)
    bufs = lambda: [torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H)]
    a, b, c = bufs(), bufs(), bufs()
    norm_rope(x[0], pos, *a, **kw)
    norm_rope(x[1], pos, *b, **kw)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    norm_rope(x[1], pos, *c, stream=st, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(b, c))
    src, out = x[0].clone(), bufs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm_rope(src, pos, *out, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, out))
    src.copy_(x[1])
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(b, out))


def test_rotary_follows_its_tensors():
    """A parameter whose memory is replaced after the Rotary was made is read where it is at the call."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    gen = torch.Generator().manual_seed(8)
    n, Hq, H, d = 5, 4, 2, 64
    rope = make_rotary(d, d, torch.bfloat16, gen, True, False)
    other = make_rotary(d, d, torch.bfloat16, gen, True, False)
    x = torch.randn(n, (Hq + 2 * H) * d, generator=gen).to(torch.bfloat16).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    out = [[torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H)] for _ in range(2)]
    kw = dict(q_heads=Hq, kv_heads=H, head_dim=d)
    rot = Rotary(**rope)
    norm_rope(x, pos, *out[0], rotary=Rotary(**other), **kw)
    for name in ("inv_freq", "q_weight", "k_weight"):
        if torch.is_tensor(rope[name]):
            rope[name].data = other[name].clone()
    norm_rope(x, pos, *out[1], rotary=rot, **kw)
    assert all(torch.equal(p, q) for p, q in zip(*out))
    rope["q_weight"].data = torch.ones(d + 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="q_weight"):
        norm_rope(x, pos, *out[1], rotary=rot, **kw)


def test_a_stream_is_an_object_or_its_handle():
    import threading
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    gen = torch.Generator().manual_seed(9)
    n, Hq, H, d = 9, 4, 2, 64
    rope = make_rotary(d, d, torch.bfloat16, gen, True, False)
    x = torch.randn(n, (Hq + 2 * H) * d, generator=gen).to(torch.bfloat16).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    kw = dict(q_heads=Hq, kv_heads=H, head_dim=d, rotary=Rotary(**rope))
    want = [torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H)]
    norm_rope(x, pos, *want, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for given in (st, st.cuda_stream, 0, None):
        out = [torch.zeros_like(w) for w in want]
        torch.cuda.synchronize()
        norm_rope(x, pos, *out, stream=given, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, out)), given
    with torch.cuda.stream(st):
        out = [torch.zeros_like(w) for w in want]
        norm_rope(x, pos, *out, **kw)
    st.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, out))
    for bad in ("0", 1.5):
        with pytest.raises(AttributeError):
            norm_rope(x, pos, *out, stream=bad, **kw)
    same = []

    def work():
        mine = [torch.zeros_like(w) for w in want]
        for _ in range(200):
            norm_rope(x, pos, *mine, **kw)
        torch.cuda.synchronize()
        same.append(all(torch.equal(p, q) for p, q in zip(want, mine)))
    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert same == [True] * 4


def test_binding_refusals():
    import torch
    from sparse_kv_cache_draft_gb300 import OkvError, Rotary, norm_rope
    kw = dict(q_heads=4, kv_heads=2, head_dim=64)
    qkv = torch.zeros(3, 8 * 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    inv = torch.ones(32, device="cuda")
    with pytest.raises(ValueError):
        norm_rope(qkv[:, :-64], pos, q, rotary=Rotary(inv), **kw)
    with pytest.raises(ValueError):
        norm_rope(qkv, pos.long(), q, rotary=Rotary(inv), **kw)
    with pytest.raises(ValueError):
        norm_rope(qkv, pos, q.float(), rotary=Rotary(inv), **kw)
    with pytest.raises(ValueError):
        norm_rope(qkv, pos, q, rotary=Rotary(inv, q_weight=torch.ones(64, device="cuda")), **kw)
    with pytest.raises(ValueError):
        Rotary(inv.double())
    with pytest.raises(TypeError):
        norm_rope(qkv.cpu(), pos, q, rotary=Rotary(inv), **kw)
    for bad in (dict(rotary=Rotary(torch.ones(33, device="cuda"))), dict(rotary=Rotary(torch.ones(40, device="cuda"))),
                dict(rotary=Rotary(inv, eps=-1.0)), dict(rotary=Rotary(inv, eps=float("nan")))):
        with pytest.raises(OkvError):
            norm_rope(qkv, pos, q, **bad, **kw)
    with pytest.raises(OkvError):  # no output at all
        norm_rope(qkv, pos, rotary=Rotary(inv), **kw)
    flat = torch.zeros(3 * 8 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(OkvError):  # rows that do not start on 16 bytes
        norm_rope(flat[4:4 + 3 * 8 * 64].view(3, 8 * 64), pos, q, rotary=Rotary(inv), **kw)
    with pytest.raises(OkvError):
        norm_rope(torch.zeros(3, 8 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :8 * 64], pos, q, rotary=Rotary(inv), **kw)
