"""Eviction by accumulated attention weight (okv_evict_static) against the definition, and a run of the calls of a bounded
cache as a decoder makes them."""
import random

import pytest

import chunk_ref

pytestmark = pytest.mark.gpu


def tables(R, H, kb, bs, lengths, rng, fill=1.0):
    """Random slot tables of requests of these lengths: past blocks, some of the next, empty slots, repeated ids."""
    import torch
    sb = torch.full((R, H, kb), -1, dtype=torch.int32)
    for r in range(R):
        nb = -(-max(0, lengths[r]) // bs)
        for h in range(H):
            ids = rng.sample(range(nb + 3), min(kb, nb + 3))
            for i in range(kb):
                if rng.random() < fill:
                    sb[r, h, i] = ids[i % len(ids)] if rng.random() < 0.95 else rng.choice([-1, -9, 2 ** 31 - 1, ids[0]])
    return sb


def weights(shape, rng):
    import torch
    w = torch.tensor([rng.choice([0.0, -0.0, 0.25, 0.5, 0.5, rng.random(), 1e-40, 3.0, -1.0]) for _ in range(int(torch.Size(shape).numel()))])
    for x in (float("inf"), float("nan"), -float("nan"), -float("inf")):
        w[rng.randrange(len(w))] = x
    return w.reshape(shape)


def run(sb, w, ln, counts, **kw):
    import torch
    from sparse_kv_cache_draft_gb300 import evict_static
    R, H, kb = sb.shape
    a, b = torch.full_like(sb, -77), torch.full_like(w, -77.0)
    evict_static(sb, w, ln, counts, a, b, kv_heads=H, slots=kb, **kw)
    return a, b


def check(sb, w, ln, counts, got, **kw):
    import torch
    table, drawn = chunk_ref.evict(sb, w, ln, counts, kw["n_new"], kw["block_size"], kw["sinks"], kw["recent"])
    assert torch.equal(got[0].cpu(), torch.tensor(table, dtype=torch.int32))
    want = torch.tensor(drawn)
    assert torch.equal(torch.isnan(got[1].cpu()), torch.isnan(want)) and torch.equal(got[1].cpu().nan_to_num(0), want.nan_to_num(0))


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("kb,bs,n_new", [(1, 16, 1), (7, 16, 40), (32, 16, 1), (33, 1, 50), (128, 16, 300), (200, 64, 5000), (256, 3, 1000), (511, 24, 900),
                                        (1024, 16, 1000), (1000, 1, 3000)])
def test_against_the_definition(kb, bs, n_new, seed):
    import torch
    rng = random.Random(kb * 10 + seed)
    R, H = rng.choice([1, 3, 9]), rng.choice([1, 2, 5])
    lengths = [rng.choice([0, 1, bs, bs + 1, kb * bs - 1, kb * bs, rng.randrange(4 * kb * bs + 1)]) for _ in range(R)]
    counts = None if seed == 0 else torch.tensor([rng.choice([0, 1, n_new, n_new + 5, -1, rng.randrange(n_new + 1)]) for _ in range(R)], dtype=torch.int32, device="cuda")
    sb, w = tables(R, H, kb, bs, lengths, rng, fill=rng.choice([0.0, 0.8, 1.0])).cuda(), weights((R, H, kb), rng).cuda()
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kw = dict(n_new=n_new, block_size=bs, sinks=rng.choice([0, 1, bs, 5 * bs]), recent=rng.choice([0, 1, bs, 3 * bs + 1, 2 ** 31 - 1 if seed == 3 else 9]))
    got = run(sb, w, ln, counts, **kw)
    check(sb, w, ln, counts, got, **kw)
    # in place
    from sparse_kv_cache_draft_gb300 import evict_static
    a, b = sb.clone(), w.clone()
    evict_static(a, b, ln, counts, kv_heads=H, slots=kb, **kw)
    assert torch.equal(a, got[0]) and torch.equal(b.view(torch.int32), got[1].view(torch.int32))


def test_ties_ends_and_left_out_requests():
    """Equal weights go by index; positions next to 2^31 - 1; requests without room for positions stay as they are."""
    import torch
    kb, bs, n_new = 40, 16, 100
    top = 2 ** 31 - 1
    lengths = [640, 640, top - n_new, top - n_new + 1, -5, -2 ** 31]
    rng = random.Random(5)
    sb = torch.arange(kb, dtype=torch.int32).repeat(6, 1, 1)
    sb[2] = torch.arange((top - n_new) // bs - kb + 1, (top - n_new) // bs + 1, dtype=torch.int64).to(torch.int32)
    sb, w = sb.cuda(), torch.ones(6, 1, kb, device="cuda")
    w[1, 0] = torch.tensor([rng.choice([1.0, 2.0]) for _ in range(kb)])
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kw = dict(n_new=n_new, block_size=bs, sinks=20, recent=40)
    got = run(sb, w, ln, None, **kw)
    check(sb, w, ln, None, got, **kw)
    assert got[0][0, 0, :12].tolist() == [0, 1] + list(range(40, 47)) + [9, 10, 11]
    assert torch.equal(got[0][3:], sb[3:])


def test_captured():
    import torch
    from sparse_kv_cache_draft_gb300 import evict_static
    rng = random.Random(1)
    sb, w = tables(4, 2, 64, 16, [900] * 4, rng).cuda(), weights((4, 2, 64), rng).cuda()
    ln = torch.full((4,), 900, dtype=torch.int32, device="cuda")
    kw = dict(n_new=70, block_size=16, sinks=16, recent=32)
    a, b = torch.zeros_like(sb), torch.zeros_like(w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        evict_static(sb, w, ln, None, a, b, kv_heads=2, slots=64, **kw)
    ln.add_(333)
    g.replay()
    torch.cuda.synchronize()
    check(sb, w, ln, None, (a, b), **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_run_of_steps(dtype):
    """A prompt in chunks, then single tokens, through a pool of fewer slots than the request has blocks: room, append, attention
    with weights; each call against its plain form on the same inputs, the pool against the tokens."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static, attend_chunk_static, evict_static
    R, Hq, H, d, bs, kb = 3, 8, 2, 64, 16, 12
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator(device="cuda").manual_seed(3)
    inv = (1e4 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)).float()
    rot = Rotary(inv)
    pool = torch.full((R, H, kb, 2, bs, d), float("nan"), dtype=dt, device="cuda")
    sb = torch.full((R, H, kb), -1, dtype=torch.int32, device="cuda")
    w, ln = torch.zeros(R, H, kb, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    kw = dict(kv_heads=H, block_size=bs, slots=kb)
    for T, counts in [(70, [70, 33, 0]), (70, [70, 70, 5]), (70, [1, 70, 70]), (1, None), (1, [1, 0, 1]), (1, None), (40, [40, 17, 16]), (1, None)]:
        cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        qkv = torch.randn(R, T, (Hq + 2 * H) * d, generator=gen, device="cuda").to(dt)
        table = chunk_ref.evict(sb, w, ln, cnt, T, bs, 4, 20)
        evict_static(sb, w, ln, cnt, n_new=T, sinks=4, recent=20, **kw)
        assert sb.tolist() == table[0] and w.tolist() == table[1]
        q, out = torch.zeros(R, T, Hq, d, dtype=dt, device="cuda"), torch.full((R, T, Hq, d), -7.0, dtype=dt, device="cuda")
        lse, before = torch.full((R, T, Hq), -7.0, device="cuda"), w.clone()
        append_qkv_static(qkv, ln, cnt, pool, sb, q, q_heads=Hq, head_dim=d, rotary=rot, **kw)
        attend_chunk_static(pool, sb, ln, cnt, q, out, lse, w, q_heads=Hq, head_dim=d, window=100, sinks=4, **kw)
        from test_gpu_chunk import check as check_chunk
        check_chunk(dict(pool=pool, slot_block=sb, lengths=ln, counts=cnt, q=q, window=100, sinks=4, weight=before), (out, lse, w))
        ln += T if cnt is None else cnt
    assert ln.tolist() == [185, 193, 95]
