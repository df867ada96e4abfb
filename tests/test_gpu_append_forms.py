"""okv_append_qkv_static in every form of okv_rotary: both orders of pairs, partial and no rotation, with and without
norms, for each group of head sizes and both types."""
import pytest

import tree_ref
from test_gpu_rows import dt_of, make_rotary, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dtype,d,rot", [("bf16", 32, 32), ("bf16", 64, 32), ("bf16", 128, 128), ("bf16", 96, 48), ("bf16", 256, 64),
                                         ("bf16", 160, 0), ("f32", 32, 16), ("f32", 64, 64), ("f32", 128, 64), ("f32", 192, 192)])
def test_forms(dtype, d, rot, inter, norm):
    """Against the plain form, and bit for bit what okv_norm_rope gives at those positions."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static, norm_rope
    gen = torch.Generator().manual_seed(d * 3 + rot)
    dt, R, T, Hq, H, bs, kb = dt_of(dtype), 3, 21, 6, 2, 16, 5
    lengths, counts = [0, 37, 1000], [21, 4, 21]
    sb = torch.full((R, H, kb), -1, dtype=torch.int32)
    for r in range(R):
        ids = torch.arange(lengths[r] // bs, (lengths[r] + T - 1) // bs + 1, dtype=torch.int32)
        for h in range(H):
            sb[r, h, torch.randperm(kb, generator=gen)[:len(ids)]] = ids
    pool = torch.full((R, H, kb, 2, bs, d), -7.0, dtype=dt, device="cuda")
    qkv = torch.randn(R, T, (Hq + 2 * H) * d, generator=gen).to(dt).cuda()
    rope = make_rotary(d, rot, dt, gen, norm, inter)
    q = torch.full((R, T, Hq, d), -7.0, dtype=dt, device="cuda")
    kw = dict(q_heads=Hq, kv_heads=H, head_dim=d, rotary=Rotary(**rope))
    to = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    append_qkv_static(qkv, to(lengths), to(counts), pool, sb.cuda(), q, block_size=bs, slots=kb, **kw)
    want = torch.full_like(pool, -7.0)
    for r in range(R):
        n = counts[r]
        pos = lengths[r] + torch.arange(n, device="cuda")
        wq, wk, wv, bq, bk = tree_ref.rows(qkv[r, :n], pos, Hq, H, d, **rope)
        rows = [torch.empty(n, h, d, dtype=dt, device="cuda") for h in (Hq, H, H)]
        norm_rope(qkv[r, :n], pos.to(torch.int32), *rows, **kw)
        near(rows[0], wq, bq, "q")
        near(rows[1], wk, bk, "key")
        assert torch.equal(rows[2].double(), wv)
        assert torch.equal(q[r, :n], rows[0]) and bool((q[r, n:] == -7.0).all())
        for h in range(H):
            for t in range(n):
                s = int((sb[r, h] == (lengths[r] + t) // bs).nonzero()[0])
                want[r, h, s, 0, (lengths[r] + t) % bs], want[r, h, s, 1, (lengths[r] + t) % bs] = rows[1][t, h], rows[2][t, h]
    assert torch.equal(pool, want)
