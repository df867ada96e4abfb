"""What passes the rows unchanged passes bit for bit."""
import pytest

from test_gpu_rows import dt_of, make_rotary

pytestmark = pytest.mark.gpu


def bits(t):
    import torch
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,d,rot", [("bf16", 128, 0), ("bf16", 128, 64), ("bf16", 96, 32), ("bf16", 256, 16), ("f32", 64, 0),
                                         ("f32", 128, 48), ("f32", 32, 16)])
def test_dims_that_are_not_turned(dtype, d, rot, inter):
    """Without a norm: zeros of both signs, infinities and the smallest numbers among them. With one: a zero keeps the
    sign of its product with the weight, and an infinite weight reaches its own dim alone."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static, norm_rope
    gen = torch.Generator().manual_seed(d + rot)
    dt, n, Hq, H = dt_of(dtype), 9, 6, 2
    x = torch.randn(n, Hq + 2 * H, d, generator=gen).to(dt)
    x[:, :, rot::7], x[:, :, rot + 1::7] = 0.0, -0.0
    x[1, :, rot + 2], x[2, :, rot + 3], x[3, :, -1] = float("inf"), float("-inf"), -torch.finfo(dt).tiny / 2
    x = x.cuda()
    kw = dict(q_heads=Hq, kv_heads=H, head_dim=d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    rope = make_rotary(d, rot, dt, gen, False, inter)
    out = [torch.full((n, h, d), -7.0, dtype=dt, device="cuda") for h in (Hq, H, H)]
    norm_rope(x.view(n, -1), pos, *out, rotary=Rotary(**rope), **kw)
    for o, part in zip(out, (x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:])):
        assert torch.equal(bits(o[..., rot:]), bits(part[..., rot:].contiguous()))
    pool = torch.full((1, H, 1, 2, 16, d), -7.0, dtype=dt, device="cuda")
    q = torch.empty(1, n, Hq, d, dtype=dt, device="cuda")
    append_qkv_static(x.view(1, n, -1), pos[:1], None, pool, torch.zeros(1, H, 1, dtype=torch.int32, device="cuda"), q, block_size=16,
                      slots=1, rotary=Rotary(**rope), **kw)
    for got, want in ((q[0], out[0]), (pool[0, :, 0, 0, :n].transpose(0, 1), out[1]), (pool[0, :, 0, 1, :n].transpose(0, 1), out[2])):
        assert torch.equal(bits(got.contiguous()), bits(want))
    rope = make_rotary(d, rot, dt, gen, True, inter)
    for w in ("q_weight", "k_weight"):
        rope[w][rot::5] *= -1
        rope[w][-1] = float("inf")
    x[1:4] = x[4]
    norm_rope(x.view(n, -1), pos, *out, rotary=Rotary(**rope), **kw)
    for o, part, w in ((out[0], x[:, :Hq], rope["q_weight"]), (out[1], x[:, Hq:Hq + H], rope["k_weight"])):
        plain = part[..., rot:].float() * w[rot:].float()
        got = o[..., rot:].float()
        zero = plain == 0
        assert bool(zero.any()) and torch.equal(got[zero], plain[zero])
        assert torch.equal(got.isinf(), plain.isinf()) and torch.equal(got.isnan(), plain.isnan())
        there = ~plain.isnan()
        assert torch.equal(got.signbit()[there], plain.signbit()[there])
