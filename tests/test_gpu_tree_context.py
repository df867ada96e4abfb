"""Drafted trees and projection rows through a context: the steps a decoder with a drafter takes,
against a twin context that appends one ready token at a time, and against the plain forms."""
import numpy as np
import pytest

import tree_ref

pytestmark = pytest.mark.gpu

R, LAYERS, BS, KB, CAP = 5, 2, 16, 12, 40
SHAPES = [("bf16", 8, 2, 128), ("f32", 4, 2, 64), ("bf16", 3, 1, 96)]


class Twin:
    """A context over its own copy of seeded host buffers: requests 0, 1 (partially staged) and 3 of
    300, 333 and 2 tokens; 2 and 4 are inactive."""

    lengths = {0: 300, 1: 333, 3: 2}

    def __init__(self, dtype, Hq, H, d, stage=True):
        import torch
        from sparse_kv_cache_draft_gb300 import BF16, F32, Config, Context, HostBuffer
        self.dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.cfg = Config(LAYERS, Hq, H, d, BS, KB * BS, R, CAP, 0.25, BF16 if dtype == "bf16" else F32)
        self.ctx = Context(self.cfg)
        self.bufs = {}
        gen = torch.Generator().manual_seed(20)
        n = self.cfg.host_bytes(CAP) // self.cfg.elem_bytes
        for r in self.lengths:
            self.bufs[r] = HostBuffer(self.cfg.host_bytes(CAP))
            x = torch.randn(n, generator=gen).to(self.dt)
            self.bufs[r].numpy(np.uint8)[:] = x.view(torch.uint8).numpy()
        self.tier = HostBuffer(self.cfg.host_bytes(8))
        self.tier.numpy(np.uint8)[:] = 0
        self.ctx.add_request(0, self.bufs[0].ptr, CAP, 300)
        self.ctx.add_request_partial(1, self.bufs[1].ptr, CAP, self.tier.ptr, 8, 333)
        self.ctx.add_request(3, self.bufs[3].ptr, CAP, 2)
        self.draft = torch.randn(LAYERS, R, Hq, d, generator=gen).to(self.dt).cuda()
        if stage:
            for layer in range(LAYERS):
                self.ctx.stage(layer, self.draft[layer], 0, 1.0)

    def state(self, layer):
        import torch
        torch.cuda.synchronize()
        c = self.ctx
        got = [c.read_lengths(layer), *c.read_slot_table(layer), *c.read_local(layer)[:1]]
        live = c.read_lengths(layer)
        for r in self.lengths:
            nb = -(-int(live[r]) // BS)
            got.append(c.read_summaries(layer, r)[:, :nb])
            sb = got[1][r]
            for h in range(self.cfg.kv_heads):
                got.append(c.read_pool(layer, r, h)[sb[h] >= 0])
        return got

    def host(self):
        return [self.bufs[r].numpy().copy() for r in self.lengths] + [self.tier.numpy().copy()]

    def pool(self, layer):
        import torch
        c = self.cfg
        x = np.stack([np.stack([self.ctx.read_pool(layer, r, h) for h in range(c.kv_heads)]) for r in range(R)])
        return torch.from_numpy(x if self.dt == torch.float32 else x.view(np.int16)).view(self.dt).cuda()

    def close(self):
        self.ctx.close()
        for b in self.bufs.values():
            b.free()
        self.tier.free()


def same(a, b):
    return all(np.array_equal(x, y) for x, y in zip(a, b)) and len(a) == len(b)


@pytest.mark.parametrize("dtype,Hq,H,d", SHAPES)
def test_draft_verify_accept_and_go_on(dtype, Hq, H, d):
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    T = 6
    a, b = Twin(dtype, Hq, H, d), Twin(dtype, Hq, H, d)
    try:
        gen = torch.Generator().manual_seed(30)
        dt = a.dt
        inv = (1e6 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
        rot = Rotary(inv, *(1 + 0.2 * torch.randn(2, d, generator=gen)).to(dt).cuda())
        kw = dict(q_heads=Hq, kv_heads=H, head_dim=d, rotary=rot)
        parent = [-1, 0, 0, 1, 3, 2]
        mask, depth = [0] * T, [0] * T
        for t, p in enumerate(parent):
            mask[t] = 1 << t | (mask[p] if p >= 0 else 0)
            depth[t] = depth[p] + 1 if p >= 0 else 0
        mask = torch.tensor([mask] * R, dtype=torch.int64, device="cuda")
        counts = torch.tensor([6, 4, 0, 6, 0], dtype=torch.int32, device="cuda")
        accepted = {0: [0, 2, 5], 1: [], 3: [0, 1, 3, 4]}
        for layer in range(LAYERS):
            # the drafted tree: rows -> queries, keys, values -> attention
            qkv = torch.randn(R, T, (Hq + 2 * H) * d, generator=gen).to(dt).cuda()
            start = torch.from_numpy(a.ctx.read_lengths(layer)).cuda()
            pos = (start[:, None] + torch.tensor(depth, device="cuda")).to(torch.int32)
            q = torch.empty(R, T, Hq, d, dtype=dt, device="cuda")
            k, v = (torch.empty(R, T, H, d, dtype=dt, device="cuda") for _ in range(2))
            norm_rope(qkv.flatten(0, 1), pos.flatten(), q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), **kw)
            out = torch.full_like(q, -7.0)
            a.ctx.attend_tree(layer, q, k, v, mask, out, counts=counts)
            torch.cuda.synchronize()
            sb, _ = a.ctx.read_slot_table(layer)
            live = torch.tensor([1 if r in a.lengths else 0 for r in range(R)], device="cuda", dtype=torch.int32)
            cnt = counts * live
            want, bound = tree_ref.attend(a.pool(layer), torch.from_numpy(sb).cuda(), start, cnt, q, k, v, mask)
            fresh = torch.arange(T, device="cuda") < cnt[:, None]
            assert float(((out.double() - want).abs() - bound)[fresh].max()) <= 0
            assert bool((out[~fresh] == -7.0).all())
            # the accepted paths, against one ready token after another in the twin: requests that
            # append fewer are taken out of the twin's batch by appending the others alone
            a.ctx.append_tree(layer, k, v, accepted)
            one = [Twin(dtype, Hq, H, d, stage=False)]  # not staged: host, summaries and lengths alone
            try:
                for r in (0, 3):
                    only = one[0]
                    for other in [x for x in only.lengths if x != r]:
                        if int(only.ctx.read_lengths(layer)[other]):
                            only.ctx.remove_request(other)
                    for t in accepted[r]:
                        only.ctx.append(layer, k[:, t].contiguous(), v[:, t].contiguous())
                    torch.cuda.synchronize()
                    n = int(only.ctx.read_lengths(layer)[r])
                    assert n == a.lengths[r] + len(accepted[r]) == int(a.ctx.read_lengths(layer)[r])
                    nb = -(-n // BS)
                    assert np.array_equal(a.ctx.read_summaries(layer, r)[:, :nb], only.ctx.read_summaries(layer, r)[:, :nb])
                    shape = (LAYERS, H, CAP, 2, BS, d)
                    st = np.float32 if dtype == "f32" else np.uint16
                    assert np.array_equal(a.bufs[r].numpy(st, shape)[layer], only.bufs[r].numpy(st, shape)[layer])
                    if r == 0:
                        only.ctx.remove_request(0)
                        only.close()
                        one[0] = Twin(dtype, Hq, H, d, stage=False)
            finally:
                one[0].close()
            assert int(a.ctx.read_lengths(layer)[1]) == 333
            # resident copies of the blocks appended to are those of the host
            sb, _ = a.ctx.read_slot_table(layer)
            for r in a.lengths:
                n = int(a.ctx.read_lengths(layer)[r])
                st = np.float32 if dtype == "f32" else np.uint16
                host = a.bufs[r].numpy(st, (LAYERS, H, CAP, 2, BS, d))[layer]
                for h in range(H):
                    pool = a.ctx.read_pool(layer, r, h)
                    for s in range(KB):
                        blk = int(sb[r, h, s])
                        if blk >= 0:
                            nv = min(BS, n - blk * BS)
                            assert np.array_equal(pool[s, :, :nv], host[h, blk, :, :nv])
            # and the next staging and attention run on what was appended
            a.ctx.stage(layer, a.draft[layer], 1)
            o = torch.zeros(R, Hq, d, dtype=dt, device="cuda")
            a.ctx.attend(layer, q[:, 0].contiguous(), o)
            torch.cuda.synchronize()
            assert a.ctx.sync(60_000) == 0
            assert bool(torch.isfinite(o.float()).all())
    finally:
        a.close()
        b.close()


@pytest.mark.parametrize("dtype,Hq,H,d", SHAPES)
def test_append_qkv_is_norm_rope_and_append(dtype, Hq, H, d):
    """Bit for bit: queries, lengths, slot tables, summaries, pools and host buffers, over enough steps
    to open new blocks; attention and staging of both contexts agree afterwards."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    a, b = Twin(dtype, Hq, H, d), Twin(dtype, Hq, H, d)
    try:
        gen = torch.Generator().manual_seed(40)
        dt = a.dt
        inv = (1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
        rot = Rotary(inv, *(1 + 0.2 * torch.randn(2, d, generator=gen)).to(dt).cuda(), interleaved=d == 96)
        for step in range(18):
            for layer in range(LAYERS):
                qkv = torch.randn(R, (Hq + 2 * H) * d + 8, generator=gen).to(dt).cuda()[:, :(Hq + 2 * H) * d]
                pos = torch.from_numpy(b.ctx.read_lengths(layer)).cuda()
                live = torch.tensor([r in a.lengths for r in range(R)], device="cuda")
                q1 = torch.full((R, Hq, d), -7.0, dtype=dt, device="cuda")
                q2 = torch.full_like(q1, -7.0)
                a.ctx.append_qkv(layer, qkv, q1, rot)
                k, v = (torch.zeros(R, H, d, dtype=dt, device="cuda") for _ in range(2))
                norm_rope(qkv, torch.where(live, pos, -1).to(torch.int32), q2, k, v, q_heads=Hq, kv_heads=H, head_dim=d, rotary=rot)
                b.ctx.append(layer, k, v)
                assert torch.equal(q1, q2)
                if step % 6 == 5:
                    for x in (a, b):
                        x.ctx.stage(layer, x.draft[layer], step)
                    o1, o2 = torch.zeros_like(q1), torch.zeros_like(q1)
                    a.ctx.attend(layer, q1, o1)
                    b.ctx.attend(layer, q2, o2)
                    torch.cuda.synchronize()
                    assert torch.equal(o1, o2)
        for layer in range(LAYERS):
            assert same(a.state(layer), b.state(layer))
        assert same(a.host(), b.host())
        assert int(a.ctx.read_lengths(0)[3]) == 20
        assert a.ctx.sync(60_000) == 0 and b.ctx.sync(60_000) == 0
    finally:
        a.close()
        b.close()


def test_refusals():
    import torch
    from sparse_kv_cache_draft_gb300 import OkvError, Rotary, binding
    a = Twin("bf16", 8, 2, 128)
    try:
        T = 4
        q = torch.zeros(R, T, 8, 128, dtype=torch.bfloat16, device="cuda")
        k = torch.zeros(R, T, 2, 128, dtype=torch.bfloat16, device="cuda")
        mask = torch.ones(R, T, dtype=torch.int64, device="cuda")
        out = torch.empty_like(q)
        qkv = torch.zeros(R, 12 * 128, dtype=torch.bfloat16, device="cuda")
        row = torch.zeros(R, 8, 128, dtype=torch.bfloat16, device="cuda")

        def refused(status, f, *args, **kw):
            with pytest.raises(OkvError) as e:
                f(*args, **kw)
            assert e.value.status == status, e.value

        refused(binding.EINVAL, a.ctx.attend_tree, LAYERS, q, k, k, mask, out)
        refused(binding.EINVAL, a.ctx.append_tree, -1, k, k, {0: [0]})
        refused(binding.EINVAL, a.ctx.append_tree, 0, k, k, {0: [4]})
        refused(binding.EINVAL, a.ctx.append_tree, 0, k, k, {0: [-1]})
        refused(binding.EINVAL, a.ctx.append_qkv, LAYERS, qkv, row, Rotary())
        with pytest.raises(ValueError):
            a.ctx.append_tree(0, k, k, {0: [0] * 5})
        with pytest.raises(ValueError):
            a.ctx.append_tree(0, k, k, {R: [0]})
        with pytest.raises(ValueError):
            a.ctx.append_qkv(0, qkv[:, :-8], row, Rotary())
        big = torch.zeros(R, 65, 8, 128, dtype=torch.bfloat16, device="cuda")
        bk = torch.zeros(R, 65, 2, 128, dtype=torch.bfloat16, device="cuda")
        refused(binding.EINVAL, a.ctx.attend_tree, 0, big, bk, bk, torch.ones(R, 65, dtype=torch.int64, device="cuda"), big.clone())
        # a request without room for all of its tokens refuses the call, and nothing is appended
        a.ctx.remove_request(3)
        a.ctx.add_request(3, a.bufs[3].ptr, CAP, CAP * BS - 2)
        torch.cuda.synchronize()
        before = a.ctx.read_lengths(0).copy()
        refused(binding.EINVAL, a.ctx.append_tree, 0, k, k, {0: [0], 3: [0, 1, 2]})
        assert np.array_equal(before, a.ctx.read_lengths(0))
        a.ctx.append_tree(0, k, k, {3: [0, 1]})
        refused(binding.EINVAL, a.ctx.append_qkv, 0, qkv, row, Rotary())
        a.ctx.append_tree(0, k, k, {0: [0], 3: []})  # a full request that appends nothing is no hindrance
        torch.cuda.synchronize()
        assert a.ctx.read_lengths(0)[0] == before[0] + 1
        # captures
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            refused(binding.ESTATE, a.ctx.append_qkv, 1, qkv, row, Rotary())
            refused(binding.ESTATE, a.ctx.append_tree, 1, k, k, {0: [0]})
            refused(binding.ESTATE, a.ctx.attend_tree, 0, q, k, k, mask, out)
            out.zero_()
        # no request at all: nothing to do
        for r in list(a.lengths):
            a.ctx.remove_request(r)
        a.ctx.attend_tree(0, q, k, k, mask, out)
        a.ctx.append_qkv(0, qkv, row, Rotary())
        a.ctx.append_tree(0, k, k, {})
        assert a.ctx.sync(60_000) == 0
    finally:
        a.close()


def test_timing_counts_the_launches():
    import torch
    a = Twin("bf16", 8, 2, 128)
    try:
        a.ctx.set_timing(True)
        q = torch.zeros(R, 3, 8, 128, dtype=torch.bfloat16, device="cuda")
        k = torch.zeros(R, 3, 2, 128, dtype=torch.bfloat16, device="cuda")
        a.ctx.attend_tree(0, q, k, k, torch.ones(R, 3, dtype=torch.int64, device="cuda"), torch.empty_like(q))
        a.ctx.append_tree(0, k, k, {0: [0, 1]})
        torch.cuda.synchronize()
        t = a.ctx.read_timing()
        assert t["launches"]["attend"] == 1 and t["launches"]["append"] == 1
        sb, _ = a.ctx.read_slot_table(0)
        live = sorted(a.lengths)
        assert t["attended_slots"] == int((sb[live] >= 0).sum())
    finally:
        a.close()
