"""Accepted paths through a context (okv_append_tree) against their definition: every place that holds a token is
compared bit for bit with the drafted vectors put there one after another."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


class Rig:
    """A context of seeded requests {id: tokens}; those in `partial` keep every block they fetch. Everything fits the
    budget, so a staging makes every block resident (and kept)."""

    def __init__(self, dtype, Hq, H, d, lengths, partial=(), R=None, layers=2, bs=16, kb=24, cap=40):
        import torch
        from sparse_kv_cache_draft_gb300 import BF16, F32, Config, Context, HostBuffer
        self.R, self.layers, self.H, self.d, self.bs, self.kb, self.cap = R or max(lengths) + 1, layers, H, d, bs, kb, cap
        self.dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.st = np.float32 if dtype == "f32" else np.uint16
        cfg = Config(layers, Hq, H, d, bs, kb * bs, self.R, cap, 1.0, BF16 if dtype == "bf16" else F32)
        self.ctx = Context(cfg)
        self.gen = torch.Generator().manual_seed(50)
        self.partial, self.buf, self.tier, self.want = tuple(partial), {}, {}, {}
        shape = (layers, H, cap, 2, bs, d)
        for r, n in lengths.items():
            self.buf[r] = HostBuffer(cfg.host_bytes(cap))
            x = torch.randn(cfg.host_bytes(cap) // cfg.elem_bytes, generator=self.gen).to(self.dt)
            self.buf[r].numpy(np.uint8)[:] = x.view(torch.uint8).numpy()
            self.want[r] = self.buf[r].numpy(self.st, shape).copy()
            if r in self.partial:
                self.tier[r] = HostBuffer(cfg.host_bytes(cap))
                self.tier[r].numpy(np.uint8)[:] = 0
                self.ctx.add_request_partial(r, self.buf[r].ptr, cap, self.tier[r].ptr, cap, n)
            else:
                self.ctx.add_request(r, self.buf[r].ptr, cap, n)
        self.length = {layer: dict(lengths) for layer in range(layers)}
        self.draft = torch.randn(layers, self.R, Hq, d, generator=self.gen).to(self.dt).cuda()

    def drafted(self, T):
        import torch
        return [torch.randn(self.R, T, self.H, self.d, generator=self.gen).to(self.dt).cuda() for _ in range(2)]

    def bits(self, t):
        import torch
        return t.cpu().view(torch.int16 if self.st == np.uint16 else torch.int32).numpy().view(self.st)

    def expect(self, layer, k, v, paths):
        """Puts the paths into the wanted host buffers."""
        k, v = self.bits(k), self.bits(v)
        for r, path in paths.items():
            for j in path:
                b, t = divmod(self.length[layer][r], self.bs)
                self.want[r][layer, :, b, 0, t], self.want[r][layer, :, b, 1, t] = k[r, j], v[r, j]
                self.length[layer][r] += 1

    def floats(self, x):
        return x if self.st == np.float32 else (x.astype(np.uint32) << 16).view(np.float32)

    def check(self, layer, kept=None):
        """Lengths, host buffers, summaries, resident and kept copies. kept: the least number of kept blocks."""
        import torch
        torch.cuda.synchronize()
        assert self.ctx.sync(60_000) == 0
        live = self.ctx.read_lengths(layer)
        sb, _ = self.ctx.read_slot_table(layer)
        _, local_of, _ = self.ctx.read_local(layer)
        for r, n in self.length[layer].items():
            assert live[r] == n, (layer, r)
            want = self.want[r][layer]
            assert np.array_equal(self.buf[r].numpy(self.st, (self.layers,) + want.shape)[layer], want), (layer, r)
            x, nb = self.floats(want[:, :, 0]), -(-n // self.bs)
            got = self.floats(self.ctx.read_summaries(layer, r).view(self.st))
            for b in range(nb):
                t = min(self.bs, n - b * self.bs)
                assert np.array_equal(got[:, b, 0], x[:, b, :t].min(1)) and np.array_equal(got[:, b, 1], x[:, b, :t].max(1)), (layer, r, b)
            held = 0
            for h in range(self.H):
                pool = self.ctx.read_pool(layer, r, h).view(self.st)
                for s in np.nonzero(sb[r, h] >= 0)[0]:
                    b = sb[r, h, s]
                    t = min(self.bs, n - b * self.bs)
                    assert np.array_equal(pool[s, :, :t], want[h, b, :, :t]), (layer, r, h, b)
                if r in self.partial:
                    tier = self.tier[r].numpy(self.st, (self.layers,) + want.shape)[layer]
                    for b in np.nonzero(local_of[r, h, :nb] >= 0)[0]:
                        t = min(self.bs, n - b * self.bs)
                        assert np.array_equal(tier[h, local_of[r, h, b], :, :t], want[h, b, :, :t]), (layer, r, h, b)
                        held += 1
            assert r not in self.partial or kept is None or held >= kept * self.H

    def close(self):
        self.ctx.close()
        for b in [*self.buf.values(), *self.tier.values()]:
            b.free()


def path(n, T, step=7):
    """n drafted tokens of T in no particular order, some of them twice where n is past T."""
    return [(5 + step * i) % T for i in range(n)]


def test_paths_of_layers_behind_a_long_kernel():
    """Calls of different paths, layers and streams queued behind work that has not ended, with nothing in between
    that waits: each appends its own path."""
    import torch
    a = Rig("bf16", 8, 2, 128, {0: 300, 1: 333, 3: 2})
    try:
        T = 40
        drafts = [a.drafted(T) for _ in range(2)]
        other = torch.cuda.Stream()
        a.ctx.append_tree(0, *drafts[0], {3: [1]})  # the kernel is loaded before the others
        a.expect(0, *drafts[0], {3: [1]})
        calls = [(0, drafts[0], {0: path(5, T), 1: path(30, T, 3), 3: path(17, T)}, None),
                 (1, drafts[0], {0: path(40, T), 1: path(2, T), 3: path(1, T)}, other),
                 (0, drafts[1], {0: path(1, T, 11), 1: path(13, T, 9)}, None),
                 (1, drafts[1], {1: path(24, T, 3), 3: path(40, T, 13)}, other),
                 (0, drafts[0], {3: path(33, T, 11)}, None)]
        torch.cuda.synchronize()
        busy, done = torch.randn(4096, 4096, device="cuda"), torch.cuda.Event()
        for st in (torch.cuda.current_stream(), other):
            with torch.cuda.stream(st):
                y = busy
                for _ in range(200):
                    y = busy @ y
        done.record()
        for layer, (k, v), paths, st in calls:
            a.ctx.append_tree(layer, k, v, paths, stream=st)
        assert not done.query(), "the calls did not return ahead of the work before them"
        for layer, (k, v), paths, _ in calls:
            a.expect(layer, k, v, paths)
        for layer in range(a.layers):
            a.check(layer)
        del y
    finally:
        a.close()


def test_paths_of_more_requests_than_one_launch_takes():
    """60 requests whose paths of up to 64 tokens pass one launch's parameters."""
    import torch
    a = Rig("f32", 2, 1, 32, {r: 1 + r % 18 for r in range(1, 70) if r % 7}, layers=1, kb=4, cap=16)
    try:
        assert len(a.length[0]) * 65 > 3584
        a.ctx.set_timing(True)
        k, v = a.drafted(64)
        paths = {r: path((r * 5) % 65, 64, 5) for r in a.length[0]}
        paths[69] = path(64, 64, 5)
        a.ctx.append_tree(0, k, v, paths)
        a.expect(0, k, v, paths)
        a.check(0)
        assert a.ctx.read_timing()["launches"]["append"] == 2
        paths = {r: p[:2] for r, p in paths.items()}
        a.ctx.append_tree(0, k, v, paths)
        a.expect(0, k, v, paths)
        a.check(0)
        assert a.ctx.read_timing()["launches"]["append"] == 3
    finally:
        a.close()


@pytest.mark.parametrize("dtype,Hq,H,d,bs", [("bf16", 8, 2, 128, 16), ("f32", 4, 2, 64, 16), ("bf16", 3, 1, 96, 5), ("bf16", 8, 1, 256, 64),
                                             ("f32", 2, 2, 32, 1)])
def test_paths_across_blocks_and_into_kept_copies(dtype, Hq, H, d, bs):
    """Paths that end inside a resident (and, for request 1, kept) block, that cross one block boundary and several, and
    that start a new block; stagings in between bring the new blocks in."""
    kb = 24 if bs > 5 else 100
    n = 15 * bs
    a = Rig(dtype, Hq, H, d, {0: n + bs // 2, 1: n + bs - 1 if bs > 1 else n, 3: 1}, partial=(1,), R=5, bs=bs, kb=kb, cap=kb)
    try:
        T = 40
        for layer in range(a.layers):
            a.ctx.stage(layer, a.draft[layer], 0)
            a.check(layer, kept=16 if bs > 1 else 15)
        plans = [{0: 3, 1: 1, 3: 4}, {0: 0, 1: 37, 3: 20}, {0: 18, 1: 9, 3: 0}] if bs > 1 else [{0: 3, 1: 20, 3: 4}, {0: 0, 1: 9, 3: 20}]
        for step, plan in enumerate(plans):
            for layer in range(a.layers):
                k, v = a.drafted(T)
                paths = {r: path(m, T, 3 + 4 * layer + 2 * step) for r, m in plan.items() if m}
                a.ctx.append_tree(layer, k, v, paths)
                a.expect(layer, k, v, paths)
                a.check(layer)
            for layer in range(a.layers):
                a.ctx.stage(layer, a.draft[layer], step + 1)
                nb = -(-a.length[layer][1] // bs)
                a.check(layer, kept=nb)
                assert all(int((a.ctx.read_slot_table(layer)[0][1, h] >= 0).sum()) == nb for h in range(H))
    finally:
        a.close()


@pytest.mark.parametrize("dtype,Hq,H,d", [("bf16", 8, 2, 128), ("f32", 4, 2, 64)])
def test_a_path_is_one_token_after_another(dtype, Hq, H, d):
    """The same state, bit for bit, as that of okv_append for each token of the paths; staging, attention and the next
    paths run on from there."""
    import torch
    a, b = (Rig(dtype, Hq, H, d, {0: 300, 1: 333, 3: 2}, partial=(1,), R=5, kb=12) for _ in range(2))
    try:
        T = 40
        for x in (a, b):
            for layer in range(x.layers):
                x.ctx.stage(layer, x.draft[layer], 0)
        for step, m in enumerate((37, 1, 16)):
            for layer in range(a.layers):
                k, v = a.drafted(T)
                paths = {r: path(m, T, 3 + 2 * r) for r in a.length[layer]}
                a.ctx.append_tree(layer, k, v, paths)
                for i in range(m):
                    pick = torch.tensor([paths[r][i] if r in paths else 0 for r in range(a.R)], device="cuda")
                    at = torch.arange(a.R, device="cuda")
                    b.ctx.append(layer, k[at, pick].contiguous(), v[at, pick].contiguous())
                for x in (a, b):
                    x.expect(layer, k, v, paths)
                    x.check(layer)
                q = torch.randn(a.R, Hq, d, generator=a.gen).to(a.dt).cuda()
                out = [torch.zeros_like(q) for _ in range(2)]
                for x, o in zip((a, b), out):
                    x.ctx.stage(layer, x.draft[layer], step + 1, 0.25)
                    x.ctx.attend(layer, q, o)
                torch.cuda.synchronize()
                assert torch.equal(*out)
                for f in ("read_slot_table", "read_local", "read_selection", "read_fetch_list"):
                    got, want = getattr(a.ctx, f)(layer), getattr(b.ctx, f)(layer)
                    live = sorted(a.length[layer])
                    if f == "read_local":
                        live, got, want = [1], got[:2], want[:2]
                    if f in ("read_selection", "read_fetch_list"):
                        got, want = got[:1], want[:1]
                    assert all(np.array_equal(x[live], y[live]) for x, y in zip(got, want)), f
    finally:
        a.close()
        b.close()
