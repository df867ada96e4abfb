"""Chunks over a paged pool in the company of other calls: behind one another, from several threads, after other kernels, and
over tables that no step of a decoder makes."""
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_gpu_chunk import call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,dtype,d,bs", [(1, "bf16", 128, 16), (3, "bf16", 64, 8), (100, "bf16", 128, 16), (20, "f32", 64, 16), (2, "bf16", 128, 12)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 5)])
def test_the_same_block_in_many_slots(T, dtype, d, bs, window, sinks):
    """Every slot counts, as in attention without a window: a table may hold a block more often than a window has blocks."""
    import torch
    kb = 120
    x = make(2, T, 8, 2, d, bs, kb, dtype, seed=31, lengths=[5 * bs, 200 * bs], holes=False, stale=0.0)
    x["slot_block"][0] = torch.arange(kb, dtype=torch.int32) % 2 + 4  # the last blocks of the first request
    x["slot_block"][1] = (200 * bs) // bs - 1
    gen = torch.Generator().manual_seed(3)
    x["pool"][:] = torch.randn(x["pool"].shape, generator=gen).to(x["pool"])
    x.update(window=window, sinks=sinks)
    check(x, call(x))


@pytest.mark.parametrize("T,dtype,d", [(3, "bf16", 128), (30, "bf16", 64), (90, "bf16", 128), (70, "bf16", 256), (90, "bf16", 96), (3, "f32", 64), (60, "f32", 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 6)])
def test_rows_past_a_count_may_hold_anything(T, dtype, d, window, sinks):
    """Queries of rows from a request's count on are no part of any other row, nor of what slots draw."""
    x = make(4, T, 6, 2, d, 16, 30, dtype, seed=51, lengths=[300, 17, 400, 0], counts=[T - 2, 1, 0, T - 1])
    x.update(window=window, sinks=sinks)
    for r, c in enumerate((T - 2, 1, 0, T - 1)):
        x["q"][r, c:, 0::2] = float("nan")
        x["q"][r, c:, 1::2] = float("inf")
    check(x, call(x))


def test_calls_behind_one_another():
    """Steps that feed one another without a wait between them give what the same steps give one at a time: room, rows,
    attention with weights in place, of every kind of kernel."""
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static, attend_chunk_static, evict_static

    def steps(wait):
        outs = []
        gen = torch.Generator(device="cuda").manual_seed(1)
        for dt, d in ((torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)):
            R, Hq, H, bs, kb = 5, 8, 2, 16, 24
            rot = Rotary((1e4 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)).float())
            pool = torch.zeros(R, H, kb, 2, bs, d, dtype=dt, device="cuda")
            sb = torch.full((R, H, kb), -1, dtype=torch.int32, device="cuda")
            w, ln = torch.zeros(R, H, kb, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
            kw = dict(kv_heads=H, block_size=bs, slots=kb)
            for T in (90, 1, 1, 200, 7, 1, 64, 1, 33):
                qkv = torch.randn(R, T, (Hq + 2 * H) * d, generator=gen, device="cuda").to(dt)
                q, out = (torch.empty(R, T, Hq, d, dtype=dt, device="cuda") for _ in range(2))
                lse = torch.empty(R, T, Hq, device="cuda")
                torch.cuda.synchronize()
                for f in (lambda: evict_static(sb, w, ln, None, n_new=T, sinks=4, recent=40, **kw),
                          lambda: append_qkv_static(qkv, ln, None, pool, sb, q, q_heads=Hq, head_dim=d, rotary=rot, **kw),
                          lambda: attend_chunk_static(pool, sb, ln, None, q, out, lse, w, q_heads=Hq, head_dim=d, window=150, sinks=4, **kw),
                          lambda: attend_chunk_static(pool, sb, ln, None, out, q, lse, w, q_heads=Hq, head_dim=d, **kw)):
                    f()
                    if wait:
                        torch.cuda.synchronize()
                ln += T
                outs += [out, q, lse, w.clone(), sb.clone()]
        return outs

    a, b = steps(True), steps(False)
    torch.cuda.synchronize()
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_every_call_of_every_thread_gives_its_result():
    import torch
    shapes = [(1, 8, 32, 8, 128, 16, 40, "bf16"), (2, 64, 16, 2, 128, 16, 20, "bf16"), (3, 5, 8, 2, 64, 32, 9, "f32"), (2, 9, 4, 2, 256, 16, 30, "bf16"),
              (2, 20, 8, 2, 96, 16, 12, "f32"), (40, 1, 8, 8, 64, 16, 6, "bf16")]
    xs = [make(*s, seed=70 + i) for i, s in enumerate(shapes)]
    want = [call(x) for x in xs]
    torch.cuda.synchronize()

    def work(i):
        st, same = torch.cuda.Stream(), 0
        with torch.cuda.stream(st):
            for _ in range(25):
                got = call(xs[i])
                st.synchronize()
                same += all(torch.equal(a, b) for a, b in zip(got, want[i]))
        return same

    with ThreadPoolExecutor(len(xs)) as ex:
        assert list(ex.map(work, range(len(xs)))) == [25] * len(xs)


@pytest.mark.parametrize("shape", [(40, 1, 8, 8, 64, 16, 6, "bf16"), (1, 1, 8, 8, 128, 16, 128, "bf16"), (3, 43, 18, 3, 128, 16, 19, "bf16"),
                                   (2, 70, 8, 1, 64, 24, 20, "bf16"), (2, 7, 4, 2, 256, 16, 30, "bf16"), (2, 50, 6, 2, 96, 7, 40, "bf16"), (5, 9, 6, 2, 64, 16, 20, "f32")],
                         ids=str)
def test_what_shared_memory_held_before_has_no_part(shape):
    import torch
    x = make(*shape, seed=80)
    x.update(window=100, sinks=3)
    want = call(x)
    for i, (s, size) in enumerate([((40, 16, 32, 8, 128, 16, 16, "bf16"), 30.0), ((30, 64, 16, 2, 128, 16, 20, "bf16"), 1e4), ((20, 32, 16, 4, 256, 16, 12, "bf16"), 0.0),
                                   ((40, 8, 16, 4, 64, 16, 8, "f32"), 1e3), ((40, 64, 16, 8, 64, 16, 16, "bf16"), float("nan"))]):
        y = make(*s, seed=81 + i, stale=0.0)
        y["q"] *= size
        y["pool"] *= 10
        for _ in range(3):
            call(y)
            assert all(torch.equal(a, b) for a, b in zip(call(x), want)), s


def test_agrees_with_the_drafted_trees():
    """A tree that is one line, verified, is a chunk: the same tokens as drafted keys and values, and in the pool."""
    import torch
    import tree_ref
    from sparse_kv_cache_draft_gb300 import attend_tree_static
    R, T, Hq, H, d, bs, kb = 3, 20, 8, 2, 128, 16, 40
    x = make(R, T, Hq, H, d, bs, kb, "bf16", seed=9, lengths=[600, 333, 0], holes=False)
    out = call(x, weigh=False)[0]
    k, v = (torch.zeros(R, T, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for r, n in enumerate(x["lengths"].tolist()):
        for t in range(T):
            for to, i in ((k, 0), (v, 1)):
                to[r, t] = x["pool"][r, :, (n + t) // bs, i, (n + t) % bs]
    mask = torch.tensor([[(1 << t + 1) - 1 for t in range(T)]] * R, dtype=torch.int64, device="cuda")
    sb = torch.where(x["slot_block"] * bs >= x["lengths"][:, None, None], -1, x["slot_block"])
    tree = torch.empty_like(out)
    attend_tree_static(x["pool"], sb, x["lengths"], None, x["q"], k, v, mask, tree, q_heads=Hq, kv_heads=H, head_dim=d, block_size=bs, slots=kb)
    _, bound = tree_ref.attend(x["pool"], sb, x["lengths"], None, x["q"], k, v, mask)
    assert bool(((out.double() - tree.double()).abs() <= 2 * bound).all())
