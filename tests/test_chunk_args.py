"""Refusals of the calls of a bounded cache that need no GPU: every bad argument is an OKV_EINVAL before anything is
launched."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_cache_draft_gb300 import build, load_library
    build.build()
    return load_library()


P = 0x10000  # a 16-byte aligned address that is never read

CHUNK_OK = dict(n_requests=2, n_new=8, q_heads=32, kv_heads=8, head_dim=128, block_size=16, slots=128, dtype=1, pool=P, slot_block=P, lengths=P,
                counts=None, window=0, sinks=0, q=P, out=P, lse=P, weight=P, weight_out=P)


@pytest.mark.parametrize("bad", [
    dict(n_requests=0), dict(n_requests=-1), dict(n_new=0), dict(n_new=-3), dict(q_heads=36), dict(q_heads=72), dict(kv_heads=0), dict(head_dim=48),
    dict(head_dim=0), dict(head_dim=288), dict(block_size=0), dict(block_size=65), dict(slots=0), dict(slots=1025), dict(dtype=2), dict(dtype=-1),
    dict(n_requests=1 << 22), dict(n_new=1 << 28), dict(n_requests=1 << 16, n_new=1 << 13), dict(n_requests=1, n_new=1 << 29, kv_heads=1, q_heads=4),
    dict(window=-1), dict(sinks=-1), dict(pool=None), dict(pool=P + 8), dict(slot_block=None), dict(lengths=None), dict(q=None), dict(q=P + 4),
    dict(out=None), dict(out=P + 2), dict(lse=None), dict(lse=None, weight=None), dict(weight_out=None),
], ids=str)
def test_attend_chunk_static_refuses(lib, bad):
    assert lib.okv_attend_chunk_static(*dict(CHUNK_OK, **bad).values(), None) == 1


EVICT_OK = dict(n_requests=2, n_new=8, kv_heads=8, block_size=16, slots=128, lengths=P, counts=None, sinks=0, recent=0, slot_block=P, weight=P,
                slot_block_out=P, weight_out=P)


@pytest.mark.parametrize("bad", [
    dict(n_requests=0), dict(n_requests=-1), dict(n_new=0), dict(n_new=-1), dict(kv_heads=0), dict(kv_heads=-8), dict(block_size=0), dict(block_size=65),
    dict(slots=0), dict(slots=1025), dict(n_requests=1 << 24), dict(sinks=-1), dict(recent=-1), dict(lengths=None), dict(slot_block=None),
    dict(weight=None), dict(slot_block_out=None), dict(weight_out=None),
], ids=str)
def test_evict_static_refuses(lib, bad):
    assert lib.okv_evict_static(*dict(EVICT_OK, **bad).values(), None) == 1


def test_calls_refuse_on_the_host(lib):
    """What a call's arguments are is seen before anything is launched."""
    import inspect
    import torch
    from sparse_kv_cache_draft_gb300 import attend_chunk_static, evict_static
    x, p, kw = torch.zeros(2, 1, 1, 8), torch.zeros(2, dtype=torch.int32), dict(q_heads=1, kv_heads=1, head_dim=8, block_size=16, slots=1)
    ev = dict(n_new=1, kv_heads=1, block_size=16, slots=1)
    for bad, why in [(lambda: attend_chunk_static(x, p, p, None, x, x, **kw), "CUDA tensor"), (lambda: attend_chunk_static(x, p, p, None, x, **kw), "'out'"),
                     (lambda: attend_chunk_static(x, p, p, x, x, x, **dict(kw, length=1)), "unexpected keyword argument 'length'"),
                     (lambda: attend_chunk_static(x, p, p, None, x, x, q_heads=1, kv_heads=1, head_dim=8, block_size=16), "'slots'"),
                     (lambda: attend_chunk_static(x, p, p, None, x, x, None, None, None, 1, **kw), "at most 9"),
                     (lambda: evict_static(p, p, p, None, **ev), "CUDA tensor"), (lambda: evict_static(p, p, p, **ev), "'counts'"),
                     (lambda: evict_static([1], p, p, None, **ev), "got list"), (lambda: evict_static(p, p, p, None, kv_heads=1, block_size=16, slots=1), "'n_new'")]:
        with pytest.raises(TypeError, match=why):
            bad()
    assert list(inspect.signature(attend_chunk_static).parameters)[:9] == ["pool", "slot_block", "lengths", "counts", "q", "out", "lse", "weight", "weight_out"]
    assert list(inspect.signature(evict_static).parameters)[:6] == ["slot_block", "weight", "lengths", "counts", "slot_block_out", "weight_out"]
