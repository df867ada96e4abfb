"""Refusals of the calls on rows and drafted trees that need no GPU: every bad argument is an
OKV_EINVAL before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_cache_draft_gb300 import build, load_library
    build.build()
    return load_library()


P = 0x10000  # a 16-byte aligned address that is never read


def rotary(**kw):
    from sparse_kv_cache_draft_gb300 import binding
    f = dict(inv_freq=P, q_weight=P, k_weight=P, eps=1e-6, rotary_dim=128, interleaved=0)
    f.update(kw)
    return binding._Rotary(**f)


def test_struct_layout(lib, tmp_path):
    import os
    import subprocess
    from sparse_kv_cache_draft_gb300 import binding
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "okv.h"', "int main(void) {",
             '  printf("%zu\\n", sizeof(okv_rotary));']
    lines += [f'  printf("%zu\\n", offsetof(okv_rotary, {f}));' for f, _ in binding._Rotary._fields_]
    src = tmp_path / "l.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c99", "-I", inc, "-o", str(tmp_path / "l"), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(binding._Rotary)] + [getattr(binding._Rotary, f).offset for f, _ in binding._Rotary._fields_]


ROWS_OK = dict(n_rows=4, q_heads=32, kv_heads=8, head_dim=128, dtype=1, qkv=P, row_stride=6144, positions=P, rotary=None, q=P, k=P,
               v=P, stream=None)


@pytest.mark.parametrize("bad", [
    dict(n_rows=-1), dict(q_heads=0), dict(q_heads=30), dict(kv_heads=0), dict(kv_heads=-8), dict(q_heads=16384, kv_heads=8), dict(q_heads=4104, kv_heads=8, row_stride=4120 * 128),
    dict(head_dim=0), dict(head_dim=100), dict(head_dim=288), dict(dtype=2), dict(qkv=None), dict(qkv=P + 8),
    dict(row_stride=6143), dict(row_stride=6148), dict(row_stride=1 << 40), dict(positions=None),
    dict(q=None, k=None, v=None), dict(q=P + 4), dict(k=P + 2), dict(v=P + 8),
    dict(rotary=dict(rotary_dim=136)), dict(rotary=dict(rotary_dim=-16)), dict(rotary=dict(rotary_dim=24)),
    dict(rotary=dict(inv_freq=None)), dict(rotary=dict(eps=-1e-6)), dict(rotary=dict(eps=float("nan"))),
    dict(rotary=dict(eps=float("inf"))), dict(rotary=dict(interleaved=2)), dict(rotary=dict(q_weight=P + 8)), dict(rotary=dict(k_weight=P + 2)),
    dict(rotary="none"),
], ids=str)
def test_norm_rope_refuses(lib, bad):
    a = dict(ROWS_OK, **bad)
    r = a["rotary"]
    r = None if r == "none" else ctypes.addressof(keep := rotary(**(r or {})))
    assert lib.okv_norm_rope(a["n_rows"], a["q_heads"], a["kv_heads"], a["head_dim"], a["dtype"], a["qkv"], a["row_stride"],
                             a["positions"], r, a["q"], a["k"], a["v"], a["stream"]) == 1


def test_rotary_is_the_struct(lib):
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, binding
    x = torch.zeros(1, 8)
    assert Rotary()._check(x, 8) == bytes(binding._Rotary(0, 0, 0, 1e-6, 0, 0))
    assert Rotary(None, None, None, 0.25, True)._check(x, 8) == bytes(binding._Rotary(0, 0, 0, 0.25, 0, 1))
    assert Rotary(interleaved=1, eps=2).tensors == (None, None, None)


def test_calls_refuse_on_the_host(lib):
    """What a call's arguments are is seen before anything is launched."""
    import copy
    import inspect
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, append_qkv_static, attend_tree_static, norm_rope
    x, p, kw = torch.zeros(2, 24), torch.zeros(2, dtype=torch.int32), dict(q_heads=1, kv_heads=1, head_dim=8, rotary=Rotary())
    for bad, why in [(lambda: norm_rope(x, p, **kw), "CUDA tensor"), (lambda: norm_rope([1.0], p, **kw), "CUDA tensor, got list"),
                     (lambda: norm_rope(x, **kw), "missing required argument: 'positions'"), (lambda: norm_rope(), "missing"),
                     (lambda: norm_rope(x, p, **dict(kw, heads=3)), "unexpected keyword argument 'heads'"),
                     (lambda: norm_rope(x, p, qkv=x, **kw), "multiple values for argument 'qkv'"),
                     (lambda: norm_rope(x, p, None, None, None, 1, **kw), "at most 5 positional"),
                     (lambda: append_qkv_static(x, p, None, x, p, None, **kw), "missing required argument: 'block_size'"),
                     (lambda: attend_tree_static(x, p, p, None, x, x, x, p, x, q_heads=1, kv_heads=1, head_dim=8, block_size=16), "'slots'"),
                     (lambda: Rotary(x[0], x[0], x[0], 1e-6, False, 0), "at most 5"), (lambda: Rotary(freq=x), "unexpected"),
                     (lambda: Rotary(eps="a"), "real number"), (lambda: Rotary(3), "expected a CUDA tensor"),
                     (lambda: Rotary.__new__(Rotary), "Rotary"), (lambda: type.__call__(Rotary), "Rotary"), (lambda: copy.copy(Rotary()), "Rotary")]:
        with pytest.raises(TypeError, match=why):
            bad()
    with pytest.raises(ValueError, match="contiguous CUDA vector"):
        Rotary(x[0])
    assert list(inspect.signature(norm_rope).parameters) == ["qkv", "positions", "q", "k", "v", "q_heads", "kv_heads", "head_dim",
                                                              "rotary", "stream"]


def test_calls_keep_no_references(lib):
    import sys
    import torch
    from sparse_kv_cache_draft_gb300 import Rotary, norm_rope
    x, p, rot, key = torch.zeros(2, 24), torch.zeros(2, dtype=torch.int32), Rotary(), "".join(["no", "_such"])

    def counts():
        return [sys.getrefcount(o) for o in (x, p, rot, key, Rotary, Rotary.tensors, norm_rope, None)][:-1]
    before = counts()
    for _ in range(50):
        for f in (lambda: norm_rope(x, p, q_heads=1, kv_heads=1, head_dim=8, rotary=rot), lambda: norm_rope(x, p, **{key: rot}),
                  lambda: Rotary(x), lambda: Rotary(p, p, p)):
            with pytest.raises((TypeError, ValueError)):
                f()
        Rotary(None, None, None)._check(x, 8)
    assert counts() == before


def test_no_rows_is_no_work(lib):
    r = rotary()
    assert lib.okv_norm_rope(0, 32, 8, 128, 1, None, 6144, None, ctypes.addressof(r), None, None, None, None) == 0


APPEND_OK = dict(n_requests=2, n_new=3, q_heads=32, kv_heads=8, head_dim=128, block_size=16, slots=128, dtype=1, qkv=P, row_stride=6144,
                 lengths=P, counts=None, pool=P, slot_block=P, q=P)


@pytest.mark.parametrize("bad", [
    dict(n_requests=0), dict(n_requests=-2), dict(n_new=0), dict(n_requests=1 << 20, n_new=1 << 12), dict(q_heads=72),
    dict(block_size=0), dict(block_size=65), dict(slots=0), dict(slots=1025), dict(n_requests=1 << 22), dict(dtype=5),
    dict(lengths=None), dict(pool=None), dict(pool=P + 8), dict(slot_block=None), dict(qkv=None), dict(row_stride=128), dict(q=P + 8),
    dict(rot=dict(rotary_dim=144)),
], ids=str)
def test_append_static_refuses(lib, bad):
    a = dict(APPEND_OK, **bad)
    r = rotary(**a.get("rot", {}))
    assert lib.okv_append_qkv_static(a["n_requests"], a["n_new"], a["q_heads"], a["kv_heads"], a["head_dim"], a["block_size"],
                                     a["slots"], a["dtype"], a["qkv"], a["row_stride"], a["lengths"], a["counts"],
                                     ctypes.addressof(r), a["pool"], a["slot_block"], a["q"], None) == 1


TREE_OK = dict(n_requests=2, n_draft=8, q_heads=32, kv_heads=8, head_dim=128, block_size=16, slots=128, dtype=1, pool=P, slot_block=P,
               lengths=P, counts=None, q=P, k=P, v=P, mask=P, out=P)


@pytest.mark.parametrize("bad", [
    dict(n_requests=0), dict(n_draft=0), dict(n_draft=65), dict(q_heads=36), dict(q_heads=72), dict(kv_heads=0), dict(head_dim=48),
    dict(head_dim=320), dict(block_size=0), dict(block_size=100), dict(slots=0), dict(slots=2000), dict(dtype=-1),
    dict(n_requests=1 << 22), dict(n_requests=1 << 26, kv_heads=1, q_heads=4, slots=1, n_draft=64), dict(pool=None), dict(pool=P + 4), dict(slot_block=None), dict(lengths=None), dict(q=None), dict(q=P + 8),
    dict(k=None), dict(k=P + 2), dict(v=None), dict(v=P + 8), dict(mask=None), dict(out=None), dict(out=P + 8),
], ids=str)
def test_attend_tree_static_refuses(lib, bad):
    a = dict(TREE_OK, **bad)
    assert lib.okv_attend_tree_static(*[a[n] for n in ("n_requests", "n_draft", "q_heads", "kv_heads", "head_dim", "block_size",
                                                       "slots", "dtype", "pool", "slot_block", "lengths", "counts", "q", "k", "v",
                                                       "mask", "out")], None) == 1


def test_null_context(lib):
    r = rotary()
    assert lib.okv_append_qkv(None, 0, P, 6144, ctypes.addressof(r), P, None) == 1
    assert lib.okv_attend_tree(None, 0, 4, None, P, P, P, P, P, None) == 1
    assert lib.okv_append_tree(None, 0, 4, P, P, P, P, None) == 1


def test_row_stride_of_views():
    import torch
    from sparse_kv_cache_draft_gb300.binding import _row_stride
    t = torch.zeros(4, 3, 40)
    assert _row_stride(t[..., :32], 32) == 40 and _row_stride(t, 40) == 40
    assert _row_stride(t[:1, :1, :8], 8) == 8            # one row: its own width
    assert _row_stride(t[:, 1:2, :8], 8) == 120          # one token per request
    assert _row_stride(t[2:3, :, :8], 8) == 40
    for bad in (t[..., ::2], t[:, :2, :20], t.transpose(1, 2)):
        with pytest.raises(ValueError):
            _row_stride(bad, bad.shape[-1])
    with pytest.raises(ValueError):
        _row_stride(t, 32)
