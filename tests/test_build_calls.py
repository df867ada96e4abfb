"""The build of the library where the Python calls on rows and drafted trees cannot be built."""
import os

import pytest


@pytest.mark.parametrize("compiler", ["false", "/no/such/compiler"])
def test_the_library_is_built_without_a_compiler_for_the_calls(tmp_path, monkeypatch, capsys, compiler):
    """A user of the other calls needs none: the library is there, the reason is said, and no module that was made for
    another library stays."""
    pytest.importorskip("torch")
    from sparse_kv_cache_draft_gb300 import build
    build.build()
    made, old = build._build_calls, tmp_path / "_calls.so"
    old.write_bytes(b"")
    monkeypatch.setattr(build, "CALLS", str(old))
    monkeypatch.setattr(build, "CXX", compiler)
    monkeypatch.setattr(build, "_build_calls", lambda nv, force: made(nv, True))
    lib = build.build()
    assert lib == build.LIB and os.path.exists(lib)
    assert not old.exists()
    assert "norm_rope" in capsys.readouterr().err
