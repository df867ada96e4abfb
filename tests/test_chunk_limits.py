"""The longest calls of okv_attend_chunk_static, refused on the host: rows are counted in 32 bits, past a group's end as well."""
import pytest

from test_chunk_args import CHUNK_OK


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_cache_draft_gb300 import build, load_library
    build.build()
    return load_library()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("heads,n_new", [(1, 2 ** 31 - 1), (1, 2 ** 31 - 100), (1, 2 ** 31 - 512), (2, 2 ** 30 - 1), (2, 2 ** 30 - 256), (8, 2 ** 28 - 1), (8, 2 ** 28 - 64)])
def test_rows_next_to_the_limit_are_refused(lib, dtype, heads, n_new):
    bad = dict(n_requests=1, kv_heads=1, q_heads=heads, n_new=n_new, head_dim=32, dtype=dtype)
    assert lib.okv_attend_chunk_static(*dict(CHUNK_OK, **bad).values(), None) == 1
