"""The log sum of a row (csrc/row_sums.h), on the CPU: of what it has seen, and where its block has given up. The weights of slots
are taken from it, so a row without one must be told from every other."""
import ctypes
import math
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "sparse_kv_cache_draft_gb300", "csrc")


@pytest.fixture(scope="module")
def sums(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("sums") / "row_sums.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, os.path.join(HERE, "row_sums.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    f = ctypes.c_float
    lib.lse_at_end.argtypes, lib.lse_at_end.restype, lib.draws.argtypes = [ctypes.c_int, f, f], f, [f]
    return lib


INF, NAN, TOP = math.inf, math.nan, 3.4028234663852886e38


@pytest.mark.parametrize("m", [-INF, -1e30, 0.0, 7.5, TOP, INF, NAN])
@pytest.mark.parametrize("l", [0.0, 1e-30, 1.0, 1e9, INF, NAN])
def test_a_row_of_a_block_that_gave_up_draws_nothing(sums, m, l):
    lse = sums.lse_at_end(1, m, l)
    assert lse == -INF and not sums.draws(lse)


@pytest.mark.parametrize("m,l", [(0.0, 1.0), (-20.0, 3.5), (1000.0, 1.0), (-1e6, 2000.0), (12.25, 1e-3)])
def test_log_sum(sums, m, l):
    """m ln 2 + ln l: the logarithm and the sum half a step of the larger part each, the product one and its constant one."""
    want, size = (m + math.log2(l)) * math.log(2), max(abs(m), abs(math.log2(l)))
    lse = sums.lse_at_end(0, m, l)
    assert abs(lse - want) <= 4 * 2.0 ** -24 * size and sums.draws(lse)


def test_what_is_not_finite(sums):
    assert sums.lse_at_end(0, -INF, 0.0) == -INF and not sums.draws(-INF)          # nothing seen
    for m in (-INF, 3.0):                                                          # a score that is not a number
        lse = sums.lse_at_end(0, m, NAN)
        assert math.isnan(lse) and sums.draws(lse)
    assert sums.lse_at_end(0, TOP, INF) == INF and sums.draws(INF)                 # an infinite one
