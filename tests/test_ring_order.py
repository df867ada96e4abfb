"""What the copy warps of an attention kernel wait for when a wait of another warp has run out (csrc/ring.h): every copy that was
started and that nobody waited for, and no barrier that has moved on. On the CPU, with copies that land only where they are waited for."""
import ctypes
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "sparse_kv_cache_draft_gb300", "csrc")


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("ring") / "ring_order.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, os.path.join(HERE, "ring_order.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def run(order, s, ring, n, rng):
    """A block that gives up somewhere: uses that its warps started, and those whose copy the MMA thread has waited for."""
    key, value = (lambda i: order.key(s, i)), (lambda i: order.value(s, i))
    uses = sorted([key(i) for i in range(n)] + [value(i) for i in range(n)])
    stop = rng.choice([0, len(uses), rng.randrange(len(uses) + 1)])         # products before the MMA thread gives up
    ends = [rng.choice([n, n, rng.randrange(n + 1)]) for _ in range(2)]     # tiles after which a copy warp gives up by itself
    issued, read = [0, 0], set()
    while True:
        # a copy warp starts its next copy once the buffer's last one has been read; the MMA thread reads in order
        can = [w for w in (0, 1) if issued[w] < ends[w] and ((u := (key, value)[w](issued[w])) < ring or u - ring in read or u - ring not in uses)]
        started = {key(i) for i in range(issued[0])} | {value(i) for i in range(issued[1])}
        nxt = uses[len(read)] if len(read) < stop else None
        if nxt is not None and nxt in started:
            can.append(2)
        if not can:
            return started, read, issued
        step = rng.choice(can)
        if step == 2:
            read.add(nxt)
        else:
            issued[step] += 1


@pytest.mark.parametrize("s", [1, 2])
def test_uses_are_each_one_copy(order, s):
    n = 40
    uses = [order.key(s, i) for i in range(n)] + [order.value(s, i) for i in range(n)]
    assert len(set(uses)) == 2 * n and min(uses) == 0
    assert all(order.key(s, i) < order.value(s, i) for i in range(n))


@pytest.mark.parametrize("s", [1, 2])
@pytest.mark.parametrize("ring", range(4, 13))
def test_every_copy_lands_before_the_memory_is_given_up(order, s, ring):
    rng = random.Random(100 * s + ring)
    left = 0
    for _ in range(400):
        n = rng.choice([0, 1, 2, 3, ring // 2, ring, rng.randrange(1, 50)])
        started, read, issued = run(order, s, ring, n, rng) if n else (set(), set(), [0, 0])
        landed = set(read)
        for w, use_of in enumerate((order.key, order.value)):
            for i in range(max(0, issued[w] - ring), issued[w]):
                u = use_of(s, i)
                if order.may_be_on_its_way(s, u, ring, *issued):
                    assert u + ring not in started, "its barrier has another phase by now"
                    landed.add(u)
        assert landed == started
        left += len(started - read)
    assert left > 0  # copies that only this wait sees to
