"""Units of many groups of rows (okv_attend_chunk_static): long chunks, and the weights of chunks whose sums do not fit shared memory."""
import pytest

from test_gpu_chunk import call, check, make

pytestmark = pytest.mark.gpu

SHAPES = [  # R, T, Hq, Hkv, d, bs, kb, dtype
    (1, 2048, 8, 2, 128, 16, 200, "bf16"),      # 32 groups of 256 rows
    (1, 1500, 8, 1, 64, 16, 150, "bf16"),       # 47
    (2, 1100, 3, 1, 96, 24, 70, "bf16"),
    (1, 700, 8, 2, 256, 16, 60, "bf16"),        # 22 groups of 128 rows
    (1, 600, 4, 2, 160, 33, 40, "bf16"),
    (1, 1000, 8, 2, 64, 16, 90, "f32"),         # 63 groups of 64 rows
    (2, 400, 5, 1, 128, 16, 60, "f32"),
    (3, 8, 8, 2, 128, 16, 300, "bf16"),         # 32 rows, and slots for which sums have no room
    (2, 16, 16, 2, 128, 16, 100, "bf16"),
    (2, 32, 8, 2, 64, 8, 200, "bf16"),
]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 20)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(v) for v in s))
def test_against_plain(shape, window, sinks, ragged):
    R, T, _, _, _, bs, kb, _ = shape
    x = make(*shape, seed=R * 1000 + T, lengths=[max(0, kb * bs - T - 37 * r) for r in range(R)], counts=[T - 1 - T // 3 * r for r in range(R)] if ragged else None,
             holes=ragged)
    x.update(window=window, sinks=sinks)
    check(x, call(x))
