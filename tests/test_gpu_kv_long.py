"""GPU: attention loops that run long: contexts in one piece, so that a wave takes hundreds of tiles and looks its pages
up again and again, holes and windows on the way; and the 32-row tiles, split and not, even and ragged."""
import numpy as np
import pytest

from gpu_util import needs_gpu
from kv_fill import Fields, Filled, check_attn

pytestmark = [pytest.mark.gpu, needs_gpu]

# D, heads on one KV head, sequences (or rows of each), rows, split: tiles of 8, 16 and 32 rows.
# A workgroup's 4 waves (8: D = 256, tiles of 8) take tiles of 32 positions in turn and look 64 pages each ahead, so
# contexts of more than 8192 (16384) positions in one piece make them look again.
FORMS = [(64, 4, 800, 800, False), (128, 6, 800, 800, False), (256, 6, 300, 300, False),
         (64, 8, 800, 1600, False), (128, 8, 800, 1600, False), (256, 6, 600, 1200, False),
         (64, 6, 2, 4096, False), (64, 4, 1, 260, True), (64, 8, [300, 2, 700], 1002, True), (64, 8, [2100, 0, 2200], 4300, False)]


def context(D, length, holes=(), mean=0.0, on=None):
    rng = np.random.default_rng(D)
    k, v = (rng.standard_normal((length, 1, D), dtype=np.float32) for _ in range(2))
    v += np.float32(mean)
    if on is not None:
        v *= on[:, None, None]
    return rng, Filled(rng, Fields(k), Fields(v), 64, holes)


@pytest.mark.parametrize("window", [0, 13001])
@pytest.mark.parametrize("D,grp,ns,rows,split", FORMS, ids=lambda x: str(x).replace(" ", ""))
def test_long_contexts_with_holes(D, grp, ns, rows, split, window):
    length = 20011  # 626 tiles of 32, 157 (79) a wave
    rng, c = context(D, length, holes=(0, 3, 140, 141, 258, 300, 312))
    q = rng.standard_normal((rows, grp, D), dtype=np.float32).astype(np.float16)
    check_attn(c, q, ns, split, [0, 1, rows // 2, rows - 2, rows - 1], window)


@pytest.mark.parametrize("part", ["noise", "all", "first half", "second half", "last tenth"])
@pytest.mark.parametrize("D,grp,ns,rows", [(64, 8, 800, 1600), (128, 6, 800, 800), (256, 6, 300, 300), (64, 6, 2, 4096)])
def test_a_quarter_of_a_million_positions_in_one_piece(D, grp, ns, rows, part):
    """Thousands of sums into one fp32 accumulator of the matrix instructions, beside those of the softmax sum: values
    around 0, or around 4 in a part of the context (a sum that lost something at every step would show)."""
    length = 262139
    at = np.arange(length)
    on = {"first half": at < length // 2, "second half": at >= length // 2, "last tenth": at >= length * 9 // 10}.get(part, at >= 0)
    rng, c = context(D, length, mean=4.0 if part != "noise" else 0.0, on=on)
    q = rng.standard_normal((rows, grp, D), dtype=np.float32).astype(np.float16)
    q[0] = 0  # equal probabilities
    check_attn(c, q, ns, False, [0, 1, rows - 1])
