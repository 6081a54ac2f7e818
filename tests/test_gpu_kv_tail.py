"""GPU: attention where one position stands far above a long tail, as a trained model's first position does: the
tail's share of the output has to be there, whatever the values' scale, in fp32 outputs against fp64."""
from functools import lru_cache

import numpy as np
import pytest

from gpu_util import needs_gpu
from kv_fill import Fields, Filled, check_attn

pytestmark = [pytest.mark.gpu, needs_gpu]

# D, tile: heads on one KV head, sequences, rows of each, whether their contexts are cut into splits.
# Tiles of 8 rows (up to 8 rows x heads a sequence), 16, and 32 (D = 64 from 1024 rows x heads on).
FORMS = {
    (64, 8): [(4, 1, 1, True), (4, 800, 1, False)], (128, 8): [(6, 1, 1, True), (6, 800, 1, False)],
    (256, 8): [(6, 1, 1, True), (6, 300, 1, False)],
    (64, 16): [(8, 1, 5, True), (8, 800, 2, False)], (128, 16): [(6, 1, 4, True), (8, 800, 2, False)],
    (256, 16): [(6, 1, 17, True), (6, 600, 2, False)],
    (64, 32): [(4, 1, 260, True), (6, 2, 2048, False)],
}


@lru_cache(maxsize=9)
def keys(D, length, gap):
    """Keys of which the first stands `gap` nats above the others for every query near `along`."""
    rng = np.random.default_rng(D + int(gap))
    along = rng.standard_normal((1, D))
    along *= np.sqrt(D) / np.linalg.norm(along)
    k = rng.standard_normal((length, 1, D), dtype=np.float32) * np.float32(0.05)
    k[0] = along * (gap / np.sqrt(D))
    return along, Fields(k)


@lru_cache(maxsize=1)
def context(D, length, gap, scale, mean, first):
    rng = np.random.default_rng(D + length)
    v = (mean + rng.standard_normal((length, 1, D), dtype=np.float32)) * np.float32(scale)
    if not first:
        v[0] = 0
    along, k = keys(D, length, gap)
    return along, Filled(rng, k, Fields(v), 64)


@pytest.mark.parametrize("D,length,gap,tile,form", [
    (D, length, gap, tile, f) for D in (64, 128, 256) for length, gap in ((4096, 8.0), (32768, 12.0), (32768, 16.0))
    for (d, tile), forms in FORMS.items() if d == D for f in forms])
@pytest.mark.parametrize("scale,mean,first", [(1.0, 0.0, False), (0.02, 1.0, True), (0.02, 0.0, False), (1e-4, 0.0, True),
                                              (3e4, 0.0, False)])
def test_one_position_above_a_tail(D, length, gap, tile, form, scale, mean, first):
    grp, nseq, n, split = form
    along, c = context(D, length, gap, scale, mean, first)
    rng = np.random.default_rng(D + n)
    q = (along + 0.05 * rng.standard_normal((nseq * n, grp, D), dtype=np.float32)).astype(np.float16)
    check_attn(c, q, nseq, split, sorted({0, nseq * n // 2, nseq * n - 1}))


def sizes(kind, length, D):
    """Factors of the values, by position or by group."""
    if kind == "rising":      # every later tile brings a larger step, up to 8734
        return np.geomspace(1e-6, 3e4, length)[:, None, None]
    if kind == "falling":
        return np.geomspace(3e4, 1e-6, length)[:, None, None]
    if kind == "late":        # nothing, then ordinary values
        return (np.arange(length) >= 100)[:, None, None] * 0.5
    if kind == "one large":   # one position of steps above 1000 among small ones
        return np.where(np.arange(length) == length // 2, 6e3, 0.01)[:, None, None]
    return np.repeat(np.geomspace(1e-4, 2e4, D // 32), 32)[None, None]  # groups of unlike sizes


@pytest.mark.parametrize("D,tile,form", [(d, tile, f) for (d, tile), forms in FORMS.items() for f in forms])
@pytest.mark.parametrize("kind", ["rising", "falling", "late", "one large", "groups"])
def test_steps_of_many_sizes(D, tile, form, kind):
    """The scaling of the steps moves along a wave's tiles, and serves groups and positions of unlike steps."""
    grp, nseq, n, split = form
    length = 5000
    rng = np.random.default_rng(D + tile)
    x = [rng.standard_normal((length, 1, D)).astype(np.float32) for _ in range(2)]
    x[1] = (x[1] * sizes(kind, length, D)).astype(np.float32)
    c = Filled(rng, *(Fields(a) for a in x), 64)
    q = rng.standard_normal((nseq * n, grp, D), dtype=np.float32).astype(np.float16)
    check_attn(c, q, nseq, split, sorted({0, nseq * n // 2, nseq * n - 1}))
