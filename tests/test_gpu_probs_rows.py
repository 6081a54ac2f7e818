"""GPU: log probabilities of rows of many batches a wave -- equal logits at any
place of a batch, and sums of flat rows."""
import numpy as np
import pytest

from gpu_util import needs_gpu, torch
from test_gpu_token import F16, F32, dev, host, laid

pytestmark = [pytest.mark.gpu, needs_gpu]

if torch is not None:
    from quant_dequant_gemv_amd import binding


# ------------------------------------------------------------------ ties

def tied(kind, rows, vocab, dt):
    rng = np.random.default_rng(rows + vocab)
    if kind == "run":  # all masked but a run of equals in a later batch
        z = np.full((rows, vocab), -np.inf, dt)
        for r in range(rows):
            at = int(rng.integers(0, vocab - 200))
            z[r, at: at + int(rng.integers(1, 120))] = 0.5
        z[0] = -np.inf
        z[0, 9000: 9040] = 0.5
        return z
    if kind == "pairs":  # the same maximum at places 1 and 20, 3 and 40, ... of later batches, rising
        z = rng.standard_normal((rows, vocab)).astype(dt)
        for i, base in enumerate(range(4096, vocab - 4096, 3000)):
            for a, b in ((1, 20), (3, 40), (700, 701)):
                z[:, base + a] = z[:, base + b] = 8 + i + a / 1024
        return z
    if kind == "coarse":  # a few levels
        return np.round(1.5 * rng.standard_normal((rows, vocab))).astype(dt)
    z = rng.standard_normal((rows, vocab)).astype(dt)  # "zeros": the largest is 0 or -0
    return np.where(z > 0, np.where(rng.random(z.shape) < 0.5, 0.0, -0.0), z).astype(dt)


@pytest.mark.parametrize("rows,vocab", [(300, 32768), (13, 160000), (2, 700001)])
@pytest.mark.parametrize("layout,dt", [("plain", F32), ("plain", F16), ("odd", F32), ("odd", F16), ("column", F32)])
@pytest.mark.parametrize("kind", ["run", "pairs", "coarse", "zeros"])
def test_equal_logits_go_by_the_lower_index(kind, layout, dt, rows, vocab):
    z = tied(kind, rows, vocab, dt)
    order = np.argsort(-z + dt(0), axis=1, kind="stable")[:, :64]
    best = np.take_along_axis(z, order, 1)
    ids = np.where(best > -np.inf, order, -1)
    zd = laid(z, layout)
    for top in (1, 5, 20, 64):
        got = binding.logprobs(zd, top=top)
        few = binding.logprobs(zd[rows // 2: rows // 2 + 1], top=top)  # (the row in more parts)
        torch.cuda.synchronize()
        assert np.array_equal(host(got.top_ids), ids[:, :top])
        assert np.array_equal(host(few.top_ids)[0], ids[rows // 2, :top])


# ------------------------------------------------------------------ sums

def flat(kind, V):
    """A row of float32 whose terms repeat, so that roundings of a sum add up where it has few bits."""
    rng = np.random.default_rng(V)
    if kind == "two":
        return np.where(rng.random(V) < 0.5, 0, -0.3).astype(F32)
    if kind == "one above":
        z = np.full(V, 2.0, F32)
        z[V // 3] = 2.37
        return z
    if kind == "some above":
        z = np.full(V, -1.7, F32)
        z[rng.permutation(V)[:4096]] = 1.1
        return z
    if kind == "rising":  # ever a new maximum
        return np.linspace(-9, 3, V).astype(F32)
    return np.linspace(3, -9, V).astype(F32)


@pytest.mark.parametrize("V", [131072, 262144, 1 << 20, 300001])
@pytest.mark.parametrize("side_by_side", [False, True])
@pytest.mark.parametrize("kind", ["two", "one above", "some above", "rising", "falling"])
def test_sums_of_flat_rows(kind, side_by_side, V):
    """In units u = 2^-24 of a sum, for rows of one kind of term: a term 2 (its power) and 3.5 of its distance (difference,
    scale, product), 16 of them summed in two halves 8, what follows compensated or in fp64 but for a power of 2 u where a
    maximum rises -- over lanes, waves and, a row in parts, again over lanes and waves, whose sums are stored in 1: 19 of 24
    in all, and 24 more where maxima rise as a lane goes, by 4 log 2 or more each (3 each, and 3.5 of the 4 log 2 that a
    lane's maximum is behind).  The logarithm 2 and one of its value; the result one."""
    z = flat(kind, V)
    for scale in (1.0, 0.7):
        t = (z.astype(np.float64) - float(z.max())) * float(F32(scale))
        p = np.exp(t)
        s = p.sum()
        lse = float(z.max()) * float(F32(scale)) + np.log(s)
        dist = -(p * t).sum() / s
        ent = np.log(s) + dist
        err = 2.0 ** -24 * (26 + 24 * (kind == "rising") + 3.5 * dist + np.log(s) + abs(lse) + abs(float(z.max())) * scale)
        zd = dev(np.repeat(z, 2))[::2] if side_by_side else dev(z)
        at = np.array([0, V // 3, V - 1])
        for rows in (1, 600, 4200):  # a row in parts, a block's, a wave's
            tok = torch.from_numpy(np.tile(at.astype(np.int32), (rows, 1))).cuda()
            got = binding.logprobs(zd.expand(rows, V), tok, scale=scale)
            torch.cuda.synchronize()
            assert np.abs(host(got.lse) - lse).max() <= err
            # (a token's own distance: difference, scale, sum)
            assert (np.abs(host(got.token_lp) - (t[at] - np.log(s))) <= err - 4.0 * 2.0 ** -24 * t[at]).all()
            assert np.abs(host(got.entropy) - ent).max() <= 2.0 ** -18 * (1 + np.log(V))
            assert (host(got.lse) == host(got.lse)[0]).all()
            assert (host(got.token_lp) <= 0).all() and (host(got.entropy) >= 0).all()
