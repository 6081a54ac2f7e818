"""GPU: log probabilities of rows of many batches a wave -- equal logits at any
place of a batch."""
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
