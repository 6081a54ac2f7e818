"""GPU: the recurrence with queries and keys whose squares leave fp32 on the
small side, with and without an eps; rows one by one and tiles alike."""
import numpy as np
import pytest

import token_ref as ref
from gpu_util import needs_gpu, torch
from test_gpu_token import F32, delta_inputs, dev, host

pytestmark = [pytest.mark.gpu, needs_gpu]

if torch is not None:
    from quant_dequant_gemv_amd import binding


def normed(t, eps):
    """Rows of length 1 in fp64; rows of zeros stay zeros."""
    t = t.astype(np.float64)
    s = (t * t).sum(-1, keepdims=True) + eps
    return t / np.sqrt(np.where(s == 0, 1, s))


@pytest.mark.parametrize("n", [1, 17, 79, 200])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30, 1e-38])
def test_rows_of_any_length(n, dk, eps):
    rng = np.random.default_rng(n + dk)
    hk, hv, dv = 2, 4, 64
    q, k, v, al, be, A, dt = delta_inputs(rng, n, hk, hv, dk, dv, F32)
    small = F32([1, 1e-8, 1e-12, 3e-13, 1e-15, 1e-18, 1e-19, 1e-20, 1e-24, 1e-30, 1e-38, 1e-41, 2e-45, 0])
    for i in range(n):
        q[i] *= small[(i + n) % small.size]
        k[i] *= small[(3 * i + n + 1) % small.size]
    k[n // 2, 0, 1:] *= F32(1e-25)  # (one element far above the others)
    pool = (0.3 * rng.standard_normal((2, hv, dv, dk))).astype(F32)
    seqs = [(0, n, 0, 1, n)]
    g = A.astype(np.float64) * np.logaddexp(al.astype(np.float64) + dt, 0)
    out, err, new, new_err = ref.delta_rule(pool, normed(q, F32(eps)), normed(k, F32(eps)), v, g, ref.sigmoid(be.astype(np.float64)),
                                            seqs, None, None, False, 0, dk ** -0.5)
    state = binding.DeltaState(2, hk, hv, dk, dv, pool=dev(pool))
    o = binding.delta_rule(state, *map(dev, (q, k, v, al, be)), dev(np.array([0], np.int32)), dev(np.array([1], np.int32)),
                           A=dev(A), dt_bias=dev(dt), eps=eps)
    torch.cuda.synchronize()
    ref.rounded(host(o), out, err, F32)
    d = np.sqrt(((host(state.pool) - new) ** 2).sum(-1))
    assert (d <= new_err + 2.0 ** -24 * np.sqrt((new ** 2).sum(-1)) + 2.0 ** -140).all()
