"""GPU: block norms under any eps that is accepted."""
import numpy as np
import pytest

import token_ref as ref
from gpu_util import needs_gpu, torch
from test_gpu_token import F32, dev, host

pytestmark = [pytest.mark.gpu, needs_gpu]

if torch is not None:
    from quant_dequant_gemv_amd import binding


@pytest.mark.parametrize("dim", [1, 3, 200, 9000])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30, 1.0, 1e37, 3.39e38])
def test_any_eps(dim, eps):
    y = np.random.default_rng(dim).uniform(1, 2, (8, 1, dim)).astype(F32)
    y *= F32([1e-20, 1e-13, 1e-3, 1, 1e6, 1e15, 1.5e18, 3e19])[:, None, None]
    w = np.ones(dim, F32)
    _, x, _, ex = ref.block_norm(y, w, None, "none", 1.0, None, w, float(F32(eps)))
    got = binding.block_norm(dev(y), dev(w), pre_norm=dev(w), eps=eps, x_out=torch.empty(8, 1, dim, device="cuda"))[1]
    torch.cuda.synchronize()
    ref.rounded(host(got), x, ex, F32)
