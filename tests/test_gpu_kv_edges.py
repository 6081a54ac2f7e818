"""GPU: places at the edges of what the attention side documents."""
import numpy as np
import pytest

import kv_ref
from gpu_util import dev, needs_gpu, torch

pytestmark = [pytest.mark.gpu, needs_gpu]

if torch is not None:
    from quant_dequant_gemv_amd import binding


@pytest.mark.parametrize("D,grp,n", [(64, 3, 1), (128, 8, 1), (256, 6, 1), (64, 6, 3), (128, 6, 3), (256, 6, 3), (64, 4, 260)])
def test_positions_before_the_window_may_hold_anything(D, grp, n):
    """A window opens inside a tile whose earlier positions were never appended: NaN and infinities, not 0 times them."""
    rng = np.random.default_rng(D + n)
    mp, window = 20, 40
    c = kv_ref.Cache(rng, 1, mp, 1, D, 32)
    length = mp * 32 - 3
    first = length - n - window + 1  # of the positions that a row sees
    assert first % 32 > 4
    fields = [[x[0].copy() for x in f] for f in c.f]
    for code, d, m in fields:
        code[:first], d[:first], m[:first] = 15, np.float16(np.nan), np.float16(-np.inf)
    for j in range(first // 32 + 1):
        at = slice(32 * j, 32 * j + 32)
        c.pool[c.pages[0, j]] = kv_ref.pack_page(*(x[at] for f in fields for x in f))
    q = rng.standard_normal((n, grp, D)).astype(np.float16)
    kv_len = np.array([length], np.int32)
    want, mass, amax = kv_ref.attention(c, q, [(0, i, n) for i in range(n)], kv_len, D ** -0.5, window)
    cache = binding.KVCache(c.num_pages, 1, D, 32, pool=dev(c.pool))
    got = binding.kv_attn(cache, dev(q), dev(c.pages), dev(kv_len), window=window, out=torch.empty(n, grp, D, device="cuda"))
    torch.cuda.synchronize()
    assert (np.abs(got.cpu().numpy() - want) <= kv_ref.attention_bound(want, mass, amax, False)).all()
