"""CPU-only: the numpy reference of the 4-bit cache against the documented
layout and error bound, by construction."""
import numpy as np
import pytest

import kv_ref


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_places_every_nibble_once(D):
    """A page of known codes, read back through the header's index formulas."""
    rng = np.random.default_rng(D)
    S, H, G = 32, 2, D // 32
    f = [(rng.integers(0, 16, (S, H, D), dtype=np.uint8), rng.standard_normal((S, H, G)).astype(np.float16),
          rng.standard_normal((S, H, G)).astype(np.float16)) for _ in range(2)]
    page = kv_ref.pack_page(*f[0], *f[1])
    assert page.size == 2 * H * S * D * 5 // 8
    for h in range(H):
        for kind in range(2):
            blk = page[(2 * h + kind) * S * D * 5 // 8:][: S * D * 5 // 8]
            codes, rest = blk[: S * D // 2], blk[S * D // 2:].view(np.float16)
            d = rest[: S * G].reshape(S // 4, G, 4)
            m = rest[S * G:].reshape(S // 4, G, 4) if kind else rest[S * G:].reshape(S, G)
            if kind == 0:
                w = codes.view(np.uint32).reshape(S, 4, G)
                got = lambda p, i: (int(w[p, i % 32 // 8, i // 32]) >> (4 * (i % 8))) & 15  # noqa: E731
            elif D == 64:
                w16 = codes.view(np.uint16).reshape(S // 4, 16, 4)
                got = lambda p, i: (int(w16[p // 4, i % 16, p % 4]) >> (4 * (i // 16))) & 15  # noqa: E731
            else:
                w4 = codes.view(np.uint32).reshape(S // 4, D // 128, 16, 4)
                got = lambda p, i: (int(w4[p // 4, i // 128, i % 16, p % 4]) >> (4 * (i % 128 // 16))) & 15  # noqa: E731
            for p in range(S):
                for i in range(D):
                    assert got(p, i) == f[kind][0][p, h, i]
                    assert d[p // 4, i // 32, p % 4] == f[kind][1][p, h, i // 32]
                    assert (m[p // 4, i // 32, p % 4] if kind else m[p, i // 32]) == f[kind][2][p, h, i // 32]


@pytest.mark.parametrize("scale,shift", [(1, 0), (1e-6, 0), (3e4, 0), (1e-3, 100), (1e9, 0), (0, 5.5), (1e-9, 1e-8)])
def test_quantisation_error(scale, shift):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, 64)) * scale + shift).astype(np.float32)
    c, d, m = kv_ref.quantise(x)
    assert np.isfinite(d).all() and np.isfinite(m).all() and c.max() <= 15
    g = np.clip(x, -65504, 65504).reshape(50, 2, 32).astype(np.float64)
    err = np.abs(kv_ref.values(c, d, m).reshape(50, 2, 32) - g)
    m64, d64 = m.astype(np.float64)[..., None], d.astype(np.float64)[..., None]
    # half a step, the minimum's rounding (values below m), 15 d short of the range by d's rounding; subnormals
    bound = d64 / 2 + 2.0 ** -11 * np.abs(m64) + 2.0 ** -11 * (g.max(-1, keepdims=True) - m64) + 16 * 2.0 ** -25
    assert (err <= bound * (1 + 1e-6)).all()


def test_nan_and_infinities_are_held_finite():
    x = np.zeros((1, 64), np.float32)
    x[0, :4] = np.nan, np.inf, -np.inf, 1
    v = kv_ref.values(*kv_ref.quantise(x))
    assert np.isfinite(v).all()
    assert v[0, 1] > 65000 and v[0, 2] == -65504 and abs(v[0, 0]) < 5000 and (v[0, 32:] == 0).all()
