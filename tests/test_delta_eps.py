"""CPU-only: the recurrence takes an eps that a row's sum of squares can be
added to (fake aligned addresses, never dereferenced: every call is refused)."""
import os

import pytest

import test_token_checks as t
from quant_dequant_gemv_amd import binding as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH),
                                reason="libqkgemv.so not built (run __graft_entry__.build())")


def test_eps_range():
    # (out over the rows of q: what is taken comes to the overlap)
    call = lambda eps: b.qk_delta_rule(t.delta(), t.seqs(), t.rows(eps=eps), t.heads(1, 256, 64), *t.WS)  # noqa: E731
    for eps in (0.0, 1e-6, 2.0 ** 126):
        assert call(eps) == t.PTR
    for eps in (-1e-30, 2.0 ** 126 * (1 + 2.0 ** -23), 3.4e38, t.INF, t.NAN):
        assert call(eps) == t.SHAPE
