"""CPU-only: copies of the recurrent layers' states work on the tensors that
they hold, not on those of the state they were made from."""
import copy
import os
import pickle
import struct

import pytest
import torch

from quant_dequant_gemv_amd import binding as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH),
                                reason="libqkgemv.so not built (run __graft_entry__.build())")


def addresses(state):
    """Those that a call passes on (fields of the packed qk_conv and qk_delta)."""
    f = struct.unpack("PqiiPP" if isinstance(state, b.ConvState) else "Pqiiii", state._c)
    return (f[0], f[4], f[5]) if isinstance(state, b.ConvState) else f[:1]


def held(state):
    names = ("pool", "weight", "bias") if isinstance(state, b.ConvState) else ("pool",)
    return tuple(0 if getattr(state, n) is None else getattr(state, n).data_ptr() for n in names)


@pytest.mark.parametrize("make", [
    lambda: b.ConvState(3, torch.randn(64, 4), torch.randn(64)),
    lambda: b.ConvState(2, torch.randn(5, 2), pool=torch.randn(2, 1, 5)),
    lambda: b.DeltaState(3, 1, 2, 64, 96, pool=torch.randn(3, 2, 96, 64)),
])
def test_copies(make):
    s = make()
    assert addresses(s) == held(s)
    for t in (copy.deepcopy(s), pickle.loads(pickle.dumps(s)), copy.deepcopy([s, {"also": s}])[0]):
        assert type(t) is type(s) and addresses(t) == held(t)
        assert t.pool.data_ptr() != s.pool.data_ptr() and torch.equal(t.pool, s.pool)
        assert t.num_slots == s.num_slots and t.pool.shape == s.pool.shape
        t.pool.fill_(7)
        assert not (s.pool == 7).any()
    t = copy.copy(s)  # (the same tensors)
    assert addresses(t) == held(t) == held(s)
