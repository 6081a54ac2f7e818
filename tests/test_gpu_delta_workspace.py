"""GPU: only calls that go in tiles take the recurrence's workspace."""
import numpy as np
import pytest

from gpu_util import needs_gpu, torch
from test_gpu_token import F32, delta_inputs, dev

pytestmark = [pytest.mark.gpu, needs_gpu]

if torch is not None:
    from quant_dequant_gemv_amd import binding as b


@pytest.mark.parametrize("norm,raw", [(True, True), (False, True), (True, False), (False, False)])
def test_rows_one_by_one_take_no_workspace(norm, raw):
    rng = np.random.default_rng(1)
    n, hk, hv, dk, dv = 3000, 4, 8, 128, 128
    q, k, v, al, be, A, dt = delta_inputs(rng, n, hk, hv, dk, dv, F32, raw)
    q, k = (t / np.sqrt((t * t).sum(-1, keepdims=True)) for t in (q, k))
    ins = [dev(t) for t in (q, k, v, al, be)]
    kw = dict(A=dev(A), dt_bias=dev(dt), norm=norm)
    slots = dev(np.array([0], np.int32))
    state, other = (b.DeltaState(1, hk, hv, dk, dv) for _ in range(2))
    out, again = torch.empty(n, hv, dv, device="cuda"), torch.empty(n, hv, dv, device="cuda")
    need = b.qk_delta_workspace_bytes(b.qk_delta(None, 1, hk, hv, dk, dv), b.qk_state_seqs(n, 1))
    assert need > 10 << 20
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    b.delta_rule(state, *ins, slots, out=out, **kw)
    took = torch.cuda.max_memory_allocated() - before
    tiles = norm and raw
    assert took >= need if tiles else took < 1 << 20
    # the C ABI without a workspace
    heads = lambda t: b._heads_arg(t, "t")  # noqa: E731
    col = lambda t: b.qk_heads(t.data_ptr(), *t.stride(), 1, 0)  # noqa: E731
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    rows = b.qk_delta_rows(*map(heads, ins[:3]), *map(col, ins[3:]), ptr(kw["A"]), ptr(kw["dt_bias"]), 1e-6, dk ** -0.5, norm)
    seqs = b.qk_state_seqs(n, 1, None, slots.data_ptr())
    rc = b.qk_delta_rule(b.qk_delta(other.pool.data_ptr(), 1, hk, hv, dk, dv), seqs, rows, heads(again), None, 0,
                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == (b.QK_EINVAL_SHAPE if tiles else b.QK_OK)
    if not tiles:
        assert torch.equal(out, again) and torch.equal(state.pool, other.pool)
