"""GPU: block norms, convolution, recurrence and log probabilities where calls
go wrong: captured and replayed, on other streams, at once, in place, in
several launches, past 32-bit offsets, with extreme and non-finite values."""
import numpy as np
import pytest

import token_ref as ref
from gpu_util import needs_gpu, torch
from test_gpu_token import F32, check_delta, delta_inputs, dev, host

pytestmark = [pytest.mark.gpu, needs_gpu]

if torch is not None:
    from quant_dequant_gemv_amd import binding

I32 = np.int32


def same_bits(a, b):
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def layer(seed, n=70, nseq=2, hk=1, hv=2, dk=64, dv=64):
    """The four operators in a row on one set of inputs: a callable that returns all they leave."""
    rng = np.random.default_rng(seed)
    rows, C = n * nseq, 2 * hk * dk + hv * dv
    conv = binding.ConvState(2 * nseq, dev(0.4 * rng.standard_normal((C, 4)).astype(F32)),
                             pool=dev(rng.standard_normal((2 * nseq, 3, C)).astype(F32)))
    state = binding.DeltaState(2 * nseq, hk, hv, dk, dv, pool=dev(0.2 * rng.standard_normal((2 * nseq, hv, dv, dk)).astype(F32)))
    x, z = dev(rng.standard_normal((rows, C)).astype(F32)), dev(rng.standard_normal((rows, hv, dv)).astype(F32))
    al, be = dev(rng.standard_normal((rows, hv)).astype(F32)), dev(rng.standard_normal((rows, hv)).astype(F32))
    A, w = dev(-np.ones(hv, F32)), dev(1 + 0.1 * rng.standard_normal(dv).astype(F32))
    head = dev(0.1 * rng.standard_normal((hv * dv, 5000)).astype(np.float16))
    slots, out_slots = dev(np.arange(nseq, dtype=I32)), dev(np.arange(nseq, 2 * nseq, dtype=I32))
    tok = dev(rng.integers(0, 5000, (rows, 2)).astype(I32))

    def run(stream=None):
        y = binding.conv_silu(conv, x, slots, out_slots, stream=stream)
        q, k, v = (t.unflatten(1, s) for t, s in zip(y.split([hk * dk, hk * dk, hv * dv], 1), ((hk, dk), (hk, dk), (hv, dv))))
        o = binding.delta_rule(state, q, k, v, al, be, slots, out_slots, A=A, stream=stream)
        _, g = binding.block_norm(o, w, z, stream=stream)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            logits = g.flatten(1) @ head
        p = binding.logprobs(logits, tok, top=7, stream=stream)
        return [y, o, g, *p, conv.pool[nseq:], state.pool[nseq:]]
    return run


@pytest.mark.parametrize("n", [1, 17, 200])
def test_captured_and_replayed(n):
    run = layer(n, n)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()  # (workspaces of the allocator's, first use of the kernels)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = run()
    for _ in range(4):
        for t in outs:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        same_bits(outs, want)
        same_bits(layer(n + 100, 3)(), layer(n + 100, 3)())  # eager work between the replays
        torch.cuda.synchronize()


def test_other_streams_and_calls_at_once():
    runs = [layer(i, n) for i, n in enumerate((90, 5, 130, 1))]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [None] * len(runs)
    for _ in range(3):
        for i, (r, s) in enumerate(zip(runs, streams)):
            got[i] = r(stream=s)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        same_bits(g, w)


@pytest.mark.parametrize("n", [3, 150])
def test_rows_of_no_sequence_and_empty_sequences(n):
    rng = np.random.default_rng(n)
    rows, hk, hv, dk, dv = 2 * n + 9, 1, 2, 64, 64
    q_start = dev(np.array([2, n + 2, n + 2, 2 * n + 2], I32))  # 2 rows before the first, 7 behind the last; one without rows
    slots = dev(np.array([0, 1, 2], I32))
    C = 128
    pool = rng.standard_normal((3, 3, C)).astype(F32)
    w, x = rng.standard_normal((C, 4)).astype(F32), rng.standard_normal((rows, C)).astype(F32)
    conv = binding.ConvState(3, dev(w), pool=dev(pool))
    out = torch.full((rows, C), 9.0, device="cuda")
    binding.conv_silu(conv, dev(x), slots, q_start=q_start, out=out)
    q, k, v, al, be, A, dt = delta_inputs(rng, rows, hk, hv, dk, dv, F32)
    sp = rng.standard_normal((3, hv, dv, dk)).astype(F32)
    state = binding.DeltaState(3, hk, hv, dk, dv, pool=dev(sp))
    o = torch.full((rows, hv, dv), 9.0, device="cuda")
    binding.delta_rule(state, *map(dev, (q, k, v, al, be)), slots, q_start=q_start, A=dev(A), dt_bias=dev(dt), out=o)
    torch.cuda.synchronize()
    seqs = [(2, n, 0, 0, n), (n + 2, 0, 1, 1, 0), (n + 2, n, 2, 2, n)]
    y, err, new = ref.conv_silu(pool, w, None, x, seqs, True)
    live = slice(2, 2 * n + 2)
    ref.rounded(host(out)[live], y[live], err[live], F32)
    assert (host(conv.pool) == new).all()
    r, e, new, ne = ref.delta_rule(sp, q, k, v, al, be, seqs, A, dt, True, 1e-6, dk ** -0.5)
    ref.rounded(host(o)[live], r[live], e[live], F32)
    assert (host(state.pool)[1] == sp[1]).all()
    for t in (out, o):
        assert (t[:2] == 9).all() and (t[2 * n + 2:] == 9).all()


@pytest.mark.parametrize("n", [8, 130])
def test_starts_that_decrease_stay_in_bounds(n):
    """Rows are undefined, memory around them is not touched."""
    rng = np.random.default_rng(n)
    guard, hk, hv, dk, dv, C = 50, 1, 1, 64, 64, 64
    for starts in ([0, n, n // 2, n], [n, 0, n, 0], [-5, n + 400, 3, 1 << 30]):
        q_start, slots = dev(np.array(starts, I32)), dev(np.array([0, 1, 2], I32))
        buf = torch.full((n + 2 * guard, C), 9.0, device="cuda")
        conv = binding.ConvState(3, dev(rng.standard_normal((C, 4)).astype(F32)))
        binding.conv_silu(conv, dev(rng.standard_normal((n, C)).astype(F32)), slots, q_start=q_start, out=buf[guard: guard + n])
        q, k, v, al, be, A, dt = (dev(t) for t in delta_inputs(rng, n, hk, hv, dk, dv, F32))
        state = binding.DeltaState(3, hk, hv, dk, dv)
        binding.delta_rule(state, q, k, v, al, be, slots, q_start=q_start, A=A, dt_bias=dt,
                           out=buf[guard: guard + n].unflatten(1, (1, 64)))
        torch.cuda.synchronize()
        assert (buf[:guard] == 9).all() and (buf[guard + n:] == 9).all()


def test_in_place_states_row_by_row():
    """n calls of a row leave the bits of one call of n rows."""
    rng = np.random.default_rng(5)
    n, hk, hv, dk, dv, C = 20, 2, 4, 128, 96, 300
    slots = dev(np.array([1], I32))
    q, k, v, al, be, A, dt = (dev(t) for t in delta_inputs(rng, n, hk, hv, dk, dv, F32))
    x, w = dev(rng.standard_normal((n, C)).astype(F32)), dev(rng.standard_normal((C, 5)).astype(F32))
    conv, state = (binding.ConvState(2, w), binding.ConvState(2, w)), [binding.DeltaState(2, hk, hv, dk, dv) for _ in range(2)]
    whole = [binding.conv_silu(conv[0], x, slots), binding.delta_rule(state[0], q, k, v, al, be, slots, A=A, dt_bias=dt)]
    parts = [torch.cat([binding.conv_silu(conv[1], x[i: i + 1], slots) for i in range(n)]),
             torch.cat([binding.delta_rule(state[1], q[i: i + 1], k[i: i + 1], v[i: i + 1], al[i: i + 1], be[i: i + 1], slots,
                                           A=A, dt_bias=dt) for i in range(n)])]
    torch.cuda.synchronize()
    same_bits(whole + [conv[0].pool, state[0].pool], parts + [conv[1].pool, state[1].pool])


def test_drafts_keep_the_state_of_the_accepted_ones():
    """The state after m of 17 drafts is that of a call of m rows, from the same slot."""
    rng = np.random.default_rng(6)
    n, hk, hv, dk, dv = 17, 1, 3, 128, 128
    q, k, v, al, be, A, dt = (dev(t) for t in delta_inputs(rng, n, hk, hv, dk, dv, F32))
    pool = dev(rng.standard_normal((3, hv, dv, dk)).astype(F32))
    a, b = dev(np.array([0], I32)), dev(np.array([2], I32))
    for m in (0, 1, 9, 17):
        two = [binding.DeltaState(3, hk, hv, dk, dv, pool=pool.clone()) for _ in range(2)]
        out = binding.delta_rule(two[0], q, k, v, al, be, a, b, commit=dev(np.array([m], I32)), A=A, dt_bias=dt)
        if m:
            short = binding.delta_rule(two[1], q[:m], k[:m], v[:m], al[:m], be[:m], a, b, A=A, dt_bias=dt)
            same_bits([short], [out[:m]])
        torch.cuda.synchronize()
        same_bits([two[0].pool], [two[1].pool])


def test_long_calls_in_several_launches():
    """More tiles than a launch's workspace holds: a sequence's state is carried, also past its neighbours'."""
    hk, hv, dk, dv = 16, 48, 128, 128
    g = torch.Generator("cuda").manual_seed(1)
    ns = [6500, 40, 3100]
    rows = sum(ns)
    x = torch.randn(rows, 2 * hk * dk + hv * dv, generator=g, device="cuda").half()
    q, k, v = (t.unflatten(1, s) for t, s in zip(x.split([hk * dk, hk * dk, hv * dv], 1), ((hk, dk), (hk, dk), (hv, dv))))
    al, be = (torch.randn(rows, hv, generator=g, device="cuda") for _ in range(2))
    A = -torch.rand(hv, generator=g, device="cuda")
    pool = torch.randn(4, hv, dv, dk, generator=g, device="cuda")
    slots = [dev(np.array(s, I32)) for s in ([0, 1, 2], [3, 1, 0])]
    commit = [6400, 40, 3100]
    q_start = dev(np.cumsum([0] + ns).astype(I32))
    whole = binding.DeltaState(4, hk, hv, dk, dv, pool=pool.clone())
    slot_out = dev(np.array([3, 1, 2], I32))
    out = binding.delta_rule(whole, q, k, v, al, be, slots[0], slot_out, q_start=q_start, commit=dev(np.array(commit, I32)), A=A)
    r0 = 0
    for s, n in enumerate(ns):
        # one by one, in pieces that end where tiles do
        one = binding.DeltaState(4, hk, hv, dk, dv, pool=pool.clone())
        src, got, m = slots[0][s: s + 1].contiguous(), [], commit[s]
        cuts = sorted({0, m, n} | set(range(0, m, 2048)))
        kept = None
        for a, b in zip(cuts, cuts[1:]):
            piece = slice(r0 + a, r0 + b)
            if n < 80:
                got.append(None)
            else:
                got.append(binding.delta_rule(one, q[piece], k[piece], v[piece], al[piece], be[piece], src, A=A))
            if b == m:
                kept = one.pool[s].clone()
        torch.cuda.synchronize()
        if n >= 80:
            same_bits([torch.cat(got), kept], [out[r0: r0 + n], whole.pool[slot_out[s].long()]])
        r0 += n
    assert torch.isfinite(out).all()


def test_offsets_past_32_bits():
    g = torch.Generator("cuda").manual_seed(2)
    # a pool of states of 4.8 GB, the last slot in use
    hk, hv, dk, dv = 1, 16, 128, 256
    state = binding.DeltaState(2300, hk, hv, dk, dv)
    small = binding.DeltaState(2, hk, hv, dk, dv)
    small.pool[1] = torch.randn(hv, dv, dk, generator=g, device="cuda")
    state.pool[2299] = small.pool[1]
    n = 100
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda") for h, d in ((hk, dk), (hk, dk), (hv, dv)))
    al = torch.randn(n, hv, generator=g, device="cuda")
    A = -torch.ones(hv, device="cuda")
    for m in (3, n):
        a = binding.delta_rule(state, q[:m], k[:m], v[:m], al[:m], al[:m], dev(np.array([2299], I32)), A=A)
        b = binding.delta_rule(small, q[:m], k[:m], v[:m], al[:m], al[:m], dev(np.array([1], I32)), A=A)
        same_bits([a, state.pool[2299]], [b, small.pool[1]])
    assert not state.pool[:2299].any()
    del state
    # 2.6 G logits in one call
    z = torch.randn(20011, 131075, generator=g, device="cuda", dtype=torch.float16)
    top = binding.logprobs(z, top=3)
    one = binding.logprobs(z[-300:], top=3)
    torch.cuda.synchronize()
    assert torch.equal(top.top_ids[-300:], one.top_ids)
    assert (top.lse[-300:] - one.lse).abs().max() <= 2.0 ** -19 + 2.0 ** -22 * 10
    # as many values through a norm
    y = z.view(-1)[: 20011 * 131072].view(20011 * 4, 1, 32768)
    w = torch.ones(32768, device="cuda")
    x = binding.block_norm(y, w, x_out=y)[1][-5:]
    torch.cuda.synchronize()
    assert ((x.double() ** 2).mean(-1) - 1).abs().max() < 2e-3


@pytest.mark.parametrize("n", [17, 200])
def test_recurrence_with_extreme_rows(n):
    """Keys and queries of any length, values of any scale, resets, steps next to 0 and 1."""
    def mutate(q, k, v, al, be, A):
        k[3] = 0
        q[4] = 0
        k[5:7] *= F32(1e-15)
        k[8] *= F32(1e15)
        q[9] *= F32(1e-12)
        q[10] *= F32(1e12)
        al[12] = 300   # a decay of e^-300 and more
        be[13] = -200  # (no step)
        be[14] = 200
        v[..., 5] *= F32(1e20)
        v[..., 6] *= F32(1e-20)
        v[..., 7] = 0
    check_delta(np.random.default_rng(n), [n], 1, 2, 128, 64, "plain", F32, mutate=mutate)


@pytest.mark.parametrize("n", [5, 200])
def test_recurrence_non_finite_rows_touch_nothing_else(n):
    rng = np.random.default_rng(n)
    nseq, hk, hv, dk, dv = 3, 2, 4, 64, 64
    rows = n * nseq
    ins = delta_inputs(rng, rows, hk, hv, dk, dv, F32)
    bad = [t.copy() for t in ins]
    bad[2][n + n // 2, 1, 3] = np.nan       # a value of sequence 1, head 1
    bad[1][2 * n + n // 2, 1, 0] = np.inf   # a key of sequence 2: heads 2 and 3
    bad[3][n + n // 2, 3] = np.nan          # a gate of sequence 1, head 3
    slots = dev(np.arange(3, dtype=I32))
    res = []
    for t in (ins, bad):
        st = binding.DeltaState(3, hk, hv, dk, dv)
        o = binding.delta_rule(st, *map(dev, t[:5]), slots, A=dev(t[5]), dt_bias=dev(t[6]))
        res.append((host(o).reshape(nseq, n, hv, dv), host(st.pool)))
    torch.cuda.synchronize()
    (a, sa), (b, sb) = res
    first = n // 2 // 64 * 64 if n >= 80 else n // 2  # rows before the tile of the bad one
    for s, h in ((0, 0), (0, 1), (0, 2), (0, 3), (1, 0), (1, 2), (2, 0), (2, 1)):
        assert (a[s, :, h] == b[s, :, h]).all() and (sa[s, h] == sb[s, h]).all()
    for s, h in ((1, 1), (1, 3), (2, 2), (2, 3)):
        assert (a[s, :first, h] == b[s, :first, h]).all()
        assert not np.isfinite(b[s, n // 2:, h]).all()


def test_conv_states_of_non_finite_rows():
    """What a row brings reaches taps rows and no other channel."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 8)).astype(F32)
    y = x.copy()
    y[10, 3], y[20, 5] = np.inf, np.nan
    w = rng.standard_normal((8, 4)).astype(F32)
    slots = dev(np.array([0], I32))
    a, b = (host(binding.conv_silu(binding.ConvState(1, dev(w)), dev(t), slots)) for t in (x, y))
    same = np.ones(a.shape, bool)
    same[10:14, 3] = same[20:24, 5] = False
    assert (a[same] == b[same]).all() and not np.isfinite(b[10:14, 3]).all() and np.isnan(b[20:24, 5]).all()


def test_zero_rows():
    slots = dev(np.array([0], I32))
    st = binding.DeltaState(1, 1, 1, 64, 64)
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    assert binding.delta_rule(st, e(0, 1, 64), e(0, 1, 64), e(0, 1, 64), e(0, 1), e(0, 1), slots, A=e(1)).shape == (0, 1, 64)
    assert binding.conv_silu(binding.ConvState(1, e(8, 4)), e(0, 8), slots).shape == (0, 8)
    assert binding.block_norm(e(0, 2, 8))[1].shape == (0, 2, 8)
    assert binding.logprobs(e(0, 9), top=2).top_ids.shape == (0, 2)


def test_logprobs_of_many_columns_and_strides():
    """Rows side by side past one block's, parts of rows of every length, logits that repeat."""
    rng = np.random.default_rng(9)
    z = rng.standard_normal((67, 5000)).astype(F32)
    for view in (dev(z.T).t(), dev(np.repeat(z, 2, 1))[:, ::2], dev(z)[:1].expand(67, 5000), dev(z)[:, 1:4098]):
        want = host(view)
        got = binding.logprobs(view, top=33, scale=0.9)
        torch.cuda.synchronize()
        _, (lse, le), (ent, ee), ids, (tl, te) = ref.logprobs(want, None, 33, 0.9)
        ref.near(host(got.lse), lse, le)
        ref.near(host(got.entropy), ent, ee)
        assert (host(got.top_ids) == ids).all()
        ref.near(host(got.top_lp), tl, te)


@pytest.mark.parametrize("dim", [256, 257, 512, 1023, 1024, 1025, 2049, 2560, 4096, 4097, 8192, 8193])
@pytest.mark.parametrize("skew", [0, 1])
def test_block_norm_lengths_where_the_threads_change(dim, skew):
    rng = np.random.default_rng(dim)
    y, r = (rng.standard_normal((5, 1, dim)).astype(F32) for _ in range(2))
    y[2], y[3, :, ::2] = 1e25, 0  # (squares beyond fp32; half a row of zeros)
    w = (1 + 0.1 * rng.standard_normal(dim)).astype(F32)
    h, x, eh, ex = ref.block_norm(y, w, None, "none", 0.5, r, w, 1e-6)
    lay = lambda a: dev(np.pad(a, ((0, 0), (0, 0), (skew, 0))))[:, :, skew:]  # noqa: E731  (rows off 16 bytes)
    ho, xo = (lay(np.zeros_like(y)) for _ in range(2))
    binding.block_norm(lay(y), dev(w), residual=lay(r), scale=0.5, pre_norm=dev(w), eps=1e-6, h_out=ho, x_out=xo)
    torch.cuda.synchronize()
    ref.rounded(host(ho), h, eh, F32)
    ref.rounded(host(xo), x, ex, F32)


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("vocab", [1000, 8200, 70001])
def test_logprobs_of_rows_side_by_side_in_unequal_groups(rows, vocab):
    rng = np.random.default_rng(rows + vocab)
    z = (4 * rng.standard_normal((rows, vocab))).astype(F32)
    z[:, 5:40] = z[:, 4:5]         # equals
    z[rows // 2, 7:] = -np.inf     # fewer than are asked for
    tok = rng.integers(-1, vocab, (rows, 70)).astype(I32)
    for zd in (dev(z), dev(z.T.copy()).t()):
        got = binding.logprobs(zd, dev(tok), top=12)
        torch.cuda.synchronize()
        m = z.max(1, keepdims=True).astype(np.float64)
        lse = m[:, 0] + np.log(np.exp(z - m).sum(1))
        order = np.lexsort((np.broadcast_to(np.arange(vocab), z.shape), -z), axis=1)[:, :12]
        best = np.take_along_axis(z, order, 1)
        ids = np.where(best > -np.inf, order, -1)
        assert np.array_equal(host(got.top_ids), ids)
        tol = 2.0 ** -20 * (1 + np.abs(lse) + np.abs(m[:, 0]))  # a logit, its maximum and a log, each off by a few 2^-23
        assert np.all(np.abs(host(got.lse) - lse) <= tol)
        want = np.where(tok >= 0, np.take_along_axis(z, np.maximum(tok, 0), 1) - lse[:, None], 0.0)
        have = host(got.token_lp)
        fin = np.isfinite(want)
        assert np.array_equal(have[~fin], want[~fin])
        assert np.all(np.abs(have[fin] - want[fin]) <= (2.0 ** -20 * (1 + np.abs(want) + np.abs(lse)[:, None] + np.abs(m)))[fin])


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("dim", [64, 9000])
def test_gates_of_any_size(act, dim):
    far = np.array([-np.inf, np.finfo(F32).min, -1e30, -65504, -1000, -104, -100, -88, -87.1, -87, -86.9, -30, -1e-30, -0.0, 0, 1e-30,
                    30, 86.9, 87, 88, 100, 65504, 1e30], F32)
    rng = np.random.default_rng(dim)
    y = rng.standard_normal((4, 1, dim)).astype(F32)
    z = rng.choice(far, (4, 1, dim))
    z[0, 0, :far.size] = far
    w = np.ones(dim, F32)
    with np.errstate(over="ignore", invalid="ignore"):
        n = y / np.sqrt((y.astype(np.float64) ** 2).mean(-1, keepdims=True) + 1e-6)
        s = 1 / (1 + np.exp(-z.astype(np.float64)))
        a = s if act == "sigmoid" else np.where(z == -np.inf, 0, z.astype(np.float64) * s)
    h = torch.empty(4, 1, dim, device="cuda")
    binding.block_norm(dev(y), dev(w), dev(z), act, eps=1e-6, h_out=h)
    torch.cuda.synchronize()
    ref.rounded(host(h), n * a, 2.0 ** -20 * np.abs(n * a) + 2.0 ** -119 * np.abs(n), F32)  # the header's terms
    z[1, 0, 3] = np.nan
    binding.block_norm(dev(y), dev(w), dev(z), act, eps=1e-6, h_out=h)
    torch.cuda.synchronize()
    assert list(zip(*np.where(np.isnan(host(h))))) == [(1, 0, 3)]


def test_convolution_far_below_zero():
    C = 256
    x = np.zeros((6, C), F32)
    x[:, 0::4], x[:, 1::4], x[:, 2::4], x[:, 3::4] = -1e30, np.finfo(F32).min, -90, -60000
    w = np.zeros((C, 4), F32)
    w[:, 3] = 1
    conv = binding.ConvState(1, dev(w))
    y = binding.conv_silu(conv, dev(x), dev(np.zeros(1, I32)))
    torch.cuda.synchronize()
    assert y.dtype == torch.float32 and np.all(np.abs(host(y)) <= 2.0 ** -119)
