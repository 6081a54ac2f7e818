"""GPU: block norms, the short convolution, the gated delta recurrence and log
probabilities against the numpy forms, through the torch helpers of the C ABI."""
import numpy as np
import pytest

import token_ref as ref
from gpu_util import needs_gpu, torch

pytestmark = [pytest.mark.gpu, needs_gpu]

if torch is not None:
    from quant_dequant_gemv_amd import binding

F16, F32 = np.float16, np.float32


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().cpu().numpy()


def laid(x, layout):
    """x [rows, ...] on the GPU in a layout, as a view of that shape."""
    if x is None:
        return None
    if layout == "column":  # [n][rows]: as a GEMV writes it
        return dev(x.reshape(len(x), -1).T).t().unflatten(1, x.shape[1:])
    if layout == "odd":  # odd strides and an offset
        b = np.full((len(x), x[0].size + 5), 7, x.dtype)
        b[:, 3:-2] = x.reshape(len(x), -1)
        return dev(b)[:, 3:-2].unflatten(1, x.shape[1:])
    if layout == "wide":  # whole pieces of 16 bytes, rows apart
        b = np.full((len(x), x[0].size + 8), 7, x.dtype)
        b[:, :-8] = x.reshape(len(x), -1)
        return dev(b)[:, :-8].unflatten(1, x.shape[1:])
    return dev(x)


# ------------------------------------------------------------------ block norm

@pytest.mark.parametrize("rows,groups,dim", [(1, 1, 5120), (17, 1, 5120), (3, 5, 128), (33, 3, 64), (2, 7, 40), (5, 2, 1),
                                             (4, 1, 513), (2, 3, 2048), (3, 1, 8191), (2, 1, 8196), (3, 1, 12345), (2, 1, 32768),
                                             (1, 4, 300), (70, 48, 128)])
@pytest.mark.parametrize("layout,dt", [("plain", F32), ("column", F32), ("odd", F16), ("wide", F16)])
@pytest.mark.parametrize("what", ["all", "residual", "heads", "pre"])
def test_block_norm(rows, groups, dim, layout, dt, what):
    rng = np.random.default_rng(rows + groups + dim)
    mk = lambda t: laid(t, layout)  # noqa: E731
    y, z = ((2 * rng.standard_normal((rows, groups, dim))).astype(dt) for _ in range(2))
    res = (3 * rng.standard_normal((rows, groups, dim))).astype(F32)
    post, pre = ((1 + 0.3 * rng.standard_normal(dim)).astype(F32) for _ in range(2))
    act, scale, eps = {"all": "silu", "heads": "sigmoid"}.get(what, "none"), 0.75, 1e-5
    if what == "residual":
        post = z = pre = None
    elif what == "heads":
        res = pre = None
    elif what == "pre":
        post = z = res = None
    h, x, eh, ex = ref.block_norm(y, post, z, act, scale, res, pre, eps)
    args = dict(post_norm=dev(post), gate=mk(z), act=act, scale=scale, residual=mk(res), pre_norm=dev(pre), eps=eps)
    none, got = binding.block_norm(mk(y), **args)
    ho = mk(np.zeros((rows, groups, dim), F32))
    xo = laid(np.zeros((rows, groups, dim), dt), layout)
    same_h, same_x = binding.block_norm(mk(y), h_out=ho, x_out=xo, **args)
    torch.cuda.synchronize()
    assert none is None and got.dtype == torch.float16 and same_h is ho and same_x is xo
    ref.rounded(host(got), x, ex, F16)
    ref.rounded(host(ho), h, eh, F32)
    ref.rounded(host(xo), x, ex, dt)


@pytest.mark.parametrize("dim", [96, 5120, 9000])
def test_block_norm_in_place_and_h_alone(dim):
    rng = np.random.default_rng(dim)
    y, z, r = (rng.standard_normal((6, 2, dim)).astype(F32) for _ in range(3))
    w = (1 + 0.1 * rng.standard_normal(dim)).astype(F32)
    h, x, eh, ex = ref.block_norm(y, w, z, "silu", 1.0, r, w, 1e-6)
    yd, rd, wd = dev(y), dev(r), dev(w)
    out = binding.block_norm(yd, wd, dev(z), residual=rd, pre_norm=wd, h_out=rd, x_out=yd)
    torch.cuda.synchronize()
    assert out[0] is rd and out[1] is yd
    ref.rounded(host(rd), h, eh, F32)
    ref.rounded(host(yd), x, ex, F32)
    ho = torch.empty(6, 2, dim, dtype=torch.float16, device="cuda")
    assert binding.block_norm(dev(y), wd, dev(z), residual=dev(r), h_out=ho) == (ho, None)
    torch.cuda.synchronize()
    ref.rounded(host(ho), h, eh, F16)


def test_block_norm_broadcast_gates_and_extreme_rows():
    rng = np.random.default_rng(3)
    y = rng.standard_normal((5, 3, 200)).astype(F32)
    y[1] *= F32(1e30)   # squares beyond fp32
    y[2] *= F32(1e-30)
    y[3] = 0
    w = np.ones(200, F32)
    channel, token = rng.standard_normal(200).astype(F32), rng.standard_normal(5).astype(F32)
    got = {}
    for name, gate in (("channel", dev(channel).expand(5, 3, 200)), ("token", dev(token)[:, None, None].expand(5, 3, 200))):
        got[name] = binding.block_norm(dev(y), dev(w), gate, act="none", eps=0.0 if name == "channel" else 1e-6,
                                       x_out=torch.empty(5, 3, 200, device="cuda"))[1]
    torch.cuda.synchronize()
    live = [0, 1, 2, 4]  # (a row of zeros without eps is 0 / 0)
    _, x, _, ex = ref.block_norm(y[live], w, np.broadcast_to(channel, (4, 3, 200)), "none", 1.0, None, None, 0.0)
    ref.rounded(host(got["channel"])[live], x, ex, F32)
    assert np.isnan(host(got["channel"])[3]).all()
    _, x, _, ex = ref.block_norm(y, w, np.broadcast_to(token[:, None, None], y.shape), "none", 1.0, None, None, 1e-6)
    ref.rounded(host(got["token"]), x, ex, F32)


def test_block_norm_non_finite_rows_stay_their_own():
    rng = np.random.default_rng(4)
    y = rng.standard_normal((9, 4, 128)).astype(F32)
    clean = y.copy()
    y[2, 1, 5], y[4, 0, 0], y[7, 3, 127] = np.nan, np.inf, -np.inf
    w = dev(np.ones(128, F32))
    a, b = (host(binding.block_norm(dev(t), w, pre_norm=w)[1]) for t in (y, clean))
    bad = np.zeros((9, 4), bool)
    bad[2, 1] = bad[4, 0] = bad[7, 3] = True
    assert np.isnan(a[2, 1]).all() and np.isnan(a[4, 0]).any() and (a[~bad] == b[~bad]).all()


# ------------------------------------------------------------------ sequences with a state

def state_case(rng, ns, spare=3, commit=None, fresh=False, holes=False):
    """Arrays of a call over sequences of ns rows, their states in one half of a pool and left in the other."""
    nseq = len(ns)
    num = 2 * (nseq + spare)
    slots = rng.permutation(nseq + spare)[:nseq].astype(np.int32)
    out = (nseq + spare + rng.permutation(nseq + spare)[:nseq]).astype(np.int32)
    kv = np.array([n + int(rng.integers(0, 3)) if fresh else n + 5 for n in ns], np.int32)
    if holes and nseq > 2:
        slots[0], out[1], slots[2] = -1, num, num + 7
    q_start = None if len(set(ns)) == 1 else np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    c = None if commit is None else np.array([int(rng.integers(-1, n + 3)) for n in ns], np.int32)
    return dict(slots=slots, slots_out=out, q_start=q_start, kv_len=kv, commit=c), num


def seq_list(a, rows, num):
    return list(ref.sequences(rows, len(a["slots"]), a["q_start"], a["slots"], a["slots_out"], a["kv_len"], a["commit"], num))


NS = [[1], [1] * 37, [17], [5, 0, 1, 33, 2, 64], [16, 48, 200, 3], [31, 31, 31]]


@pytest.mark.parametrize("ns", NS)
@pytest.mark.parametrize("C,taps,bias,act", [(256, 4, False, "silu"), (1028, 2, True, "none"), (37, 8, True, "silu"),
                                             (2052, 3, False, "silu"), (5, 5, False, "silu"), (320, 6, True, "silu"), (64, 7, False, "none")])
@pytest.mark.parametrize("layout,dt", [("plain", F32), ("column", F32), ("odd", F16), ("wide", F16)])
def test_conv(ns, C, taps, bias, act, layout, dt):
    rng = np.random.default_rng(C + len(ns))
    rows = sum(ns)
    a, num = state_case(rng, ns, commit=taps % 2 or None, fresh=C != 37, holes=True)
    pool = rng.standard_normal((num, taps - 1, C)).astype(F32)
    w, b = rng.standard_normal((C, taps)).astype(F32), rng.standard_normal(C).astype(F32) if bias else None
    x = (2 * rng.standard_normal((rows, C))).astype(dt)
    y, err, new = ref.conv_silu(pool, w, b, x, seq_list(a, rows, num), act == "silu")
    conv = binding.ConvState(num, dev(w), dev(b), pool=dev(pool))
    got = binding.conv_silu(conv, laid(x, layout), **{k: dev(v) for k, v in a.items()}, act=act)
    torch.cuda.synchronize()
    ref.rounded(host(got), y, err, dt)
    assert (host(conv.pool) == new).all()


def delta_inputs(rng, rows, hk, hv, dk, dv, dt, raw=True):
    q, k, v = (rng.standard_normal((rows, h, d)).astype(dt) for h, d in ((hk, dk), (hk, dk), (hv, dv)))
    al, be = (rng.standard_normal((rows, hv)).astype(dt) for _ in range(2))
    if raw:
        A = -np.exp(rng.uniform(-1, 2.8, hv)).astype(F32)
        return q, k, v, al, be, A, np.log(np.expm1(np.exp(rng.uniform(-7, -2, hv)))).astype(F32)
    return q, k, v, -np.abs(al), ref.sigmoid(be.astype(np.float64)).astype(dt), None, None


def check_delta(rng, ns, hk, hv, dk, dv, layout, dt, raw=True, out_dt=F32, commit=None, fresh=False, holes=False, mutate=None,
                eps=1e-6, scale=None):
    rows = sum(ns)
    a, num = state_case(rng, ns, commit=commit, fresh=fresh, holes=holes)
    q, k, v, al, be, A, dt_b = delta_inputs(rng, rows, hk, hv, dk, dv, dt, raw)
    if mutate:
        mutate(q, k, v, al, be, A)
    pool = (0.3 * rng.standard_normal((num, hv, dv, dk))).astype(F32)
    out, err, new, new_err = ref.delta_rule(pool, q, k, v, al, be, seq_list(a, rows, num), A, dt_b, True, eps,
                                            dk ** -0.5 if scale is None else scale)
    state = binding.DeltaState(num, hk, hv, dk, dv, pool=dev(pool))
    mk = lambda t: laid(t, layout)  # noqa: E731
    ins = [mk(t) for t in (q, k, v, al, be)]
    arr = {n: dev(t) for n, t in a.items()}
    o = laid(np.full((rows, hv, dv), 9, out_dt), layout)
    got = binding.delta_rule(state, *ins, **arr, A=dev(A), dt_bias=dev(dt_b), eps=eps, scale=scale, out=o)
    torch.cuda.synchronize()
    assert got is o
    ref.rounded(host(o), out, err, out_dt)
    after = host(state.pool).astype(np.float64)
    d = np.sqrt(((after - new) ** 2).sum(-1))
    assert (d <= new_err + 2.0 ** -24 * np.sqrt((new ** 2).sum(-1)) + 2.0 ** -140).all()
    untouched = np.setdiff1d(np.arange(num), [s[3] for s in seq_list(a, rows, num) if s[3] is not None and s[4] > 0])
    assert (host(state.pool)[untouched] == pool[untouched]).all()
    # the state alone, and again: the same bits
    again = binding.DeltaState(num, hk, hv, dk, dv, pool=dev(pool))
    assert binding.delta_rule(again, *ins, **arr, A=dev(A), dt_bias=dev(dt_b), eps=eps, scale=scale, state_only=True) is None
    torch.cuda.synchronize()
    assert (host(again.pool) == host(state.pool)).all()
    return host(o)


@pytest.mark.parametrize("ns", NS)
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 1, 128, 128), (2, 6, 128, 64), (3, 3, 64, 96), (1, 2, 64, 256), (2, 2, 128, 32)])
@pytest.mark.parametrize("layout,dt", [("plain", F32), ("column", F32), ("odd", F16), ("wide", F16)])
def test_delta(ns, hk, hv, dk, dv, layout, dt):
    rng = np.random.default_rng(len(ns) + hv + dv)
    check_delta(rng, ns, hk, hv, dk, dv, layout, dt, raw=hv != 3, out_dt=F16 if layout == "wide" else F32,
                commit=True if dk == 128 else None, fresh=hv != 1, holes=dv != 96)


LONG = [[64], [65], [200], [63, 130, 0, 64, 129], [128] * 3, [700, 1, 66]]


@pytest.mark.parametrize("ns", LONG)
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 1, 128, 128), (2, 6, 128, 64), (9, 9, 64, 96), (1, 2, 64, 256)])
@pytest.mark.parametrize("layout,dt", [("plain", F32), ("column", F32), ("odd", F16), ("wide", F16)])
def test_delta_long(ns, hk, hv, dk, dv, layout, dt):
    rng = np.random.default_rng(len(ns) + hv + dv)
    check_delta(rng, ns, hk, hv, dk, dv, layout, dt, out_dt=F16 if layout == "wide" else F32, commit=True if dk == 128 else None,
                fresh=hv != 1, holes=dv != 96)


# ------------------------------------------------------------------ log probabilities

def check_probs(z, tokens, top, scale, layout):
    tok = None if tokens is None else tokens.astype(np.int32)
    (t, te), (lse, le), (ent, ee), ids, (tl, tle) = ref.logprobs(z, tok, top, scale)
    got = binding.logprobs(laid(z, layout), dev(tok), top=top, scale=scale)
    again = binding.logprobs(laid(z, layout), dev(tok), top=top, scale=scale)
    torch.cuda.synchronize()
    ref.near(host(got.lse), lse, le)
    ref.near(host(got.entropy), ent, ee)
    if tok is not None:
        ref.near(host(got.token_lp), t, te)
    if top:
        assert (host(got.top_ids) == ids).all()
        ref.near(host(got.top_lp), tl, tle)
    for a, b in zip(got, again):
        assert a is None and b is None or (host(a).view(np.int32) == host(b).view(np.int32)).all()


@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 5), (1, 1000), (17, 4099), (1, 160001), (33, 257), (70, 2048), (3, 32768),
                                        (600, 300)])
@pytest.mark.parametrize("layout,dt", [("plain", F32), ("column", F32), ("odd", F16), ("plain", F16), ("column", F16)])
@pytest.mark.parametrize("ntok,top,scale", [(1, 20, 1.0), (0, 64, 0.5), (3, 1, 1.7), (70, 0, 1.0)])
def test_logprobs(rows, vocab, layout, dt, ntok, top, scale):
    rng = np.random.default_rng(rows + vocab)
    z = (3 * rng.standard_normal((rows, vocab)) - 2).astype(dt)
    tokens = rng.integers(-2, vocab + 2, (rows, ntok)) if ntok else None
    check_probs(z, tokens, top, scale, layout)


@pytest.mark.parametrize("layout", ["plain", "column", "odd"])
@pytest.mark.parametrize("dt", [F32, F16])
def test_logprobs_masks_ties_and_non_finite(layout, dt):
    rng = np.random.default_rng(8)
    V = 3001
    z = (2 * rng.standard_normal((14, V))).astype(dt)
    z[0] = -np.inf                       # nothing left
    z[1, :-1] = -np.inf                  # one token left
    z[2, 7:] = -np.inf                   # fewer than asked for
    z[3] = 1.5                           # all equal
    z[4, ::2], z[4, 1::2] = 0.0, -0.0    # equal too
    z[5] = np.finfo(dt).min              # masks by the type's lowest value
    z[5, 100:103] = 3
    z[6] = np.finfo(dt).min
    z[7, 11] = np.nan
    z[8, 2000] = np.inf
    z[9] = np.sort(z[9])                 # ever larger
    z[10] = np.sort(z[10])[::-1]
    z[11, 5] = np.finfo(dt).max / 2      # one far above the others
    z[12] = -np.inf
    z[12, 3000] = np.nan
    tokens = rng.integers(0, V, (14, 4))
    tokens[:, 0] = [5, 3000, 3, 0, 1, 100, 0, 11, 2000, 3000, 0, 5, 0, 0]
    check_probs(z, tokens, 20, 1.0, layout)


# ------------------------------------------------------------------ a layer, as it is used

@pytest.mark.parametrize("ncols", [1, 5])
def test_a_recurrent_layer_behind_its_gemvs(ncols):
    """norm -> qkv and gates' GEMVs -> convolution -> recurrence -> gated head norm -> output GEMV + residual -> norm ->
    head -> log probabilities, feature-major throughout; step by step against the numpy forms on the GPU's own inputs."""
    import oracle
    from quant_dequant_gemv_amd import synth
    H, hk, hv, dk, dv, V = 512, 2, 4, 64, 64, 768
    C = 2 * hk * dk + hv * dv
    rng = np.random.default_rng(ncols)
    W = {n: synth.superblocks(synth.Q4_K, N, K, i) for i, (n, N, K) in enumerate(
        [("qkv", C, H), ("z", hv * dv, H), ("ab", 256, H), ("out", H, hv * dv), ("head", V, H)])}
    gemv = lambda n, x, N, K, **kw: binding.gemv_ex(binding.Q4_K, dev(W[n].reshape(-1)), x, N, K, **kw)  # noqa: E731
    h0 = rng.standard_normal((H, ncols)).astype(F32)
    wn, wo = (1 + 0.1 * rng.standard_normal(n).astype(F32) for n in (H, dv))
    A, dtb = -np.exp(rng.uniform(0, 1, hv)).astype(F32), rng.uniform(-3, -1, hv).astype(F32)
    conv = binding.ConvState(3, dev(0.4 * rng.standard_normal((C, 4)).astype(F32)))
    conv.pool.copy_(dev(rng.standard_normal((3, 3, C)).astype(F32)))
    state = binding.DeltaState(3, hk, hv, dk, dv, pool=dev(0.2 * rng.standard_normal((3, hv, dv, dk)).astype(F32)))
    slots, out_slots = dev(np.array([1], np.int32)), dev(np.array([2], np.int32))
    cp, sp = host(conv.pool).copy(), host(state.pool).copy()
    rows_of = lambda y, *s: y.view(*s, ncols).movedim(-1, 0)  # noqa: E731
    hid = dev(h0)
    x = torch.empty(H, ncols, dtype=torch.float16, device="cuda")
    binding.block_norm(rows_of(hid, 1, H), pre_norm=dev(wn), x_out=rows_of(x, 1, H))
    qkv, z, ab = gemv("qkv", x, C, H), gemv("z", x, hv * dv, H), gemv("ab", x, 256, H)
    y = binding.conv_silu(conv, rows_of(qkv, C), slots, out_slots)
    q, k, v = (t.unflatten(1, s) for t, s in zip(y.split([hk * dk, hk * dk, hv * dv], 1), ((hk, dk), (hk, dk), (hv, dv))))
    al, be = rows_of(ab[:hv], hv) * 1e-2, rows_of(ab[hv: 2 * hv], hv) * 1e-2
    o = binding.delta_rule(state, q, k, v, al, be, slots, out_slots, A=dev(A), dt_bias=dev(dtb))
    g = torch.empty(hv * dv, ncols, dtype=torch.float16, device="cuda")
    binding.block_norm(o, dev(wo), rows_of(z, hv, dv), act="silu", x_out=rows_of(g, hv, dv))
    h1 = gemv("out", g, H, hv * dv, residual=hid)
    x2 = torch.empty_like(x)
    binding.block_norm(rows_of(h1, 1, H), pre_norm=dev(wn), x_out=rows_of(x2, 1, H))
    logits = gemv("head", x2, V, H)
    probs = binding.logprobs(rows_of(logits, V), top=4)
    torch.cuda.synchronize()

    at = lambda t, *s: np.moveaxis(host(t).reshape(*s, ncols), -1, 0)  # noqa: E731
    seqs = [(0, ncols, 1, 2, ncols)]
    _, r, _, e = ref.block_norm(at(hid, 1, H), None, None, "none", 1.0, None, wn, 1e-6)
    ref.rounded(at(x, 1, H), r, e, F16)
    r, e, new = ref.conv_silu(cp, host(conv.weight), None, at(qkv, C), seqs, True)
    ref.rounded(host(y), r, e, F32)
    assert (host(conv.pool) == new).all()
    r, e, new, ne = ref.delta_rule(sp, *(host(t) for t in (q, k, v, al, be)), seqs, A, dtb, True, 1e-6, dk ** -0.5)
    ref.rounded(host(o), r, e, F32)
    assert (np.sqrt(((host(state.pool) - new) ** 2).sum(-1)) <= ne + 2.0 ** -24 * np.sqrt((new ** 2).sum(-1))).all()
    _, r, _, e = ref.block_norm(host(o), wo, at(z, hv, dv), "silu", 1.0, None, None, 1e-6)
    ref.rounded(at(g, hv, dv), r, e, F16)
    yo, S = oracle.gemv(synth.Q4_K, W["out"], host(g), hv * dv)
    assert (np.abs(host(h1) - (host(hid) + yo)) <= 1e-4 * S + 2.0 ** -23 * np.abs(yo + host(hid))).all()
    _, r, _, e = ref.block_norm(at(h1, 1, H), None, None, "none", 1.0, None, wn, 1e-6)
    ref.rounded(at(x2, 1, H), r, e, F16)
    _, (lse, le), _, ids, _ = ref.logprobs(at(logits, V), None, 4, 1.0)
    ref.near(host(probs.lse), lse, le)
    assert (host(probs.top_ids) == ids).all()
