"""GPU: norm + rotation, the paged 4-bit cache and attention over it against
the numpy reference, through the torch helpers of the C ABI."""
import numpy as np
import pytest

import kv_ref
from gpu_util import needs_gpu, torch

pytestmark = [pytest.mark.gpu, needs_gpu]

if torch is not None:
    from quant_dequant_gemv_amd import binding


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def freqs(half, base=1e7):
    return (base ** (-np.arange(half) / max(1, half))).astype(np.float32)


def make_rope(rng, D, rot, interleaved, norm):
    f = freqs(rot // 2)
    w = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in range(2)]
    rope = binding.Rope(dev(f) if rot else None, interleaved, *(None if x is None else dev(x) for x in w), eps=1e-5)
    return rope, f if rot else None, w


def close_to_rounding(got, ref, dtype):
    """One rounding of the fp64 value (through fp32 for fp16: a double rounding), 2^-40 relative for fp64's own."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref)
    half = 2.0 ** -11 * np.abs(ref) * (1 + 2.0 ** -12) + 2.0 ** -25 if dtype == np.float16 else 2.0 ** -24 * np.abs(ref)
    assert (np.abs(got - ref) <= half + 2.0 ** -40 * np.abs(ref).max() + 2.0 ** -140).all()


def strided(x, layout, np_dtype):
    """x [rows, heads, D] in memory of a layout, as a torch view of that shape (and its buffer)."""
    rows, heads, D = x.shape
    x = x.astype(np_dtype)
    if layout == "token":
        return dev(x)
    if layout == "column":  # [heads * D][rows]: as a GEMV writes it
        return dev(x.transpose(1, 2, 0)).permute(2, 0, 1)
    if layout == "gated":  # [heads][2][D][rows]: every head's gate behind it
        b = np.full((heads, 2, D, rows), 7, np_dtype)
        b[:, 0] = x.transpose(1, 2, 0)
        return dev(b)[:, 0].permute(2, 0, 1)
    b = np.full((rows, heads + 3, D + 5), 7, np_dtype)  # odd strides and an offset
    b[:, 2:-1, 1:D + 1] = x
    return dev(b)[:, 2:-1, 1:D + 1]


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 0), (128, 2), (128, 128), (256, 64), (256, 256), (256, 22)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,hq,hk,layout,dt", [(1, 24, 4, "gated", np.float32), (17, 6, 2, "column", np.float32),
                                                  (131, 3, 1, "odd", np.float16), (1, 1, 0, "token", np.float16)])
def test_norm_rope(D, rot, interleaved, rows, hq, hk, layout, dt):
    rng = np.random.default_rng(D + rot + rows)
    rope, f, (wq, wk) = make_rope(rng, D, rot, interleaved, norm=rows != 131)
    pos = rng.integers(-5, 1 << 20, rows).astype(np.int32)
    q = (rng.standard_normal((rows, hq, D)) * 3).astype(dt)
    k = rng.standard_normal((rows, hk, D)).astype(dt) if hk else None
    qo, ko = binding.norm_rope(rope, dev(pos), strided(q, layout, dt), None if k is None else strided(k, layout, dt))
    out32 = torch.full((hq, D, rows + 1), 9.0, device="cuda")
    binding.norm_rope(rope, dev(pos), strided(q, layout, dt), q_out=out32[:, :, :rows].permute(2, 0, 1))
    torch.cuda.synchronize()
    ref = kv_ref.norm_rope(q, pos, f, interleaved, wq, 1e-5)
    close_to_rounding(qo.cpu().numpy(), ref, np.float16)
    close_to_rounding(out32[:, :, :rows].permute(2, 0, 1).cpu().numpy(), ref, np.float32)
    assert (out32[:, :, rows] == 9).all()
    if hk:
        close_to_rounding(ko.cpu().numpy(), kv_ref.norm_rope(k, pos, f, interleaved, wk, 1e-5), np.float16)
    else:
        assert ko is None


def test_norm_rope_in_place_keys_alone_and_non_finite_rows():
    rng = np.random.default_rng(5)
    rope, f, (_, wk) = make_rope(rng, 128, 128, False, True)
    k = rng.standard_normal((9, 4, 128)).astype(np.float32)
    k[3, 1] = 0
    k[5, 2, 7] = np.nan
    pos = np.arange(9, dtype=np.int32)
    kd = dev(k)
    none, same = binding.norm_rope(rope, dev(pos), None, kd, k_out=kd)
    torch.cuda.synchronize()
    assert none is None and same is kd
    got = kd.cpu().numpy()
    assert np.isnan(got[5, 2]).all()
    got[5, 2] = k[5, 2] = 0
    close_to_rounding(got, kv_ref.norm_rope(k, pos, f, False, wk, 1e-5), np.float32)


# ------------------------------------------------------------------ append and read

def rows_of(ns):
    return [(s, i, n) for s, n in enumerate(ns) for i in range(n)]


@pytest.mark.parametrize("D,hkv,ps,rot,interleaved", [(64, 1, 32, 64, True), (64, 5, 128, 20, False),
                                                      (128, 8, 32, 128, False), (128, 3, 64, 0, False),
                                                      (256, 4, 64, 64, False), (256, 1, 1024, 256, True)])
@pytest.mark.parametrize("layout,dt", [("column", np.float32), ("odd", np.float16)])
@pytest.mark.parametrize("ns", [[1], [17], [3, 0, 1, 40, 2], [1] * 70])
def test_append_writes_the_documented_bytes(D, hkv, ps, rot, interleaved, layout, dt, ns):
    rng = np.random.default_rng(D + hkv + ps + len(ns))
    nseq, rows = len(ns), sum(ns)
    rope, f, (wq, wk) = make_rope(rng, D, rot, interleaved, norm=D != 64)
    mp = max(2, -(-64 // ps) + 1)
    kv_len = np.array([n + rng.integers(0, mp * ps - n) for n in ns], np.int32)
    pages = rng.permutation(nseq * mp + 2)[: nseq * mp].reshape(nseq, mp).astype(np.int32)
    k, v = (rng.standard_normal((rows, hkv, D)).astype(dt) * dt(2) for _ in range(2))
    q = rng.standard_normal((rows, 2 * hkv, D)).astype(dt)
    pb = 2 * hkv * ps * D * 5 // 8
    before = rng.integers(0, 256, (nseq * mp + 2, pb), dtype=np.uint8)
    cache = binding.KVCache(nseq * mp + 2, hkv, D, ps, pool=dev(before))
    q_start = dev(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)) if len(set(ns)) > 1 else None
    args = (strided(k, layout, dt), strided(v, layout, dt), dev(pages), dev(kv_len))
    qo = binding.kv_append(cache, *args, q_start=q_start, q=strided(q, layout, dt), rope=rope)
    rk, rv = binding.kv_read(cache, rows, dev(pages), dev(kv_len), q_start=q_start)
    torch.cuda.synchronize()

    where = rows_of(ns)
    pos = np.array([kv_len[s] - n + i for s, i, n in where])
    kr = kv_ref.norm_rope(k, pos, f, interleaved, wk, 1e-5).astype(np.float32)
    close_to_rounding(qo.cpu().numpy(), kv_ref.norm_rope(q, pos, f, interleaved, wq, 1e-5), np.float16)
    fk, fv = kv_ref.quantise(kr), kv_ref.quantise(v.astype(np.float32))
    assert np.array_equal(rk.cpu().numpy(), kv_ref.values(*fk).astype(np.float32))
    assert np.array_equal(rv.cpu().numpy(), kv_ref.values(*fv).astype(np.float32))
    # the bytes of the written positions, and no others: unwritten bytes of every touched page are as they were
    after = cache.pool.cpu().numpy()
    zero = np.zeros((ps, hkv, D), np.uint8), np.zeros((ps, hkv, D // 32), np.float16)
    touched = {}
    for t, (s, i, n) in enumerate(where):
        touched.setdefault(int(pages[s, pos[t] // ps]), []).append((t, pos[t] % ps))
    for page, items in list(touched.items())[:6]:
        want = [zero[0].copy(), zero[1].copy(), zero[1].copy(), zero[0].copy(), zero[1].copy(), zero[1].copy()]
        mask = [w.copy() for w in want]
        for t, p in items:
            for x, src in zip(want, (*fk, *fv)):
                x[p] = src[t]
            for x, ones in zip(mask, (15, 0, 0, 15, 0, 0)):
                x[p] = ones if ones else np.uint16(0xffff).view(np.float16)
        m = kv_ref.pack_page(*mask)
        assert np.array_equal(after[page] & m, kv_ref.pack_page(*want) & m)
        assert np.array_equal(after[page] & ~m, before[page] & ~m)
    rest = [p for p in range(len(before)) if p not in touched]
    assert np.array_equal(after[rest], before[rest])


def test_append_values_of_the_whole_range():
    """Groups of zeros, constants, NaN, infinities, fp32 values beyond fp16, subnormals."""
    D, ps = 64, 32
    x = np.zeros((9, 1, D), np.float32)
    x[1] = 5.4321
    x[2, 0, 3], x[2, 0, 40] = np.nan, np.inf
    x[3, 0, 0], x[3, 0, 1] = -np.inf, np.inf
    x[4] = np.linspace(-1e30, 1e30, D)
    x[5] = np.linspace(0, 1e-7, D)
    x[6] = np.linspace(-1e-41, 1e-41, D)
    x[7] = -65504 + np.arange(D)
    x[8] = np.nan
    cache = binding.KVCache(1, 1, D, ps, pool=torch.zeros(1, 2 * ps * 40, dtype=torch.uint8, device="cuda"))
    pages, kv_len = dev(np.zeros((1, 1), np.int32)), dev(np.array([9], np.int32))
    binding.kv_append(cache, dev(x), dev(x), pages, kv_len)
    k, v = binding.kv_read(cache, 9, pages, kv_len)
    k16, v16 = torch.empty(9, 1, D, dtype=torch.float16, device="cuda"), torch.empty(9, 1, D, dtype=torch.float16, device="cuda")
    binding.kv_read(cache, 9, pages, kv_len, k_out=k16, v_out=v16)
    torch.cuda.synchronize()
    want = kv_ref.values(*kv_ref.quantise(x)).astype(np.float32)
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want)
    assert np.array_equal(k16.cpu().numpy(), want.astype(np.float16)) and torch.equal(k16, v16)


def test_rows_that_have_no_place():
    """Rows behind the last sequence, positions below 0 and past the table, pages not held: not stored, read as 0, and
    rows of no sequence keep what the outputs held."""
    rng = np.random.default_rng(8)
    D, ps, mp, hkv = 128, 32, 2, 2
    k = rng.standard_normal((12, hkv, D)).astype(np.float32)
    before = rng.integers(0, 256, (5, 2 * hkv * ps * 80), dtype=np.uint8)
    cache = binding.KVCache(5, hkv, D, ps, pool=dev(before))
    # sequence 0: positions -2..1; 1: 62..65 (the table ends at 64); 2: on a page not held, then one too high
    q_start = dev(np.array([1, 5, 9, 11], np.int32))
    kv_len = dev(np.array([2, 66, 33], np.int32))
    pages = np.array([[0, -1], [1, 2], [-1, 5]], np.int32)
    q_out = torch.full((12, 4, D), 3.0, device="cuda")
    q = rng.standard_normal((12, 4, D)).astype(np.float32)
    binding.kv_append(cache, dev(k), dev(k), dev(pages), kv_len, q_start=q_start, q=dev(q), q_out=q_out)
    ko = torch.full((12, hkv, D), 3.0, device="cuda")
    vo = ko.clone()
    binding.kv_read(cache, 12, dev(pages), kv_len, q_start=q_start, k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    want = kv_ref.values(*kv_ref.quantise(k)).astype(np.float32)
    want[[1, 2, 7, 8, 9, 10]] = 0
    want[[0, 11]] = 3
    assert np.array_equal(ko.cpu().numpy(), want) and torch.equal(ko, vo)
    q[[0, 11]] = 3
    assert np.array_equal(q_out.cpu().numpy(), q)
    after = cache.pool.cpu().numpy()
    assert np.array_equal(after[[3, 4]], before[[3, 4]])


# ------------------------------------------------------------------ attention

def check_attn(c, q, ns, kv_len, scale, window=0, behind=0, f32=False, out_layout="token", cache=None):
    where = rows_of(ns) + [None] * behind
    out, mass, amax = kv_ref.attention(c, q, where, kv_len, scale, window)
    q_start = None if len(set(ns)) == 1 and not behind else dev(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32))
    cache = cache or binding.KVCache(c.num_pages, c.hkv, c.D, c.ps, pool=dev(c.pool))
    rows, hq = q.shape[:2]
    dt = torch.float32 if f32 else torch.float16
    if out_layout == "token":
        buf = torch.full((rows, hq, c.D), 77.0, dtype=dt, device="cuda")
        o = buf
    else:
        buf = torch.full((hq, c.D, rows), 77.0, dtype=dt, device="cuda")
        o = buf.permute(2, 0, 1)
    args = (cache, dev(q), dev(c.pages), dev(kv_len))
    binding.kv_attn(*args, q_start=q_start, scale=scale, window=window, out=o)
    again = binding.kv_attn(*args, q_start=q_start, scale=scale, window=window) if not behind else None
    torch.cuda.synchronize()
    got = o.cpu().numpy().astype(np.float64)
    live = [t for t, r in enumerate(where) if r is not None]
    err = np.abs(got - out)[live]
    bound = kv_ref.attention_bound(out, mass, amax, not f32)[live]
    assert np.isfinite(got).all()
    assert (err <= bound).all(), f"worst {np.max(err / bound):.3g} of the bound"
    for t, r in enumerate(where):
        if r is None:
            assert (got[t] == 77).all()
        elif not mass[t].any():
            assert (got[t] == 0).all()
    if again is not None and not f32:
        assert torch.equal(again, o)  # the same bits on every call
    return np.max(err / bound) if len(live) else 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 255, 1000, 2049])
def test_attn_lengths(D, length):
    rng = np.random.default_rng(D + length)
    c = kv_ref.Cache(rng, 1, -(-length // 64) + 1, 2, D, 64)
    c.spoil(0, length)
    q = rng.standard_normal((1, 12, D)).astype(np.float16)
    check_attn(c, q, [1], np.array([length], np.int32), D ** -0.5)
    check_attn(c, q * np.float16(4), [1], np.array([length], np.int32), D ** -0.5, f32=True)


@pytest.mark.parametrize("D,ps", [(64, 32), (128, 32), (128, 256), (256, 128)])
@pytest.mark.parametrize("hkv,grp", [(1, 1), (3, 5), (2, 8), (1, 17), (1, 40)])
@pytest.mark.parametrize("n", [1, 2, 7, 17, 33])
def test_attn_head_and_row_counts(D, ps, hkv, grp, n):
    rng = np.random.default_rng(D + hkv * grp + n)
    length = 150 + n
    c = kv_ref.Cache(rng, 1, -(-length // ps), hkv, D, ps)
    c.spoil(0, length)
    q = rng.standard_normal((n, hkv * grp, D)).astype(np.float16)
    check_attn(c, q, [n], np.array([length], np.int32), D ** -0.5, out_layout="column")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 5, 32, 100])
def test_attn_ragged_batch(D, window):
    """Sequences of 0..40 rows and 0..400 positions, shared pages, rows behind the last."""
    rng = np.random.default_rng(D + window)
    ns = [3, 0, 1, 40, 2, 1, 0, 9]
    kv_len = np.array([400, 5, 1, 130, 2, 0, 0, 5], np.int32)  # sequences 5 and 7: rows before position 0
    c = kv_ref.Cache(rng, len(ns), 13, 2, D, 32)
    c.pages[2], c.held[2] = c.pages[0], True
    for f in c.f:
        for x in f:
            x[2] = x[0]
    for s in (0, 1, 3, 4, 5, 6, 7):
        if s != 0:
            c.spoil(s, int(kv_len[s]))
    q = rng.standard_normal((sum(ns) + 5, 6, D)).astype(np.float16)
    check_attn(c, q, ns, kv_len, D ** -0.5, window=window, behind=5)


@pytest.mark.parametrize("D", [64, 256])
def test_attn_pages_not_held(D):
    """Holes inside a sequence and a sequence of holes alone: their positions are not attended to."""
    rng = np.random.default_rng(D)
    c = kv_ref.Cache(rng, 3, 6, 2, D, 32, holes=[(0, 0, -1), (0, 3, 1 << 30), (0, 4, -7), (2, 0, -1), (2, 1, 99999)])
    q = rng.standard_normal((6, 4, D)).astype(np.float16)
    check_attn(c, q, [2, 2, 2], np.array([180, 64, 40], np.int32), D ** -0.5)
    check_attn(c, q, [2, 2, 2], np.array([192, 192, 64], np.int32), D ** -0.5, window=33)


def test_attn_lengths_past_the_table():
    """kv_len beyond max_pages * page_size: the positions that the table has."""
    rng = np.random.default_rng(2)
    c = kv_ref.Cache(rng, 1, 2, 1, 128, 32)
    q = rng.standard_normal((3, 2, 128)).astype(np.float16)
    check_attn(c, q, [3], np.array([1000], np.int32), 0.1)
    check_attn(c, q, [3], np.array([2 ** 31 - 1], np.int32), 0.1)
    check_attn(c, q, [3], np.array([65], np.int32), 0.1, window=2)


@pytest.mark.parametrize("qs,vs,scale", [(1e-3, 1, 1.0), (300.0, 1, 1e-3), (1.0, 1e4, 0.01), (1.0, 1e-3, 0.06),
                                         (1.0, 1.0, -0.06), (1.0, 1.0, 0.0), (6e4, 1.0, 1e-6), (1.0, 1.0, 3.0),
                                         (1e-6, 1.0, 1e5), (6e-8, 1.0, 1e6), (3e-5, 1.0, 3e3)])
def test_attn_ranges(qs, vs, scale):
    rng = np.random.default_rng(4)
    c = kv_ref.Cache(rng, 1, 5, 1, 128, 64, scale=vs)
    q = np.clip(rng.standard_normal((2, 4, 128)) * qs, -65504, 65504).astype(np.float16)
    check_attn(c, q, [2], np.array([300], np.int32), scale / max(vs, 1), f32=True)
    check_attn(c, np.tile(q, (1, 4, 1)), [2], np.array([300], np.int32), scale / max(vs, 1), f32=True)


def test_attn_non_finite_queries_stay_in_their_rows():
    rng = np.random.default_rng(11)
    c = kv_ref.Cache(rng, 1, 4, 1, 128, 32)
    q = rng.standard_normal((3, 4, 128)).astype(np.float16)
    bad = q.copy()
    bad[1, 2, 5], bad[1, 3, 0] = np.nan, np.inf
    cache = binding.KVCache(c.num_pages, 1, 128, 32, pool=dev(c.pool))
    good, got = (binding.kv_attn(cache, dev(x), dev(c.pages), dev(np.array([100], np.int32))) for x in (q, bad))
    torch.cuda.synchronize()
    assert not torch.isfinite(got[1, 2:]).any()
    got[1, 2:] = good[1, 2:]
    assert torch.equal(good, got)


def test_attn_long_context():
    """Enough positions for every split of the work, checked in fp64 on the device."""
    D, hkv, ps, length, n = 128, 2, 64, 40007, 3
    g = torch.Generator("cuda").manual_seed(1)
    cache = binding.KVCache(-(-length // ps), hkv, D, ps)
    k, v = (torch.randn(length, hkv, D, generator=g, device="cuda") for _ in range(2))
    pages = torch.randperm(cache.num_pages, generator=g, device="cuda").int()[None].contiguous()
    kv_len = dev(np.array([length], np.int32))
    binding.kv_append(cache, k, v, pages, kv_len)
    kk, vv = binding.kv_read(cache, length, pages, kv_len)
    q = (2 * torch.randn(n, 4, D, generator=g, device="cuda")).half()
    out = torch.empty(n, 4, D, device="cuda")
    binding.kv_attn(cache, q, pages, kv_len, out=out)
    for t in range(n):
        for h in range(4):
            end = length - n + t + 1
            p = torch.softmax(kk[:end, h // 2].double() @ q[t, h].double() * D ** -0.5, 0)
            want = p @ vv[:end, h // 2].double()
            # the fp32 sums of a split: rms error far below the worst case; 2^-16 of sum p (|V| + 2|m|) with |m| < 5
            assert ((out[t, h] - want).abs() <= 2.0 ** -16 * (p @ vv[:end, h // 2].double().abs() + 10)).all()


def test_attn_many_sequences():
    """More sequences than a wave has lanes, some without rows or positions, tables far longer than they need."""
    rng = np.random.default_rng(50)
    nseq, D = 200, 64
    ns = [int(x) for x in rng.integers(0, 4, nseq)]
    kv_len = np.array([n + int(rng.integers(0, 90)) if n else 7 for n in ns], np.int32)
    kv_len[5] = 96
    c = kv_ref.Cache(rng, nseq, 3, 1, D, 32)
    for s in range(0, nseq, 3):
        c.spoil(s, int(kv_len[s]))
    wide = np.full((nseq, 700), -1, np.int32)  # held pages, then nothing
    wide[:, :3] = c.pages
    wide[:, 3:] = rng.integers(0, c.num_pages, (nseq, 697))  # pages of others behind the end: never read
    c.pages, c.held, c.mp = wide, np.ones((nseq, 700), bool), 700
    q = rng.standard_normal((sum(ns), 3, D)).astype(np.float16)
    check_attn(c, q, ns, kv_len, 0.125)
    check_attn(c, q, ns, kv_len, 0.125, window=40)


def test_more_sequences_than_are_shared_out():
    """A batch so wide that no context is split, ragged and even, with empty sequences: append and attention."""
    rng = np.random.default_rng(51)
    D, ps, hkv = 64, 32, 1
    for even in (False, True):
        nseq = 5000
        ns = [1] * nseq if even else [int(x) for x in (rng.random(nseq) < 0.3) * rng.integers(1, 4, nseq)]
        rows = sum(ns)
        kv_len = np.array([n + int(rng.integers(0, 9)) for n in ns], np.int32)
        table = np.zeros((nseq, 12), np.int32)
        table[:, 0] = rng.permutation(nseq)
        pool = torch.zeros(nseq, 2 * hkv * ps * 40, dtype=torch.uint8, device="cuda")
        cache = binding.KVCache(nseq, hkv, D, ps, pool=pool)
        q_start = None if even else dev(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32))
        k, v = (rng.standard_normal((rows, hkv, D)).astype(np.float32) for _ in range(2))
        q = rng.standard_normal((rows, 2, D)).astype(np.float16)
        binding.kv_append(cache, dev(k), dev(v), dev(table), dev(kv_len), q_start=q_start)
        out = binding.kv_attn(cache, dev(q), dev(table), dev(kv_len), q_start=q_start, out=torch.empty(rows, 2, D, device="cuda"))
        torch.cuda.synchronize()
        where = rows_of(ns)
        fk, fv = kv_ref.quantise(k), kv_ref.quantise(v)
        first = np.concatenate([[0], np.cumsum(ns)])
        for t in rng.choice(rows, 60, replace=False):
            s, i, n = where[t]
            old = int(kv_len[s]) - n  # positions that hold zeros, then this call's rows
            c = kv_ref.Cache.__new__(kv_ref.Cache)
            c.hkv, c.D, c.ps, c.mp, c.held = hkv, D, old + n, 1, np.ones((1, 1), bool)
            c.f = [tuple(np.concatenate([np.zeros((old,) + x.shape[1:], x.dtype), x[first[s]:first[s] + n]])[None] for x in f)
                   for f in (fk, fv)]
            want, mass, amax = kv_ref.attention(c, q[t:t + 1], [(0, i, n)], [old + n], 0.125)
            assert (np.abs(out[t].cpu().numpy() - want[0]) <= kv_ref.attention_bound(want, mass, amax, False)[0]).all()


@pytest.mark.parametrize("nseq", [79, 80, 81, 130])
def test_few_live_sequences_among_many(nseq):
    """Contexts shared out over workgroups and, from a few sequences more on, one piece each; most sequences have no rows."""
    rng = np.random.default_rng(52)
    c = kv_ref.Cache(rng, nseq, 20, 1, 64, 32)
    ns = [0] * nseq
    ns[0], ns[nseq // 2], ns[nseq - 1] = 2, 1, 3
    kv_len = np.where(np.array(ns) > 0, 640, rng.integers(0, 640, nseq)).astype(np.int32)
    kv_len[nseq // 2] = 97
    q = rng.standard_normal((6, 3, 64)).astype(np.float16)
    for window in (0, 100):
        check_attn(c, q, ns, kv_len, 0.125, window=window, f32=True)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_splits_with_windows_and_holes(D):
    """Contexts that are shared out over workgroups, by a table of the right length and by one 30 times as long."""
    rng = np.random.default_rng(60 + D)
    c = kv_ref.Cache(rng, 2, 47, 1, D, 64, holes=[(0, 3, -1), (0, 20, -1), (1, 46, -1), (1, 0, -1)])
    q = rng.standard_normal((5, 4, D)).astype(np.float16)
    kv_len = np.array([2990, 3008], np.int32)
    for window in (0, 1500, 70):
        check_attn(c, q, [2, 3], kv_len, D ** -0.5, window=window)
        check_attn(c, q[:4], [2, 2], kv_len, D ** -0.5, window=window, f32=True)
    c.pages = np.concatenate([c.pages, np.full((2, 1400), -1, np.int32)], 1)
    c.held = np.concatenate([c.held, np.zeros((2, 1400), bool)], 1)
    c.mp += 1400
    check_attn(c, q, [2, 3], kv_len, D ** -0.5, window=0)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("layout,dt", [("token", np.float16), ("column", np.float32), ("token", np.float32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_rows(D, layout, dt, interleaved):
    """Rows enough for a wave to take several heads of each: prepared alone, and appended."""
    rng = np.random.default_rng(70 + D)
    rows, hq, hkv, ps = 1203, 11, 5, 64
    rope, f, (wq, wk) = make_rope(rng, D, D // 2, interleaved, True)
    q, k, v = (rng.standard_normal((rows, h, D)).astype(dt) for h in (hq, hkv, hkv))
    pos = np.arange(rows, dtype=np.int32) + 1000
    qo, ko = binding.norm_rope(rope, dev(pos), strided(q, layout, dt), strided(k, layout, dt))
    cache = binding.KVCache(20, hkv, D, ps, pool=torch.zeros(20, 2 * hkv * ps * D * 5 // 8, dtype=torch.uint8, device="cuda"))
    pages, kv_len = dev(rng.permutation(20)[None, :19].astype(np.int32)), dev(np.array([rows], np.int32))
    qa = binding.kv_append(cache, strided(k, layout, dt), strided(v, layout, dt), pages, kv_len, q=strided(q, layout, dt),
                           rope=rope, positions=dev(pos))
    rk, rv = binding.kv_read(cache, rows, pages, kv_len)
    torch.cuda.synchronize()
    kr = kv_ref.norm_rope(k, pos, f, interleaved, wk, 1e-5)
    close_to_rounding(qo.cpu().numpy(), kv_ref.norm_rope(q, pos, f, interleaved, wq, 1e-5), np.float16)
    close_to_rounding(ko.cpu().numpy(), kr, np.float16)
    assert torch.equal(qo, qa)
    assert np.array_equal(rk.cpu().numpy(), kv_ref.values(*kv_ref.quantise(kr.astype(np.float32))).astype(np.float32))
    assert np.array_equal(rv.cpu().numpy(), kv_ref.values(*kv_ref.quantise(v.astype(np.float32))).astype(np.float32))


def test_far_positions_and_wide_frequencies():
    """Angles up to 2^31, and beyond where the exact reduction ends: still the cosine of the fp64 product."""
    rng = np.random.default_rng(80)
    f = np.array([1.0, 0.3, 1e-3, 123.5, 3e4, 0.0, 0.999999, 2.5e-7], np.float32)
    rope = binding.Rope(dev(f))
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 262139, 12345678], np.int32)
    x = rng.standard_normal((7, 2, 64)).astype(np.float32)
    got, _ = binding.norm_rope(rope, dev(pos), dev(x), q_out=torch.empty(7, 2, 64, device="cuda"))
    torch.cuda.synchronize()
    close_to_rounding(got.cpu().numpy(), kv_ref.norm_rope(x, pos, f), np.float32)


def test_append_in_place_and_at_given_positions():
    rng = np.random.default_rng(90)
    D, rows = 128, 5
    rope, f, (wq, wk) = make_rope(rng, D, 64, False, True)
    q, k = (rng.standard_normal((rows, h, D)).astype(np.float32) for h in (6, 2))
    pos = np.array([900, 3, 77, 5, 100000], np.int32)
    cache = binding.KVCache(2, 2, D, 32)
    pages, kv_len = dev(np.array([[1, 0]], np.int32)), dev(np.array([40], np.int32))
    qd = dev(q)
    same = binding.kv_append(cache, dev(k), dev(k), pages, kv_len, q=qd, q_out=qd, rope=rope, positions=dev(pos))
    rk, _ = binding.kv_read(cache, rows, pages, kv_len)
    torch.cuda.synchronize()
    assert same is qd
    close_to_rounding(qd.cpu().numpy(), kv_ref.norm_rope(q, pos, f, False, wq, 1e-5), np.float32)
    kr = kv_ref.norm_rope(k, pos, f, False, wk, 1e-5).astype(np.float32)
    assert np.array_equal(rk.cpu().numpy(), kv_ref.values(*kv_ref.quantise(kr)).astype(np.float32))


def test_pool_beyond_four_gib():
    """Pages whose byte offsets pass 32 bits: written, read back and attended to."""
    rng = np.random.default_rng(100)
    D, hkv, ps = 128, 8, 1024
    pb = 2 * hkv * ps * D * 5 // 8  # 1.25 MiB
    n = (1 << 32) // pb + 40
    cache = binding.KVCache(n, hkv, D, ps)
    cache.pool[:3] = 0
    pages = np.array([[n - 1, 1, n - 20]], np.int32)
    L = 2 * ps + 100
    k, v = (rng.standard_normal((L, hkv, D)).astype(np.float32) for _ in range(2))
    kv_len = np.array([L], np.int32)
    binding.kv_append(cache, dev(k), dev(v), dev(pages), dev(kv_len))
    rk, rv = binding.kv_read(cache, L, dev(pages), dev(kv_len))
    c = kv_ref.Cache.__new__(kv_ref.Cache)
    c.hkv, c.D, c.ps, c.mp, c.held = hkv, D, ps, 3, np.ones((1, 3), bool)
    c.f = [tuple(np.concatenate([x, np.zeros((3 * ps - L,) + x.shape[1:], x.dtype)])[None] for x in kv_ref.quantise(t)) for t in (k, v)]
    assert np.array_equal(rk.cpu().numpy(), c.kv()[0][0, :L].astype(np.float32))
    assert np.array_equal(rv.cpu().numpy(), c.kv()[1][0, :L].astype(np.float32))
    c.pages, c.num_pages = pages, n
    q = rng.standard_normal((2, 16, D)).astype(np.float16)
    check_attn(c, q, [2], kv_len, D ** -0.5, cache=cache)
    assert not cache.pool[0].any() and not cache.pool[2].any()


def test_calls_at_once():
    """Host threads on streams of their own, each with its own workspace and cache: the bits of single calls."""
    import threading
    rng = np.random.default_rng(110)
    jobs = []
    for i, D in enumerate((64, 128, 256, 128)):
        c = kv_ref.Cache(rng, 1, 40, 2, D, 64)
        cache = binding.KVCache(c.num_pages, 2, D, 64, pool=dev(c.pool))
        args = (cache, dev(rng.standard_normal((1 + i, 8, D)).astype(np.float16)), dev(c.pages), dev(np.array([2500 - i], np.int32)))
        jobs.append((args, binding.kv_attn(*args)))
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream, (args, want) = torch.cuda.Stream(), jobs[i]
        for _ in range(20):
            got = binding.kv_attn(*args, stream=stream)
            stream.synchronize()
            if not torch.equal(got, want):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_workspace_of_the_caller():
    rng = np.random.default_rng(120)
    c = kv_ref.Cache(rng, 1, 40, 2, 128, 64)
    cache = binding.KVCache(c.num_pages, 2, 128, 64, pool=dev(c.pool))
    args = (cache, dev(rng.standard_normal((1, 8, 128)).astype(np.float16)), dev(c.pages), dev(np.array([2500], np.int32)))
    want = binding.kv_attn(*args)
    need = binding.qk_kv_attn_workspace_bytes(cache._c, binding._seqs_arg(1, args[2], args[3], None), 8)
    assert need > 0
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(2):  # whatever it held
        assert torch.equal(binding.kv_attn(*args, workspace=ws[:need]), want)
    torch.cuda.synchronize()
    assert (ws[need:] == 0xff).all()
    with pytest.raises(binding.QKError):
        binding.kv_attn(*args, workspace=ws[: need - 16])


# ------------------------------------------------------------------ together

def test_a_layer_step_from_gemv_to_gemv():
    """q, k and v by GEMVs of three drafted columns, append, attention into the x of the output projection's GEMV --
    twice, the second token's rows after the first's -- against the same path in numpy."""
    from quant_dequant_gemv_amd import synth
    rng = np.random.default_rng(21)
    Kin, D, hq, hkv, ps, T = 512, 128, 4, 2, 32, 3
    Ws = {n: synth.superblocks(binding.Q4_K, N, Kin, i) for i, (n, N) in
          enumerate((("q", hq * D), ("k", hkv * D), ("v", hkv * D)))}
    rope, f, (wq, wk) = make_rope(rng, D, 64, False, True)
    cache = binding.KVCache(4, hkv, D, ps)
    pages = dev(np.array([[2, 0, 3]], np.int32))
    kv_len = torch.zeros(1, dtype=torch.int32, device="cuda")
    wd = {n: dev(W.reshape(-1)) for n, W in Ws.items()}
    hist, length = {"k": [], "v": []}, 0
    for step in range(2):
        x = (rng.standard_normal((Kin, T)) * 0.05).astype(np.float16)
        y = {n: binding.gemv(binding.Q4_K, wd[n], dev(x), N, Kin) for n, N in (("q", hq * D), ("k", hkv * D), ("v", hkv * D))}
        heads = {n: t.view(-1, D, T).permute(2, 0, 1) for n, t in y.items()}
        kv_len += T
        xo = torch.empty(hq * D, T, dtype=torch.float16, device="cuda")
        q = binding.kv_append(cache, heads["k"], heads["v"], pages, kv_len, q=heads["q"], rope=rope)
        binding.kv_attn(cache, q, pages, kv_len, out=xo.view(hq, D, T).permute(2, 0, 1))
        torch.cuda.synchronize()
        host = {n: t.cpu().numpy() for n, t in heads.items()}
        pos = length + np.arange(T)
        length += T
        hist["k"].append(kv_ref.quantise(kv_ref.norm_rope(host["k"], pos, f, False, wk, 1e-5).astype(np.float32)))
        hist["v"].append(kv_ref.quantise(host["v"]))
        c = kv_ref.Cache.__new__(kv_ref.Cache)
        c.hkv, c.D, c.ps, c.mp, c.held = hkv, D, length, 1, np.ones((1, 1), bool)
        c.f = [tuple(np.concatenate([r[i] for r in hist[n]])[None] for i in range(3)) for n in "kv"]
        out, mass, amax = kv_ref.attention(c, q.cpu().numpy(), rows_of([T]), [length], D ** -0.5)
        got = xo.view(hq, D, T).permute(2, 0, 1).cpu().numpy()
        assert (np.abs(got - out) <= kv_ref.attention_bound(out, mass, amax, True)).all()


def test_captured_and_replayed():
    """A token's append and attention as a graph, replayed while kv_len moves on, with eager work between replays."""
    rng = np.random.default_rng(31)
    D, hq, hkv, ps, mp = 256, 12, 2, 32, 8
    rope = binding.Rope(dev(freqs(32)))
    caches = [binding.KVCache(mp, hkv, D, ps) for _ in range(2)]
    for c in caches:
        c.pool.zero_()
    pages = dev(rng.permutation(mp)[None].astype(np.int32))
    q, k, v = (torch.empty(1, h, D, device="cuda") for h in (hq, hkv, hkv))
    kv_len = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(1, hq, D, dtype=torch.float16, device="cuda")

    def step(cache):
        qo = binding.kv_append(cache, k, v, pages, kv_len, q=q, rope=rope)
        return binding.kv_attn(cache, qo, pages, kv_len, out=out)

    kv_len.fill_(1)
    step(caches[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0])
    kv_len.zero_()
    for i in range(70):
        for x in (q, k, v):
            x.copy_(dev(rng.standard_normal(tuple(x.shape)).astype(np.float32)))
        kv_len += 1
        graph.replay()
        replayed = out.clone()
        eager = step(caches[1]).clone()
        assert torch.equal(replayed, eager), i
    torch.cuda.synchronize()
    assert torch.equal(caches[0].pool, caches[1].pool)


def test_on_another_stream():
    rng = np.random.default_rng(41)
    c = kv_ref.Cache(rng, 1, 3, 2, 128, 64)
    q = rng.standard_normal((1, 8, 128)).astype(np.float16)
    cache = binding.KVCache(c.num_pages, 2, 128, 64, pool=dev(c.pool))
    args = (cache, dev(q), dev(c.pages), dev(np.array([150], np.int32)))
    want = binding.kv_attn(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [binding.kv_attn(*args, stream=s), binding.kv_attn(*args, stream=int(s.cuda_stream))]
    s.synchronize()
    assert all(torch.equal(want, g) for g in got)
