"""The cases that the attention-side operators are measured on: norm + rotation of
query and key heads, appending to the 4-bit paged cache, and attention over it.

``run`` computes them in plain torch, or with ``own`` through the public helpers of
``quant_dequant_gemv_amd.binding``.  Inputs are what the projections' GEMVs leave in
memory: fp32 ``[N][ncols]`` (feature-major, with the gate of each query head between the
heads) for decode and verify widths, fp16 or fp32 token-major rows for batches and prompts.

Cache pages, for every head a block of keys and one of values (ps positions a page, G = D/32
groups): codes, then the fp16 steps d, then the fp16 minima m; value = d * code + m.
  keys    codes [ps][4][G] words: nibble n of word (a, g) is dim 32g + 8a + n
          d [ps/4][G][4], m [ps][G]
  values  codes [ps/4][W][16][4] pieces: nibble n of piece (w, l) is dim 128w + 16n + l
          (D = 64: W = 1 and a piece has 4 nibbles), d and m [ps/4][G][4]
"""
import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def _case(name, op, **kw):
    c = dict(name=name, op=op, nseq=1, n=1, ragged=False, hq=24, hkv=4, d=256, rot=64, interleaved=False, norm=True,
             f16=False, fm=False, gate=False, ps=64, len_lo=1, len_hi=1, window=0)
    c.update(kw)
    return c


def listed():
    return [
        # a decode token: the head norms and the partial rotation on their own, as the GEMVs leave q (with its gate) and k
        _case("norm_rope 1 token d256", "norm_rope", fm=True, gate=True, len_lo=40001, len_hi=40001),
        # a prompt's rows, fp16 token-major, full interleaved rotation
        _case("norm_rope 2048 rows d128", "norm_rope", n=2048, hq=32, hkv=8, d=128, rot=128, interleaved=True, f16=True,
              len_lo=9000, len_hi=9000),
        # a decode token's keys and values into the cache, its queries made ready in the same call
        _case("append 1 token d256", "append", fm=True, gate=True, len_lo=32773, len_hi=32773),
        # 17 drafted tokens at once: the widest verify width that the callers ask for
        _case("append 17 drafts d256", "append", n=17, fm=True, gate=True, len_lo=8191, len_hi=8191),
        # one step of a batch of sequences of very different lengths, some with drafts
        _case("append 64 seqs d128", "append", nseq=64, n=5, ragged=True, hq=32, hkv=8, d=128, rot=128, f16=True, ps=32,
              len_lo=1, len_hi=16384),
        # a prompt written to an empty cache: small heads, no norms, interleaved pairs
        _case("append 4096 rows d64", "append", n=4096, hq=32, hkv=8, d=64, rot=64, interleaved=True, norm=False, f16=True,
              ps=128, len_lo=4096, len_hi=4096),
        # the shortest whole step: norm + rotation + append, then attention over 67 positions
        _case("step 1 token len 67 d256", "step", fm=True, gate=True, len_lo=67, len_hi=67),
        # the verify step of 17 drafts over a cache of 8191 positions
        _case("step 17 drafts len 8191 d256", "step", n=17, fm=True, gate=True, len_lo=8191, len_hi=8191),
        # single-stream decode in a long context
        _case("attn 1 token len 32773 d256", "attn", fm=True, len_lo=32773, len_hi=32773),
        # the longest context: a quarter of a million positions
        _case("attn 1 token len 262139 d256", "attn", fm=True, len_lo=262139, len_hi=262139, ps=256),
        # a ragged batch: a token each, contexts from one position to 16384
        _case("attn 48 seqs d128", "attn", nseq=48, hq=32, hkv=8, d=128, ps=32, len_lo=1, len_hi=16384),
        # a prompt's chunk under a sliding window
        _case("attn 509 rows window d64", "attn", n=509, hq=32, hkv=4, d=64, len_lo=8200, len_hi=8200, window=4096, ps=128),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    most = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:  # at most the cost of the listed ones
        c = _drawn(rng)
        w = work(c)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return c


def _drawn(rng):
    op = rng.choice(["norm_rope", "append", "attn", "attn", "step"])
    d = rng.choice([64, 128, 256])
    hkv = rng.randint(1, 8)
    hq = hkv * rng.randint(1, 8)
    few = rng.random() < 0.6  # one stream, or a batch / a prompt
    nseq = 1 if few else _log(rng, 1, 64)
    n = _log(rng, 1, 32) if few else _log(rng, 1, 8) if nseq > 1 else _log(rng, 33, 1024)
    ragged = nseq > 1 and rng.random() < 0.5
    hi = _log(rng, n + 1, max(n + 1, min(262144 * 4 * 256 // (hkv * d * nseq), 262144)))
    lo = rng.randint(n, hi) if nseq > 1 else hi
    fm = few and rng.random() < 0.7
    return _case("drawn", op, nseq=nseq, n=n, ragged=ragged, hq=hq, hkv=hkv, d=d, rot=2 * rng.randint(1, d // 2),
                 interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, f16=not fm and rng.random() < 0.6, fm=fm,
                 gate=fm and rng.random() < 0.5, ps=rng.choice([32, 64, 128, 256]), len_lo=lo, len_hi=hi,
                 window=_log(rng, 1, 8192) if rng.random() < 0.25 else 0)


def _sizes(c):
    """Rows and cache length (with those rows) of each sequence: of the case alone."""
    r = random.Random("%d %d %d %d" % (c["nseq"], c["n"], c["len_lo"], c["len_hi"]))
    ns = [r.randint(1, c["n"]) if c["ragged"] else c["n"] for _ in range(c["nseq"])]
    lens = [max(n, _log(r, c["len_lo"], c["len_hi"]) if c["len_lo"] < c["len_hi"] else c["len_lo"]) for n in ns]
    return ns, lens


def _visible(c):
    """Sum over rows of the positions they see, and the positions that some row of a sequence sees."""
    ns, lens = _sizes(c)
    pairs = seen = 0
    for n, ln in zip(ns, lens):
        w = c["window"] or ln
        first = max(0, ln - n - w + 1)
        seen += ln - first
        if c["window"]:
            pairs += sum(min(ln - n + i + 1, w) for i in range(n))
        else:
            pairs += n * (ln - n) + n * (n + 1) // 2
    return pairs, seen


def work(c):
    rows = sum(_sizes(c)[0])
    x = 2 if c["f16"] else 4
    q, kv = rows * c["hq"] * c["d"], rows * c["hkv"] * c["d"]
    pairs, seen = _visible(c)
    if c["op"] == "norm_rope":
        return {"bytes": q * (x + 2) + kv * (x + 2), "flops": 10 * (q + kv)}
    append = {"bytes": q * (x + 2) + 2 * kv * (x + 0.625), "flops": 10 * (q + 2 * kv)}
    if c["op"] == "append":
        return append
    attn = {"bytes": 2 * seen * c["hkv"] * c["d"] * 0.625 + q * 4, "flops": 4 * c["d"] * c["hq"] * pairs}
    if c["op"] == "attn":
        return attn
    return {k: append[k] + attn[k] for k in attn}


# ------------------------------------------------------------------ inputs

def _projection(g, c, rows, heads, gate):
    """What a projection leaves: heads of d values for each row, [rows][heads][d] as a view of its buffer."""
    d, m = c["d"], 2 if gate else 1
    t = torch.randn(heads * m * d * rows, generator=g, device="cuda")
    scale = torch.exp(0.5 * torch.randn(heads * m * d, generator=g, device="cuda"))
    if c["fm"]:  # [N][ncols], as qk_gemv writes y
        t = (t.view(heads * m * d, rows) * scale[:, None]).view(heads, m, d, rows)[:, 0].permute(2, 0, 1)
    else:
        t = (t.view(rows, heads * m * d) * scale).view(rows, heads, m, d)[:, :, 0]
    return t.half() if c["f16"] else t


def _fields(c, g, ns, lens):
    """A filled cache as its fields: for keys and values [nseq][L][hkv] rows of codes, steps and minima."""
    ps, length = c["ps"], max(lens)
    pages = -(-length // ps)
    out = []
    for _ in range(2):
        x = torch.randn(c["nseq"] * pages * ps, c["hkv"], c["d"] // 32, 32, generator=g, device="cuda")
        x *= torch.exp(0.4 * torch.randn(c["hkv"], c["d"] // 32, 32, generator=g, device="cuda"))
        m = x.amin(-1).half()
        step = ((x.amax(-1) - m.float()) / 15).half()
        code = ((x - m.float()[..., None]) / step.float()[..., None]).round_().clamp_(0, 15).to(torch.uint8)
        out.append((code, step, m))
    return pages, out


def _words(codes, n):
    """Nibbles [..., n] to bytes [..., n/2]."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _pack(c, fields):
    """[pages][bytes] of a cache's fields, in the order of the positions."""
    ps, h, d, grp = c["ps"], c["hkv"], c["d"], c["d"] // 32
    blocks = []
    for values, (code, step, m) in enumerate(fields):
        p = code.shape[0] // ps
        if not values:
            x = _words(code.view(p, ps, h, grp, 4, 8).permute(0, 2, 1, 4, 3, 5), 8)
        else:
            w, nib = max(1, d // 128), min(8, d // 16)
            x = _words(code.view(p, ps // 4, 4, h, w, nib, 16).permute(0, 3, 1, 4, 6, 2, 5), nib)
        by4 = lambda t: t.view(p, ps // 4, 4, h, grp).permute(0, 3, 1, 4, 2).reshape(p, h, -1).contiguous().view(torch.uint8)  # noqa: E731
        mm = by4(m) if values else m.view(p, ps, h, grp).permute(0, 2, 1, 3).reshape(p, h, -1).contiguous().view(torch.uint8)
        blocks.append(torch.cat([x.reshape(p, h, -1), by4(step), mm], -1))
    return torch.stack(blocks, 2).reshape(blocks[0].shape[0], -1)


def _make(c, seed):
    """Everything of a case from its seed: inputs, the cache's fields, and the page table."""
    g = torch.Generator("cuda").manual_seed(int(seed))
    ns, lens = _sizes(c)
    rows = sum(ns)
    half = c["rot"] // 2
    s = {"ns": ns, "lens": lens, "rows": rows}
    s["inv_freq"] = (10000000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
    pos = [ln - n + i for n, ln in zip(ns, lens) for i in range(n)]
    s["positions"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    if c["norm"]:
        s["q_norm"], s["k_norm"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda") for _ in range(2))
    else:
        s["q_norm"] = s["k_norm"] = None
    if c["op"] != "attn":
        s["q"] = _projection(g, c, rows, c["hq"], c["gate"])
        s["k"] = _projection(g, c, rows, c["hkv"], False)
        s["v"] = _projection(g, c, rows, c["hkv"], False)
    else:
        s["q"] = torch.randn(rows, c["hq"], c["d"], generator=g, device="cuda").half()
    if c["op"] == "norm_rope":
        return s
    ps = c["ps"]
    if c["op"] == "append":  # the cache's older rows are not read: an empty pool of the size that the table needs
        pages = -(-max(lens) // ps)
        s["fields"] = None
    else:
        pages, s["fields"] = _fields(c, g, ns, lens)
    spare = 1 + c["nseq"] * pages // 16
    s["order"] = torch.randperm(c["nseq"] * pages + spare, generator=g, device="cuda")[: c["nseq"] * pages]
    s["num_pages"] = c["nseq"] * pages + spare
    table = s["order"].view(c["nseq"], pages).int()
    # pages that a sequence has not reached are not allocated yet
    need = torch.tensor([-(-ln // ps) for ln in lens], device="cuda")[:, None]
    s["pages"] = torch.where(torch.arange(pages, device="cuda")[None] < need, table, -1).contiguous()
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor(np.cumsum([0] + ns), dtype=torch.int32, device="cuda") if c["ragged"] else None
    return s


def prepare(case, seed):
    c = case
    s = _make(c, seed)
    s["case"] = c
    s["scale"] = c["d"] ** -0.5
    page_bytes = 2 * c["hkv"] * c["ps"] * c["d"] * 5 // 8
    if c["op"] != "norm_rope":
        s["pool"] = torch.zeros(s["num_pages"], page_bytes, dtype=torch.uint8, device="cuda")
        if s["fields"] is not None:
            s["pool"][s["order"]] = _pack(c, s["fields"])
        s["row_seq"] = torch.repeat_interleave(torch.arange(c["nseq"], device="cuda"), torch.tensor(s["ns"], device="cuda"))
    del s["fields" if "fields" in s else "ns"]
    if own:
        from quant_dequant_gemv_amd import binding
        s["rope"] = binding.Rope(s["inv_freq"], interleaved=c["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6)
        if c["op"] != "norm_rope":
            s["cache"] = binding.KVCache(s["num_pages"], c["hkv"], c["d"], c["ps"], pool=s["pool"])
    return s


# ------------------------------------------------------------------ the operators

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "norm_rope":
        return tuple(_norm_rope(c, s, s[x], s[x + "_norm"]).half() for x in "qk")
    if c["op"] == "attn":
        k, v = _unpack(c, s["pool"], s["pages"])
        return _layout(c, _attend(c, s, s["q"], k, v))
    q = _norm_rope(c, s, s["q"], s["q_norm"]).half()
    k = _quantise(_norm_rope(c, s, s["k"], s["k_norm"]))
    v = _quantise(s["v"])
    if c["op"] == "append":
        return q, k, v
    kc, vc = _unpack(c, s["pool"], s["pages"])
    at = (s["row_seq"], s["positions"].long())
    kc[at], vc[at] = k, v
    return _layout(c, _attend(c, s, q, kc, vc)), k, v


def _run_own(s, c):
    from quant_dequant_gemv_amd import binding
    if c["op"] == "norm_rope":
        return binding.norm_rope(s["rope"], s["positions"], s["q"], s["k"])
    if c["op"] == "attn":
        return _out(binding, s, c, s["q"])
    q = binding.kv_append(s["cache"], s["k"], s["v"], s["pages"], s["kv_len"], q_start=s["q_start"], q=s["q"], rope=s["rope"])
    out = _out(binding, s, c, q) if c["op"] == "step" else q
    k, v = binding.kv_read(s["cache"], s["rows"], s["pages"], s["kv_len"], q_start=s["q_start"])
    return out, k, v


def _out(binding, s, c, q):
    """The heads' outputs, feature-major where a GEMV of few columns reads them as its x."""
    out = None
    if c["fm"]:
        out = torch.empty(c["hq"] * c["d"], s["rows"], dtype=torch.float16, device="cuda")
    o = binding.kv_attn(s["cache"], q, s["pages"], s["kv_len"], q_start=s["q_start"], scale=s["scale"], window=c["window"],
                        out=None if out is None else out.view(c["hq"], c["d"], s["rows"]).permute(2, 0, 1))
    return o if out is None else out


def _layout(c, o):
    o = o.half()
    return o.permute(1, 2, 0).reshape(c["hq"] * c["d"], -1).contiguous() if c["fm"] else o


def _norm_rope(c, s, x, w):
    """fp64: angles of far positions, and keys next to a code's border."""
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
    half = c["rot"] // 2
    a = (s["positions"].double()[:, None] * s["inv_freq"].double())[:, None]
    cos, sin = torch.cos(a), torch.sin(a)
    r = x[..., : c["rot"]]
    u, v = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
    y = (u * cos - v * sin, u * sin + v * cos)
    y = torch.stack(y, -1).flatten(-2) if c["interleaved"] else torch.cat(y, -1)
    return torch.cat([y, x[..., c["rot"]:]], -1)


def _quantise(x):
    """The values that fp32 rows are held as."""
    shape = x.shape
    x = x.float().reshape(*shape[:-1], -1, 32).clamp(-65504, 65504)
    m = x.amin(-1, keepdim=True).half().float()
    d = ((x.amax(-1, keepdim=True) - m) / x.new_full((1,), 15)).half().float()  # a quotient: by a number, torch multiplies
    code = torch.where(d > 0, (x - m) / d, torch.zeros_like(x)).round().clamp(0, 15)
    return (code.double() * d.double() + m.double()).float().reshape(shape)


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _unpack(c, pool, pages):
    """fp32 keys and values [nseq][max_pages * ps][hkv][d] of the paged cache."""
    ps, h, d, grp = c["ps"], c["hkv"], c["d"], c["d"] // 32
    x = pool[pages.clamp(min=0).long().flatten()].view(-1, h, 2, ps * d * 5 // 8)
    p = x.shape[0]
    codes, steps, mins = x.split([ps * d // 2, ps * d // 16, ps * d // 16], -1)
    by4 = lambda t: t.contiguous().view(torch.float16).view(p, h, ps // 4, grp, 4).permute(0, 2, 4, 1, 3).reshape(p * ps, h, grp, 1).float()  # noqa: E731
    k = _nibbles(codes[:, :, 0].reshape(p, h, ps, 4, grp, 4)).permute(0, 2, 1, 4, 3, 5).reshape(p * ps, h, grp, 32).float()
    km = mins[:, :, 0].contiguous().view(torch.float16).view(p, h, ps, grp).permute(0, 2, 1, 3).reshape(p * ps, h, grp, 1).float()
    k = k * by4(steps[:, :, 0]) + km
    w, nib = max(1, d // 128), min(8, d // 16)
    v = _nibbles(codes[:, :, 1].reshape(p, h, ps // 4, w, 16, 4, nib // 2)).permute(0, 2, 5, 1, 3, 6, 4).reshape(p * ps, h, grp, 32).float()
    v = v * by4(steps[:, :, 1]) + by4(mins[:, :, 1])
    return k.view(c["nseq"], -1, h, d), v.view(c["nseq"], -1, h, d)


def _attend(c, s, q, k, v):
    """fp32 attention of every row over its sequence, in rows padded to the longest sequence's."""
    n, hq, d = c["n"], c["hq"], c["d"]
    nseq, length = k.shape[:2]
    pos = s["positions"].long()
    if c["ragged"]:
        first = s["q_start"].long()[:-1]
        slot = torch.arange(s["rows"], device="cuda") - first[s["row_seq"]]
    else:
        slot = torch.arange(s["rows"], device="cuda") % n
    at = (s["row_seq"], slot)
    qp = torch.zeros(nseq, n, hq, d, device="cuda")
    pp = torch.full((nseq, n), -1, dtype=torch.long, device="cuda")
    qp[at], pp[at] = q.float(), pos
    qp = qp.view(nseq, n, c["hkv"], -1, d).permute(0, 2, 1, 3, 4).reshape(nseq, c["hkv"], -1, d)
    sc = torch.matmul(qp, k.permute(0, 2, 3, 1).contiguous()).view(nseq, c["hkv"], n, -1, length) * s["scale"]
    j = torch.arange(length, device="cuda")
    see = j <= pp[..., None]
    if c["window"]:
        see &= j > pp[..., None] - c["window"]
    sc = sc.masked_fill(~see[:, None, :, None], -math.inf)
    e = torch.exp(sc - sc.amax(-1, keepdim=True))
    e = torch.where(see[:, None, :, None], e, torch.zeros_like(e))
    den = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(nseq, c["hkv"], -1, length), v.permute(0, 2, 1, 3).contiguous()).view(nseq, c["hkv"], n, -1, d)
    o = o / torch.where(den > 0, den, torch.ones_like(den))
    return o.permute(0, 2, 1, 3, 4).reshape(nseq, n, hq, d)[at]


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    c, s = case, _make(case, seed)

    def turned(x, w):
        x = x.to(torch.float64)
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * w.to(torch.float64)
        y, half = x.clone(), c["rot"] // 2
        lo = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
        hi = lo + (1 if c["interleaved"] else half)
        angle = torch.outer(s["positions"].to(torch.float64), s["inv_freq"].to(torch.float64))
        z = torch.complex(x[..., lo], x[..., hi]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    def held(x):
        """The values of the 4-bit groups: the operator takes fp32 rows and makes its groups in that type, numpy's here."""
        f = np.float32
        x = np.clip(x.float().cpu().numpy().reshape(s["rows"], c["hkv"], -1, 32), f(-65504), f(65504))
        m = x.min(-1, keepdims=True).astype(np.float16).astype(f)
        d = ((x.max(-1, keepdims=True) - m) / f(15)).astype(np.float16).astype(f)
        code = np.clip(np.rint(np.divide(x - m, d, out=np.zeros_like(x), where=d > 0)), 0, 15)
        held = d.astype(np.float64) * code + m
        return torch.from_numpy(held.reshape(s["rows"], c["hkv"], c["d"])).cuda()

    if c["op"] == "norm_rope":
        return turned(s["q"], s["q_norm"]), turned(s["k"], s["k_norm"])
    if c["op"] == "attn":
        q = s["q"].to(torch.float64)
    else:
        q, k, v = turned(s["q"], s["q_norm"]), held(turned(s["k"], s["k_norm"])), held(s["v"])
        if c["op"] == "append":
            return q, k, v
        q = q.half().to(torch.float64)  # the queries that the append leaves
    out = torch.zeros(s["rows"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    span = s["fields"][0][0].shape[0] // c["nseq"]
    r0 = 0
    for i, (n, ln) in enumerate(zip(s["ns"], s["lens"])):
        rows = slice(r0, r0 + n)
        r0 += n
        for h in range(c["hkv"]):
            kv = []
            for x, (code, step, m) in enumerate(s["fields"]):
                at = slice(i * span, i * span + ln)
                t = (code[at, h].double() * step[at, h, :, None].double() + m[at, h, :, None].double()).reshape(ln, c["d"])
                if c["op"] == "step":
                    t[ln - n:] = (k, v)[x][rows, h]
                kv.append(t)
            for hh in range(h * c["hq"] // c["hkv"], (h + 1) * c["hq"] // c["hkv"]):
                a = q[rows, hh] @ kv[0].T * c["d"] ** -0.5
                j, p = torch.arange(ln, device="cuda")[None], torch.arange(ln - n, ln, device="cuda")[:, None]
                a[(j > p) | (j <= p - (c["window"] or ln + 1))] = -math.inf
                out[rows, hh] = torch.softmax(a, -1) @ kv[1]
    if c["fm"]:
        out = out.permute(1, 2, 0).reshape(c["hq"] * c["d"], -1)
    return out if c["op"] == "attn" else (out, k, v)
