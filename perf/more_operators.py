"""The cases that the rest of a decode token is measured on: norms around a block with its
gate and residual, the short convolution and the gated delta recurrence of the DeltaNet
layers, and log probabilities of tokens with their entropy and the top alternatives.

``run`` computes them in plain torch, or with ``own`` through the public helpers of
``quant_dequant_gemv_amd.binding``.  Inputs lie as the projections' GEMVs leave them: fp32
``[N][ncols]`` (feature-major) for decode and verify widths, token-major rows for batches and
prompts.  Recurrent states live in slots of a pool; a call reads a sequence's state from one
slot and leaves the new one in another, as a server does that may still go back.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases

_NONE = dict(rows=1, groups=1, dim=5120, f16=False, fm=False, post=False, gate="", residual=True, pre=True, scale=1.0)
_CONV = dict(nseq=1, n=1, ragged=False, drafts=False, fresh=False, channels=10240, taps=4, bias=False, fm=False, f16=False)
_DELTA = dict(nseq=1, n=1, ragged=False, drafts=False, fresh=False, hk=16, hv=48, dk=128, dv=128, fm=False, f16=False)
_PROBS = dict(rows=1, vocab=160000, f16=False, fm=False, ntok=1, top=20, scale=1.0, masked=False)


def _case(name, op, **kw):
    return {"name": name, "op": op, **{"norm": _NONE, "conv": _CONV, "delta": _DELTA, "probs": _PROBS}[op], **kw}


def listed():
    return [
        # a decode token, before a block: the projection's output joins the residual stream, which is normed for the next
        _case("norm 1 token 5120", "norm", fm=True),
        # 17 drafted tokens with a norm behind the block too, its output scaled
        _case("norm 17 drafts 5120", "norm", rows=17, fm=True, post=True, scale=0.7),
        # a prompt's head outputs of the recurrence: each head normed, then gated by the silu of its own projection
        _case("norm 2048 rows 48 heads gated", "norm", rows=2048, groups=48, dim=128, post=True, gate="silu",
              residual=False, pre=False),
        # 17 drafted tokens through the short convolution, its state kept after those that were accepted
        _case("conv 17 drafts", "conv", n=17, drafts=True, fm=True),
        # a prompt's first 4096 rows
        _case("conv 4096 rows", "conv", n=4096, fresh=True),
        # one token of one stream: latency
        _case("delta 1 token", "delta", fm=True),
        # one token each of 64 sequences: the states' way to the chip and back
        _case("delta 64 seqs", "delta", nseq=64),
        # a prompt of 4096 rows in one call
        _case("delta 4096 rows", "delta", n=4096, fresh=True),
        # a batch of prompts of unlike lengths that continue, fp16 rows
        _case("delta 12 seqs ragged", "delta", nseq=12, n=701, ragged=True, hk=4, hv=8, f16=True),
        # one token's logits: its log probability, the entropy and 20 alternatives
        _case("probs 1 token", "probs", fm=True),
        # verification of 17 drafts under a temperature, as the head's GEMV leaves the logits
        _case("probs 17 drafts", "probs", rows=17, fm=True, scale=1 / 0.7, masked=True),
        # a text's log probabilities in one call, fp16 logits
        _case("probs 1021 rows f16", "probs", rows=1021, vocab=131071, f16=True, top=5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    most = {}
    for c in listed():
        for k, v in work(c).items():
            most[c["op"], k] = max(v, most.get((c["op"], k), 0))
    while True:  # at most the cost of the operator's listed ones
        c = _drawn(rng)
        if all(v <= most[c["op"], k] for k, v in work(c).items()):
            return c


def _drawn(rng):
    op = rng.choice(["norm", "conv", "delta", "delta", "probs"])
    few = rng.random() < 0.5  # a few columns of one stream, or a batch / a prompt
    fm = few and rng.random() < 0.7
    f16 = not fm and rng.random() < 0.5
    if op == "norm":
        heads = rng.random() < 0.5
        return _case("drawn", op, rows=_log(rng, 1, 32 if few else 8192), groups=rng.randint(1, 64) if heads else 1,
                     dim=rng.choice([64, 128, 256, rng.randint(1, 300)]) if heads else _log(rng, 64, 16384), fm=fm, f16=f16,
                     post=rng.random() < 0.6, gate=rng.choice(["", "silu", "sigmoid", "none"]), residual=rng.random() < 0.6,
                     pre=rng.random() < 0.6, scale=rng.choice([1.0, 0.25, 1.5]))
    if op == "probs":
        return _case("drawn", op, rows=_log(rng, 1, 32 if few else 1024), vocab=_log(rng, 1000, 262144), fm=fm, f16=f16,
                     ntok=rng.randint(0, 4), top=rng.choice([0, 1, 5, 20, 50]), scale=rng.choice([1.0, 0.5, 1 / 0.7]),
                     masked=rng.random() < 0.3)
    nseq = 1 if few else _log(rng, 1, 64)
    n = _log(rng, 1, 32) if few else _log(rng, 1, 4096 if nseq == 1 else 512)
    kw = dict(nseq=nseq, n=n, ragged=nseq > 1 and rng.random() < 0.5, drafts=n <= 32 and rng.random() < 0.5,
              fresh=rng.random() < 0.3, fm=fm, f16=f16)
    if op == "conv":
        return _case("drawn", op, channels=_log(rng, 64, 16384), taps=rng.randint(2, 6), bias=rng.random() < 0.3, **kw)
    hk = rng.randint(1, 16)
    return _case("drawn", op, hk=hk, hv=hk * rng.randint(1, 4), dk=rng.choice([64, 128]), dv=rng.choice([64, 96, 128, 256]), **kw)


def _counts(c):
    """Rows of each sequence, and after how many of them its state is kept: of the case alone."""
    r = random.Random("%d %d" % (c["nseq"], c["n"]))
    ns = [r.randint(1, c["n"]) if c["ragged"] else c["n"] for _ in range(c["nseq"])]
    return ns, [r.randint(0, n) if c["drafts"] else n for n in ns]


def work(c):
    x = 2 if c["f16"] else 4
    if c["op"] == "norm":
        n = c["rows"] * c["groups"] * c["dim"]
        return {"bytes": n * (x + x * bool(c["gate"]) + 8 * c["residual"] + 2), "flops": 10 * n}
    if c["op"] == "probs":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * x, "flops": 6 * n}
    rows = sum(_counts(c)[0])
    if c["op"] == "conv":
        state = c["nseq"] * (c["taps"] - 1) * c["channels"] * 4
        return {"bytes": rows * c["channels"] * (x + x) + state * (1 if c["fresh"] else 2),
                "flops": rows * c["channels"] * (2 * c["taps"] + 4)}
    state = c["nseq"] * c["hv"] * c["dk"] * c["dv"] * 4
    row = x * (2 * c["hk"] * c["dk"] + 2 * c["hv"] * c["dv"] + 2 * c["hv"])
    return {"bytes": rows * row + state * (1 if c["fresh"] else 2), "flops": rows * c["hv"] * 7 * c["dk"] * c["dv"]}


# ------------------------------------------------------------------ inputs

def _values(g, c, rows, *shape):
    """Rows of a projection: [rows, *shape] as a view of what it leaves, channels of unlike scale."""
    n = math.prod(shape)
    t = torch.randn(rows, n, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(n, generator=g, device="cuda"))
    t = t.half() if c["f16"] else t
    t = t.t().contiguous().t() if c["fm"] else t
    return t.unflatten(1, shape)


def _make(c, seed):
    """Everything of a case from its seed."""
    g = torch.Generator("cuda").manual_seed(int(seed))
    rand = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    s = {}
    if c["op"] == "norm":
        shape = (c["groups"], c["dim"])
        s["y"] = _values(g, c, c["rows"], *shape)
        s["gate"] = _values(g, c, c["rows"], *shape) if c["gate"] else None
        s["residual"] = _values(g, {**c, "f16": False}, c["rows"], *shape) * 3 if c["residual"] else None
        s["post"] = 1 + 0.2 * rand(c["dim"]) if c["post"] else None
        s["pre"] = 1 + 0.2 * rand(c["dim"]) if c["pre"] else None
        return s
    if c["op"] == "probs":
        z = _values(g, {**c, "f16": False}, c["rows"], c["vocab"])
        z = z.mul_(2).add_(3 * rand(c["rows"], 1)).clamp_(-60, 60)
        if c["masked"]:  # a grammar leaves some of the tokens
            z.masked_fill_(torch.rand(c["vocab"], generator=g, device="cuda") < 0.6, -math.inf)
        s["logits"] = z.half() if c["f16"] else z
        tok = torch.randint(0, c["vocab"], (c["rows"], c["ntok"]), generator=g, device="cuda").int()
        s["tokens"] = tok if c["ntok"] else None
        return s
    ns, commit = _counts(c)
    rows, nseq = sum(ns), c["nseq"]
    s["ns"], s["kept"], s["rows"] = ns, commit, rows
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s["q_start"] = i32([sum(ns[:i]) for i in range(nseq + 1)]) if c["ragged"] else None
    s["kv_len"] = i32([n if c["fresh"] else n + 100 for n in ns])
    s["commit"] = i32(commit) if c["drafts"] else None
    s["slots"] = torch.randperm(nseq + 3, generator=g, device="cuda")[:nseq].int()  # states are read from here
    s["slots_out"] = torch.arange(nseq + 3, 2 * nseq + 3, device="cuda").int()      # and left here
    num = 2 * nseq + 3
    if c["op"] == "conv":
        s["x"] = _values(g, c, rows, c["channels"])
        s["weight"] = 0.4 * rand(c["channels"], c["taps"])
        s["bias"] = 0.1 * rand(c["channels"]) if c["bias"] else None
        s["pool"] = rand(num, c["taps"] - 1, c["channels"])
        return s
    hk, hv, dk, dv = c["hk"], c["hv"], c["dk"], c["dv"]
    x = _values(g, c, rows, 2 * hk * dk + hv * dv)  # q, k and v side by side, as the convolution leaves them
    x *= torch.sigmoid(x)
    s["q"] = x[:, : hk * dk].unflatten(1, (hk, dk))
    s["k"] = x[:, hk * dk: 2 * hk * dk].unflatten(1, (hk, dk))
    s["v"] = x[:, 2 * hk * dk:].unflatten(1, (hv, dv))
    s["alpha"], s["beta"] = _values(g, c, rows, hv), _values(g, c, rows, hv)
    u = torch.rand(2, hv, generator=g, device="cuda")
    s["A"] = -torch.exp(u[0] * math.log(16))
    s["dt_bias"] = torch.log(torch.expm1(torch.exp(math.log(1e-3) + u[1] * math.log(100))))
    s["pool"] = 0.2 * rand(num, hv, dv, dk)
    return s


def prepare(case, seed):
    s = _make(case, seed)
    s["case"] = case
    if case["op"] == "norm" and case["residual"]:
        s["h"] = torch.empty_like(s["residual"])
    if own:
        from quant_dequant_gemv_amd import binding
        if case["op"] == "conv":
            s["state"] = binding.ConvState(s["pool"].shape[0], s["weight"], s["bias"], pool=s["pool"])
        elif case["op"] == "delta":
            s["state"] = binding.DeltaState(s["pool"].shape[0], case["hk"], case["hv"], case["dk"], case["dv"], pool=s["pool"])
    return s


# ------------------------------------------------------------------ the operators

def run(state):
    s, c = state, state["case"]
    return {"norm": _norm, "conv": _conv, "delta": _delta, "probs": _probs}[c["op"]](s, c)


def _norm(s, c):
    if own:
        from quant_dequant_gemv_amd import binding
        x = torch.empty_like(s["y"], dtype=torch.float16)
        binding.block_norm(s["y"], post_norm=s["post"], gate=s["gate"], act=c["gate"] or "none", scale=c["scale"],
                           residual=s["residual"], pre_norm=s["pre"], h_out=s.get("h"), x_out=x)
        return (s["h"], x) if c["residual"] else x
    t = s["y"].float()
    if c["post"]:
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * s["post"]
    if c["gate"]:
        z = s["gate"].float()
        t = t * {"silu": z * torch.sigmoid(z), "sigmoid": torch.sigmoid(z), "none": z}[c["gate"]]
    h = t * c["scale"]
    if c["residual"]:
        h = s["residual"] + h
    x = h
    if c["pre"]:
        x = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["pre"]
    return (h, x.half()) if c["residual"] else x.half()


def _conv(s, c):
    if own:
        from quant_dequant_gemv_amd import binding
        y = binding.conv_silu(s["state"], s["x"], s["slots"], s["slots_out"], q_start=s["q_start"], kv_len=s["kv_len"],
                              commit=s["commit"])
        return y, s["pool"][c["nseq"] + 3:]
    back = c["taps"] - 1
    old = s["pool"][s["slots"].long()]
    if c["fresh"]:
        old = torch.zeros_like(old)
    rows = torch.split(s["x"].float(), s["ns"])
    x = torch.cat([t for i, r in enumerate(rows) for t in (old[i], r)])  # every sequence behind what came before it
    first = torch.repeat_interleave(torch.arange(c["nseq"], device="cuda") * back, torch.tensor(s["ns"], device="cuda"))
    at = torch.arange(s["rows"], device="cuda") + first
    y = torch.zeros(s["rows"], c["channels"], device="cuda")
    for j in range(c["taps"]):
        y = y + s["weight"][:, j] * x[at + j]
    if c["bias"]:
        y = y + s["bias"]
    y = y * torch.sigmoid(y)
    starts = [sum(s["ns"][:i]) + i * back + m for i, m in enumerate(s["kept"])]
    new = torch.stack([x[p: p + back] for p in starts])
    keep = torch.tensor(s["kept"], device="cuda")[:, None, None] == 0  # nothing kept: the slot as it was
    return y.to(s["x"].dtype), torch.where(keep, s["pool"][c["nseq"] + 3:], new)


def _delta(s, c):
    if own:
        from quant_dequant_gemv_amd import binding
        o = binding.delta_rule(s["state"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["slots"], s["slots_out"],
                               q_start=s["q_start"], kv_len=s["kv_len"], commit=s["commit"], A=s["A"],
                               dt_bias=s["dt_bias"])
        return o, s["pool"][c["nseq"] + 3:]
    nseq, n, hv, dk = c["nseq"], max(s["ns"]), c["hv"], c["dk"]
    ns = torch.tensor(s["ns"], device="cuda")
    at = (torch.cumsum(ns, 0) - ns)[:, None] + torch.arange(n, device="cuda")  # rows in steps, padded to the longest
    there = torch.arange(n, device="cuda") < ns[:, None]
    at = at.clamp(max=s["rows"] - 1)
    unit = lambda x: x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)  # noqa: E731
    rep = hv // c["hk"]
    q = (unit(s["q"].float()) * dk ** -0.5).repeat_interleave(rep, 1)[at].unsqueeze(-1)
    k = unit(s["k"].float()).repeat_interleave(rep, 1)[at].unsqueeze(-2)
    v = s["v"].float()[at].unsqueeze(-1)
    w = s["alpha"].float() + s["dt_bias"]
    decay = s["A"] * (torch.clamp(w, min=0) + torch.log1p(torch.exp(-w.abs())))  # log(1 + e^w)
    a = torch.exp(decay)[at].masked_fill(~there[..., None], 1)[..., None, None]
    b = torch.sigmoid(s["beta"].float())[at].masked_fill(~there[..., None], 0)[..., None, None]
    st = s["pool"][s["slots"].long()]
    if c["fresh"]:
        st = torch.zeros_like(st)
    kept = s["pool"][nseq + 3:]
    commit = torch.tensor(s["kept"], device="cuda")[:, None, None, None]
    out = []
    for t in range(n):  # st: [nseq, hv, dv, dk]
        st = st * a[:, t]
        kt = k[:, t]
        u = b[:, t] * (v[:, t] - (st * kt).sum(-1, keepdim=True))
        st = st + u * kt
        out.append(torch.matmul(st, q[:, t])[..., 0])
        if c["drafts"]:
            kept = torch.where(commit == t + 1, st, kept)
    o = torch.stack(out, 1)[there]
    return o, kept if c["drafts"] else st


def _probs(s, c):
    if own:
        from quant_dequant_gemv_amd import binding
        return tuple(x for x in binding.logprobs(s["logits"], s["tokens"], top=c["top"], scale=c["scale"]) if x is not None)
    outs = []
    for r in range(0, c["rows"], 256):  # as many rows at once as leave room for the sort keys
        z = s["logits"][r: r + 256]
        zf = z.float()
        m = zf.amax(-1, keepdim=True)
        t = (zf - m) * c["scale"]
        e = torch.exp(t)
        den = e.sum(-1, keepdim=True)
        logden = torch.log(den)
        ent = (logden - (e * t.clamp(min=-1e4)).sum(-1, keepdim=True) / den)[:, 0]
        lse = (m * c["scale"] + logden)[:, 0]
        part = [lse, ent]
        if c["ntok"]:
            part.insert(0, (torch.gather(zf, 1, s["tokens"][r: r + 256].long()) - m) * c["scale"] - logden)
        if c["top"]:
            bits = (zf + 0.0).view(torch.int32).long()
            key = torch.where(bits < 0, -2147483648 - bits, bits) * 4294967296 - torch.arange(c["vocab"], device="cuda")
            best = torch.topk(key, c["top"], -1).values  # ties: the lowest index
            ids = (-best) % 4294967296
            top = (torch.gather(zf, 1, ids) - m) * c["scale"] - logden
            part += [torch.where(top == -math.inf, -1, ids).int(), top]
        outs.append(part)
    return tuple(torch.cat(x) for x in zip(*outs))


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    c, s = case, _make(case, seed)
    d = torch.float64
    if c["op"] == "norm":
        x = s["y"].to(d)
        rms = lambda x: (x.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt()  # noqa: E731
        if c["post"]:
            x = x / rms(x) * s["post"].to(d)
        if c["gate"]:
            z = s["gate"].to(d)
            x = x * (z if c["gate"] == "none" else (z if c["gate"] == "silu" else 1) / (1 + torch.exp(-z)))
        h = c["scale"] * x + (s["residual"].to(d) if c["residual"] else 0)
        x = h / rms(h) * s["pre"].to(d) if c["pre"] else h
        return (h, x) if c["residual"] else x
    if c["op"] == "probs":
        return _exact_probs(c, s)
    outs, states = [], []
    back, r0 = c.get("taps", 1) - 1, 0
    for i, (n, m) in enumerate(zip(s["ns"], s["kept"])):
        st = s["pool"][s["slots"][i].long()].to(d)
        if c["fresh"]:
            st = torch.zeros_like(st)
        kept = s["pool"][c["nseq"] + 3 + i].to(d)
        rows = slice(r0, r0 + n)
        r0 += n
        if c["op"] == "conv":
            x = torch.cat([st, s["x"][rows].to(d)])
            y = (x.unfold(0, c["taps"], 1) * s["weight"].to(d)).sum(-1) + (s["bias"].to(d) if c["bias"] else 0)
            outs.append(y / (1 + torch.exp(-y)))
            states.append(x[m: m + back] if m else kept)
            continue
        q, k, v = (s[x][rows].to(d) for x in "qkv")
        q, k = (x / (x.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
        head = torch.arange(c["hv"], device="cuda") // (c["hv"] // c["hk"])
        q, k = q[:, head] / math.sqrt(c["dk"]), k[:, head]
        a = torch.exp(s["A"].to(d) * torch.logaddexp(s["alpha"][rows].to(d) + s["dt_bias"].to(d), torch.zeros((), dtype=d, device="cuda")))
        b = 1 / (1 + torch.exp(-s["beta"][rows].to(d)))
        st = st.transpose(1, 2).contiguous()  # [hv, dk, dv]
        for t in range(n):
            seen = torch.matmul(k[t].unsqueeze(1), st)[:, 0] * a[t][:, None]
            u = (v[t] - seen) * b[t][:, None]
            st = st * a[t][:, None, None] + k[t].unsqueeze(2) * u.unsqueeze(1)
            outs.append(torch.matmul(q[t].unsqueeze(1), st)[:, 0])
            if t + 1 == m:
                kept = st.transpose(1, 2).clone()
        states.append(kept)
    return (torch.cat(outs) if c["op"] == "conv" else torch.stack(outs)), torch.stack(states)


def _exact_probs(c, s):
    outs = []
    for r in range(0, c["rows"], 64):
        z = s["logits"][r: r + 64].to(torch.float64)
        lse = torch.logsumexp(z * c["scale"], -1)
        p = z * c["scale"] - lse[:, None]
        ent = -torch.where(p > -1e300, torch.exp(p) * p, torch.zeros_like(p)).sum(-1)
        part = [lse, ent]
        if c["ntok"]:
            part.insert(0, p[torch.arange(z.shape[0], device="cuda")[:, None], s["tokens"][r: r + 64].long()])
        if c["top"]:
            ids, left, place = [], z.clone(), torch.arange(c["vocab"], device="cuda")
            for _ in range(c["top"]):
                best = left.amax(-1, keepdim=True)
                i = torch.where(left == best, place, c["vocab"]).amin(-1, keepdim=True)
                ids.append(torch.where(best == -math.inf, -1, i))
                left.scatter_(1, i, -math.inf)
            ids = torch.cat(ids, 1)
            top = torch.gather(p, 1, ids.clamp(min=0)).masked_fill(ids < 0, -math.inf)
            part += [ids.int(), top]
        outs.append(part)
    return tuple(torch.cat(x) for x in zip(*outs))
