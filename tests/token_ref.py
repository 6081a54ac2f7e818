"""Plain numpy fp64 forms of the rest of a token -- block norms, the short
convolution, the gated delta recurrence, log probabilities -- written from
their formulas, row after row, with the bounds that the header states."""
import numpy as np

HALF = {np.float16: 2.0 ** -11, np.float32: 2.0 ** -24}
TINY = {np.float16: 2.0 ** -25, np.float32: 2.0 ** -140}


def rounded(got, ref, err, dtype):
    """got is ref within err and one rounding to dtype (beyond its range +-inf)."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape
    big = np.abs(ref) + err >= np.finfo(dtype).max
    ok = np.abs(got - ref) <= err + HALF[dtype] * (np.abs(ref) + err) + TINY[dtype]
    ok |= big & (np.sign(got) == np.sign(ref)) & (np.abs(got) >= np.finfo(dtype).max * (1 - 2.0 ** -10))
    assert ok.all(), (np.argwhere(~ok)[:4], got[~ok][:4], ref[~ok][:4])


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


# ------------------------------------------------------------------ block norm

def block_norm(y, post, gate, act, scale, residual, pre, eps):
    """h, x [..., dim] in fp64, and the errors that fp32 may add to each, in units u = 2^-24 of a value: a thread's sum of
    8 squares 8 (the root half of that), the mean 0.5, the root 1, two products and the weight 2: 7.5 of 8 u for n; with
    the gate's function (6) and two products more 15.5 of 16 u for what is added to the residual."""
    y = y.astype(np.float64)
    rms = lambda x: np.sqrt((x * x).mean(-1, keepdims=True) + eps)  # noqa: E731
    n = y if post is None else y / rms(y) * post.astype(np.float64)
    if gate is not None:
        z = gate.astype(np.float64)
        n = n * {"none": z, "silu": z * sigmoid(z), "sigmoid": sigmoid(z)}[act]
    h = scale * n + (0 if residual is None else residual.astype(np.float64))
    e = 2.0 ** -20 * np.abs(scale * n) + 2.0 ** -23 * np.abs(h) + 2.0 ** -126
    if pre is None:
        return h, h, e, e
    r, w = rms(h), np.abs(pre.astype(np.float64))
    x = h / r * pre.astype(np.float64)
    ex = 2.0 ** -21 * np.abs(x) + w * e / r + 2.0 ** -20 * np.abs(x) * (e / r).max(-1, keepdims=True)
    return h, x, e, ex


# ------------------------------------------------------------------ sequences with a state

def sequences(rows, nseq, q_start, slots, slots_out, kv_len, commit, num_slots):
    """(first, n, slot to read or None, slot to write or None, rows committed) of each."""
    for s in range(nseq):
        first, n = (s * (rows // nseq), rows // nseq) if q_start is None else (q_start[s], q_start[s + 1] - q_start[s])
        src = slots[s] if kv_len is None or kv_len[s] > n else -1
        dst = (slots if slots_out is None else slots_out)[s]
        m = n if commit is None else min(max(commit[s], 0), n)
        yield int(first), int(n), int(src) if 0 <= src < num_slots else None, int(dst) if 0 <= dst < num_slots else None, int(m)


def conv_silu(pool, weight, bias, x, seqs, act):
    """y and its error bound [rows, C], and the new pool."""
    taps = weight.shape[1]
    y, err, new = np.zeros(x.shape), np.zeros(x.shape), pool.copy()
    w = weight.astype(np.float64)
    for first, n, src, dst, m in seqs:
        old = np.zeros(pool.shape[1:]) if src is None else pool[src].astype(np.float64)
        xs = np.concatenate([old, x[first: first + n].astype(np.float64)])
        for i in range(n):
            terms = xs[i: i + taps] * w.T
            b = 0 if bias is None else bias.astype(np.float64)
            s, e = terms.sum(0) + b, 2.0 ** -20 * (np.abs(terms).sum(0) + np.abs(b))
            if act:
                s = s * sigmoid(s)
            y[first + i], err[first + i] = s, e + 2.0 ** -22 * np.abs(s)
        if dst is not None and m:
            new[dst] = xs[m: m + taps - 1]
    return y, err, new


def delta_rule(pool, q, k, v, alpha, beta, seqs, A, dt, norm, eps, scale, unit=2.0 ** -18, floor=2.0 ** -26):
    """out, its bound, the new pool and its bound (columns), in fp64.

    Every step's error, at most `unit` of what it adds up, then shrinks with the state: a (I - b k k^T) has norm <= a
    for 0 <= b <= 2 and |k| <= 1.

    floor: where 64 rows are worked on together, V - K S0 and U are fp16 pairs on one scale a column, set by m <= max|v| + 24
    max|S0| over those rows so that m is below 2^15 (U: 64 m): a pair ends at 2^-25, 2^-39 m (2^-33 m) of a value.  U = T R
    sums 64 entries up to 1: 2^-33 m; with its own end 2^-32 m; a state and an output sum 64 rows of U: 2^-26 m.  Nothing of
    that shrinks with the decays inside the 64 rows."""
    q, k, v, alpha, beta = (t.astype(np.float64) for t in (q, k, v, alpha, beta))
    rows, hv, dv = v.shape
    rep = hv // k.shape[1]
    if norm:
        q, k = (t / np.sqrt((t * t).sum(-1, keepdims=True) + eps) for t in (q, k))
    q, k = q.repeat(rep, 1), k.repeat(rep, 1)
    g, b = alpha, beta
    if A is not None:
        g = A.astype(np.float64) * np.logaddexp(alpha + (0 if dt is None else dt.astype(np.float64)), 0)
        b = sigmoid(beta)
    g = np.where(g > 0, 0, g)
    out, err = np.zeros(v.shape), np.zeros(v.shape)
    new, new_err = pool.astype(np.float64), np.zeros(pool.shape[:3])
    for first, n, src, dst, m in seqs:
        S = np.zeros(pool.shape[1:]) if src is None else pool[src].astype(np.float64)
        E = np.zeros(S.shape[:2])  # of a column, in its norm
        last = []                  # of the last 64 rows: |v| and 24 |S|
        for i in range(n):
            t = first + i
            a = np.exp(g[t])[:, None]
            before = np.abs(S).max(-1)
            size = a * np.sqrt((S * S).sum(-1)) * (1 + np.abs(np.maximum(g[t], -200))[:, None])
            u = b[t][:, None] * (v[t] - a * np.einsum("hvk,hk->hv", S, k[t]))
            S = a[..., None] * S + u[..., None] * k[t][:, None]
            E = a * E + unit * (size + np.abs(b[t][:, None] * v[t])) + 2.0 ** -130
            out[t] = scale * np.einsum("hvk,hk->hv", S, q[t])
            last = last[-63:] + [np.maximum(np.abs(v[t]), 24 * before)]
            F = 2 * floor * np.max(last, 0)
            if i % 64 == 63 or i + 1 == m:
                E = E + F  # (a tile's end)
            err[t] = abs(scale) * np.sqrt((q[t] ** 2).sum(-1))[:, None] * (E + F + unit * np.sqrt((S * S).sum(-1)))
            if dst is not None and i + 1 == m:
                new[dst], new_err[dst] = S, E
    return out, err, new, new_err


# ------------------------------------------------------------------ log probabilities

def logprobs(z, tokens, top, scale):
    """token_lp, lse, entropy, ids, top_lp and the bounds of the first three and the last."""
    z = z.astype(np.float64)
    rows, vocab = z.shape
    lse, ent = np.empty(rows), np.empty(rows)
    lp, dist = np.empty(z.shape), np.zeros(z.shape)
    ids = np.full((rows, top), -1, np.int64)
    for r in range(rows):
        row = z[r]
        live = row > -np.inf
        m = np.where(np.isnan(row), -np.inf, row).max()
        if np.isnan(row).any() or m == np.inf:
            lse[r] = ent[r] = np.nan
            lp[r] = np.nan
        elif m == -np.inf:
            lse[r], ent[r], lp[r] = -np.inf, 0, -np.inf
        else:
            t = (row[live] - m) * scale
            ls = np.log(np.exp(t).sum())
            lse[r] = m * scale + ls
            p = t - ls
            e = np.exp(p)
            ent[r] = -(e * np.where(e > 0, p, 0)).sum()
            lp[r] = -np.inf
            lp[r][live] = p
            dist[r][live] = -t
        order = [i for i in np.lexsort((np.arange(vocab), np.where(live, -(row + 0.0), np.inf))) if live[i]][:top]
        ids[r, : len(order)] = order
    unit = 2.0 ** -20
    token = token_err = None
    if tokens is not None:
        held = (tokens >= 0) & (tokens < vocab)
        at = np.where(held, tokens, 0)
        token = np.where(held, np.take_along_axis(lp, at, 1), 0.0)
        token_err = unit * (1 + np.take_along_axis(dist, at, 1))
    at = np.maximum(ids, 0)
    top_lp = np.where(ids >= 0, np.take_along_axis(lp, at, 1), -np.inf)
    peak = np.where(np.isfinite(z), z, -np.inf).max(-1)
    lse_err = unit + 2.0 ** -23 * np.where(np.isfinite(peak), np.abs(peak) * scale, 0)
    return ((token, token_err), (lse, lse_err), (ent, np.full(rows, 2.0 ** -18 * (1 + np.log(vocab)))), ids,
            (top_lp, unit * (1 + np.take_along_axis(dist, at, 1))))


def near(got, ref, err):
    """got is ref within err; NaN and infinities where ref has them."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape
    with np.errstate(invalid="ignore"):
        ok = (np.isnan(ref) & np.isnan(got)) | (got == ref) | (np.abs(got - ref) <= err)
    assert ok.all(), (np.argwhere(~ok)[:4], got[~ok][:4], ref[~ok][:4])
