"""A cache filled through qk_kv_append from given rows, and fp64 attention over it by matrix products: long contexts
without packing pages one nibble at a time (the bytes that an append writes are tested by themselves)."""
from __future__ import annotations

import numpy as np

import kv_ref


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Fields:
    """Keys or values x, fp32 [length, hkv, D], and what the cache holds of them: values and d * code + |m| by KV
    head, [hkv, length, D]; steps and |minima| [hkv, length, D/32]."""

    def __init__(self, x):
        self.x = x
        code, d, m = (np.ascontiguousarray(np.swapaxes(t, 0, 1)) for t in kv_ref.quantise(x))
        self.values, self.sizes = kv_ref.values(code, d, m), kv_ref.values(code, d, np.abs(m))
        self.d, self.m = d, np.abs(m)


class Filled:
    """One context on shuffled pages.  `table(nseq)` is a page table of nseq sequences that all see it.  holes: pages
    of the context that the table does not hold."""

    def __init__(self, rng, keys, values, ps, holes=()):
        from quant_dequant_gemv_amd import binding
        self.length, self.hkv, self.D = keys.x.shape
        self.ps, self.mp = ps, -(-self.length // ps)
        self.pages = rng.permutation(self.mp + 2)[None, :self.mp].astype(np.int32)
        self.cache = binding.KVCache(self.mp + 2, self.hkv, self.D, ps)
        binding.kv_append(self.cache, _dev(keys.x), _dev(values.x), _dev(self.pages), _dev(np.array([self.length], np.int32)))
        self.pages[0, list(holes)] = -1
        self.k, self.v = keys, values
        self.held = np.repeat(self.pages[0] >= 0, ps)[:self.length]

    def table(self, nseq):
        return _dev(np.repeat(self.pages, nseq, 0))


def attention(c, q, pos, seen, scale, window=0):
    """One row of queries q [hq, D] at position pos, in fp64: its output, and how far the kernel may be from it in
    fp32.  seen: positions that the rows of its sequence see, as a slice.

    The bound is kv_ref.attention_bound's, and what the two fp16 terms of a probability and of its product with a
    step may lose.  With P the row's largest probability, both are held in units of 2^-37 P (fp16's last place 2^-24
    where P is 2^13 or more), the product in units of a power of two U above the largest step S, at most 16 S (2^-14 at
    the least): a position loses up to half a unit of its weight, for the sum of the weights and for its minimum, and
    for a code of 15 at most 15 P (2^-25 d + 1.5 * 2^-24 U) 2^-13 < 2^-28 P S.  Steps brought down because S >= 1 (U is
    then 2 S at most) are rounded by 2^-25 U, once for all positions: 15 * 2^-24 S < 2^-20 S."""
    j = np.arange(max(0, pos - window + 1) if window else 0, pos + 1)
    j = j[c.held[j]]
    at = slice(None) if len(j) == c.length else j
    q = np.asarray(q, np.float64)
    g = q.shape[0] // c.hkv
    out, bound = np.zeros_like(q), np.zeros_like(q)
    every = np.arange(c.length)[seen]
    every = every[c.held[every]]
    for h in range(c.hkv if len(j) else 0):
        x = q[h * g:(h + 1) * g]
        e = scale * (x @ c.k.values[h, at].T)
        e = np.exp(e - e.max(-1, keepdims=True))
        e /= e.sum(-1, keepdims=True)
        o = e @ c.v.values[h, at]
        amax = abs(scale) * (np.abs(x) @ c.k.sizes[h, at].T).max(-1)
        step, low = max(float(c.v.d[h, every].max()), 2.0 ** -15), float(c.v.m[h, every].max())
        out[h * g:(h + 1) * g] = o
        mass, most = e @ c.v.sizes[h, at], len(j) * e.max(-1, keepdims=True)
        bound[h * g:(h + 1) * g] = kv_ref.attention_bound(o, mass, amax, False) + \
            most * (2.0 ** -38 * mass + 2.0 ** -28 * step + 2.0 ** -38 * low) + (2.0 ** -20 * step if step >= 1 else 0)
    return out, bound


def check_attn(c, q, ns, split, picks, window=0, length=None):
    """q [rows, hq, D], ns[s] rows for sequence s (or the number of sequences, of as many rows each), every sequence
    over the context c, into fp32; the rows `picks` against fp64.  split: whether the call has to be one that cuts
    contexts into splits."""
    import torch
    from quant_dequant_gemv_amd import binding
    rows, hq = q.shape[:2]
    even = isinstance(ns, int)
    ns = [rows // ns] * ns if even else ns
    first = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    length, scale = length or c.length, c.D ** -0.5
    out = torch.full((rows, hq, c.D), 77.0, device="cuda")
    lens, pages, q_start = _dev(np.full(len(ns), length, np.int32)), c.table(len(ns)), None if even else _dev(first)
    need = binding.qk_kv_attn_workspace_bytes(c.cache._c, binding._seqs_arg(rows, pages, lens, q_start), hq)
    assert (need > 0) == split, "not the form that this case is for"
    binding.kv_attn(c.cache, _dev(q), pages, lens, q_start=q_start, out=out, window=window)
    torch.cuda.synchronize()
    got = out[list(picks)].cpu().numpy().astype(np.float64)
    worst = 0
    for t, y in zip(picks, got):
        s = int(np.searchsorted(first, t, "right")) - 1
        n, i = ns[s], t - first[s]
        seen = slice(max(0, length - n - window + 1) if window else 0, length)
        want, bound = attention(c, q[t], length - n + i, seen, scale, window)
        err = np.abs(y - want)
        assert (err <= bound).all(), \
            f"row {t}: {np.max(err / bound):.3g} of the bound, {np.max(err) / np.max(np.abs(want)):.3g} of the output"
        worst = max(worst, np.max(err / bound))
    return worst
