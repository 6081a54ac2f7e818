"""Plain numpy reference of the attention side: fp64 norm + rotation, the
4-bit groups in fp32 as the header defines them, the page layout bit by bit,
and fp64 attention.  Shares nothing with the kernels."""
from __future__ import annotations

import numpy as np


def norm_rope(x, pos, inv_freq=None, interleaved=False, w=None, eps=0.0):
    """x [rows, heads, D] -> fp64."""
    y = np.asarray(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * np.asarray(w, np.float64)
    if inv_freq is None or len(inv_freq) == 0:
        return y
    half = len(inv_freq)
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    out = y.copy()
    iu = 2 * np.arange(half) if interleaved else np.arange(half)
    iv = iu + 1 if interleaved else iu + half
    out[..., iu] = y[..., iu] * c - y[..., iv] * s
    out[..., iv] = y[..., iu] * s + y[..., iv] * c
    return out


def quantise(x):
    """fp32 rows [..., D] -> codes [..., D] uint8, d and m fp16 [..., D/32]."""
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-65504), np.float32(65504)))
    g = x.reshape(*x.shape[:-1], -1, 32)
    m = g.min(-1).astype(np.float16)
    d = ((g.max(-1) - m.astype(np.float32)) / np.float32(15)).astype(np.float16)
    m32, d32 = m.astype(np.float32)[..., None], d.astype(np.float32)[..., None]
    z = np.divide(g - m32, d32, out=np.zeros_like(g), where=d32 > 0)
    return np.clip(np.rint(z), 0, 15).astype(np.uint8).reshape(x.shape), d, m


def values(codes, d, m):
    """fp64 values of the groups (their fp32 rounding is what the cache reads as)."""
    g = codes.reshape(*codes.shape[:-1], -1, 32).astype(np.float64)
    return (g * d.astype(np.float64)[..., None] + m.astype(np.float64)[..., None]).reshape(codes.shape)


def pack_page(kc, kd, km, vc, vd, vm):
    """One page: codes [S, H, D], d and m [S, H, G] of keys and values -> bytes, nibble by nibble."""
    S, H, D = kc.shape
    G = D // 32
    out = np.zeros((H, 2, S * D * 5 // 8), np.uint8)
    dims = np.arange(D)
    g, a, n = dims // 32, dims % 32 // 8, dims % 8
    k_byte, k_nib = 4 * (a * G + g) + n // 2, n % 2
    if D == 64:
        l, n = dims % 16, dims // 16
        v_byte, v_nib = lambda p: (p // 4 * 16 + l) * 8 + (p % 4) * 2 + n // 2, n % 2
    else:
        w, n, l = dims // 128, dims % 128 // 16, dims % 16
        v_byte, v_nib = lambda p: (((p // 4) * (D // 128) + w) * 16 + l) * 16 + (p % 4) * 4 + n // 2, n % 2
    for h in range(H):
        for p in range(S):
            np.add.at(out[h, 0], p * D // 2 + k_byte, kc[p, h] << (4 * k_nib))
            np.add.at(out[h, 1], v_byte(p), vc[p, h] << (4 * v_nib))
        by4 = lambda x: np.ascontiguousarray(x[:, h].reshape(S // 4, 4, G).transpose(0, 2, 1)).view(np.uint8).ravel()  # noqa: E731
        at = S * D // 2
        for kind, (d, m) in enumerate(((kd, km), (vd, vm))):
            out[h, kind, at:at + 2 * S * G] = by4(d)
            out[h, kind, at + 2 * S * G:] = by4(m) if kind else np.ascontiguousarray(m[:, h]).view(np.uint8).ravel()
    return out.ravel()


class Cache:
    """A filled cache of nseq sequences: fields by position, and the pool."""

    def __init__(self, rng, nseq, pages_per_seq, hkv, D, ps, holes=(), spare=3, scale=1.0):
        self.nseq, self.mp, self.hkv, self.D, self.ps = nseq, pages_per_seq, hkv, D, ps
        cap = pages_per_seq * ps
        self.f = []
        for _ in range(2):
            x = rng.standard_normal((nseq, cap, hkv, D)) * np.exp(0.5 * rng.standard_normal((hkv, D))) * scale
            self.f.append(quantise(x.astype(np.float32)))
        self.num_pages = nseq * pages_per_seq + spare
        self.pages = rng.permutation(self.num_pages)[: nseq * pages_per_seq].reshape(nseq, pages_per_seq).astype(np.int32)
        pb = 2 * hkv * ps * D * 5 // 8
        # whatever was never written is garbage: NaN and infinite steps among it
        self.pool = rng.integers(0, 256, (self.num_pages, pb), dtype=np.uint8)
        self.pool[::2] = 0xff
        for s in range(nseq):
            for j in range(pages_per_seq):
                r = slice(j * ps, (j + 1) * ps)
                self.pool[self.pages[s, j]] = pack_page(*(x[s, r] for f in self.f for x in f))
        self.held = np.ones((nseq, pages_per_seq), bool)
        for s, j, bad in holes:
            self.pages[s, j] = bad
            self.held[s, j] = False

    def kv(self):
        return values(*self.f[0]), values(*self.f[1])

    def spoil(self, s, first):
        """Garbage in the pool's places of sequence s from position `first` on, as on a page only part written."""
        codes_d_m = [[np.array(x[s]) for x in f] for f in self.f]
        for c, d, m in codes_d_m:
            c[first:], d[first:], m[first:] = 15, np.float16(np.nan), np.float16(-np.inf)
        for j in range(first // self.ps, self.mp):
            r = slice(j * self.ps, (j + 1) * self.ps)
            if self.held[s, j]:
                self.pool[self.pages[s, j]] = pack_page(*(x[r] for f in codes_d_m for x in f))


def attention(c: Cache, q, rows, kv_len, scale, window=0):
    """fp64 outputs, sum_j p_j (d code + |m|) of the values, and max_j |scale| sum_i |q_i| (d code + |m|) of the keys.
    q [rows, hq, D]; rows: (sequence, index in it, count) of every row, or None for rows of no sequence."""
    hq = q.shape[1]
    g = hq // c.hkv
    K, V = c.kv()
    absv = [values(f[0], f[1], np.abs(f[2])) for f in c.f]
    out = np.zeros((len(rows), hq, c.D))
    mass = np.zeros_like(out)
    amax = np.zeros((len(rows), hq))
    for t, r in enumerate(rows):
        if r is None:
            continue
        s, i, n = r
        p = int(kv_len[s]) - n + i
        j = np.arange(max(0, p - window + 1) if window else 0, min(p + 1, c.mp * c.ps))
        j = j[c.held[s, j // c.ps]] if len(j) else j
        if not len(j):
            continue
        for h in range(hq):
            x = np.asarray(q[t, h], np.float64)
            sc = scale * (K[s, j, h // g] @ x)
            e = np.exp(sc - sc.max())
            e /= e.sum()
            out[t, h] = e @ V[s, j, h // g]
            mass[t, h] = e @ absv[1][s, j, h // g]
            amax[t, h] = abs(scale) * (absv[0][s, j, h // g] @ np.abs(x)).max()
    return out, mass, amax


def attention_bound(out, mass, amax, f16):
    """How far fp32 arithmetic may be from the fp64 outputs.  A score is a sum of exact products in fp32 (32 to a
    group, 8 groups, the minima's terms with 22 bits): off by less than 64 * 2^-24 of |scale| sum |q| (d code + |m|)
    = amax at most.  So each p_j is off by that plus the exponential's and the two-term split's 2^-19 relative, the
    quotient by twice that; summing adds less than 2^-16 over the lengths here; then the output's rounding."""
    rel = 2.0 ** -16 + 2.0 ** -18 + 2 * amax[..., None] * 2.0 ** -18
    b = rel * mass
    return b + (2.0 ** -11 * np.abs(out) + 2.0 ** -25 if f16 else 2.0 ** -24 * np.abs(out)) + 1e-30
