"""Plain forms of the key/value cache operators and the adapters, for the tests: numpy, row by row,
sharing no code with the kernels.  The append is in f32 with every operation rounded on its own
(its codes hang on those roundings); attention and adapters are in 64 bits."""
import numpy as np

F = np.float32
BLOCK = 16


class Cache:
    """Host copy of a cache: codes int8 [pages, heads, tokens, dim], scales f32 [pages, heads, tokens / 16]."""

    def __init__(self, k, v, ks, vs):
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        self.tokens, self.dim, self.heads = k.shape[2], k.shape[3], k.shape[1]

    def copy(self):
        return Cache(self.k.copy(), self.v.copy(), self.ks.copy(), self.vs.copy())

    def values(self, table, s, lo, hi):
        """K and V of positions lo .. hi - 1 of sequence s in 64 bits: [positions, heads, dim]."""
        p = np.arange(lo, hi)
        pg, tok = table[s][p // self.tokens], p % self.tokens
        return [c[pg, :, tok].astype(np.float64) * d[pg, :, tok // BLOCK].astype(np.float64)[..., None]
                for c, d in ((self.k, self.ks), (self.v, self.vs))]


def rotate(x, row, rot, halves):
    """One row's heads [heads, dim] f32 rotated by a table row (rot / 2 cosines, rot / 2 sines)."""
    y = x.copy()
    h = rot // 2
    c, s = row[:h].astype(F), row[h:rot].astype(F)
    a, b = (x[:, :h], x[:, h:rot]) if halves else (x[:, 0:rot:2], x[:, 1:rot:2])
    na, nb = a * c - b * s, b * c + a * s
    if halves:
        y[:, :h], y[:, h:rot] = na, nb
    else:
        y[:, 0:rot:2], y[:, 1:rot:2] = na, nb
    return y


def codes(x, d):
    if d == 0:
        return np.zeros(x.shape, np.int8)
    return np.clip(np.rint(x * (F(1) / d)), -127, 127).astype(np.int8)


def append(cache, table, lens, q_start, k, v, rope=None, q=None, rot=0, halves=True):
    """Appends into `cache` in place; returns the rotated queries.  k, v [rows, heads, dim] f32."""
    q_out = None if q is None else np.full_like(q, np.nan)
    for s in range(len(lens)):
        r0, n = q_start[s], q_start[s + 1] - q_start[s]
        start = lens[s] - n
        kr = [rotate(k[r0 + i], rope[start + i], rot, halves) if rope is not None else k[r0 + i] for i in range(n)]
        for i in range(n):
            if q is not None:
                q_out[r0 + i] = rotate(q[r0 + i], rope[start + i], rot, halves) if rope is not None else q[r0 + i]
        for which, (cc, dd) in enumerate(((cache.k, cache.ks), (cache.v, cache.vs))):
            rows = kr if which == 0 else [v[r0 + i] for i in range(n)]
            i = 0
            while i < n:
                pos = start + i
                m = min(n - i, BLOCK - pos % BLOCK)
                pg, t0 = table[s][pos // cache.tokens], pos % cache.tokens
                b, first = t0 // BLOCK, t0 // BLOCK * BLOCK
                for h in range(cache.heads):
                    top = max(np.abs(rows[i + j][h]).max() for j in range(m))
                    d0 = dd[pg, h, b] if t0 > first else F(0)
                    d = max(d0, F(0) if top < F(1e-30) else F(top) / F(127))
                    if d > d0:
                        for t in range(first, t0):
                            cc[pg, h, t] = codes(cc[pg, h, t].astype(F) * d0, d)
                    for j in range(m):
                        cc[pg, h, t0 + j] = codes(rows[i + j][h], d)
                    dd[pg, h, b] = d
                i += m
    return q_out


def attention(cache, table, lens, q_start, q, scale, window=0, out=None):
    """(out, bound): the rows' attention in 64 bits, [rows, heads, dim], NaN where no sequence owns the
    row, and how far a result may be off per element (see `bound_of`)."""
    rows, heads, dim = q.shape
    G = heads // cache.heads
    out = np.full(q.shape, np.nan)
    bound = np.zeros(q.shape)
    for s in range(len(lens)):
        n = q_start[s + 1] - q_start[s]
        if n == 0:
            continue
        K, V = cache.values(table, s, 0, lens[s])
        for i in range(n):
            r, end = q_start[s] + i, lens[s] - n + 1 + i
            begin = max(0, end - window) if window else 0
            if end <= begin:
                out[r] = 0
                continue
            for h in range(heads):
                x, kk, vv = q[r, h].astype(np.float64), K[begin:end, h // G], V[begin:end, h // G]
                sc = kk @ x * scale
                w = np.exp(sc - sc.max())
                out[r, h] = w @ vv / w.sum()
                mass = np.abs(kk) @ np.abs(x) * abs(scale)
                bound[r, h] = bound_of(dim, end - begin, mass.max(), np.abs(sc).max(), np.abs(vv).max())
    return out, bound


def bound_of(dim, keys, mass, top, vmax):
    """A rigorous bound on the error of one output.  u = 2^-24 is half a step of f32; an accumulation
    step of the tensor cores may truncate, so it counts 2 u.
      score:   q in two f16 parts is off by at most 4 u max |q| per element, products are exact,
               dim / 8 + 8 accumulation steps (2 u each, on sums of at most `mass`), and four
               roundings of the scaled result: (dim / 8 + 8 + 4 + 8) 2 u mass, and the exponent's
               argument s log2(e) - m is rounded at its own size: 4 u (top + mass)
      weight:  e^(error) - 1, exp2 itself 4 u, two f16 parts 4 u, products with the block scale 2 u
      sums:    over the keys at 2 u a step for numerator and denominator (chains as long as the
               keys in the worst case), their merges within that; one division
    A relative error e of the weights moves a weighted mean by at most 2 e max |v|."""
    u = 2.0 ** -24
    score = (dim / 8 + 20) * 2 * u * mass + 4 * u * (top + mass)
    rel = np.expm1(score) + 10 * u + 2 * u * (keys / 8 + 16)
    return 2 * rel * vmax + 4 * u * vmax


def adapters(x, base, A, B, idx, scale):
    """(out, bound) of the adapters in 64 bits; A, B as float64 arrays of the exact f16 / bf16 values.
    Bound: every f32 product and sum rounds once (u = 2^-24): at most K + rank + 4 of them touch a term."""
    out = base.astype(np.float64).copy()
    bound = np.abs(out) * 2.0 ** -23
    for v, a in enumerate(idx):
        if a >= 0:
            t = A[a] @ x[v].astype(np.float64)
            out[v] += scale[a] * (B[a] @ t)
            most = np.abs(scale[a]) * (np.abs(B[a]) @ (np.abs(A[a]) @ np.abs(x[v].astype(np.float64))))
            bound[v] = (np.abs(base[v]) + np.abs(out[v])) * 2.0 ** -23 + (A.shape[2] + A.shape[1] + 4) * 2.0 ** -24 * most
    return out, bound
