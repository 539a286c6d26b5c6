"""Plain forms of the 4-bit key/value cache's operators, for the tests: numpy, row by row, sharing no code
with the kernels.  The append is in f32 with every operation rounded on its own (its codes hang on those
roundings); attention, its log-sum-exp and its weights are in 64 bits; eviction is on whole numbers."""
import numpy as np

from tests.kv_plain import rotate

F = np.float32
GROUP = 32
U = 2.0 ** -24  # half a step of f32, relative


class Cache:
    """Host copy: codes uint8 [pages, heads, tokens, dim / 2], scales f16 [pages, heads, tokens, dim / 32]."""

    def __init__(self, k, v, ks, vs):
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        self.tokens, self.dim, self.heads = k.shape[2], 2 * k.shape[3], k.shape[1]

    def copy(self):
        return Cache(self.k.copy(), self.v.copy(), self.ks.copy(), self.vs.copy())

    def at(self, table, s, lo, hi):
        p = np.arange(lo, hi)
        return table[s][p // self.tokens], p % self.tokens

    def values(self, table, s, lo, hi):
        """K and V of slots lo .. hi - 1 of sequence s in 64 bits: [slots, heads, dim]."""
        pg, tok = self.at(table, s, lo, hi)
        return [values(c[pg, :, tok], d[pg, :, tok]) for c, d in ((self.k, self.ks), (self.v, self.vs))]


def values(codes, scales):
    c = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), np.float64)
    c[..., 0::2], c[..., 1::2] = codes & 15, codes >> 4
    return (c - 8) * np.repeat(scales.astype(np.float64), GROUP, -1)


def quantise(x):
    """Codes and scales of one row of heads x [heads, dim] f32."""
    heads, dim = x.shape
    codes, scales = np.zeros((heads, dim // 2), np.uint8), np.zeros((heads, dim // GROUP), np.float16)
    for h in range(heads):
        for g in range(dim // GROUP):
            v = x[h, GROUP * g:GROUP * (g + 1)]
            top = v[np.argmax(np.abs(v))]  # the first of the largest
            d = np.float16(np.clip(F(top) * F(-0.125), F(-65504), F(65504)))
            inv = F(1) / F(d) if d != 0 else F(0)
            c = (np.clip(np.rint(v * inv), -8, 7) + 8).astype(np.uint8)
            codes[h, GROUP // 2 * g:GROUP // 2 * (g + 1)] = c[0::2] | c[1::2] << 4
            scales[h, g] = d
    return codes, scales


def append(cache, table, lens, q_start, k, v, rope=None, q=None, rot=0, halves=True, positions=None):
    """Appends into `cache` in place; returns the rotated queries.  k, v [rows, heads, dim] f32."""
    q_out = None if q is None else np.full_like(q, np.nan)
    for s in range(len(lens)):
        r0, n = q_start[s], q_start[s + 1] - q_start[s]
        for i in range(n):
            r, slot = r0 + i, lens[s] - n + i
            at = slot if positions is None else positions[r]
            turn = (lambda x: rotate(x, rope[at], rot, halves)) if rope is not None else (lambda x: x)  # noqa: B023
            if q is not None:
                q_out[r] = turn(q[r])
            pg, tok = table[s][slot // cache.tokens], slot % cache.tokens
            cache.k[pg, :, tok], cache.ks[pg, :, tok] = quantise(turn(k[r]))
            cache.v[pg, :, tok], cache.vs[pg, :, tok] = quantise(v[r])
    return q_out


def span(lens, q_start, s, i, window):
    """The slots [begin, end) that row i of sequence s sees."""
    n = q_start[s + 1] - q_start[s]
    end = max(0, lens[s] - n + 1 + i)
    return (max(0, end - window) if window else 0), end


def score_bound(dim, mass, top):
    """How far a score may be off: q in two f16 parts is off by at most 4 u max |q| per element; products are
    exact; dim / 8 + 8 accumulation steps of the tensor cores, which may truncate (2 u each), one product with
    a scale and one sum for each group, roundings of the scaled result; the exponent's argument is
    rounded at its own size."""
    return (dim / 8 + dim / 32 * 4 + 20) * 2 * U * mass + 4 * U * (top + mass)


def attention(cache, table, lens, q_start, q, scale, window=0):
    """(out, bound, lse, lse_bound): the rows' attention and log-sum-exp in 64 bits, [rows, heads, dim] and
    [rows, heads], NaN where no sequence owns the row, and how far a result may be off.

    A relative error e of the weights moves a weighted mean by at most 2 e max |v|: the scores' error, exp2
    4 u, the product with a scale u, two f16 parts 4 u; sums over the keys at 2 u a step (chains as long as
    the keys in the worst case), merges within that, one division.  What the parts cannot hold is 2^-25 under a
    reference that the row's largest weight times scale was at least 2^11 of: 8 steps of it for each key."""
    rows, heads, dim = q.shape
    G = heads // cache.heads
    out, bound = np.full(q.shape, np.nan), np.zeros(q.shape)
    lse, lse_bound = np.full((rows, heads), np.nan), np.zeros((rows, heads))
    for s in range(len(lens)):
        n = q_start[s + 1] - q_start[s]
        if n == 0:
            continue
        K, V = cache.values(table, s, 0, lens[s])
        pg, tok = cache.at(table, s, 0, lens[s])
        D = np.abs(cache.vs[pg, :, tok].astype(np.float64)).max(-1)  # [slots, heads]
        for i in range(n):
            r = q_start[s] + i
            begin, end = span(lens, q_start, s, i, window)
            if end <= begin:
                out[r], lse[r] = 0, -np.inf
                continue
            for h in range(heads):
                x, kk, vv = q[r, h].astype(np.float64), K[begin:end, h // G], V[begin:end, h // G]
                sc = kk @ x * scale
                w = np.exp(sc - sc.max())
                out[r, h] = w @ vv / w.sum()
                lse[r, h] = sc.max() + np.log(w.sum())
                mass = (np.abs(kk) @ np.abs(x) * abs(scale)).max()
                keys = end - begin
                e = score_bound(dim, mass, np.abs(sc).max())
                rel = np.expm1(e) + 11 * U + 2 * U * (keys / 8 + 16)
                low = keys * 8 * 2.0 ** -36 * (w * D[begin:end, h // G]).max() / w.sum()
                bound[r, h] = 2 * rel * np.abs(vv).max() + 4 * U * np.abs(vv).max() + low
                lse_bound[r, h] = e + 2 * U * (keys / 8 + 16) + 8 * U + 6 * U * max(abs(lse[r, h]), abs(sc).max())
    return out, bound, lse, lse_bound


def weigh(cache, table, lens, q_start, q, scale, lse, weight, window=0):
    """(weight, bound) after the rows' weights are added, 64 bits, from the given lse (f32).
    Bound: the scores' error and the argument's rounding (|s| + |lse| at 4 u), exp2 4 u, and one rounding for
    each of the rows x heads terms and of the sum with the old weight; a term under 2^-126, the least normal f32,
    may be 0."""
    rows, heads, dim = q.shape
    G = heads // cache.heads
    new, bound = weight.astype(np.float64), np.zeros(weight.shape)
    for s in range(len(lens)):
        n = q_start[s + 1] - q_start[s]
        if n == 0:
            continue
        K = cache.values(table, s, 0, lens[s])[0]
        pg, tok = cache.at(table, s, 0, lens[s])
        own = max(0, lens[s] - n)
        new[pg[own:], :, tok[own:]] = 0
        for i in range(n):
            r = q_start[s] + i
            begin, end = span(lens, q_start, s, i, window)
            for h in range(heads):
                if end <= begin:
                    continue
                x, kk = q[r, h].astype(np.float64), K[begin:end, h // G]
                sc = kk @ x * scale
                arg = sc - np.float64(lse[r, h])
                p = np.exp(arg)
                mass = np.abs(kk) @ np.abs(x) * abs(scale)
                e = score_bound(dim, mass, np.abs(sc)) + 4 * U * (abs(np.float64(lse[r, h])) + np.abs(arg))
                at = (pg[begin:end], h // G, tok[begin:end])
                new[at] += p
                bound[at] += p * (np.expm1(e) + 4 * U) + 2.0 ** -126
    return new, bound + (rows * G + 2) * U * np.abs(np.nan_to_num(new))


def evict(cache, table, lens, weight, keep, sinks, recent):
    """In place; returns (lens, kept).  weight f32 [pages, heads, tokens]."""
    kept = np.full((len(lens), cache.heads, keep), -1, np.int32)
    for s, n in enumerate(lens):
        pg, tok = cache.at(table, s, 0, n)
        for h in range(cache.heads):
            stay = list(range(n))
            if n > keep:
                w = weight[pg, h, tok]
                key = np.where(np.isnan(w), -np.inf, w.astype(np.float64))
                # a NaN is less than everything, minus infinity included
                order = sorted(range(sinks, n - recent), key=lambda j: (np.isnan(w[j]), -key[j], j))  # noqa: B023
                stay = sorted(list(range(sinks)) + list(range(n - recent, n)) + order[:keep - sinks - recent])
                for t in (cache.k, cache.v, cache.ks, cache.vs, weight):
                    t[pg[:keep], h, tok[:keep]] = t[pg[stay], h, tok[stay]]
            kept[s, h, :len(stay)] = stay
    return np.minimum(lens, keep), kept
