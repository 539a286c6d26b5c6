"""How far attention over the 4-bit cache, and the weights of its tokens, may be off where values of different sizes meet: bounds
that are relative to what each dimension's own group holds, in numpy, sharing no code with the kernels."""
import numpy as np

from tests.kv4_plain import GROUP, U, score_bound, span, values


def pack(c):
    """Codes 0 .. 15 [.., dim] as bytes."""
    c = np.asarray(c).astype(np.uint8)
    return c[..., 0::2] | c[..., 1::2] << 4


def two_parts(x):
    """x as a kernel of two f16 parts holds it: the first 11 bits, and the rest, each a multiple of 2^-24."""
    m, e = np.frexp(x)
    hi = np.ldexp(np.trunc(m * 2.0 ** 11) / 2.0 ** 11, e)
    return hi.astype(np.float16).astype(np.float64) + (x - hi).astype(np.float16).astype(np.float64)


def one_part(x):
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(m * 2.0 ** 11) / 2.0 ** 11, e)


def attend(c, table, lens, q_start, x, scale, chain, window=0, hold=None, top=2.0 ** 13):
    """(out, bound, mean) in 64 bits, [rows, heads, dim]: mean is sum w |v| / sum w.  hold: what a weight times scale
    becomes, when the largest that the row meets is `top` (nothing, by default).  The bound:
      weights   score_bound for the scores, exp2 and its argument 8 u, two f16 parts 4 u, the product with a scale u
      sums      `chain` steps of 2 u; numerator (of sum w |v|) and denominator
      floor     each of a product's two parts is a multiple of 2^-24, off by half of it, so a product by 2^-24, under a
                reference that leaves the largest product over 2^12 (2^-36 of it) and the largest weight under
                2^(44 + 1) at the least (2^-67 of it: 2^-24 over 2^43), for every code of the dimension"""
    rows, heads, dim = x.shape
    G = heads // c.heads
    out, bound, mean = (np.zeros(x.shape) for _ in range(3))
    for s in range(len(lens)):
        if q_start[s + 1] == q_start[s]:
            continue
        K, V = c.values(table, s, 0, lens[s])
        pg, tok = c.at(table, s, 0, lens[s])
        D = np.repeat(c.vs[pg, :, tok].astype(np.float64), GROUP, -1)
        C = values(c.v[pg, :, tok], np.ones(c.vs[pg, :, tok].shape))
        for i in range(q_start[s + 1] - q_start[s]):
            r = q_start[s] + i
            a, b = span(lens, q_start, s, i, window)
            for h in range(heads):
                g, xq = h // G, x[r, h].astype(np.float64)
                kk, vv, dd, cc = K[a:b, g], V[a:b, g], D[a:b, g], C[a:b, g]
                sc = kk @ xq * scale
                w = np.exp(sc - sc.max())
                p, largest = w[:, None] * dd, (w[:, None] * np.abs(dd)).max()
                if hold is not None:
                    p = hold(p * (top / largest)) * (largest / top)
                out[r, h] = (p * cc).sum(0) / w.sum()
                mean[r, h] = w @ np.abs(vv) / w.sum()
                seen = w > 1e-30
                mass = (np.abs(kk[seen]) @ np.abs(xq)).max() * abs(scale)
                rel = np.expm1(score_bound(dim, mass, np.abs(sc[seen]).max())) + 13 * U + 2 * U * chain
                floor = (2.0 ** -36 * largest + 2.0 ** -67 * w.max()) * np.abs(cc).sum(0) / w.sum()
                bound[r, h] = 2 * rel * mean[r, h] + 4 * U * mean[r, h] + floor
    return out, bound, mean


def weigh_bound(c, table, lens, q_start, x, scale, lse, new):
    """The bound on weights `new` (64 bits) that the interface states: 2^-24 ((dim / 2 + 52) M + 8 |lse| + 8 + T) of itself, M
    the largest |scale| sum |q| |K| of the slot (without the 2^-15 for queries of uneven sizes), T the rows times heads;
    2^-126 a term.  It is score_bound's: dim / 8 steps
    and dim / 8 products and sums of groups and 20 more at 2 u, then 4 u (|s| + M), and 4 u (|lse| + |s - lse|) for the
    argument, with |s| at most M; exp2 4 u, and a rounding for each term."""
    rows, heads, dim = x.shape
    G = heads // c.heads
    bound, mass = np.zeros(new.shape), np.zeros(new.shape)
    for s in range(len(lens)):
        n = q_start[s + 1] - q_start[s]
        if n == 0:
            continue
        K = c.values(table, s, 0, lens[s])[0]
        pg, tok = c.at(table, s, 0, lens[s])
        own = x[q_start[s]:q_start[s + 1]].astype(np.float64)
        far = np.abs(lse[q_start[s]:q_start[s + 1]])
        for g in range(c.heads):
            M = np.abs(scale) * np.einsum("jd,rhd->jrh", np.abs(K[:, g]), np.abs(own[:, g * G:(g + 1) * G])).max((1, 2))
            mass[pg, g, tok] = M
            of_row = np.where(np.isfinite(far[:, g * G:(g + 1) * G]), far[:, g * G:(g + 1) * G], 0).max()
            bound[pg, g, tok] = U * ((dim / 2 + 52) * M + 8 * of_row + 8 + n * G) * np.abs(new[pg, g, tok]) + n * G * 2.0 ** -126
    return bound, mass
