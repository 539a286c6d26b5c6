"""How far the weights of the 4-bit cache's tokens may be off, in numpy, sharing no code with the kernels."""
import numpy as np

from tests.kv4_plain import U


def pack(c):
    """Codes 0 .. 15 [.., dim] as bytes."""
    c = np.asarray(c).astype(np.uint8)
    return c[..., 0::2] | c[..., 1::2] << 4


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
