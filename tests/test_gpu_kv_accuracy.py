"""How exact attention is where it is hard: value blocks whose scales and weights lie far apart, scales
that are not finite in blocks that some rows of a group do not see, long sequences.  Errors are measured
against the weighted mean of |V| (what the sum itself keeps), not against the largest value around."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from tests.test_gpu_kv import Scene, dev  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]
DEV = "cuda"
U = 2.0 ** -24
# (query heads, key/value heads, rows): 4, 8 and 16 rows to a key/value head
LAYOUTS = [(4, 2, 2), (8, 1, 1), (8, 2, 4)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from quantised_decode_mat_gb300 import build as qbuild
    qbuild.build()
    q.lib()
    q.get_device_error()
    yield


@pytest.fixture(scope="module")
def ws():
    return q.kv_workspace()


def attend(s, x, scale, window=0, chain=64):
    """(out, bound, mean) in 64 bits, [rows, heads, dim]: mean is sum w |v| / sum w.  The bound, with
    U = 2^-24 and an accumulation step of the tensor cores counted as 2 U (it may truncate):
      score     f32 queries as two f16 parts (4 U max |q| an element), dim / 8 + 20 steps on sums of at
                most `mass`, the exponent's argument rounded at its own size
      weight    e^error - 1, exp2 and its argument's rounding against the running maximum 8 U, two f16
                parts 4 U, the block scale 2 U
      sums      `chain` steps of 2 U: blocks of a warp's range, parts of a join
      floor     the second part of a weight is a multiple of 2^-24 under 2^6 times a reference of at most
                4 times the largest weight times scale: 4 * 2^-31 of that for every code that is summed
    The relative part enters numerator (of sum w |v|) and denominator."""
    out, bound, mean = (np.zeros(x.shape) for _ in range(3))
    G = s.heads // s.kv
    for i, l in enumerate(s.lens):
        with np.errstate(invalid="ignore"):
            K, V = s.c.values(s.table, i, 0, l)
        n = s.n[i]
        tok = np.arange(l)
        vs = np.abs(s.c.vs[s.table[i][tok // s.page], :, tok % s.page // 16].astype(np.float64))
        codes = np.abs(s.c.v[s.table[i][tok // s.page], :, tok % s.page].astype(np.float64))
        for j in range(n):
            r, end = s.q_start[i] + j, l - n + 1 + j
            a = max(0, end - window) if window else 0
            for h in range(s.heads):
                g, xq = h // G, x[r, h].astype(np.float64)
                kk, vv = K[a:end, g], V[a:end, g]
                sc = kk @ xq * scale
                w = np.exp(sc - sc.max())
                out[r, h], mean[r, h] = w @ vv / w.sum(), w @ np.abs(vv) / w.sum()
                seen = w > 1e-30
                mass = (np.abs(kk[seen]) @ np.abs(xq)).max() * abs(scale)
                part = (np.abs(kk[seen]).sum(1) * np.abs(xq).max()).max() * abs(scale)
                score = (s.dim / 8 + 20) * 2 * U * mass + 4 * U * part + 4 * U * np.abs(sc[seen]).max()
                rel = np.expm1(score) + 14 * U + 2 * U * chain
                floor = 4 * 2.0 ** -31 * (w * vs[a:end, g]).max() * codes[a:end, g].sum(0) / w.sum()
                bound[r, h] = 2 * rel * mean[r, h] + 4 * U * mean[r, h] + floor
    return out, bound, mean


def close(s, x, ws, scale, window=0, chain=64, copies=1):
    """The scene's sequences `copies` times over (on the same pages): with thousands of items a warp's range
    holds several blocks of one, cut at ever other places."""
    ref, bound, mean = attend(s, x, scale, window, chain)
    n = len(s.lens)
    start = np.concatenate([s.q_start[:-1] + i * s.T for i in range(copies)] + [[copies * s.T]])
    batch = q.KVBatch(s.table_d.repeat(copies, 1), s.len_d.repeat(copies), dev(start.astype(np.int32)), max(s.n), copies * s.T)
    assert batch.kv_len.shape[0] == copies * n
    got = q.kv_attention(s.cache, batch, dev(x).repeat(copies, 1, 1), scale, ws, window=window)
    q.get_device_error()
    got = got.view(copies, *x.shape).double().cpu().numpy()
    err = np.abs(got - ref)
    assert (err <= bound).all(), f"{np.nanmax(err / bound)} times the bound"
    return err, mean


@pytest.mark.parametrize("heads,kv,rows", LAYOUTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ratio", [2.0 ** 12, 2.0 ** 18, 2.0 ** 24, 2.0 ** 40, 2.0 ** 100, 2.0 ** 150])
@pytest.mark.parametrize("first", [True, False])
def test_a_large_scale_without_weight_beside_the_block_that_has_it(ws, heads, kv, rows, dim, ratio, first):
    """One block holds all the weight, the others' scores lie far below (weight times scale under 2^-10 of
    the block's) under a value scale `ratio` times as large, and come first or last."""
    s = Scene([96, 96], [rows] * 2, heads, kv, dim, 32, seed=int(np.log2(ratio)) + dim)
    sign = s.rng.choice([-1.0, 1.0], (kv, dim))
    far = np.log(ratio) + 14.0  # how far the scores lie apart
    for i in range(2):
        for b in range(6):
            pg, t0 = s.table[i, b // 2], b % 2 * 16
            heavy = b == (4 if first else 1)
            s.c.k[pg, :, t0:t0 + 16] = np.rint((60 if heavy else -60) * sign)[:, None] + s.rng.integers(-2, 3, (kv, 16, dim))
            s.c.ks[pg, :, t0 // 16] = 1 / 64
            s.c.vs[pg, :, t0 // 16] = s.rng.uniform(0.01, 0.02, kv) * (1 if heavy else ratio) / ratio ** 0.6
    s.place()
    x = (sign.repeat(heads // kv, 0) * s.rng.uniform(0.9, 1.1, (s.T, heads, dim))).astype(np.float32)
    close(s, x, ws, far / (2 * 60 / 64 * dim), copies=1000)


@pytest.mark.parametrize("heads,kv,rows", LAYOUTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scales_that_rise_and_fall(ws, heads, kv, rows, dim):
    """Scales wander over 2^60 while scores wander the other way, so that every block's part of the sum
    counts for some while."""
    s = Scene([700, 333], [rows] * 2, heads, kv, dim, 32, seed=dim)
    sign = s.rng.choice([-1.0, 1.0], (kv, dim))
    for i, l in enumerate(s.lens):
        level = np.cumsum(s.rng.uniform(-1, 1, -(-l // 16)))
        level = level / np.abs(level).max()  # -1 .. 1
        for b, z in enumerate(level):
            pg, t0, m = s.table[i, b * 16 // 32], b % 2 * 16, min(16, l - b * 16)
            s.c.k[pg, :, t0:t0 + m] = np.rint(-100 * z * sign)[:, None] + s.rng.integers(-2, 3, (kv, m, dim))
            s.c.ks[pg, :, t0 // 16] = 1 / 64
            s.c.vs[pg, :, t0 // 16] = 0.01 * 2.0 ** (30 * z)
    s.place()
    x = (sign.repeat(heads // kv, 0) * s.rng.uniform(0.9, 1.1, (s.T, heads, dim))).astype(np.float32)
    close(s, x, ws, 30 * np.log(2) / (100 / 64 * dim), copies=300)


@pytest.mark.parametrize("heads", [2, 4, 8])  # of 2 key/value heads and 4 rows: 4, 8 and 16 rows to one
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_scales_that_are_not_finite_stay_with_the_rows_that_see_them(ws, heads, dim, bad, which):
    # sequence 0: the last row alone sees block 4; sequence 1, window 20: rows see 14 + i .. 33 + i, so
    # the first two alone see block 0
    s = Scene([65, 37], [4, 4], heads, 2, dim, 16, seed=dim + heads)
    x = s.queries()
    ref, bound, _ = attend(s, x, 0.1, 20)
    getattr(s.c, which)[s.table[0, 4]] = bad
    getattr(s.c, which)[s.table[1, 0]] = bad
    s.place()
    got = q.kv_attention(s.cache, s.batch, dev(x), 0.1, ws, window=20).view(x.shape).cpu().numpy()
    q.get_device_error()
    clear = [0, 1, 2, 6, 7]
    assert (np.abs(got - ref) <= bound)[clear].all()


@pytest.mark.parametrize("heads,kv,rows,dim", [(4, 1, 1, 64), (8, 1, 1, 64), (8, 2, 4, 64), (32, 8, 1, 128), (16, 2, 1, 128),
                                               (16, 2, 2, 128), (4, 2, 2, 256), (8, 1, 1, 256), (4, 2, 4, 256)])
def test_long_sequences_to_f32(ws, heads, kv, rows, dim):
    """20011 tokens.  No chain of sums is longer than a warp's range and its joins: at most 13 blocks (with
    132 SMs or more of 6 warps or more), 16 parts in a CTA and 152 in all, which round once (U), so the
    bound counts 100 steps of 2 U.  The root mean square is what the header says, with sums |q| |K| of 15
    to 28."""
    s = Scene([20011], [rows], heads, kv, dim, 64, seed=dim + heads, uniform=True)
    err, mean = close(s, s.queries(), ws, dim ** -0.5, chain=100)
    assert np.sqrt(((err / mean) ** 2).mean()) <= 2.0 ** -20
