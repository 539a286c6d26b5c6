"""How exact attention over the 4-bit cache is where it is hard: groups of a head, and tokens, whose value scales lie far
apart, each held to a bound of its own; scores up to 32; long sequences."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from tests import kv4_bounds as B  # noqa: E402
from tests.test_gpu_kv4 import Scene, dev  # noqa: E402
from tests.test_gpu_kv4_weight_accuracy import LAYOUTS, aligned  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]


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


def close(s, x, ws, scale, chain, window=0):
    ref, bound, mean = B.attend(s.c, s.table, s.lens, s.q_start, x, scale, chain, window)
    got = q.kv4_attention(s.cache, s.batch, dev(x), scale, ws, window=window)
    q.get_device_error()
    err = np.abs(got.reshape(x.shape).double().cpu().numpy() - ref)
    assert (err <= bound).all(), f"{np.nanmax(err / bound)} times the bound"
    return err, mean


def chain_of(lens):
    """A warp's range has at most as many units of 32 slots as the sequence (two steps of 16 each), and 16 parts are joined in
    a CTA, some more between CTAs."""
    return max(lens) // 16 + 40


@pytest.mark.parametrize("heads,kv,rows", LAYOUTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_small_groups_keep_their_bits(ws, heads, kv, rows, dim):
    """Groups of 32 dimensions 2^10 to 2^19 apart: each is exact to its own size."""
    s = Scene([200, 33, 90], [rows] * 3, heads, kv, dim, 32, seed=dim + heads)
    for g, f in zip(range(dim // 32), 2 * (1.0, 2.0 ** -10, 2.0 ** 6, 2.0 ** -13)):
        s.c.vs[..., g] = np.where(np.isnan(s.c.vs[..., g]), np.nan, s.c.vs[..., g] * np.float16(f))
    s.place()
    close(s, s.queries(0.3), ws, 0.16 / dim, chain_of(s.lens))


@pytest.mark.parametrize("heads,kv,rows", LAYOUTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("depth", [20, 40, 60])
def test_a_token_without_value_that_has_all_the_weight(ws, heads, kv, rows, dim, depth):
    """16 tokens whose value scales are zero, their scores 2^depth above all others': what the others add is still exact
    to its own size, as far down as 2^-67 of the largest weight (which the bound counts)."""
    s = Scene([400, 70], [rows] * 2, heads, kv, dim, 32, seed=depth + dim)
    way = s.rng.choice([-1.0, 1.0], (kv, dim))
    for i, n in enumerate(s.lens):
        pg, tok = s.c.at(s.table, i, 0, n)
        heavy = (np.arange(n) // 16 == 1)[:, None, None]
        c = np.rint(way * np.where(heavy, 6, -6)) + s.rng.integers(-1, 2, (n, kv, dim))
        s.c.k[pg, :, tok] = B.pack(c + 8)
        s.c.ks[pg, :, tok] = 0.125
        s.c.vs[pg, :, tok] = np.where(heavy, 0, s.c.vs[pg, :, tok])
    s.place()
    x = (way.repeat(heads // kv, 0) * s.rng.uniform(0.9, 1.1, (s.T, heads, dim))).astype(np.float32)
    scale = depth * np.log(2) / (2 * 6 * 0.125 * dim)
    err, mean = close(s, x, ws, scale, chain_of(s.lens))
    assert mean.max() < 2.0 ** -(depth - 12)


@pytest.mark.parametrize("heads,kv,rows", LAYOUTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_up_to_32(ws, heads, kv, rows, dim, sign):
    """Attention's root mean square of 2^-20 of the weighted mean of |V|, which is stated for sums |scale| |q| |K| up to
    32, over sequences of a few tokens to 300, where no mean over many scores hides their errors."""
    lens = [4, 5, 9, 17, 33, 70, 140, 300]
    s = Scene(lens, [rows] * 8, heads, kv, dim, 32, seed=dim + heads + rows)
    x, scale = aligned(s, 31.0, sign)
    err, mean = close(s, x, ws, scale, chain_of(lens))
    at = mean > 0  # (a row that sees one token, whose value is 0)
    assert np.sqrt(((err[at] / mean[at]) ** 2).mean()) <= 2.0 ** -20


@pytest.mark.parametrize("heads,kv,rows,dim", [(4, 1, 1, 64), (8, 1, 1, 64), (8, 2, 4, 64), (32, 8, 1, 128), (16, 2, 1, 128),
                                               (16, 2, 2, 128), (4, 2, 2, 256), (8, 1, 1, 256), (4, 2, 4, 256)])
def test_long_sequences_to_f32(ws, heads, kv, rows, dim):
    """20011 tokens, 626 units of 32.  A warp's range is at most 626 * 8 * 2 / (132 * 6) = 13 units (two steps of 16 tokens each),
    then 16 parts in a CTA and up to 152 in all, which round once (U): 26 + 8 + 66 steps of 2 U.  The root mean square is
    what is stated for attention, with sums |scale| |q| |K| of up to 32."""
    s = Scene([20011], [rows], heads, kv, dim, 64, seed=dim + heads, uniform=True)
    err, mean = close(s, s.queries(), ws, dim ** -0.5, chain=100)
    assert np.sqrt(((err / mean) ** 2).mean()) <= 2.0 ** -20
