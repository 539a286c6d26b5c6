"""How exact the weights of the 4-bit cache's tokens are, with scores and log-sum-exps up to 32."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from tests import kv4_bounds as B  # noqa: E402
from tests import kv4_plain as P  # noqa: E402
from tests.test_gpu_kv4 import Scene, dev  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]
# (query heads, key/value heads, rows): 4, 8 and 16 rows to a key/value head
LAYOUTS = [(4, 1, 1), (4, 2, 2), (8, 1, 1), (8, 2, 4)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from quantised_decode_mat_gb300 import build as qbuild
    qbuild.build()
    q.lib()
    q.get_device_error()
    yield


def aligned(s, mass, sign=1):
    """Keys that lie along a pattern of signs, codes 4 +- 1.5 of it, and queries along it: every score is a large part of its sum
    |q| |K|, of which the largest is `mass`.  Returns (queries, scale)."""
    way = s.rng.choice([-1.0, 1.0], (s.kv, s.dim))
    for i, n in enumerate(s.lens):
        pg, tok = s.c.at(s.table, i, 0, n)
        c = np.rint(s.rng.normal(4, 1.5, (n, s.kv, s.dim)) * way)
        s.c.k[pg, :, tok] = B.pack(np.clip(c, -8, 7) + 8)
        s.c.ks[pg, :, tok] = s.rng.uniform(0.1, 0.4, (n, s.kv, s.dim // 32))
    s.place()
    x = (way.repeat(s.heads // s.kv, 0) * s.rng.uniform(0.2, 1.8, (s.T, s.heads, s.dim))).astype(np.float32)
    most = 0.0
    for i, n in enumerate(s.lens):
        K = np.abs(s.c.values(s.table, i, 0, n)[0])
        for r in range(s.q_start[i], s.q_start[i + 1]):
            for h in range(s.heads):
                most = max(most, (K[:, h // (s.heads // s.kv)] @ np.abs(x[r, h].astype(np.float64))).max())
    return x, sign * mass / most


@pytest.mark.parametrize("heads,kv,rows", LAYOUTS + [(16, 1, 1), (16, 1, 5), (8, 1, 20)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sign", [1, -1])
def test_weights_to_what_is_stated(heads, kv, rows, dim, sign):
    """The bound that the interface states for a weight, and its root mean square of 2^-18 (3.8e-6) while sums |scale| |q| |K| and
    log-sum-exps are up to 32: the argument's two terms lie near 46 in log2 units, where half a step of f32 is 2^-19, a
    rounding each (0.8 * 2^-20 root mean square of a weight), one of the scale that all share (2 at most), a product of
    each group (1.5 together) and the steps of the tensor cores' sums (3 if they cut off): 4 together."""
    s = Scene([300, 60, 41], [rows] * 3, heads, kv, dim, 32, seed=dim + heads + rows)
    x, scale = aligned(s, 26.0, sign)
    lse = P.attention(s.c, s.table, s.lens, s.q_start, x, scale)[2].astype(np.float32)
    assert np.abs(lse).max() <= 32
    ref, _ = P.weigh(s.c, s.table, s.lens, s.q_start, x, scale, lse, s.w)
    bound, mass = B.weigh_bound(s.c, s.table, s.lens, s.q_start, x, scale, lse, ref)
    got = q.kv4_weigh(s.cache, s.batch, dev(x), scale, dev(lse), s.weight.clone()).cpu().numpy()
    q.get_device_error()
    at = mass > 0
    err = np.abs(got - ref)[at]
    assert (err <= bound[at]).all(), f"{(err / bound[at]).max()} times the bound"
    # over weights that begin at zero, nothing of the old ones in them
    zero = np.where(np.isnan(s.w), np.nan, 0).astype(np.float32)
    ref, _ = P.weigh(s.c, s.table, s.lens, s.q_start, x, scale, lse, zero)
    got = q.kv4_weigh(s.cache, s.batch, dev(x), scale, dev(lse), dev(zero)).cpu().numpy()
    q.get_device_error()
    at &= ref > 1e-30
    assert at.sum() > 100 and np.sqrt(((got[at] / ref[at] - 1) ** 2).mean()) <= 2.0 ** -18
