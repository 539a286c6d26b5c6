"""Appending to blocks whose scale and codes the caller wrote: of either sign, far smaller and far larger
than what the append itself makes; bit for bit against a plain form of the header's steps."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from tests.test_gpu_kv import bits, dev  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]
F = np.float32
HEADS, DIM = 2, 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from quantised_decode_mat_gb300 import build as qbuild
    qbuild.build()
    q.lib()
    q.get_device_error()
    yield


def codes(x, inv):
    return np.clip(np.rint(x * inv), -127, 127).astype(np.int8)


def block_after(old, d0, new):
    """One head's block: earlier codes [t, dim], its scale, new rows [m, dim] -> (codes, scale)."""
    with np.errstate(over="ignore"):
        top = np.abs(new).max()
        d = max(abs(F(d0)), F(0) if top < F(1e-30) else top / F(127))
        inv = min(F(1) / d, np.finfo(F).max) if d > 0 else F(0)
        if d != F(d0):
            old = codes(old.astype(F) * F(d0), inv)
        return np.concatenate((old, codes(new, inv))), d


def blocks(earlier, scales, rows, seed=0):
    """A sequence to a scale, `earlier` tokens each in a block with it, and the given new rows [m, dim]
    appended: every (codes, scale) against the plain form."""
    rng = np.random.default_rng(seed)
    n, m = len(scales), len(rows)
    k = rng.integers(-128, 128, (n, HEADS, 16, DIM)).astype(np.int8)
    ks = np.repeat(np.array(scales, F)[:, None, None], HEADS, 1)
    new = np.broadcast_to(rows.astype(F)[None, :, None], (n, m, HEADS, DIM)) * np.array([1, -1], F)[:, None]
    cache = q.KVCache(dev(k), dev(k), dev(ks), dev(ks))
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1)
    batch = q.KVBatch(table, torch.full((n,), earlier + m, dtype=torch.int32, device="cuda"), max_q=m)
    x = dev(new.reshape(n * m, HEADS, DIM))
    q.kv_append(cache, batch, x, x)
    q.get_device_error()
    for i in range(n):
        for h in range(HEADS):
            want, d = block_after(k[i, h, :earlier], ks[i, h, 0], new[i, :, h])
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
                got = c[i, h].cpu().numpy()
                assert np.array_equal(got[:earlier + m], want), (scales[i], h)
                assert np.array_equal(got[earlier + m:], k[i, h, earlier + m:])
                assert bits(s[i, h].cpu().numpy()) == bits(np.array([d], F)), (scales[i], h)
    return k, cache


def rows_of(m, top, seed=1):
    x = np.random.default_rng(seed).uniform(-1, 1, (m, DIM)).astype(F)
    x[0, 3] = 1
    return x * F(top)


@pytest.mark.parametrize("earlier,m", [(1, 1), (9, 3), (15, 1)])
@pytest.mark.parametrize("top", [1.27, 0.0, 1e-36, 1e-30, 200.0])
def test_scales_of_either_sign(earlier, m, top):
    # 0.01 is what the rows of 1.27 ask for: below, at and above it, and none
    blocks(earlier, [-0.5, -0.02, -0.0101, -0.01, -0.0099, -1e-4, 0.5, 0.02, 0.01, 0.0099, 1e-4, -3.0, 0.0, -0.0], rows_of(m, top))


def test_earlier_values_under_a_negative_scale_are_kept():
    k, cache = blocks(8, [-0.5, -0.02], rows_of(1, 1.27))
    got = cache.k.cpu().numpy()[:, :, :8].astype(F) * cache.k_scale.cpu().numpy()[..., None]
    was = np.clip(-k[:, :, :8].astype(F), -127, 127) * np.array([0.5, 0.02], F)[:, None, None, None]
    assert np.array_equal(got, was)


@pytest.mark.parametrize("top", [9e-31, 1e-33, 1e-38, 0.0, 1.0])
def test_scales_far_below_what_an_append_makes(top):
    blocks(5, [1e-35, 7e-33, 1e-37, 2e-39, 1e-42, 1e-45, -1e-35, -1e-39], rows_of(2, top))


@pytest.mark.parametrize("top", [1.0, 1e36, 3e38])
def test_huge_scales(top):
    blocks(7, [1e30, -1e30, 1e36, -1e36, 3e36], rows_of(2, top))
