"""The 4-bit cache's calls at the ends of what they take: a pool whose offsets pass 32 bits, 2048 sequences, pages of 65536
tokens, page tables much wider than the sequences need, with no page in what they do not need."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from tests import kv4_plain as P  # noqa: E402
from tests.test_gpu_kv4 import DEV, Scene, dev, evict_case  # noqa: E402

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


def test_a_pool_past_4_gb(ws):
    """The same sequences at the end of a pool of 4.9 GB of keys: every call gives the same bits as in a small one."""
    s = Scene([500, 100, 70], [1, 3, 2], 8, 2, 256, 64, seed=5)
    few, n = s.cache.pages, 300000
    far, wfar = q.KV4Cache.empty(n, 2, 64, 256), torch.zeros((n, 2, 64), device=DEV)
    tensors = lambda c: (c.k, c.v, c.k_scale, c.v_scale)  # noqa: E731
    for a, b in zip(tensors(far) + (wfar,), tensors(s.cache) + (s.weight,)):
        a[n - few:] = b
    x = dev(s.queries())
    k, v = (torch.randn((s.T, 512), device=DEV) for _ in "kv")
    got = []
    for cache, weight, first in ((s.cache, s.weight, 0), (far, wfar, n - few)):
        batch = q.KVBatch((s.table_d + first).int(), s.len_d, s.start_d, 3, s.T)
        q.kv4_append(cache, batch, k, v)
        lse = torch.zeros((s.T, 8), device=DEV)
        out = q.kv4_attention(cache, batch, x, 0.06, ws, lse=lse)
        q.kv4_weigh(cache, batch, x, 0.06, lse, weight)
        held = weight[first:].clone()
        left = q.kv4_evict(cache, batch, weight, 60, 2, 8)
        back = q.KVBatch(batch.page_table, left, torch.arange(4, dtype=torch.int32, device=DEV) * 60, 60, 180)
        got.append([t.contiguous().view(torch.uint8) for t in (out, lse, held, left, *q.kv4_read(cache, back), weight[first:]) +
                    tuple(t[first:] for t in tensors(cache))])
    q.get_device_error()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert not far.k[:n - few].any() and not wfar[:n - few].any()


@pytest.mark.parametrize("dim,heads,kv,rows", [(64, 4, 2, 1), (128, 4, 1, 1), (256, 8, 1, 3), (128, 16, 1, 1), (64, 9, 1, 2)])
def test_2048_sequences(ws, dim, heads, kv, rows):
    s = Scene(np.random.default_rng(dim + heads).integers(0, 40, 2048).tolist(), [rows] * 2048, heads, kv, dim, 16, seed=1)
    s.check(s.queries(), ws)


def test_eviction_of_2048_sequences():
    evict_case(np.random.default_rng(3).integers(0, 60, 2048).tolist(), 20, 2, 4, 1, 64, 16, seed=2)


def test_pages_of_65536_tokens(ws):
    s = Scene([1500, 300], [1, 3], 8, 2, 64, 65536, seed=3)
    s.check(s.queries(), ws)
    evict_case([1500, 300], 200, 2, 4, 1, 64, 65536, seed=4)


@pytest.mark.parametrize("slots", [4096, 4160, 32768, 65536, 65600, 262144])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_tables_wider_than_the_sequences(ws, slots, dim):
    """Columns that no sequence needs hold -1: looked at, they would be index errors."""
    lens = [0, 1, 90, 700, 333, 1088]
    s = Scene(lens, [0, 1, 2, 1, 30, 3], 4, 2, dim, 64, seed=slots + dim)
    s.table = np.concatenate([s.table, np.full((6, slots // 64 - s.table.shape[1]), -1, np.int32)], 1)
    for i, n in enumerate(lens):
        s.table[i, -(-n // 64):] = -1
    s.place()
    s.check(s.queries(), ws)
    want, w = s.c.copy(), s.w.copy()
    wlen, wkept = P.evict(want, s.table, lens, w, 300, 4, 64)
    kept = torch.zeros((6, 2, 300), dtype=torch.int32, device=DEV)
    n = q.kv4_evict(s.cache, s.batch, s.weight, 300, 4, 64, kept=kept)
    q.get_device_error()
    assert np.array_equal(n.cpu().numpy(), wlen) and np.array_equal(kept.cpu().numpy(), wkept)
    for a, b in ((s.cache.k, want.k), (s.cache.v, want.v), (s.cache.k_scale.view(torch.int16), want.ks.view(np.int16)),
                 (s.cache.v_scale.view(torch.int16), want.vs.view(np.int16)), (s.weight.view(torch.int32), w.view(np.int32))):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("window", [1, 16, 50, 200])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows_over_many_rows(ws, window, dim):
    """More rows to a head than a warp takes (a team of them adds the weights up), some of which see nothing."""
    s = Scene([200, 45, 3, 90], [60, 45, 5, 1], 8, 2, dim, 16, seed=window + dim, extra_rows=2)
    s.check(s.queries(), ws, window=window)
