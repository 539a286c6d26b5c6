"""Low-rank adapters beside a shared projection on the GPU, against the formula in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from quantised_decode_mat_gb300 import synth  # noqa: E402
from tests import kv_plain as P  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from quantised_decode_mat_gb300 import build as qbuild
    qbuild.build()
    q.lib()
    q.get_device_error()
    yield


def make(batch, n, rank, K, rows, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, base = r(batch, K), r(batch, rows)
    A, B = (r(n, rank, K) / K ** 0.5).to(dtype), (r(n, rows, rank) / rank ** 0.5).to(dtype)
    scale = r(n) + 2
    idx = torch.randint(0, n, (batch,), generator=g, dtype=torch.int32)
    return x, base, A, B, idx, scale


def check(t, out, idx=None):
    x, base, A, B, i, scale = t
    ref, bound = P.adapters(x.numpy(), base.numpy(), A.double().numpy(), B.double().numpy(),
                            (i if idx is None else idx).tolist(), scale.double().numpy())
    err = np.abs(out.cpu().numpy() - ref)
    assert (err <= bound).all(), f"{(err / bound).max()} times the bound"


CASES = [(1, 1, 8, 256, 1), (1, 4, 8, 4096, 4096), (2, 3, 16, 512, 77), (3, 5, 24, 768, 1001), (8, 16, 64, 4096, 6144),
         (8, 2, 128, 2304, 333), (5, 9, 40, 14336, 4097), (4, 4, 16, 65536, 50), (8, 8, 8, 256, 28672), (7, 7, 72, 1280, 2049)]


@pytest.mark.parametrize("batch,n,rank,K,rows", CASES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_adapters(batch, n, rank, K, rows, dtype):
    t = make(batch, n, rank, K, rows, dtype, seed=rank + K)
    d = [a.to(DEV) for a in t]
    out = torch.full((batch, rows), float("nan"), device=DEV)
    q.lora_add(*d[:4], d[4], d[5], out=out)
    q.get_device_error()
    check(t, out)
    check(t, q.lora_add(*d[:4], d[4], d[5], out=d[1]))  # in place


def test_vectors_without_an_adapter_and_a_bad_index():
    t = make(6, 4, 16, 1024, 500, torch.bfloat16, seed=1)
    idx = torch.tensor([-1, 2, 2, -7, 0, 2], dtype=torch.int32)
    d = [a.to(DEV) for a in t]
    out = q.lora_add(*d[:4], idx.to(DEV), d[5])
    q.get_device_error()
    check(t, out, idx)
    assert torch.equal(out[0], d[1][0]) and torch.equal(out[3], d[1][3])
    bad = idx.clone()
    bad[4] = 4
    got = q.lora_add(*d[:4], bad.to(DEV), d[5])
    with pytest.raises(q.QmdError, match="QMD_ERR_INDEX"):
        q.get_device_error()
    bad[4] = -1
    check(t, got, bad)
    assert torch.equal(got[4], d[1][4])


def test_bad_numbers_stay_with_their_vector():
    t = make(4, 3, 8, 512, 300, torch.float16, seed=2)
    t[0][2, 5] = float("nan")
    idx = torch.tensor([0, 1, 1, 2], dtype=torch.int32)
    d = [a.to(DEV) for a in t]
    out = q.lora_add(*d[:4], idx.to(DEV), d[5]).cpu()
    assert out[2].isnan().all() and out[[0, 1, 3]].isfinite().all()


def test_beside_a_quantised_projection_and_in_a_graph():
    """The shared projection, then the adapters on its output in place: eagerly and replayed with
    other adapters chosen."""
    K, rows, B = 1024, 640, 4
    t = make(B, 6, 16, K, rows, torch.float16, seed=3)
    W = torch.from_numpy(synth.q4k_weights(3, rows, K)).to(DEV)
    x, _, A, Bm, idx, scale = [a.to(DEV) for a in t]
    y = torch.empty((B, rows), device=DEV)

    def step():
        q.qmatvec_x(q.Q4_K, W, None, x, y)
        q.lora_add(x, y, A, Bm, idx, scale, out=y)

    shared = q.qmatvec_x(q.Q4_K, W, None, x)
    t = (t[0], shared.cpu(), *t[2:])
    step()
    q.get_device_error()
    check(t, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for choice in ([5, -1, 0, 0], [1, 2, 3, 4]):
        c = torch.tensor(choice, dtype=torch.int32)
        idx.copy_(c)
        x.copy_(t[0])
        g.replay()
        q.get_device_error()
        check(t, y, c)


def test_two_streams_and_large_and_small_values():
    """Two calls at once (a call holds no state), with sums far above and below f16's range."""
    jobs = []
    for i, f in enumerate((1e20, 1e-20, 1.0)):
        t = list(make(8, 5, 32, 2048, 3001, torch.float16 if i % 2 else torch.bfloat16, seed=10 + i))
        t[0] *= f
        t[1] *= f
        jobs.append((t, [a.to(DEV) for a in t], torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[q.lora_add(*d[:4], d[4], d[5], stream=st) for t, d, st in jobs] for _ in range(8)][-1]
    torch.cuda.synchronize()
    for (t, _, _), o in zip(jobs, outs):
        check(t, o)


def test_refusals_of_the_binding():
    x, base, A, B, idx, scale = [a.to(DEV) for a in make(2, 3, 8, 512, 40, torch.float16)]
    wide = torch.zeros((2, 80), device=DEV)
    for bad in ((x.double(), base, A, B, idx, scale), (x[:1], base, A, B, idx, scale), (x, base[:, :39], A, B, idx, scale),
                (x, wide[:, :40], A, B, idx, scale), (x, base, A.bfloat16(), B, idx, scale), (x, base, A.float(), B, idx, scale),
                (x, base, A, B[:2], idx, scale), (x, base, A, B.transpose(1, 2), idx, scale), (x, base, A, B, idx.long(), scale),
                (x, base, A, B, idx[:1], scale), (x, base, A, B, idx, scale[:2]), (x, base, A, B, idx, scale.cpu()),
                (x, base, A[0], B, idx, scale), (x, base.cpu(), A, B, idx, scale)):
        with pytest.raises(q.QmdError):
            q.lora_add(*bad)
    for out in (torch.empty((2, 41), device=DEV), torch.empty((2, 40), dtype=torch.float64, device=DEV), wide[:, 40:], x[:, :40]):
        with pytest.raises(q.QmdError):
            q.lora_add(x, base, A, B, idx, scale, out=out)
    q.get_device_error()
