"""Adapters whose sums lie far from 1: finite results through large and small A x and scales, ranks far
apart; one-hot A and x, so that A x is exact and what B does with it shows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]
DEV = "cuda"
U = 2.0 ** -24
HALVES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from quantised_decode_mat_gb300 import build as qbuild
    qbuild.build()
    q.lib()
    q.get_device_error()
    yield


def run(t, B, base, s, dtype, K=512):
    """t f64 [batch, rank] as A x exactly (A picks values of x), B [rows, rank], base [batch, rows]:
    the result, its 64-bit value and a bound."""
    batch, rank = t.shape
    A = torch.zeros((1, rank, K))
    A[0, torch.arange(rank), torch.arange(rank) * (K // rank)] = 1
    x = torch.zeros((batch, K))
    x[:, torch.arange(rank) * (K // rank)] = torch.from_numpy(t).float()
    t = x[:, torch.arange(rank) * (K // rank)].double().numpy()
    Bh, base = torch.from_numpy(B).to(dtype), torch.from_numpy(base).float()
    Bv, basev = Bh.double().numpy(), base.double().numpy()
    got = q.lora_add(x.to(DEV), base.to(DEV), A.to(dtype).to(DEV), Bh[None].contiguous().to(DEV),
                     torch.zeros(batch, dtype=torch.int32, device=DEV), torch.tensor([s], device=DEV))
    q.get_device_error()
    add = np.float32(s).astype(np.float64) * (t @ Bv.T)
    most = abs(s) * (np.abs(t) @ np.abs(Bv).T)
    # t's parts: 2 U each value (two f16 parts: 4 U, and multiples of 2^-36 of twice the largest; the tensor
    # cores align products to the largest, a zero of B counting as 2^-14 of its value of t: 2^-38 a rank);
    # rank + 8 steps of sums at 2 U (they may truncate); scale and base: 4 roundings of the result
    floor = abs(s) * np.abs(t).max(1, keepdims=True) * (2.0 ** -35 * np.abs(Bv).sum(1) + rank * 2.0 ** -38)
    if dtype is torch.bfloat16:
        floor = abs(s) * np.abs(t).max(1, keepdims=True) * rank * 2.0 ** -126 * np.ones(len(Bv))
    return got.double().cpu().numpy(), basev + add, (rank + 12) * 2 * U * most + 4 * U * np.abs(basev + add) + floor + 1e-44


def check(*a, **k):
    got, ref, bound = run(*a, **k)
    err = np.abs(got - ref)
    assert np.isfinite(ref.astype(np.float32)).all()
    assert (err <= bound).all(), f"{np.nanmax(err / bound)} times the bound, {np.isnan(got).sum()} NaN"
    return got


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("rank", [8, 24, 64, 128])
@pytest.mark.parametrize("ex,s,small", [(120, 1000.0, 2.0 ** -10), (126, 30000.0, 2.0 ** -14), (110, 2.0 ** 30, 2.0 ** -14),
                                        (-100, 2.0 ** 90, 1.0), (-120, 2.0 ** 120, 1.0), (100, 2.0 ** -90, 1.0), (0, 1.0, 1.0)])
def test_large_and_small_sums_with_finite_results(dtype, rank, ex, s, small):
    rng = np.random.default_rng(rank + ex + 200)
    t = rng.uniform(0.5, 1, (3, rank)) * rng.choice([-1, 1], (3, rank)) * 2.0 ** ex / rank
    B = rng.uniform(0.5, 1, (70, rank)) * rng.choice([-1, 1], (70, rank)) * small
    B[::7] = 0
    got = check(t, B, np.zeros((3, 70)), s, dtype)
    assert not got[:, ::7].any()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("rank", [8, 40, 128])
@pytest.mark.parametrize("ratio", [10, 20, 24])
def test_ranks_far_apart(dtype, rank, ratio):
    """The largest value of A x meets zeros of B: the others, 2^ratio smaller, are what counts."""
    # (f16 has two parts, so its floor shows from 2^12 on; bf16's exponents reach as far as f32's)
    rng = np.random.default_rng(rank)
    t = rng.standard_normal((2, rank)) * 2.0 ** -ratio
    B = rng.standard_normal((300, rank))
    big = rank // 2
    t[:, big], B[:, big] = 1.0, 0.0
    check(t, B, np.zeros((2, 300)), 1.5, dtype)


@pytest.mark.parametrize("dtype", HALVES)
def test_each_rank_and_row_alone(dtype):
    """One-hot B: row r holds a 1 at rank r % rank, so an output is one value of A x and the base."""
    rng = np.random.default_rng(1)
    for rank in (8, 64, 120):
        rows = 4099
        B = np.zeros((rows, rank))
        B[np.arange(rows), np.arange(rows) % rank] = 1
        check(rng.standard_normal((5, rank)), B, rng.standard_normal((5, rows)), -2.0, dtype, K=1024)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("batch,rank,K,rows", [(1, 8, 65536, 300), (8, 24, 14336, 1001), (5, 128, 2304, 4100), (8, 64, 256, 29)])
def test_whole_numbers_are_exact(dtype, batch, rank, K, rows):
    """x, A, B and base of small whole numbers: A x is below 2^17 and the outputs below 2^24, so every product,
    part and sum is a whole number that f32 holds, in whatever order; a lost or doubled term is off by 1."""
    g = torch.Generator().manual_seed(K + rank)
    whole = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g)  # noqa: E731
    x, A = whole(-1, 2, batch, K), whole(-1, 2, 3, rank, K)
    B, base = torch.zeros((3, rows, rank), dtype=torch.int64), whole(-99, 100, batch, rows)
    for a in range(3):  # up to 8 ranks to a row
        B[a].scatter_(1, whole(0, rank, rows, 8), whole(-8, 9, rows, 8))
    idx = whole(0, 3, batch).int()
    want = torch.stack([base[v] + 2 * (B[i] @ (A[i] @ x[v])) for v, i in enumerate(idx.tolist())])
    assert want.abs().max() < 1 << 24
    d = lambda t, ty: t.to(ty).to(DEV)  # noqa: E731
    got = q.lora_add(d(x, torch.float32), d(base, torch.float32), d(A, dtype), d(B, dtype), idx.to(DEV),
                     torch.full((3,), 2.0, device=DEV))
    q.get_device_error()
    assert torch.equal(got.cpu().long(), want)
