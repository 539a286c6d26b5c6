"""The bounds that attention over the 4-bit cache is held to let pass what the kernel does and catch what it must not do:
mistakes planted in the plain form, on the CPU."""
import numpy as np
import pytest

from tests import kv4_bounds as B
from tests import kv4_plain as P

# (of the groups of 32 dimensions, as often as there are groups)
FACTORS = (1.0, 2.0 ** -10, 2.0 ** 6, 2.0 ** -13)


def scene(dim, heads, lens=(200, 33), seed=0):
    rng = np.random.default_rng(seed)
    pages = -(-max(lens) // 32)
    shape = (pages * len(lens), 1, 32)
    k, v = (rng.integers(0, 256, shape + (dim // 2,)).astype(np.uint8) for _ in "kv")
    ks, vs = ((rng.uniform(0.1, 0.4, shape + (dim // 32,)) * rng.choice([-1, 1], shape + (dim // 32,))).astype(np.float16) for _ in "kv")
    for g in range(dim // 32):
        vs[..., g] *= np.float16(FACTORS[g % 4])
    x = (rng.standard_normal((len(lens), heads, dim)) * 0.3).astype(np.float32)
    table = np.arange(pages * len(lens), dtype=np.int32).reshape(len(lens), pages)
    return P.Cache(k, v, ks, vs), table, list(lens), np.arange(len(lens) + 1), x


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_second_part_that_is_missing_is_seen_in_every_group(dim):
    args = scene(dim, 4)
    ref, bound, mean = B.attend(*args, 0.16 / dim, 41)
    got = B.attend(*args, 0.16 / dim, 41, hold=B.two_parts)[0]
    assert (np.abs(got - ref) <= bound).all()
    got = B.attend(*args, 0.16 / dim, 41, hold=B.one_part)[0]
    wrong = np.abs(got - ref) > bound
    for g in range(dim // 32):
        assert wrong[..., 32 * g:32 * g + 32].mean() > 0.5, f"group {g}: a bound of {(bound / mean)[..., 32 * g].max()}"


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_reference_that_is_too_high_is_seen_in_the_small_groups(dim):
    args = scene(dim, 4)
    ref, bound, mean = B.attend(*args, 0.16 / dim, 41)
    got = B.attend(*args, 0.16 / dim, 41, hold=B.two_parts, top=2.0 ** -4)[0]  # 2^17 under where it belongs
    wrong = np.abs(got - ref) > bound
    small = [g for g in range(dim // 32) if FACTORS[g % 4] < 1]
    assert all(wrong[..., 32 * g:32 * g + 32].mean() > 0.5 for g in small)


def test_plain_form_agrees_with_the_other():
    c, table, lens, start, x = scene(128, 4, seed=3)
    ref, bound, _ = B.attend(c, table, lens, start, x, 0.05, 41)
    other, wide, _, _ = P.attention(c, table, lens, start, x, 0.05)
    assert np.allclose(ref, other, rtol=1e-12, atol=1e-18)
    # ... and is the narrower where a group is small
    assert (bound[..., 96:] < 1e-3 * wide[..., 96:]).all()
