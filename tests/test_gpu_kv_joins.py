"""Attention's ranges and joins: every instance on sequences that are cut between warps and between CTAs,
with values laid out so that a block that is lost, doubled or put into another row shows at full size;
many sequences, some without rows; what a call leaves in the workspace."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from tests import kv_plain as P  # noqa: E402
from tests.test_gpu_kv import Scene, dev  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]
DEV = "cuda"
# (query heads, key/value heads, rows): 4, 8, 16 and more rows to a key/value head
LAYOUTS = [(4, 1, 1), (8, 2, 1), (8, 1, 1), (6, 2, 2), (16, 1, 1), (8, 2, 4), (8, 1, 5)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from quantised_decode_mat_gb300 import build as qbuild
    qbuild.build()
    q.lib()
    q.get_device_error()
    yield


def counters(ws):
    return ws[:torch.cuda.get_device_properties(0).multi_processor_count]


def comb(lens, n, heads, kv, dim, page, seed):
    """A scene whose values are 1 in dimension b % dim for positions of block b (and of head h in
    dimension (b + 5 h) % dim), 0 elsewhere: with queries of 0 an output counts positions."""
    s = Scene(lens, n, heads, kv, dim, page, seed=seed)
    s.c.vs[:] = 1.0
    for i, l in enumerate(s.lens):
        p = np.arange(l)
        pg, t = s.table[i][p // page], p % page
        s.c.v[pg, :, t] = 0
        for h in range(kv):
            s.c.v[pg, h, t, (p // 16 + 5 * h) % dim] = 1
    s.place()
    return s


def counts(s, window):
    """What comb's outputs are: the share of a row's positions that lie in each dimension's blocks."""
    out = np.full((s.T, s.heads, s.dim), np.nan)
    for i, l in enumerate(s.lens):
        for j in range(s.n[i]):
            end = l - s.n[i] + 1 + j
            p = np.arange(max(0, end - window) if window else 0, max(0, end))
            for h in range(s.heads):
                d = (p // 16 + 5 * (h // (s.heads // s.kv))) % s.dim
                out[s.q_start[i] + j, h] = np.bincount(d, minlength=s.dim) / max(1, len(p))
    return out


def check_counts(s, ws, window=0):
    out = torch.full((s.T, s.heads * s.dim), np.nan, device=DEV)
    q.kv_attention(s.cache, s.batch, torch.zeros((s.T, s.heads, s.dim), device=DEV), 0.1, ws, window=window, out=out)
    q.get_device_error()
    got, want = out.view(s.T, s.heads, s.dim).double().cpu().numpy(), counts(s, window)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    keep = ~np.isnan(want)
    # weights are 1 and codes 0 or 1: sums below 2^24 are whole numbers and exact; the sum's reciprocal,
    # its product and the joins' round: 2^-20
    assert (np.abs(got - want)[keep] <= 2.0 ** -20 * want[keep]).all()
    assert not counters(ws).any(), "a counter was left"
    return out


@pytest.mark.parametrize("heads,kv,rows", LAYOUTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_every_block_once(heads, kv, rows, dim):
    ws = q.kv_workspace()
    check_counts(comb([20011], [rows], heads, kv, dim, 64, 1), ws)
    check_counts(comb([3000, rows, 17, 9001, 2500, 700], [rows, rows, 1, rows, 0, rows], heads, kv, dim, 32, 2), ws)
    check_counts(comb([9001, 5003], [rows] * 2, heads, kv, dim, 16, 3), ws, window=4099)


@pytest.mark.parametrize("heads,kv,rows", LAYOUTS)
@pytest.mark.parametrize("seqs", [32, 33, 200])
def test_many_sequences_some_without_rows(heads, kv, rows, seqs):
    """More and fewer than 32 sequences; runs without rows at the start, between and at the end; one that
    is cut between CTAs."""
    rng = np.random.default_rng(seqs + heads)
    n = rng.choice([0, 0, 1, rows, 2 * rows], seqs)
    n[:2] = n[-3:] = n[10:15] = 0
    n[20] = rows
    lens = [int(v) for v in rng.integers(0, 90, seqs)]
    lens[20] = 4100
    ws = q.kv_workspace()
    check_counts(comb(lens, n.tolist(), heads, kv, 64, 16, seqs), ws)
    lens[20] = 300
    s = Scene(lens, n.tolist(), heads, kv, 128, 16, seed=seqs)
    s.check(s.queries(), ws)
    assert not counters(ws).any()


def test_one_workspace_for_calls_of_other_shapes():
    """A call that cuts items elsewhere, after every other kind of call, gives the bits that it gives on a
    fresh workspace."""
    scenes = [Scene([5000 + 700 * i, 17, 900], [r, r, r], h, kv, dim, 32, seed=i)
              for i, (h, kv, r) in enumerate(LAYOUTS) for dim in (64, 128, 256)]
    xs = [dev(s.queries()) for s in scenes]
    fresh = [q.kv_attention(s.cache, s.batch, x, 0.09, q.kv_workspace()) for s, x in zip(scenes, xs)]
    ws = q.kv_workspace()
    order = np.random.default_rng(0).permutation(2 * len(scenes)) % len(scenes)
    for i in order:
        assert torch.equal(q.kv_attention(scenes[i].cache, scenes[i].batch, xs[i], 0.09, ws), fresh[i])
        assert not counters(ws).any()
    q.get_device_error()


def test_workspace_after_a_bad_index():
    ws = q.kv_workspace()
    s = Scene([5000, 4000, 300], [1] * 3, 8, 2, 128, 32, seed=5)
    x = dev(s.queries())
    want = q.kv_attention(s.cache, s.batch, x, 0.1, ws)
    s.table_d[0, 70] = -1
    s.len_d[1] = -3
    q.kv_attention(s.cache, s.batch, x, 0.1, ws)
    with pytest.raises(q.QmdError, match="QMD_ERR_INDEX"):
        q.get_device_error()
    assert not counters(ws).any()
    s.table_d.copy_(dev(s.table))
    s.len_d.copy_(dev(np.array(s.lens, np.int32)))
    assert torch.equal(q.kv_attention(s.cache, s.batch, x, 0.1, ws), want)
    q.get_device_error()


def test_bounds_of_the_plain_form_hold_over_cut_sequences():
    s = Scene([4100, 17, 2300], [2, 1, 3], 8, 2, 256, 32, seed=6)
    ref, bound = P.attention(s.c, s.table, s.lens, s.q_start, s.queries(), 0.1)
    assert ref.shape == bound.shape and np.isfinite(bound).all()
