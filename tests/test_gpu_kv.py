"""The paged 8-bit key/value cache on the GPU: append (bit for bit), read back, attention (within a
bound derived from the arithmetic), against plain forms; graphs, streams, bad indexes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
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


@pytest.fixture(scope="module")
def ws():
    return q.kv_workspace()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def bits(a):
    return np.ascontiguousarray(a).view(np.uint32)


class Scene:
    """Sequences with lens[s] tokens of which the last rows[s] are the call's, their pages strewn over
    a pool.  Whatever no sequence may look at holds the largest codes, and a NaN scale where a whole
    block is out of reach, so that a value that leaks in is seen."""

    def __init__(self, lens, rows, heads=4, kv=2, dim=64, page=32, seed=0, uniform=False, extra_rows=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.n = rng, list(lens), list(rows)
        self.heads, self.kv, self.dim, self.page = heads, kv, dim, page
        need = [max(1, -(-max(l, 1) // page)) for l in lens]
        pages = sum(need) + 2
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(need) + 1), 0, np.int32)
        at = 0
        for s, k in enumerate(need):
            self.table[s, :k] = order[at:at + k]
            self.table[s, k:] = order[-1]  # a page that no sequence uses
            at += k
        shape = (pages, kv, page, dim)
        self.c = P.Cache(np.full(shape, 127, np.int8), np.full(shape, -127, np.int8),
                         np.full((pages, kv, page // 16), np.nan, np.float32),
                         np.full((pages, kv, page // 16), np.nan, np.float32))
        for s, l in enumerate(lens):
            for p0 in range(0, l, 16):
                pg, t0, m = self.table[s, p0 // page], p0 % page, min(16, l - p0)
                for codes, sc in ((self.c.k, self.c.ks), (self.c.v, self.c.vs)):
                    codes[pg, :, t0:t0 + m] = rng.integers(-128, 128, (kv, m, dim))
                    sc[pg, :, t0 // 16] = rng.uniform(0.005, 0.03, kv) * spread ** rng.uniform(-1, 1, kv)
        self.q_start = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
        self.T = int(self.q_start[-1]) + extra_rows
        self.uniform = uniform
        self.place()

    def place(self):
        c = self.c
        self.cache = q.KVCache(dev(c.k), dev(c.v), dev(c.ks), dev(c.vs))
        self.len_d, self.table_d, self.start_d = dev(np.array(self.lens, np.int32)), dev(self.table), dev(self.q_start)
        if self.uniform:
            self.batch = q.KVBatch(self.table_d, self.len_d, max_q=self.n[0], rows=self.T)
        else:
            self.batch = q.KVBatch(self.table_d, self.len_d, self.start_d, max(1, max(self.n)), self.T)

    def queries(self, scale=1.0):
        return (self.rng.standard_normal((self.T, self.heads, self.dim)) * scale).astype(np.float32)

    def check(self, x, ws, scale=None, window=0, out=None, **kw):
        scale = self.dim ** -0.5 if scale is None else scale
        ref, bound = P.attention(self.c, self.table, self.lens, self.q_start, x, scale, window)
        if out is None:
            out = torch.full((self.T, self.heads * self.dim), np.nan, device=DEV)
        got = q.kv_attention(self.cache, self.batch, dev(x), scale, ws, window=window, out=out, **kw)
        q.get_device_error()
        self.close(got, ref, bound)
        return got

    def close(self, got, ref, bound):
        got = got.reshape(self.T, self.heads, self.dim).cpu().numpy()
        nan = np.isnan(ref)
        assert np.array_equal(np.isnan(got), nan), "rows written where none should be, or the other way round"
        err = np.abs(got - ref)[~nan]
        assert (err <= bound[~nan]).all(), f"{(err / np.maximum(bound[~nan], 1e-300)).max()} times the bound"


# ---- attention ---------------------------------------------------------------------------------

LENS = [1, 15, 16, 17, 33, 100, 31, 64]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv", [(4, 1), (2, 2), (14, 2), (8, 1), (16, 4), (9, 3)])
def test_one_row_each(ws, dim, heads, kv):
    s = Scene(LENS, [1] * 8, heads, kv, dim, seed=dim + heads, uniform=True)
    s.check(s.queries(), ws)


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 16), (128, 48), (128, 128), (256, 32)])
@pytest.mark.parametrize("n", [2, 3, 5, 8])
def test_several_rows_each(ws, dim, page, n):
    s = Scene([n, n + 1, 16, 20, 47, 130], [n] * 6, 8, 2, dim, page, seed=n, uniform=n % 2 == 0)
    s.check(s.queries(), ws)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 40, 1000])
@pytest.mark.parametrize("n", [1, 4])
def test_window(ws, window, n):
    s = Scene([5, 16, 33, 90, 200], [n] * 5, 6, 2, 128, 32, seed=window)
    s.check(s.queries(), ws, window=window)


def test_ragged_rows_none_and_empty(ws):
    # sequences without rows, rows that see nothing (fewer tokens than rows), no tokens at all,
    # and rows behind the last sequence, which stay as they were
    s = Scene([40, 0, 2, 17, 0, 300], [3, 0, 5, 1, 2, 8], 8, 2, 128, 16, seed=1, extra_rows=3)
    x = s.queries()
    got = s.check(x, ws).reshape(s.T, 8, 128).cpu().numpy()
    assert (got[3:6] == 0).all() and (got[9:11] == 0).all()  # rows of sequences 2 (the first three) and 4
    assert np.isnan(got[-3:]).all()


@pytest.mark.parametrize("heads,kv,dim,n", [(32, 8, 128, 1), (8, 8, 64, 1), (16, 2, 128, 3), (4, 1, 256, 2)])
def test_long(ws, heads, kv, dim, n):
    s = Scene([20011], [n], heads, kv, dim, 64, seed=5, uniform=True)
    s.check(s.queries(), ws)


def test_long_beside_short(ws):
    s = Scene([1, 9001, 3, 257, 1, 1, 4100, 16], [1] * 8, 8, 2, 128, 64, seed=6, uniform=True)
    s.check(s.queries(), ws)


@pytest.mark.parametrize("seqs", [300, 700])
def test_many_sequences(ws, seqs):
    lens = np.random.default_rng(seqs).integers(0, 40, seqs).tolist()
    s = Scene(lens, [1] * seqs, 4, 2, 64, 16, seed=7)
    s.check(s.queries(), ws)


@pytest.mark.parametrize("heads,kv,n", [(64, 1, 3), (24, 2, 8), (5, 1, 33), (8, 2, 70)])
def test_many_rows_for_a_head(ws, heads, kv, n):
    s = Scene([n + 50, n, 200], [n, n, n], heads, kv, 64, 32, seed=8)
    s.check(s.queries(), ws)


def test_sharp_and_flat_weights(ws):
    s = Scene([50, 333, 1000], [1] * 3, 8, 2, 128, 32, seed=9)
    s.check(s.queries(12.0), ws)             # one position takes nearly all the weight
    s.check(s.queries(1e-3), ws)             # an average
    s.check(s.queries(), ws, scale=-0.5)     # a negative scale is a scale
    s.check(s.queries(), ws, scale=0.0)


def test_tiny_and_huge_values(ws):
    s = Scene([77, 160], [1] * 2, 8, 2, 128, 32, seed=10)
    # queries down to where f32 has few bits, and up
    s.check(s.queries(1e-30), ws, scale=1e28)
    s.check(s.queries(1e18), ws, scale=1e-18)
    for f in (1e-18, 1e18):
        t = Scene([77, 160], [1] * 2, 8, 2, 128, 32, seed=11)
        t.c.vs *= np.float32(f)
        t.place()
        t.check(t.queries(), ws)


def test_block_scales_far_apart(ws):
    # value blocks whose scales differ by up to 2^12 within a sequence, blocks of zeros among them
    s = Scene([500, 90], [2] * 2, 8, 2, 128, 32, seed=12, spread=64.0)
    s.c.vs[s.table[0, 2], :, 0] = 0
    s.c.ks[s.table[0, 3], :, 1] = 0
    s.c.vs[s.table[1, :3]] = 0  # a sequence of nothing but zeros
    s.c.vs[s.table[0, 5]] *= -1  # a scale is a factor, whatever its sign
    s.c.ks[s.table[0, 6]] *= -1
    s.place()
    got = s.check(s.queries(), ws)
    assert (got[2:] == 0).all()


def test_rows_strided(ws):
    s = Scene([40, 90, 3], [2, 1, 1], 8, 2, 128, 32, seed=13)
    x = s.queries()
    wide = torch.full((s.T, 8 * 128 + 96), np.nan, device=DEV)
    wide[:, 32:32 + 1024] = dev(x).reshape(s.T, -1)
    out = torch.full((s.T, 1024 + 64), 7.0, device=DEV)
    got = q.kv_attention(s.cache, s.batch, wide[:, 32:32 + 1024], 128 ** -0.5, ws, out=out[:, 64:])
    q.get_device_error()
    ref, bound = P.attention(s.c, s.table, s.lens, s.q_start, x, 128 ** -0.5)
    s.close(got, ref, bound)
    assert (out[:, :64] == 7.0).all()


def test_bad_numbers_stay_in_their_row_and_head(ws):
    s = Scene([40, 90, 300], [1] * 3, 8, 2, 128, 32, seed=14)
    x = s.queries()
    ref, bound = P.attention(s.c, s.table, s.lens, s.q_start, x, 0.1)
    x[1, 3, 7], x[2, 0, 5] = np.nan, np.inf
    got = q.kv_attention(s.cache, s.batch, dev(x), 0.1, ws).reshape(3, 8, 128).cpu().numpy()
    q.get_device_error()
    assert np.isnan(got[1, 3]).all()
    keep = np.ones((3, 8), bool)
    keep[1, 3] = keep[2, 0] = False
    assert (np.abs(got - ref)[keep] <= bound[keep]).all()


def test_same_bits_twice_and_workspace_left_zeroed(ws):
    s = Scene([5000, 17, 900], [2, 1, 1], 32, 8, 128, 64, seed=15)
    x = dev(s.queries())
    a = q.kv_attention(s.cache, s.batch, x, 0.09, ws).clone()
    for _ in range(5):
        assert torch.equal(a, q.kv_attention(s.cache, s.batch, x, 0.09, ws))


def test_pool_past_four_gigabytes(ws):
    page, kv, dim = 64, 8, 128
    pages = (1 << 32) // (page * kv * dim) + 3
    codes = torch.zeros((pages, kv, page, dim), dtype=torch.int8, device=DEV)
    scale = torch.ones((pages, kv, page // 16), device=DEV)
    cache = q.KVCache(codes, codes, scale, scale)
    codes[-1, :, :5] = 3
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    batch = q.KVBatch(table, torch.tensor([5], dtype=torch.int32, device=DEV))
    got = q.kv_attention(cache, batch, torch.randn((1, 32, dim), device=DEV), 0.1, ws)
    q.get_device_error()
    assert (got - 3).abs().max() < 1e-5
    q.kv_append(cache, q.KVBatch(table, torch.tensor([64], dtype=torch.int32, device=DEV)),
                torch.full((1, kv, dim), 2.0, device=DEV), torch.full((1, kv, dim), 2.0, device=DEV))
    k, _ = q.kv_read(cache, q.KVBatch(table, torch.tensor([64], dtype=torch.int32, device=DEV)))
    q.get_device_error()
    assert (k - 2).abs().max() < 1e-5 and (codes[:-1] == 0).all()


def test_bad_indexes_are_reported_and_touch_nothing(ws):
    s = Scene([40, 90, 30, 20], [1, 2, 1, 1], 8, 2, 128, 32, seed=16)
    x = s.queries()
    ref, bound = P.attention(s.c, s.table, s.lens, s.q_start, x, 0.1)

    def run(expect, rows):
        out = torch.full((s.T, 1024), np.nan, device=DEV)
        q.kv_attention(s.cache, s.batch, dev(x), 0.1, ws, out=out)
        with pytest.raises(q.QmdError, match=expect):
            q.get_device_error()
        q.get_device_error()  # reported once
        got = out.reshape(s.T, 8, 128).cpu().numpy()
        for r in range(s.T):
            if r in rows:
                assert (np.abs(got[r] - ref[r]) <= bound[r]).all()
        return got

    s.table_d[1, 1] = len(s.c.k)           # past the pool: those positions are left out
    assert np.isfinite(run("QMD_ERR_INDEX", [0, 3, 4])).all()
    s.table_d[1, 1] = -1
    run("QMD_ERR_INDEX", [0, 3, 4])
    s.table_d.copy_(dev(s.table))
    s.len_d[2] = s.table.shape[1] * 32 + 1  # longer than its table: the sequence is left out
    assert np.isnan(run("QMD_ERR_INDEX", [0, 1, 2, 4])[3]).all()
    s.len_d[2] = -5
    assert np.isnan(run("QMD_ERR_INDEX", [0, 1, 2, 4])[3]).all()
    s.len_d[2] = 30
    s.start_d[4] = s.T + 1                  # rows past the tensors
    assert np.isnan(run("QMD_ERR_INDEX", [0, 1, 2, 3])[4]).all()
    s.start_d.copy_(dev(s.q_start))
    s.start_d[0] = -1
    run("QMD_ERR_INDEX", [1, 2, 3, 4])
    s.start_d.copy_(dev(s.q_start))
    s.check(x, ws, scale=0.1)


def test_graph_replay_sees_new_lengths_and_pages(ws):
    s = Scene([40, 90, 700], [1] * 3, 8, 2, 128, 32, seed=17)
    x = s.queries()
    xd, out = dev(x), torch.zeros((3, 1024), device=DEV)
    q.kv_attention(s.cache, s.batch, xd, 0.1, ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.kv_attention(s.cache, s.batch, xd, 0.1, ws, out=out)
    for lens in ([40, 90, 700], [3, 90, 1], [40, 1, 33]):
        s.lens = lens
        s.len_d.copy_(dev(np.array(lens, np.int32)))
        g.replay()
        q.get_device_error()
        s.close(out, *P.attention(s.c, s.table, lens, s.q_start, x, 0.1))
    s.table[[0, 1]] = s.table[[1, 0]]
    s.table_d.copy_(dev(s.table))
    s.lens = [80, 30, 33]
    s.len_d.copy_(dev(np.array(s.lens, np.int32)))
    g.replay()
    q.get_device_error()
    s.close(out, *P.attention(s.c, s.table, s.lens, s.q_start, x, 0.1))


def test_two_streams_with_their_own_workspaces():
    s = Scene([3000, 4000], [1] * 2, 32, 8, 128, 64, seed=18)
    t = Scene([2500, 17, 900], [1] * 3, 32, 8, 128, 64, seed=19)
    jobs = [(u, dev(u.queries()), torch.cuda.Stream(), q.kv_workspace()) for u in (s, t)]
    torch.cuda.synchronize()
    want = [q.kv_attention(u.cache, u.batch, x, 0.1, w).clone() for u, x, _, w in jobs]
    torch.cuda.synchronize()
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for (u, x, st, w), o in zip(jobs, outs):
            q.kv_attention(u.cache, u.batch, x, 0.1, w, out=o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_lengths_past_what_positions_count_are_reported(ws):
    # a table that puts 2^31 positions on one page: the sequence is left out, the other is not
    s = Scene([40, 20], [1, 1], 4, 2, 64, 16, seed=21)
    x = s.queries()
    ref, bound = P.attention(s.c, s.table, s.lens, s.q_start, x, 0.1)
    wide = torch.zeros((2, 1 << 24), dtype=torch.int32, device=DEV)
    wide[1, :2] = s.table_d[1, :2]
    batch = q.KVBatch(wide, torch.tensor([(1 << 28) - 1 + (1 << 30), 20], dtype=torch.int32, device=DEV), s.start_d, 1, 2)
    out = torch.full((2, 256), np.nan, device=DEV)
    q.kv_attention(s.cache, batch, dev(x), 0.1, ws, out=out)
    with pytest.raises(q.QmdError, match="QMD_ERR_INDEX"):
        q.get_device_error()
    got = out.reshape(2, 4, 64).cpu().numpy()
    assert np.isnan(got[0]).all() and (np.abs(got[1] - ref[1]) <= bound[1]).all()


def test_outputs_on_another_stream(ws):
    s = Scene([300, 41], [1, 1], 8, 2, 128, 32, seed=22)
    x = s.queries()
    xd = dev(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = q.kv_attention(s.cache, s.batch, xd, 0.1, ws, stream=side)
    k, v = q.kv_read(s.cache, s.batch, stream=side.cuda_stream)
    side.synchronize()
    s.close(got, *P.attention(s.c, s.table, s.lens, s.q_start, x, 0.1))
    K, V = s.c.values(s.table, 0, 299, 300)
    assert np.array_equal(bits(k[0:1].cpu().numpy()), bits(K.astype(np.float32)))
    assert np.array_equal(bits(v[0:1].cpu().numpy()), bits(V.astype(np.float32)))


def test_graphs_that_overlap_with_their_own_workspaces():
    s = Scene([5000, 300, 77], [1] * 3, 32, 8, 128, 64, seed=23)
    x = dev(s.queries())
    want = q.kv_attention(s.cache, s.batch, x, 0.1, q.kv_workspace())
    graphs = []
    for _ in range(2):
        w, o, st = q.kv_workspace(), torch.zeros_like(want), torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(4):
                q.kv_attention(s.cache, s.batch, x, 0.1, w, out=o)
        graphs.append((g, o, st, w))
    for _ in range(10):
        for g, _, st, _ in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for _, o, _, _ in graphs)


# ---- append and read ---------------------------------------------------------------------------

def rope_np(n, rot):
    return q.rope_table(n, rot, 500000.0, device="cpu").numpy()


def run_append(s, rope, rot, pairs, x, in_place=False):
    """Appends s.n new rows per sequence on the device and on the host; compares every byte."""
    k = s.rng.standard_normal((s.T, s.kv, s.dim)).astype(np.float32)
    v = (s.rng.standard_normal((s.T, s.kv, s.dim)) * s.rng.uniform(0.1, 5, (s.T, 1, 1))).astype(np.float32)
    ref = P.append(s.c, s.table, s.lens, s.q_start, k, v, rope, x, rot, pairs == q.ROPE_HALVES)
    rope_d = None if rope is None else dev(rope)
    if x is None:
        assert q.kv_append(s.cache, s.batch, dev(k), dev(v), rope=rope_d, pairs=pairs) is None
    else:
        xd = dev(x)
        o = xd if in_place else torch.full_like(xd, np.nan)
        q.kv_append(s.cache, s.batch, dev(k), dev(v), rope=rope_d, q=xd, q_out=o, pairs=pairs)
        own = ~np.isnan(ref[:, 0, 0])
        got = o.cpu().numpy()
        assert np.array_equal(bits(got[own]), bits(ref[own]))
        assert np.array_equal(bits(got[~own]), bits(x[~own])) if in_place else np.isnan(got[~own]).all()
    q.get_device_error()
    same_cache(s)


def same_cache(s):
    differ = [int((got.cpu().numpy() != want).sum()) for got, want in ((s.cache.k, s.c.k), (s.cache.v, s.c.v))]
    differ += [int((bits(got.cpu().numpy()) != bits(want)).sum())
               for got, want in ((s.cache.k_scale, s.c.ks), (s.cache.v_scale, s.c.vs))]
    assert differ == [0] * 4


@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 96), (256, 256), (256, 32), (128, 0)])
@pytest.mark.parametrize("pairs", [q.ROPE_HALVES, q.ROPE_ADJACENT])
@pytest.mark.parametrize("rows", [[1, 1, 1, 1, 1, 1], [5, 0, 40, 16, 3, 8]])
def test_append_bit_exact(dim, rot, pairs, rows):
    before = [0, 7, 15, 16, 30, 100]
    s = Scene([b + n for b, n in zip(before, rows)], rows, 6, 2, dim, 32, seed=dim + rot + pairs,
              extra_rows=2, uniform=max(rows) == 1 and rot == 64)
    run_append(s, rope_np(200, rot) if rot else None, rot, pairs, s.queries(), in_place=rot == dim)


def test_append_without_queries():
    s = Scene([20, 33], [4, 1], 6, 3, 128, 16, seed=3)
    run_append(s, rope_np(64, 128), 128, q.ROPE_HALVES, None)


def test_append_token_by_token_as_blocks_fill_and_scales_grow():
    s = Scene([1, 14, 47], [1] * 3, 4, 2, 128, 16, seed=4)
    wide = np.zeros((3, 9), np.int32)
    pages = np.random.default_rng(0).permutation(30)[:27].reshape(3, 9)
    wide[:] = pages
    s.table = wide
    s.c = P.Cache(np.zeros((30, 2, 16, 128), np.int8), np.zeros((30, 2, 16, 128), np.int8),
                  np.full((30, 2, 1), 9.0, np.float32), np.full((30, 2, 1), 9.0, np.float32))
    rope = rope_np(200, 128)
    s.lens = [0, 0, 0]
    for step in range(70):
        s.lens = [step + 1, step // 2 + 1, step + 1]
        if step % 2 == 0:
            s.place()
        else:
            s.len_d.copy_(dev(np.array(s.lens, np.int32)))
        run_append(s, rope, 128, q.ROPE_HALVES, s.queries())


def test_append_zeros_tiny_and_large():
    s = Scene([20, 9, 33], [5, 3, 2], 4, 2, 128, 32, seed=5)
    k = s.rng.standard_normal((s.T, 2, 128)).astype(np.float32)
    k[:5] = 0
    k[5:8] *= np.float32(1e-36)  # under the smallest value that has a scale
    k[8:] *= np.float32(1e30)
    v = k[::-1].copy()
    P.append(s.c, s.table, s.lens, s.q_start, k, v)
    q.kv_append(s.cache, s.batch, dev(k), dev(v))
    q.get_device_error()
    same_cache(s)


def test_padded_batch_keeps_quiet(ws):
    # slots without a request: kv_len 0, a row each, and a page table of rubbish
    s = Scene([21, 1, 1, 60], [1] * 4, 8, 2, 128, 16, seed=24, uniform=True)
    real = [0, 3]
    s.len_d[1:3] = 0
    s.table_d[1:3] = 12345
    k, v = (s.rng.standard_normal((4, 2, 128)).astype(np.float32) for _ in "kv")
    x = s.queries()
    want = s.c
    rope = rope_np(64, 128)
    ref = P.append(want, s.table[real], [21, 60], [0, 1, 2], k[real], v[real], rope, x[real], 128)
    qr = torch.full((4, 8, 128), np.nan, device=DEV)
    q.kv_append(s.cache, s.batch, dev(k), dev(v), dev(rope), dev(x), qr)
    out = q.kv_attention(s.cache, s.batch, qr, 0.1, ws)
    ko = torch.full((4, 2, 128), 5.0, device=DEV)
    q.kv_read(s.cache, s.batch, ko, torch.empty_like(ko))
    q.get_device_error()
    same_cache(s)
    assert np.array_equal(bits(qr.cpu().numpy()[real]), bits(ref)) and qr[1:3].isnan().all() and (ko[1:3] == 5).all()
    att, bound = P.attention(want, s.table[real], [21, 60], [0, 1, 2], ref, 0.1)
    got = out.reshape(4, 8, 128).cpu().numpy()
    assert (np.abs(got[real] - att) <= bound).all() and (got[1:3] == 0).all()


def test_append_parts_of_a_fused_projection_and_read_back():
    s = Scene([33, 70, 1], [3, 9, 1], 8, 2, 128, 32, seed=6)
    qkv = s.rng.standard_normal((s.T, 12 * 128)).astype(np.float32)
    x, k, v = qkv[:, :1024].reshape(-1, 8, 128), qkv[:, 1024:1280].reshape(-1, 2, 128), qkv[:, 1280:].reshape(-1, 2, 128)
    rope = rope_np(100, 128)
    ref = P.append(s.c, s.table, s.lens, s.q_start, k, v, rope, x, 128, False)
    d = dev(qkv)
    got = q.kv_append(s.cache, s.batch, d[:, 1024:1280].unflatten(1, (2, 128)), d[:, 1280:], dev(rope),
                      d[:, :1024], d[:, :1024], pairs=q.ROPE_ADJACENT)
    q.get_device_error()
    assert got.data_ptr() == d.data_ptr()
    assert np.array_equal(bits(d[:, :1024].cpu().numpy()), bits(ref.reshape(s.T, -1)))
    assert np.array_equal(bits(d[:, 1024:].cpu().numpy()), bits(qkv[:, 1024:]))
    same_cache(s)
    ks, vs = q.kv_read(s.cache, s.batch)
    for i, l in enumerate(s.lens):
        K, V = s.c.values(s.table, i, l - s.n[i], l)
        a, b = s.q_start[i], s.q_start[i + 1]
        assert np.array_equal(bits(ks[a:b].cpu().numpy()), bits(K.astype(np.float32)))
        assert np.array_equal(bits(vs[a:b].cpu().numpy()), bits(V.astype(np.float32)))


@pytest.mark.parametrize("dim,page,rows", [(64, 16, [40, 1, 17]), (128, 128, [300, 0, 5]), (256, 48, [1, 1, 90])])
def test_read(dim, page, rows):
    s = Scene([n + 11 for n in rows], rows, 6, 3, dim, page, seed=dim, extra_rows=2)
    k = torch.full((s.T, 3 * dim + 32), 5.0, device=DEV)
    v = torch.full((s.T, 3, dim), 5.0, device=DEV)
    q.kv_read(s.cache, s.batch, k[:, 32:], v)
    q.get_device_error()
    for i, l in enumerate(s.lens):
        K, V = s.c.values(s.table, i, l - rows[i], l)
        a, b = s.q_start[i], s.q_start[i + 1]
        assert np.array_equal(bits(k[a:b, 32:].reshape(-1, 3, dim).cpu().numpy()), bits(K.astype(np.float32)))
        assert np.array_equal(bits(v[a:b].cpu().numpy()), bits(V.astype(np.float32)))
    assert (k[:, :32] == 5).all() and (k[-2:] == 5).all() and (v[-2:] == 5).all()


def test_append_and_read_bad_indexes():
    s = Scene([40, 20, 30], [2, 2, 2], 4, 2, 64, 16, seed=7)
    rope = rope_np(200, 64)
    k = s.rng.standard_normal((s.T, 2, 64)).astype(np.float32)

    def run(**kw):
        q.kv_append(s.cache, s.batch, dev(k), dev(k), **kw)
        with pytest.raises(q.QmdError, match="QMD_ERR_INDEX"):
            q.get_device_error()

    # a page outside the pool: sequence 1's rows are not stored, the others are
    s.table_d[1, 1] = 10_000
    want = s.c.copy()
    P.append(want, s.table[[0, 2]], [40, 30], [0, 2, 4], k[[0, 1, 4, 5]], k[[0, 1, 4, 5]])
    run()
    s.c = want
    same_cache(s)
    s.table_d.copy_(dev(s.table))
    # a sequence shorter than its rows
    s.len_d[0] = 1
    want = s.c.copy()
    P.append(want, s.table[1:], [20, 30], [0, 2, 4], k[2:], k[2:])
    out = torch.full((s.T, 2, 64), 5.0, device=DEV)
    run()
    s.c = want
    same_cache(s)
    q.kv_read(s.cache, s.batch, out, torch.empty_like(out))
    with pytest.raises(q.QmdError, match="QMD_ERR_INDEX"):
        q.get_device_error()
    assert (out[:2] == 5).all()
    s.len_d.copy_(dev(np.array(s.lens, np.int32)))
    # positions past the rotation table: 29 of sequence 2 and both of sequence 0 are not stored
    want = s.c.copy()
    P.append(want, s.table[1:], [20, 29], [0, 2, 3], k[2:5], k[2:5], rope, rot=64)
    run(rope=dev(rope[:29]))
    s.c = want
    same_cache(s)


def test_append_then_attention_in_one_stream_and_in_a_graph(ws):
    """Steps of a decode as they are used: append, attention, no wait between, eagerly and replayed."""
    s = Scene([64, 64], [1] * 2, 8, 2, 128, 16, seed=20)
    rope, x = rope_np(128, 128), np.zeros((2, 8, 128), np.float32)
    rope_d = dev(rope)
    xd, kd, vd = dev(x), torch.zeros((2, 2, 128), device=DEV), torch.zeros((2, 2, 128), device=DEV)
    qr, out = torch.zeros_like(xd), torch.zeros((2, 1024), device=DEV)
    s.lens = [30, 5]
    s.len_d.copy_(dev(np.array(s.lens, np.int32)))

    def step():
        q.kv_append(s.cache, s.batch, kd, vd, rope_d, xd, qr)
        q.kv_attention(s.cache, s.batch, qr, 128 ** -0.5, ws, out=out)

    for i in range(24):
        x, k, v = (s.rng.standard_normal(t.shape).astype(np.float32) for t in (xd, kd, vd))
        s.lens = [l + 1 for l in s.lens]
        for a, b in ((xd, x), (kd, k), (vd, v), (s.len_d, np.array(s.lens, np.int32))):
            a.copy_(dev(b))
        if i < 3:
            step()
        else:
            if i == 3:
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    step()
            g.replay()
        q.get_device_error()
        xr = P.append(s.c, s.table, s.lens, s.q_start, k, v, rope, x, 128, True)
        same_cache(s)
        s.close(out, *P.attention(s.c, s.table, s.lens, s.q_start, xr, 128 ** -0.5))
