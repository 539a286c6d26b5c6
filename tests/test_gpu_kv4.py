"""The paged 4-bit key/value cache on the GPU: append (bit for bit), read back, attention with its
log-sum-exp, weights and eviction, against plain forms; graphs, streams, bad indexes; a run of them together."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from tests import kv4_plain as P  # noqa: E402

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
    return np.ascontiguousarray(a).view({2: np.uint16, 4: np.uint32, 8: np.uint64}[a.dtype.itemsize])


class Scene:
    """Sequences with lens[s] tokens of which the last rows[s] are the call's, their pages strewn over a
    pool.  Every slot that no sequence holds has the largest codes and a NaN scale and weight, so that a value
    that leaks in is seen.  spread: how far apart (a power) the scales of groups and tokens lie."""

    def __init__(self, lens, rows, heads=4, kv=2, dim=64, page=32, seed=0, uniform=False, extra_rows=0, spread=2.0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.n = rng, list(lens), list(rows)
        self.heads, self.kv, self.dim, self.page = heads, kv, dim, page
        need = [max(1, -(-max(n, 1) // page)) for n in lens]
        pages = sum(need) + 2
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(need) + 1), 0, np.int32)
        at = 0
        for s, k in enumerate(need):
            self.table[s, :k] = order[at:at + k]
            self.table[s, k:] = order[-1]  # a page that no sequence uses
            at += k
        shape = (pages, kv, page)
        nan16 = lambda: np.full(shape + (dim // 32,), np.nan, np.float16)  # noqa: E731
        self.c = P.Cache(np.full(shape + (dim // 2,), 255, np.uint8), np.full(shape + (dim // 2,), 0, np.uint8), nan16(), nan16())
        self.w = np.full(shape, np.nan, np.float32)
        for s, n in enumerate(lens):
            pg, tok = self.c.at(self.table, s, 0, n)
            for codes, sc in ((self.c.k, self.c.ks), (self.c.v, self.c.vs)):
                codes[pg, :, tok] = rng.integers(0, 256, (n, kv, dim // 2))
                sc[pg, :, tok] = rng.uniform(0.1, 0.4, (n, kv, dim // 32)) * rng.choice([-1, 1], (n, kv, dim // 32)) * \
                    spread ** rng.uniform(-1, 1, (n, kv, dim // 32))
            old = max(0, n - rows[s])
            self.w[pg[:old], :, tok[:old]] = rng.exponential(1.0, (old, kv))
        self.q_start = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
        self.T = int(self.q_start[-1]) + extra_rows
        self.uniform = uniform
        self.place()

    def place(self):
        c = self.c
        self.cache = q.KV4Cache(dev(c.k), dev(c.v), dev(c.ks), dev(c.vs))
        self.weight = dev(self.w)
        self.len_d, self.table_d, self.start_d = dev(np.array(self.lens, np.int32)), dev(self.table), dev(self.q_start)
        if self.uniform:
            self.batch = q.KVBatch(self.table_d, self.len_d, max_q=self.n[0], rows=self.T)
        else:
            self.batch = q.KVBatch(self.table_d, self.len_d, self.start_d, max(1, max(self.n)), self.T)

    def queries(self, scale=0.7):
        return (self.rng.standard_normal((self.T, self.heads, self.dim)) * scale).astype(np.float32)

    def check(self, x, ws, scale=None, window=0, weigh=True):
        """Attention, its log-sum-exp, and the weights that follow from it."""
        scale = self.dim ** -0.5 if scale is None else scale
        ref, bound, lref, lbound = P.attention(self.c, self.table, self.lens, self.q_start, x, scale, window)
        out = torch.full((self.T, self.heads * self.dim), np.nan, device=DEV)
        lse = torch.full((self.T, self.heads), np.nan, device=DEV)
        xd = dev(x)
        assert q.kv4_attention(self.cache, self.batch, xd, scale, ws, window=window, out=out, lse=lse) is out
        plain = torch.full_like(out, np.nan)
        q.kv4_attention(self.cache, self.batch, xd, scale, ws, window=window, out=plain)
        q.get_device_error()
        assert torch.equal(plain.nan_to_num(9e9), out.nan_to_num(9e9)), "the log-sum-exp changes the output"
        close(out.reshape(ref.shape).cpu().numpy(), ref, bound, "attention")
        close(lse.cpu().numpy(), lref, lbound, "log-sum-exp")
        if weigh:
            self.check_weights(x, lse, scale, window)
        return out

    def check_weights(self, x, lse, scale, window):
        ref, bound = P.weigh(self.c, self.table, self.lens, self.q_start, x, scale, lse.cpu().numpy(), self.w, window)
        weight = self.weight.clone()
        assert q.kv4_weigh(self.cache, self.batch, dev(x), scale, lse, weight, window=window) is weight
        q.get_device_error()
        got = weight.cpu().numpy()
        close(got, ref, bound, "weights")
        same = bound == 0
        assert np.array_equal(bits(got[same & np.isnan(ref)]), bits(self.w[same & np.isnan(ref)])), "weights that nobody owns"


def close(got, ref, bound, what):
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{what}: written where nothing should be, or the other way round"
    assert np.array_equal(np.isinf(got), np.isinf(ref)) and (got[np.isinf(ref)] == ref[np.isinf(ref)]).all(), what
    at = ~nan & ~np.isinf(ref)
    err = np.abs(got[at] - ref[at])
    assert (err <= bound[at]).all(), f"{what}: {(err / np.maximum(bound[at], 1e-300)).max()} times the bound"


# ---- attention and weights ---------------------------------------------------------------------

LENS = [1, 15, 16, 17, 33, 100, 31, 64]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv", [(4, 1), (2, 2), (14, 2), (8, 1), (16, 4), (9, 3)])
def test_one_row_each(ws, dim, heads, kv):
    s = Scene(LENS, [1] * 8, heads, kv, dim, seed=dim + heads, uniform=True)
    s.check(s.queries(), ws)


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 16), (128, 48), (128, 128), (256, 32), (256, 80)])
@pytest.mark.parametrize("n", [2, 3, 5, 8, 21])
def test_several_rows_each(ws, dim, page, n):
    s = Scene([n, n + 1, n + 16, 20 + n, 47, 130], [n] * 6, 8, 2, dim, page, seed=n, uniform=n % 2 == 0)
    s.check(s.queries(), ws)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 40, 1000])
@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("page", [16, 32])
def test_window(ws, window, n, page):
    s = Scene([5, 16, 33, 90, 200], [n] * 5, 6, 2, 128, page, seed=window)
    s.check(s.queries(), ws, window=window)


def test_window_leaves_pages_before_it_alone(ws):
    """Table entries of slots that no row sees may hold anything: a recycled page's place, or -1."""
    s = Scene([200, 90], [2, 1], 4, 2, 128, 16, seed=3)
    x = s.queries()
    want = s.check(x, ws, window=20)
    for p in range((200 - 1 - 20) // 16):
        s.table_d[0, p] = -1
    got = q.kv4_attention(s.cache, s.batch, dev(x), 128 ** -0.5, ws, window=20)
    q.get_device_error()
    assert torch.equal(got, want)


def test_ragged_rows_none_and_empty(ws):
    # sequences without rows, rows that see nothing (fewer tokens than rows), no tokens at all,
    # and rows behind the last sequence, which stay as they were
    s = Scene([40, 0, 2, 17, 0, 300], [3, 0, 5, 1, 2, 8], 8, 2, 128, 16, seed=1, extra_rows=3)
    got = s.check(s.queries(), ws).reshape(s.T, 8, 128).cpu().numpy()
    assert (got[3:6] == 0).all() and (got[9:11] == 0).all()  # rows of sequences 2 (the first three) and 4
    assert np.isnan(got[-3:]).all()


@pytest.mark.parametrize("heads,kv,dim,n", [(32, 8, 128, 1), (8, 8, 64, 1), (16, 2, 128, 3), (4, 1, 256, 2), (5, 1, 64, 7)])
def test_long(ws, heads, kv, dim, n):
    s = Scene([5000, 333, 20011 // max(1, kv // 2)], [n] * 3, heads, kv, dim, 64, seed=heads + n)
    s.check(s.queries(), ws, weigh=n < 7)


def test_many_sequences(ws):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 90, 150).tolist()
    s = Scene(lens, [min(n, int(rng.integers(0, 3))) for n in lens], 4, 2, 64, 32, seed=9)
    s.check(s.queries(), ws)


@pytest.mark.parametrize("heads", [64, 36])
def test_many_heads_to_one(ws, heads):
    s = Scene([70, 3], [2, 1], heads, 1, 64, 16, seed=heads)
    s.check(s.queries(), ws)


@pytest.mark.parametrize("big", [3e4, 1e-6, 0.0])
def test_query_sizes(ws, big):
    s = Scene([50, 20], [1, 2], 4, 2, 128, 32, seed=7)
    x = s.queries()
    x[0] *= big
    s.check(x, ws, scale=0.05 if big <= 1 else 0.05 / big)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_of_scores(ws, scale):
    s = Scene([50, 20], [1, 2], 4, 2, 64, 32, seed=8)
    s.check(s.queries(0.3), ws, scale=scale)


@pytest.mark.parametrize("heads,dim", [(4, 64), (4, 128), (8, 128), (16, 128), (4, 256), (8, 256)])
@pytest.mark.parametrize("n", [1, 2])
def test_value_scales_far_apart(ws, heads, dim, n):
    """Tokens of one sequence whose value scales lie 2^24 apart, the largest with hardly any weight."""
    s = Scene([300, 40], [n, n], heads, 1, dim, 32, seed=dim + n)
    rng = np.random.default_rng(4)
    pg, tok = s.c.at(s.table, 0, 0, 300)
    s.c.vs[pg, :, tok] = (rng.uniform(1, 2, (300, 1, 1)) * 2.0 ** rng.integers(-13, 12, (300, 1, 1))).astype(np.float16)
    s.place()
    x = s.queries()
    s.check(x, ws, weigh=False)
    # the last of them far larger than all others, with a score far below
    far = 299 - n
    s.c.vs[pg[far], 0, tok[far]] = 3e4
    for codes in (s.c.k,):
        codes[pg[far], 0, tok[far]] = 0
    s.c.ks[pg[far], 0, tok[far]] = 1.0
    x[:] = np.abs(x)
    s.place()
    s.check(x, ws, weigh=False)


@pytest.mark.parametrize("size", [2.0 ** -22, 2.0 ** -14, 2.0 ** -6, 2.0 ** 12])
@pytest.mark.parametrize("heads,dim", [(4, 128), (8, 64), (16, 128)])
def test_values_of_all_sizes(ws, size, heads, dim):
    """The error is relative to the values, from scales that are subnormal in f16 to the largest."""
    s = Scene([2000, 45], [1, 2], heads, 1, dim, 32, seed=heads)
    with np.errstate(invalid="ignore"):
        s.c.vs = (s.c.vs.astype(np.float32) * np.float32(size)).astype(np.float16)
    s.place()
    s.check(s.queries(), ws, weigh=False)


@pytest.mark.parametrize("heads", [4, 8, 16])
def test_groups_far_apart_and_scales_of_zero(ws, heads):
    """Groups of a head 2^10 apart, one whose scales are all zero, and keys of zero."""
    s = Scene([200, 33], [1, 2], heads, 1, 128, 32, seed=heads)
    for i, f in enumerate((1.0, 2.0 ** -10, 0.0, 2.0 ** 6)):
        s.c.vs[..., i] = np.where(np.isnan(s.c.vs[..., i]), np.nan, s.c.vs[..., i] * np.float16(f))
    pg, tok = s.c.at(s.table, 0, 30, 90)
    s.c.ks[pg, :, tok] = 0
    s.place()
    s.check(s.queries(), ws)


@pytest.mark.parametrize("at", ["q", "ks", "vs"])
@pytest.mark.parametrize("heads", [4, 8, 16])
def test_not_finite_stays_where_it_is(ws, at, heads):
    """A NaN or infinite query reaches its own row and head only, a scale only the rows that see its slot."""
    s = Scene([120, 70], [3, 2], heads, 2, 128, 32, seed=11)
    x = s.queries()
    want = s.check(x, ws, weigh=False).reshape(s.T, heads, 128).cpu().numpy()
    hit = np.zeros((s.T, heads), bool)
    G = heads // 2
    for bad in (np.nan, np.inf):
        if at == "q":
            x[1, 2, 5] = bad
            hit[1, 2] = True
        else:  # the last slot but one of sequence 0, head 1: its last two rows see it
            pg, tok = s.table[0][118 // 32], 118 % 32
            (s.c.ks if at == "ks" else s.c.vs)[pg, 1, tok, 2] = bad
            hit[1:3, G:] = True
        s.place()
        lse = torch.zeros((s.T, heads), device=DEV)
        got = q.kv4_attention(s.cache, s.batch, dev(x), 128 ** -0.5, ws, lse=lse).reshape(s.T, heads, 128).cpu().numpy()
        q.get_device_error()
        assert np.array_equal(bits(got[~hit]), bits(want[~hit]))
        if at == "ks" and bad == np.inf:
            continue  # (a score of minus infinity is no weight at all: a finite result is right then)
        if at != "vs":
            assert not np.isfinite(got[hit]).any()
        else:  # in the dimensions of its group at least
            assert not np.isfinite(got[hit][:, 64:96]).any()
            assert np.isfinite(lse.cpu().numpy()).all()


# ---- append and read ---------------------------------------------------------------------------

def append_case(lens, rows, heads, kv, dim, page, seed, rot, halves, with_q, positions, fused=True, extra=0, values=None):
    s = Scene(lens, rows, heads, kv, dim, page, seed=seed, extra_rows=extra)
    rng = s.rng
    wide = rng.standard_normal((s.T, (heads + 2 * kv) * dim)).astype(np.float32)
    if values is not None:
        wide = values(wide)
    k = wide[:, heads * dim:(heads + kv) * dim].reshape(s.T, kv, dim)
    v = wide[:, (heads + kv) * dim:].reshape(s.T, kv, dim)
    x = wide[:, :heads * dim].reshape(s.T, heads, dim) if with_q else None
    top = max(lens) + 60
    rope = q.rope_table(top, rot, 10000.0, device="cpu").numpy() if rot else None
    at = None
    if positions:
        at = np.zeros(s.T, np.int32)
        for i, n in enumerate(lens):
            r0, m = s.q_start[i], rows[i]
            at[r0:r0 + m] = np.arange(n - m, n) + (7 * i + 5) % 55
    want = s.c.copy()
    want_q = P.append(want, s.table, s.lens, s.q_start, k, v, rope, x, rot, halves, at)
    wd = dev(wide)
    kd, vd = wd[:, heads * dim:(heads + kv) * dim], wd[:, (heads + kv) * dim:]
    qd = wd[:, :heads * dim] if with_q else None
    out = torch.full((s.T, heads * dim), np.nan, device=DEV) if with_q else None
    got_q = q.kv4_append(s.cache, s.batch, kd, vd, None if rope is None else dev(rope), qd, out,
                         q.ROPE_HALVES if halves else q.ROPE_ADJACENT, None if at is None else dev(at))
    q.get_device_error()
    for a, b, what in ((s.cache.k, want.k, "keys"), (s.cache.v, want.v, "values")):
        assert np.array_equal(a.cpu().numpy(), b), what
    for a, b, what in ((s.cache.k_scale, want.ks, "key scales"), (s.cache.v_scale, want.vs, "value scales")):
        a = a.cpu().numpy()
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(bits(a)[~np.isnan(b)], bits(b)[~np.isnan(b)]), what
    if with_q:
        g = got_q.reshape(s.T, heads, dim).cpu().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(want_q)) and np.array_equal(g[~np.isnan(g)], want_q[~np.isnan(g)])
    # read back: exact
    s.c = want
    kr, vr = (t.cpu().numpy() for t in q.kv4_read(s.cache, s.batch, torch.full((s.T, kv, dim), np.nan, device=DEV),
                                                   torch.full((s.T, kv, dim), np.nan, device=DEV)))
    q.get_device_error()
    for i, n in enumerate(lens):
        r0, m = s.q_start[i], rows[i]
        wk, wv = want.values(s.table, i, n - m, n)
        assert np.array_equal(kr[r0:r0 + m], wk.astype(np.float32)) and np.array_equal(vr[r0:r0 + m], wv.astype(np.float32))
    assert np.isnan(kr[s.q_start[-1]:]).all()
    return s, k, v


@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (128, 128), (128, 64), (256, 256), (256, 64), (128, 0)])
@pytest.mark.parametrize("halves", [True, False])
@pytest.mark.parametrize("positions", [True, False])
def test_append(dim, rot, halves, positions):
    append_case([1, 17, 40, 90, 33], [1, 3, 40, 33, 17], 4, 2, dim, 32, dim + rot, rot, halves, True, positions and rot > 0)


@pytest.mark.parametrize("heads,kv,dim", [(9, 3, 64), (7, 7, 64), (5, 1, 128), (11, 11, 128), (3, 1, 256), (5, 5, 256)])
def test_append_odd_heads(heads, kv, dim):
    append_case([5, 70], [2, 70], heads, kv, dim, 16, heads, dim, True, True, True, extra=3)
    append_case([5, 70], [2, 70], heads, kv, dim, 16, heads, 0, True, False, False)


def test_append_is_within_half_a_step():
    """... of the scale, a whole step where a value comes within half a step of -top, which has no code."""
    s, k, v = append_case([64], [64], 2, 2, 128, 32, 77, 0, True, False, False)
    got = s.c.values(s.table, 0, 0, 64)[1]
    pg, tok = s.c.at(s.table, 0, 0, 64)
    d = np.repeat(np.abs(s.c.vs[pg, :, tok].astype(np.float64)), 32, -1)
    x = v.astype(np.float64)
    top = np.abs(x.reshape(64, 2, 4, 32)).max(-1).repeat(32, -1).reshape(x.shape)
    err = np.abs(got - x)
    assert (err <= d * 0.5 * (1 + 2.0 ** -9) + top * 2.0 ** -11)[np.abs(x) < 7.4 * d].all()
    assert (err <= d * (1 + 2.0 ** -7)).all()


def test_append_values_of_all_sizes():
    """Zeros, ties between signs (the first counts), scales held at the largest f16, subnormal ones, and none."""
    def values(w):
        w = w.copy()
        w[0] = 0
        w[1] *= 1e7          # d is held at 65504
        w[2] *= 1e-6         # subnormal scales
        w[3] *= 1e-9         # none
        w[4] = np.where(np.arange(w.shape[1]) % 2 == 0, 1.5, -1.5)
        w[5] = np.where(np.arange(w.shape[1]) % 2 == 0, -1.5, 1.5)
        w[6, ::2] = -0.0
        return w
    append_case([9], [9], 2, 2, 64, 32, 3, 0, True, True, False, values=values)


def test_append_in_place_and_without_rows():
    s = Scene([40, 7, 0], [2, 0, 3], 4, 2, 128, 32, seed=4)  # sequence 2 pads the batch
    before = [t.clone() for t in (s.cache.k, s.cache.v, s.cache.k_scale, s.cache.v_scale)]
    x = torch.randn((s.T, 8 * 128), device=DEV)
    x0 = x.clone()
    rope = q.rope_table(64, 128)
    got = q.kv4_append(s.cache, s.batch, x[:, 512:768], x[:, 768:], rope, x[:, :512], x[:, :512])
    q.get_device_error()
    assert got.data_ptr() == x.data_ptr() and not torch.equal(x[:2, :512], x0[:2, :512])
    assert torch.equal(x[2:], x0[2:]) and torch.equal(x[:, 512:], x0[:, 512:])
    pg = int(s.table[0][38 // 32])
    for a, b in zip((s.cache.k, s.cache.v, s.cache.k_scale, s.cache.v_scale), before):
        a, b = a.view(torch.uint8).clone(), b.view(torch.uint8)
        a[pg, :, 6:8] = b[pg, :, 6:8]
        assert torch.equal(a, b), "written outside the two rows' slots"


# ---- eviction ----------------------------------------------------------------------------------

def evict_case(lens, keep, sinks, recent, kv=2, dim=64, page=16, seed=0, weights=None, kept=True):
    s = Scene(lens, [0] * len(lens), 2 * kv, kv, dim, page, seed=seed)
    if weights is not None:
        s.w = weights(s)
        s.place()
    want, w = s.c.copy(), s.w.copy()
    want_len, want_kept = P.evict(want, s.table, lens, w, keep, sinks, recent)
    k = torch.full((len(lens), kv, keep), -7, dtype=torch.int32, device=DEV) if kept else None
    n = q.kv4_evict(s.cache, s.batch, s.weight, keep, sinks, recent, kept=k)
    q.get_device_error()
    assert np.array_equal(n.cpu().numpy(), want_len)
    if kept:
        assert np.array_equal(k.cpu().numpy(), want_kept)
    for a, b in ((s.cache.k, want.k), (s.cache.v, want.v), (s.cache.k_scale.view(torch.int16), want.ks.view(np.int16)),
                 (s.cache.v_scale.view(torch.int16), want.vs.view(np.int16)), (s.weight.view(torch.int32), w.view(np.int32))):
        assert np.array_equal(a.cpu().numpy(), b)
    return s, n


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("keep,sinks,recent", [(40, 4, 8), (33, 0, 0), (17, 17, 0), (16, 0, 16), (1, 0, 0), (1, 1, 0), (50, 20, 29),
                                               (500, 3, 3)])
def test_evict(dim, keep, sinks, recent):
    evict_case([0, 1, 16, 17, 41, 90, 200, 333], keep, sinks, recent, 2, dim, 16 if dim == 64 else 48, seed=keep)


@pytest.mark.parametrize("kv,page,lens,keep", [(1, 64, [5000], 4097), (8, 128, [3000, 1500], 1024), (3, 16, [2100] * 5, 2048),
                                               (2, 32, [40000], 100), (1, 16, [1025, 513, 2049], 512)])
def test_evict_long(kv, page, lens, keep):
    evict_case(lens, keep, 4, min(keep - 4, 300), kv, 64, page, seed=kv)
    evict_case(lens, keep, 0, 0, kv, 64, page, seed=kv, kept=False)


def tied(s):
    """Few different weights, zeros of both signs, and ones that are not numbers."""
    w = s.rng.choice(np.array([0.0, -0.0, 0.5, 1.0, 1.0000001, 3.0], np.float32), s.w.shape)
    w[s.rng.random(w.shape) < 0.05] = np.nan
    w[s.rng.random(w.shape) < 0.05] = np.inf
    w[s.rng.random(w.shape) < 0.05] = -np.inf
    w[s.rng.random(w.shape) < 0.05] = -1.0
    return w


@pytest.mark.parametrize("keep", [20, 100, 290])
def test_evict_ties(keep):
    evict_case([300, 120, 301], keep, 3, 5, 2, 64, 32, seed=keep, weights=tied)
    evict_case([300, 2000], keep, 0, 0, 2, 64, 32, seed=keep, weights=lambda s: np.zeros_like(s.w))
    evict_case([300, 2000], keep, 0, 0, 2, 64, 32, seed=keep, weights=lambda s: np.full_like(s.w, np.nan))


def test_evict_more_than_a_block():
    """More slots than are worked on together, few and many of them kept, ties among them."""
    for keep, weights in ((70, None), (40000, None), (40000, tied)):
        evict_case([50000, 70000], keep, 4, 30, 1, 64, 128, seed=keep, weights=weights)


def test_evict_rising_and_falling():
    """Everything at the front stays, or everything moves."""
    for sign in (1, -1):
        def weights(s):
            w = np.zeros_like(s.w)
            for i, n in enumerate(s.lens):
                pg, tok = s.c.at(s.table, i, 0, n)
                w[pg, :, tok] = (sign * np.arange(n, dtype=np.float32))[:, None]
            return w
        evict_case([700, 1300], 600, 0, 0, 2, 128, 64, weights=weights)


# ---- bad entries, streams, graphs --------------------------------------------------------------

def index_error():
    with pytest.raises(q.QmdError, match="QMD_ERR_INDEX"):
        q.get_device_error()


@pytest.mark.parametrize("what", ["page", "page_low", "len", "len_neg", "start", "rows"])
def test_bad_entries_are_left_out(ws, what):
    s = Scene([70, 40, 33], [1, 2, 1], 4, 2, 128, 32, seed=2)
    x = s.queries()
    good = s.check(x, ws, weigh=False).cpu().numpy()
    if what == "page":
        s.table_d[1, 0] = s.cache.pages
    elif what == "page_low":
        s.table_d[1, 0] = -1
    elif what == "len":
        s.len_d[1] = s.table.shape[1] * 32 + 1
    elif what == "len_neg":
        s.len_d[1] = -1
    elif what == "start":
        s.start_d[2] = 100
    else:
        s.start_d[1] = 3
        s.start_d[2] = 3  # sequence 0 has more than max_q rows
    before = [t.clone() for t in (s.cache.k, s.cache.k_scale)]
    out = torch.full((s.T, 512), 7.0, device=DEV)
    lse = torch.zeros((s.T, 4), device=DEV)
    q.kv4_attention(s.cache, s.batch, dev(x), 128 ** -0.5, ws, out=out, lse=lse)
    index_error()
    got = out.cpu().numpy()
    if what in ("page", "page_low", "len", "len_neg"):
        assert np.array_equal(bits(got[[0, 3]]), bits(good[[0, 3]]))
    q.kv4_weigh(s.cache, s.batch, dev(x), 128 ** -0.5, lse, s.weight)
    index_error()
    if what not in ("page", "page_low"):  # (the rows of the append lie in a good page)
        q.kv4_append(s.cache, s.batch, torch.randn((s.T, 256), device=DEV), torch.randn((s.T, 256), device=DEV))
        index_error()
        q.kv4_read(s.cache, s.batch)
        index_error()
    if what in ("page", "page_low", "len", "len_neg"):
        s.cache.k.copy_(before[0])
        s.cache.k_scale.copy_(before[1])
        kept = torch.zeros((3, 2, 20), dtype=torch.int32, device=DEV)
        n = q.kv4_evict(s.cache, s.batch, s.weight, 20, kept=kept)
        index_error()
        assert n.tolist() == [20, 40 if what in ("page", "page_low") else 0, 20]
        assert (kept[1] == -1).all() and (kept[0] >= 0).all()
        pg, tok = s.c.at(s.table, 1, 0, 40)
        assert np.array_equal(s.cache.k.cpu().numpy()[pg, :, tok], s.c.k[pg, :, tok]), "the bad sequence was touched"


def test_bad_positions():
    s = Scene([30, 9], [2, 2], 4, 2, 64, 32, seed=6)
    before = s.cache.k.clone()
    k = torch.randn((4, 128), device=DEV)
    rope, x = q.rope_table(100, 64), torch.randn((4, 256), device=DEV)
    out = torch.full_like(x, np.nan)
    at = torch.tensor([99, 100, -1, 3], dtype=torch.int32, device=DEV)
    q.kv4_append(s.cache, s.batch, k, k, rope, x, out, positions=at)
    index_error()
    assert out.isnan().all(1).tolist() == [False, True, True, False]
    for slot, s_, stored in ((28, 0, True), (29, 0, False), (7, 1, False), (8, 1, True)):
        pg = int(s.table[s_][slot // 32])
        assert torch.equal(s.cache.k[pg, :, slot % 32], before[pg, :, slot % 32]) != stored
    # a table with too few rows for the slots; without rope positions are not read
    q.kv4_append(s.cache, s.batch, k, k, rope[:10])
    index_error()
    q.kv4_append(s.cache, s.batch, k, k, positions=at)
    q.get_device_error()


def test_same_bits_again_and_in_graphs(ws):
    """The same inputs give the same bits, eager, again, and replayed after lengths and pages changed."""
    s = Scene([3000, 77, 513], [1, 1, 1], 32, 8, 128, 64, seed=12)
    x, w0 = dev(s.queries()), s.weight.clone()
    lse, out = torch.zeros((3, 32), device=DEV), torch.zeros((3, 4096), device=DEV)
    kept, n = torch.zeros((3, 8, 64), dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    own = q.kv_workspace()
    keep = [t.clone() for t in (s.cache.k, s.cache.v, s.cache.k_scale, s.cache.v_scale)]

    def run():
        q.kv4_attention(s.cache, s.batch, x, 128 ** -0.5, own, out=out, lse=lse)
        q.kv4_weigh(s.cache, s.batch, x, 128 ** -0.5, lse, s.weight)
        q.kv4_evict(s.cache, s.batch, s.weight, 64, 4, 16, n, kept)

    def restore():
        for a, b in zip((s.cache.k, s.cache.v, s.cache.k_scale, s.cache.v_scale), keep):
            a.copy_(b)
        s.weight.copy_(w0)

    def result():
        torch.cuda.synchronize()
        return [t.clone().view(torch.uint8) for t in (out, lse, s.weight, kept, n, s.cache.k, s.cache.v)]

    run()
    first = result()
    restore()
    run()
    assert all(torch.equal(a, b) for a, b in zip(first, result()))
    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run()
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, result()))
    s.len_d.copy_(torch.tensor([200, 77, 60], dtype=torch.int32))
    restore()
    g.replay()
    replayed = result()
    restore()
    run()
    assert all(torch.equal(a, b) for a, b in zip(replayed, result()))
    q.get_device_error()


def test_streams_of_their_own():
    """Two streams at once, each with its workspace; outputs made by the call belong to its stream."""
    a, b = (Scene([900, 64 + i], [1, 1], 8, 2, 128, 32, seed=20 + i) for i in range(2))
    xs = [dev(s.queries()) for s in (a, b)]
    wss = [q.kv_workspace() for _ in range(2)]
    want = [q.kv4_attention(s.cache, s.batch, x, 0.1, w) for s, x, w in zip((a, b), xs, wss)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate((a, b)):
            got[i].append(q.kv4_attention(s.cache, s.batch, xs[i], 0.1, wss[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in got[i])
    n = q.kv4_evict(a.cache, a.batch, a.weight, 100, stream=streams[0])
    k, v = q.kv4_read(b.cache, b.batch, stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert n.tolist() == [100, 64] and k.shape == (2, 2, 128)
    q.get_device_error()


# ---- a run of them together --------------------------------------------------------------------

def test_a_request_that_is_kept_short(ws):
    """A prompt is appended, its last rows weigh it, it is thinned out, and decoding goes on with positions that
    run ahead of the slots; every step against the formulas, on the cache as the calls left it."""
    heads, kv, dim, page, keep = 8, 2, 128, 16, 48
    rng = np.random.default_rng(0)
    table = rng.permutation(40)[:20].reshape(2, 10).astype(np.int32)
    cache = q.KV4Cache.empty(40, kv, page, dim)
    weight, ws = cache.new_weights(), q.kv_workspace()
    rope = q.rope_table(400, dim)
    lens, gone = [120, 70], [0, 0]

    def rows(n):
        return dev(rng.standard_normal((sum(n), (heads + 2 * kv) * dim)).astype(np.float32))

    def step(x, n, weigh_last=None):
        start = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
        length = dev(np.array(lens, np.int32))
        batch = q.KVBatch(dev(table), length, dev(start), max(n), sum(n))
        at = np.concatenate([np.arange(l - m, l) + g for l, m, g in zip(lens, n, gone)]).astype(np.int32)  # noqa: E741
        qr = q.kv4_append(cache, batch, x[:, heads * dim:(heads + kv) * dim], x[:, (heads + kv) * dim:], rope, x[:, :heads * dim],
                          positions=dev(at))
        lse = torch.full((sum(n), heads), np.nan, device=DEV)
        out = q.kv4_attention(cache, batch, qr, dim ** -0.5, ws, lse=lse)
        host = P.Cache(*(t.cpu().numpy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
        xq = qr.reshape(-1, heads, dim).cpu().numpy()
        ref, bound, lref, lbound = P.attention(host, table, lens, start, xq, dim ** -0.5)
        close(out.reshape(ref.shape).cpu().numpy(), ref, bound, "attention")
        close(lse.cpu().numpy(), lref, lbound, "log-sum-exp")
        if weigh_last:  # only the last rows of the prompt, over weights of zero
            pick = np.concatenate([np.arange(e - weigh_last, e) for e in start[1:]])
            start = (np.arange(len(n) + 1) * weigh_last).astype(np.int32)
            batch = q.KVBatch(dev(table), length, max_q=weigh_last)
            qr, lse, xq = qr[dev(pick)].contiguous(), lse[dev(pick)].contiguous(), xq[pick]
        old = weight.cpu().numpy()
        q.kv4_weigh(cache, batch, qr, dim ** -0.5, lse, weight)
        wref, wbound = P.weigh(host, table, lens, start, xq, dim ** -0.5, lse.cpu().numpy(), old)
        close(weight.cpu().numpy(), wref, wbound, "weights")
        host_w = weight.cpu().numpy()
        n_d = q.kv4_evict(cache, batch, weight, keep, 2, 16)
        new, _ = P.evict(host, table, lens, host_w, keep, 2, 16)
        assert n_d.tolist() == new.tolist()
        for a, b in ((cache.k, host.k), (cache.v, host.v), (weight, host_w)):
            assert np.array_equal(a.cpu().numpy(), b)
        for i in range(2):
            gone[i] += lens[i] - int(new[i])
            lens[i] = int(new[i])

    step(rows(lens), list(lens), weigh_last=5)
    assert lens == [48, 48] and gone == [72, 22]
    for i in range(6):
        n = [1, 1] if i % 2 else [3, 1]
        lens = [l + m for l, m in zip(lens, n)]  # noqa: E741
        step(rows(n), n)
    q.get_device_error()
