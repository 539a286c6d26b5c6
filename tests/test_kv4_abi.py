"""Refusals of the 4-bit cache's calls: named statuses before anything touches the device (no GPU needed)."""
import pytest

import quantised_decode_mat_gb300 as q
from quantised_decode_mat_gb300 import build as qbuild
from tests.test_kv_abi import A, BAD_BATCH, BAD_CACHE, STEP, batch

W = A + 8 * STEP  # weights


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return q.lib()


def cache(**kw):
    f = dict(k=A, v=A + STEP, k_scale=A + 2 * STEP, v_scale=A + 3 * STEP, pages=10, kv_heads=2, page_tokens=32, head_dim=128)
    f.update(kw)
    return q.KV4CachePtrs(*[f[n] for n, _ in q.KV4CachePtrs._fields_])


def st_append(L, c=None, b=None, k=A, ks=256, v=A + STEP, vs=256, x=A + 2 * STEP, xs=512, heads=4, o=A + 3 * STEP, os_=512,
              rope=A, n=100, rot=128, pairs=0, at=A + 4 * STEP):
    return L.qmd_kv4_append(c or cache(), b or batch(), k, ks, v, vs, x, xs, heads, o, os_, rope, n, rot, pairs, at, None)


def st_read(L, c=None, b=None, k=A, ks=256, v=A + STEP, vs=256):
    return L.qmd_kv4_read(c or cache(), b or batch(), k, ks, v, vs, None)


def st_attn(L, c=None, b=None, x=A, xs=512, heads=4, scale=0.1, window=0, o=A + STEP, os_=512, lse=A + 2 * STEP, ws=A):
    return L.qmd_kv4_attention(c or cache(), b or batch(), x, xs, heads, scale, window, o, os_, lse, ws, None)


def st_weigh(L, c=None, b=None, x=A, xs=512, heads=4, scale=0.1, window=0, lse=A + STEP, w=W):
    return L.qmd_kv4_weigh(c or cache(), b or batch(), x, xs, heads, scale, window, lse, w, None)


def st_evict(L, c=None, b=None, w=W, keep=40, sinks=4, recent=8, out=A + STEP, kept=A + 2 * STEP):
    return L.qmd_kv4_evict(c or cache(), b or batch(), w, keep, sinks, recent, out, kept, None)


ALL = (st_append, st_read, st_attn, st_evict)


@pytest.mark.parametrize("kw,status", [c for c in BAD_CACHE if "k_scale" not in c[0] or c[0]["k_scale"] is None] + [
    (dict(k_scale=A + 8), 5), (dict(v_scale=A + 4), 5)])
def test_caches(L, kw, status):
    for call in ALL:
        assert call(L, cache(**kw)) == status
    if not any(f in kw for f in ("v", "v_scale")):
        assert st_weigh(L, cache(**kw)) == status


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_batches(L, kw, status):
    for call in ALL[:3] + (st_weigh,):
        assert call(L, b=batch(**kw)) == status
    if not any(f in kw for f in ("rows", "max_q", "q_start")):  # what eviction does not read
        assert st_evict(L, b=batch(**kw)) == status


def test_no_struct(L):
    assert st_read(L, None, q.KVBatchPtrs()) == 1
    for call, args in ((L.qmd_kv4_read, (A, 256, A + STEP, 256, None)), (L.qmd_kv4_evict, (W, 4, 0, 0, A, None, None)),
                       (L.qmd_kv4_weigh, (A, 512, 4, 0.1, 0, A, W, None))):
        assert call(None, batch(), *args) == 1
        assert call(cache(), None, *args) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=A + 4), 5), (dict(v=A + 8), 5), (dict(ks=255), 6), (dict(ks=258), 6),
    (dict(vs=128), 6), (dict(x=None), 10), (dict(o=None), 10), (dict(heads=0), 10), (dict(heads=-1), 6), (dict(xs=510), 6),
    (dict(os_=508), 6), (dict(x=A + 4), 5), (dict(o=A + 8), 5), (dict(rope=A + 4), 5), (dict(rot=0), 6), (dict(rot=48), 6),
    (dict(rot=160), 6), (dict(n=0), 6), (dict(rope=None), 6), (dict(pairs=2), 10), (dict(at=A + 4 * STEP + 2), 5),
    (dict(o=A + 2 * STEP, os_=516), 10), (dict(o=A + 2 * STEP + 16), 10), (dict(o=A + 64), 10), (dict(o=A + STEP), 10),
    (dict(o=A + 4 * STEP), 10), (dict(at=A + 3 * STEP + 2048 * 4), 10)])
def test_append_refusals(L, kw, status):
    assert st_append(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None, v=None), 1), (dict(k=A + 4), 5), (dict(v=A + 8), 5), (dict(ks=252), 6), (dict(vs=257), 6),
    (dict(v=A + 256), 10)])
def test_read_refusals(L, kw, status):
    assert st_read(L, **kw) == status


QUERIES = [(dict(x=None), 1), (dict(heads=3), 6), (dict(heads=0), 6), (dict(heads=130), 6), (dict(xs=508), 6), (dict(x=A + 4), 5),
           (dict(scale=float("nan")), 10), (dict(scale=float("inf")), 10), (dict(window=-1), 10)]


@pytest.mark.parametrize("kw,status", QUERIES + [
    (dict(o=None), 1), (dict(ws=None), 1), (dict(os_=513), 6), (dict(o=A + STEP + 8), 5), (dict(ws=A + 8), 5),
    (dict(lse=A + 2 * STEP + 2), 5), (dict(o=A), 10), (dict(o=A + 512 * 4), 10), (dict(lse=A + 16), 10),
    (dict(lse=A + STEP + 16), 10)])
def test_attention_refusals(L, kw, status):
    assert st_attn(L, **kw) == status


@pytest.mark.parametrize("kw,status", QUERIES + [
    (dict(lse=None), 1), (dict(w=None), 1), (dict(lse=A + STEP + 2), 5), (dict(w=W + 4), 5), (dict(w=A), 10),
    (dict(w=A + STEP), 10)])
def test_weigh_refusals(L, kw, status):
    assert st_weigh(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), 1), (dict(out=None), 1), (dict(w=W + 4), 5), (dict(out=A + STEP + 2), 5), (dict(kept=A + 1), 5),
    (dict(keep=0), 10), (dict(keep=(1 << 24) + 1), 10), (dict(sinks=-1), 10), (dict(recent=-1), 10),
    (dict(sinks=33), 10), (dict(recent=37), 10), (dict(sinks=1 << 40), 10), (dict(recent=1 << 62, sinks=1 << 62), 10),
    (dict(out=A), 10), (dict(out=A + 8), 10), (dict(kept=A), 10), (dict(kept=A + STEP + 8), 10)])
def test_evict_refusals(L, kw, status):
    assert st_evict(L, **kw) == status


def test_valid_arguments_reach_the_device_check(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    assert st_append(L) == 9 and st_append(L, at=None) == 9
    assert st_append(L, x=None, o=None, heads=0, rope=None, rot=0, at=None) == 9
    assert st_append(L, o=A + 2 * STEP) == 9  # in place
    assert st_read(L) == 9 and st_read(L, k=None) == 9
    assert st_read(L, cache(k=None, k_scale=None), k=None) == 9
    assert st_attn(L) == 9 and st_attn(L, lse=None) == 9
    assert st_attn(L, heads=128, xs=1 << 14, os_=1 << 14) == 9
    assert st_weigh(L) == 9 and st_weigh(L, cache(v=None, v_scale=None)) == 9
    assert st_evict(L) == 9 and st_evict(L, kept=None) == 9 and st_evict(L, keep=12) == 9
    assert st_evict(L, b=batch(rows=0, max_q=0, q_start=None)) == 9


def test_python_side_refuses_what_the_library_cannot_see(monkeypatch):
    import torch
    k = torch.zeros((3, 2, 32, 32), dtype=torch.uint8)
    s = torch.zeros((3, 2, 32, 2), dtype=torch.float16)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    c, b = q.KV4Cache(k, k, s, s), q.KVBatch(i32(2, 3), i32(2))
    assert c.head_dim == 64 and c.new_weights().shape == (3, 2, 32)
    e = q.KV4Cache.empty(3, 2, 16, 128, "cpu")
    assert e.k.shape == (3, 2, 16, 64) and e.v_scale.shape == (3, 2, 16, 4)
    for bad in ((k.char(), k, s, s), (k, k[:, :1], s, s), (k, k, s.float(), s), (k, k, s[..., :1], s),
                (k.transpose(0, 1), k, s, s), (k[0], k[0], s[0], s[0])):
        with pytest.raises(q.QmdError):
            q.KV4Cache(*bad)
    x, r, w = torch.zeros((2, 4, 64)), torch.zeros((2, 2, 64)), c.new_weights()
    with pytest.raises(q.QmdError, match="QMD_ERR_DEVICE"):
        q.kv4_attention(c, b, x, 0.1, i32(1))
    monkeypatch.setattr(q, "_stream_on", lambda stream, index, what: 0)
    eight = q.KVCache.empty(3, 2, 16, 64, "cpu")
    lse = torch.zeros((2, 4))
    for call in (lambda c: q.kv4_append(c, b, r, r), lambda c: q.kv4_read(c, b), lambda c: q.kv4_weigh(c, b, x, 0.1, lse, w),
                 lambda c: q.kv4_attention(c, b, x, 0.1, i32(1)), lambda c: q.kv4_evict(c, b, w, 4)):
        with pytest.raises(q.QmdError, match="FORMAT"):
            call(eight)
    for match, call in (("SHAPE", lambda: q.kv4_append(c, b, r, r, positions=i32(3))),
                        ("FORMAT", lambda: q.kv4_append(c, b, r, r, positions=i32(2).long())),
                        ("VALUE", lambda: q.kv4_append(c, b, r, r, pairs=1 << 32)),
                        ("SHAPE", lambda: q.kv4_weigh(c, b, x, 0.1, lse[:1], w)),
                        ("FORMAT", lambda: q.kv4_weigh(c, b, x, 0.1, lse.double(), w)),
                        ("SHAPE", lambda: q.kv4_weigh(c, b, x, 0.1, lse, w[:, :1])),
                        ("VALUE", lambda: q.kv4_weigh(c, b, x, 0.1, lse, w, window=1 << 64)),
                        ("VALUE", lambda: q.kv4_attention(c, b, x, 0.1, i32(1), window=-1)),
                        ("SHAPE", lambda: q.kv4_evict(c, b, w, 4, kept=i32(2, 2, 5))),
                        ("SHAPE", lambda: q.kv4_evict(c, b, w, 4, len_out=i32(3))),
                        ("FORMAT", lambda: q.kv4_evict(c, b, w.double(), 4)),
                        ("VALUE", lambda: q.kv4_evict(c, b, w, (1 << 64) + 4)),
                        ("VALUE", lambda: q.kv4_evict(c, b, w, 4, sinks=-1))):
        with pytest.raises(q.QmdError, match=match):
            call()
