"""Refusals of the key/value cache calls and the adapters: named statuses before anything touches
the device (no GPU needed)."""
import ctypes

import pytest

import quantised_decode_mat_gb300 as q
from quantised_decode_mat_gb300 import build as qbuild

A = 0x10000  # aligned fake device addresses: validation must fail before any of them is used
STEP = 1 << 30


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return q.lib()


def cache(**kw):
    f = dict(k=A, v=A + STEP, k_scale=A + 2 * STEP, v_scale=A + 3 * STEP, pages=10, kv_heads=2, page_tokens=32, head_dim=128)
    f.update(kw)
    return q.KVCachePtrs(*[f[n] for n, _ in q.KVCachePtrs._fields_])


def batch(**kw):
    f = dict(page_table=A, kv_len=A, q_start=A, table_stride=4, rows=5, seqs=3, max_q=2)
    f.update(kw)
    return q.KVBatchPtrs(*[f[n] for n, _ in q.KVBatchPtrs._fields_])


BAD_CACHE = [(dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(k=A + 8), 5),
             (dict(v=A + 4), 5), (dict(k_scale=A + 2), 5), (dict(pages=0), 6), (dict(pages=1 << 31), 6),
             (dict(kv_heads=0), 6), (dict(kv_heads=1025), 6), (dict(page_tokens=0), 6), (dict(page_tokens=24), 6),
             (dict(page_tokens=65552), 6), (dict(head_dim=96), 6), (dict(head_dim=0), 6)]
BAD_BATCH = [(dict(page_table=None), 1), (dict(kv_len=None), 1), (dict(seqs=0), 6), (dict(seqs=2049), 6), (dict(max_q=0), 6),
             (dict(max_q=(1 << 20) + 1), 6), (dict(rows=0), 6), (dict(rows=(1 << 24) + 1), 6), (dict(table_stride=0), 6),
             (dict(q_start=None), 6),  # three sequences of two rows in five rows
             (dict(kv_len=A + 2), 5), (dict(page_table=A + 1), 5), (dict(q_start=A + 2), 5)]


def st_append(L, c=None, b=None, k=A, ks=256, v=A + STEP, vs=256, x=A + 2 * STEP, xs=512, heads=4, o=A + 3 * STEP, os_=512,
              rope=A, n=100, rot=128, pairs=0):
    return L.qmd_kv_append(c or cache(), b or batch(), k, ks, v, vs, x, xs, heads, o, os_, rope, n, rot, pairs, None)


def st_read(L, c=None, b=None, k=A, ks=256, v=A + STEP, vs=256):
    return L.qmd_kv_read(c or cache(), b or batch(), k, ks, v, vs, None)


def st_attn(L, c=None, b=None, x=A, xs=512, heads=4, scale=0.1, window=0, o=A + STEP, os_=512, ws=A):
    return L.qmd_kv_attention(c or cache(), b or batch(), x, xs, heads, scale, window, o, os_, ws, None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_caches(L, kw, status):
    assert st_append(L, cache(**kw)) == status
    assert st_read(L, cache(**kw)) == status
    assert st_attn(L, cache(**kw)) == status


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_batches(L, kw, status):
    assert st_append(L, b=batch(**kw)) == status
    assert st_read(L, b=batch(**kw)) == status
    assert st_attn(L, b=batch(**kw)) == status


def test_no_struct(L):
    assert L.qmd_kv_read(None, batch(), A, 256, A + STEP, 256, None) == 1
    assert L.qmd_kv_read(cache(), None, A, 256, A + STEP, 256, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=A + 4), 5), (dict(v=A + 8), 5), (dict(ks=255), 6), (dict(ks=258), 6),
    (dict(vs=128), 6), (dict(x=None), 10), (dict(o=None), 10), (dict(heads=0), 10), (dict(heads=-1), 6), (dict(xs=510), 6),
    (dict(os_=508), 6), (dict(x=A + 4), 5), (dict(o=A + 8), 5), (dict(rope=A + 4), 5), (dict(rot=0), 6), (dict(rot=48), 6),
    (dict(rot=160), 6), (dict(n=0), 6), (dict(rope=None), 6), (dict(pairs=2), 10),
    # q_out may be q with q's stride, and overlaps nothing else
    (dict(o=A + 2 * STEP, os_=516), 10), (dict(o=A + 2 * STEP + 16), 10), (dict(o=A + 64), 10), (dict(o=A + STEP), 10),
])
def test_append_refusals(L, kw, status):
    assert st_append(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None, v=None), 1), (dict(k=A + 4), 5), (dict(v=A + 8), 5), (dict(ks=252), 6), (dict(vs=257), 6),
    (dict(v=A + 256), 10)])
def test_read_refusals(L, kw, status):
    assert st_read(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(o=None), 1), (dict(ws=None), 1), (dict(heads=3), 6), (dict(heads=0), 6), (dict(heads=130), 6),
    (dict(xs=508), 6), (dict(os_=513), 6), (dict(x=A + 4), 5), (dict(o=A + STEP + 8), 5), (dict(ws=A + 8), 5),
    (dict(scale=float("nan")), 10), (dict(scale=float("inf")), 10), (dict(window=-1), 10), (dict(o=A), 10),
    (dict(o=A + 512 * 4), 10)])
def test_attention_refusals(L, kw, status):
    assert st_attn(L, **kw) == status


def st_lora(L, type_=q.F16, x=A, base=A + STEP, a=A, b=A, scale=A, adapter=A, out=A + 2 * STEP, K=512, rows=100, rank=16,
            n=4, B=2):
    return L.qmd_lora_add(type_, x, base, a, b, scale, adapter, out, K, rows, rank, n, B, None)


@pytest.mark.parametrize("kw,status", [
    (dict(type_=0), 2), (dict(type_=3), 2), (dict(x=None), 1), (dict(base=None), 1), (dict(a=None), 1), (dict(b=None), 1),
    (dict(scale=None), 1), (dict(adapter=None), 1), (dict(out=None), 1), (dict(K=0), 6), (dict(K=300), 3),
    (dict(K=65792), 6), (dict(B=0), 4), (dict(B=9), 4), (dict(rows=0), 6), (dict(rank=0), 6), (dict(rank=12), 6),
    (dict(rank=136), 6), (dict(n=0), 6), (dict(x=A + 4), 5), (dict(a=A + 8), 5), (dict(b=A + 2), 5), (dict(base=A + STEP + 2), 5),
    (dict(out=A + 2 * STEP + 1), 5), (dict(adapter=A + 2), 5), (dict(out=A), 10), (dict(out=A + STEP + 4), 10)])
def test_adapter_refusals(L, kw, status):
    assert st_lora(L, **kw) == status


def test_valid_arguments_reach_the_device_check(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    assert st_append(L) == 9
    assert st_append(L, x=None, o=None, heads=0, rope=None, rot=0) == 9
    assert st_append(L, o=A + 2 * STEP) == 9  # in place
    assert st_read(L) == 9 and st_read(L, k=None) == 9
    assert st_read(L, cache(k=None, k_scale=None), k=None) == 9
    assert st_attn(L) == 9 and st_attn(L, b=batch(q_start=None, rows=6)) == 9 and st_attn(L, heads=128, xs=1 << 14, os_=1 << 14) == 9
    assert st_lora(L) == 9 and st_lora(L, out=A + STEP) == 9
    assert L.qmd_kv_workspace_bytes() == 0


def test_python_side_refuses_what_the_library_cannot_see():
    import torch
    k = torch.zeros((3, 2, 32, 64), dtype=torch.int8)
    s = torch.zeros((3, 2, 2))
    t, n = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    c, b = q.KVCache(k, k, s, s), q.KVBatch(t, n)
    for bad in ((k.float(), k, s, s), (k, k[:, :1], s, s), (k, k, s.double(), s), (k, k, s[:, :, :1], s),
                (k.transpose(0, 1), k, s, s)):
        with pytest.raises(q.QmdError):
            q.KVCache(*bad)
    for bad in ((t.long(), n), (t, n[:1]), (t[0], n), (t, n, torch.zeros(2, dtype=torch.int32), 1, 2),
                (t, n, torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(q.QmdError):
            q.KVBatch(*bad)
    with pytest.raises(q.QmdError, match="QMD_ERR_DEVICE"):
        q.kv_attention(c, b, torch.zeros((2, 4, 64)), 0.1, n)
    with pytest.raises(q.QmdError, match="QMD_ERR_DEVICE"):
        q.kv_append(c, b, torch.zeros((2, 2, 64)), torch.zeros((2, 2, 64)))
    with pytest.raises(q.QmdError, match="QMD_ERR_DEVICE"):
        q.lora_add(torch.zeros((1, 256)), torch.zeros((1, 8)), torch.zeros((1, 8, 256)), torch.zeros((1, 8, 8)), n[:1], torch.zeros(1))
    rows = torch.zeros((2, 4 * 64 + 8))
    assert q._rows_of(rows[:, :256], 2, 4, 64, -1, "x") == (4, 264)
    for bad in (rows[:, :250], rows[:1, :256], rows[:, :256].double(), rows[:, 0:256:2], rows[:, :256].unflatten(1, (4, 64)).transpose(1, 2)):
        with pytest.raises(q.QmdError):
            q._rows_of(bad, 2, None, 64, -1, "x")


def test_rope_table():
    import math
    t = q.rope_table(70000, 64, 10000.0, device="cpu")
    assert t.shape == (70000, 64)
    for p, i in ((0, 0), (1, 0), (69999, 0), (69999, 31), (12345, 7)):
        a = p * 10000.0 ** (-2 * i / 64)
        assert abs(t[p, i] - math.cos(a)) <= 2.0 ** -25 + 1e-10 and abs(t[p, 32 + i] - math.sin(a)) <= 2.0 ** -25 + 1e-10
    assert q.rope_table(3, 4, inv_freq=[1.0, 0.5], device="cpu")[2, 1] == pytest.approx(math.cos(1.0), abs=1e-7)
    with pytest.raises(q.QmdError):
        q.rope_table(3, 4, inv_freq=[1.0], device="cpu")
