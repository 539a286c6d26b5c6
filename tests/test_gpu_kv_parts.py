"""Row tensors that are parts of one wider buffer give what separate tensors give, and what lies between
and behind them stays as it was; keys or values read alone."""
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from tests.test_gpu_kv import Scene, dev, rope_np  # noqa: E402

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


def scene(seed):
    return Scene([40, 17, 90], [5, 1, 2], 8, 2, 128, 32, seed=seed, extra_rows=1)


def test_keys_and_values_read_into_one_buffer():
    s = scene(1)
    w = 2 * 128
    k, v = (torch.full((s.T, w), 5.0, device=DEV) for _ in "kv")
    q.kv_read(s.cache, s.batch, k, v)
    for a, b, width in ((0, w, 2 * w), (w, 0, 2 * w), (8, w + 16, 2 * w + 24)):
        buf = torch.full((s.T, width), 5.0, device=DEV)
        q.kv_read(s.cache, s.batch, buf[:, a:a + w], buf[:, b:b + w])
        q.get_device_error()
        want = torch.full_like(buf, 5.0)
        want[:, a:a + w], want[:, b:b + w] = k, v
        assert torch.equal(buf, want)


def test_attention_beside_its_queries():
    s = scene(2)
    x = dev(s.queries()).view(s.T, -1)
    ws = q.kv_workspace()
    want = q.kv_attention(s.cache, s.batch, x, 0.1, ws, out=torch.full_like(x, 5.0))
    buf = torch.full((s.T, 2 * 1024 + 32), 5.0, device=DEV)
    buf[:, :1024] = x
    q.kv_attention(s.cache, s.batch, buf[:, :1024], 0.1, ws, out=buf[:, 1024:2048])
    q.get_device_error()
    assert torch.equal(buf[:, :1024], x) and torch.equal(buf[:, 1024:2048], want) and (buf[:, 2048:] == 5).all()


def test_queries_rotated_into_the_buffer_of_keys_and_values():
    rope = dev(rope_np(100, 128))
    results = []
    for fused in (False, True):
        s = scene(3)
        qkv = torch.full((s.T, 12 * 128), 5.0, device=DEV)
        x = dev(s.queries()).view(s.T, -1)
        qkv[:, 1024:] = torch.randn((s.T, 512), device=DEV, generator=torch.Generator(DEV).manual_seed(3))
        k, v = qkv[:, 1024:1280], qkv[:, 1280:]
        if not fused:
            k, v = k.clone(), v.clone()
        o = qkv[:, :1024] if fused else torch.full((s.T, 1024), 5.0, device=DEV)
        q.kv_append(s.cache, s.batch, k, v, rope, x, o)
        q.get_device_error()
        results.append([o.clone(), qkv[:, 1024:].clone(), s.cache.k, s.cache.v])
    assert all(torch.equal(a, b) for a, b in zip(*results)) and (results[0][0][-1] == 5).all()


def test_keys_or_values_read_alone():
    s = scene(4)
    k, v = q.kv_read(s.cache, s.batch)
    own = s.T - 1  # the last row is no sequence's
    a, none = q.kv_read(s.cache, s.batch, values=False)
    assert none is None and torch.equal(a[:own], k[:own])
    none, b = q.kv_read(s.cache, s.batch, keys=False)
    assert none is None and torch.equal(b[:own], v[:own])
    out = torch.full_like(v, 5.0)
    assert q.kv_read(s.cache, s.batch, v_out=out, keys=False)[1] is out
    q.get_device_error()
    assert torch.equal(out[:own], v[:own]) and (out[own] == 5).all()
    for bad in (dict(keys=False, values=False), dict(keys=False, k_out=out), dict(values=False, v_out=out)):
        with pytest.raises(q.QmdError):
            q.kv_read(s.cache, s.batch, **bad)
