"""What the binding makes of arguments before the library sees them (no GPU needed but for one)."""
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402


def test_rope_table_from_a_parameter():
    """A model's own frequencies: a parameter that wants gradients."""
    freq = torch.nn.Parameter(torch.tensor([1.0, 0.25]))
    t = q.rope_table(5, 4, inv_freq=freq, device="cpu")
    assert not t.requires_grad and torch.equal(t, q.rope_table(5, 4, inv_freq=[1.0, 0.25], device="cpu"))


def test_counts_past_the_c_types_are_refused(monkeypatch):
    """ctypes takes numbers modulo their type: max_q = 2^32 + 1 was 1, a window of 2^64 none."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for kw in (dict(max_q=(1 << 32) + 1, rows=5), dict(max_q=1, rows=(1 << 64) + 5)):
        with pytest.raises(q.QmdError, match="SHAPE"):
            q.KVBatch(i32(2, 3), i32(2), i32(3), **kw)
    monkeypatch.setattr(q, "_stream_on", lambda stream, index, what: 0)
    cache, batch, x = q.KVCache.empty(3, 2, 16, 64, "cpu"), q.KVBatch(i32(2, 3), i32(2)), torch.zeros((2, 2, 64))
    for window in (1 << 64, -1):
        with pytest.raises(q.QmdError, match="VALUE"):
            q.kv_attention(cache, batch, x, 0.1, i32(1), window=window)
    for pairs in (1 << 32, 2, -1):
        with pytest.raises(q.QmdError, match="VALUE"):
            q.kv_append(cache, batch, x, x, pairs=pairs)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_rope_table_from_frequencies_on_the_gpu():
    t = q.rope_table(5, 4, inv_freq=torch.tensor([1.0, 0.25], device="cuda"))
    assert torch.equal(t.cpu(), q.rope_table(5, 4, inv_freq=[1.0, 0.25], device="cpu"))
