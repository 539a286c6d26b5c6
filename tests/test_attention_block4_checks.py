"""AttentionBlock over a 4-bit cache: which calls it makes, and what it refuses before any of them (no GPU
needed: the calls are replaced)."""
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from quantised_decode_mat_gb300 import step as S  # noqa: E402
from tests.test_attention_block_checks import D, HIDDEN, KV, ROWS, batch, block  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("qmatvec_x", "lora_add", "kv_append", "kv_attention", "kv4_append", "kv4_attention", "kv4_weigh", "kv4_evict"):
        monkeypatch.setattr(S, name, lambda *a, _n=name, **k: seen.append(_n))
    monkeypatch.setattr(S, "kv_workspace", lambda device: torch.zeros(4, dtype=torch.int32))
    return seen


def test_the_calls_of_each_cache(calls):
    x, four = torch.zeros((ROWS, HIDDEN)), q.KV4Cache.empty(4, KV, 16, D, "cpu")
    block(cache=four).run(x, batch())
    assert calls == ["qmatvec_x", "kv4_append", "kv4_attention", "qmatvec_x"]
    calls.clear()
    b = block(cache=four, weights=four.new_weights())
    b.run(x, batch(), positions=torch.zeros(ROWS, dtype=torch.int32))
    b.evict(batch(), 4)
    assert calls == ["qmatvec_x", "kv4_append", "kv4_attention", "kv4_weigh", "qmatvec_x", "kv4_evict"]
    calls.clear()
    block().run(x, batch())
    assert calls == ["qmatvec_x", "kv_append", "kv_attention", "qmatvec_x"]


def test_what_is_refused(calls):
    x, four = torch.zeros((ROWS, HIDDEN)), q.KV4Cache.empty(4, KV, 16, D, "cpu")
    with pytest.raises(q.QmdError, match="VALUE"):
        block().run(x, batch(), positions=torch.zeros(ROWS, dtype=torch.int32))
    for bad in (torch.zeros(ROWS + 1, dtype=torch.int32), torch.zeros(ROWS)):
        with pytest.raises(q.QmdError, match="SHAPE"):
            block(cache=four).run(x, batch(), positions=bad)
    with pytest.raises(q.QmdError, match="FORMAT"):
        block(weights=four.new_weights())
    with pytest.raises(q.QmdError, match="NULL"):
        block(cache=four).evict(batch(), 4)
    with pytest.raises(q.QmdError, match="VALUE"):
        S.make_attention_block(1, 1, 16, 4, 2, 64, 256, kv_bits=3, device="cpu")
    assert calls == []
