"""What AttentionBlock refuses before anything is launched: its mat-vecs take addresses, so rows, types
and sizes that do not fit its buffers must not reach them (no GPU needed: the calls are replaced)."""
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from quantised_decode_mat_gb300 import step as S  # noqa: E402

HEADS, KV, D, HIDDEN, ROWS = 4, 2, 64, 512, 3
WIDTH = (HEADS + 2 * KV) * D


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("qmatvec_x", "lora_add", "kv_append", "kv_attention"):
        monkeypatch.setattr(S, name, lambda *a, _n=name, **k: seen.append(_n))
    monkeypatch.setattr(S, "kv_workspace", lambda device: torch.zeros(4, dtype=torch.int32))
    return seen


def weights(rows, K):
    return torch.zeros((rows, K // 256 * 144), dtype=torch.uint8)


def block(**kw):
    f = dict(heads=HEADS, W_qkv=weights(WIDTH, HIDDEN), W_o=weights(HIDDEN, HEADS * D), rope=None,
             cache=q.KVCache.empty(4, KV, 16, D, "cpu"), rows=ROWS, hidden=HIDDEN)
    f.update(kw)
    return S.AttentionBlock(**f)


def batch(rows=ROWS):
    return q.KVBatch(torch.zeros((ROWS, 2), dtype=torch.int32), torch.ones(ROWS, dtype=torch.int32),
                     torch.arange(ROWS + 1, dtype=torch.int32), 1, rows)


def test_a_call_that_fits_runs_every_stage(calls):
    b = block()
    assert b.run(torch.zeros((ROWS, HIDDEN)), batch()) is b.y
    assert b.run(torch.zeros((ROWS, HIDDEN)), batch(2)) is b.y  # rows behind the batch's
    assert b.run(torch.zeros((2, HIDDEN)), batch(2)) is b.y
    assert calls == ["qmatvec_x", "kv_append", "kv_attention", "qmatvec_x"] * 3


@pytest.mark.parametrize("x,rows,status", [
    (torch.zeros((ROWS + 1, HIDDEN)), ROWS, "SHAPE"),          # would write past the block's rows
    (torch.zeros((ROWS + 1, HIDDEN)), ROWS + 1, "SHAPE"),
    (torch.zeros((ROWS, HIDDEN)), ROWS + 1, "SHAPE"),
    (torch.zeros((ROWS - 1, HIDDEN)), ROWS, "SHAPE"),
    (torch.zeros((ROWS, 2 * HIDDEN)), ROWS, "SHAPE"),          # would read past the weights
    (torch.zeros((ROWS, 2 * HIDDEN))[:, ::2], ROWS, "SHAPE"),
    (torch.zeros((ROWS, 2 * HIDDEN))[:, :HIDDEN], ROWS, "SHAPE"),
    (torch.zeros((1, HIDDEN)).expand(ROWS, HIDDEN), ROWS, "SHAPE"),
    (torch.zeros(ROWS * HIDDEN), ROWS, "SHAPE"),
    (torch.zeros((ROWS, HIDDEN), dtype=torch.float16), ROWS, "FORMAT"),
    (torch.zeros((ROWS, HIDDEN), device="meta"), ROWS, "DEVICE"),
])
def test_rows_that_do_not_fit(calls, x, rows, status):
    with pytest.raises(q.QmdError, match=status):
        block().run(x, batch(rows))
    assert not calls


def test_adapters_need_a_choice_for_every_row(calls):
    a = S.Adapters(torch.zeros((2, 8, HIDDEN)).half(), torch.zeros((2, WIDTH, 8)).half(), torch.ones(2))
    b, x = block(qkv_adapters=a), torch.zeros((ROWS, HIDDEN))
    for bad, status in ((None, "NULL"), (torch.zeros(ROWS - 1, dtype=torch.int32), "SHAPE")):
        with pytest.raises(q.QmdError, match=status):
            b.run(x, batch(), bad)
    with pytest.raises(q.QmdError, match="SHAPE"):
        b.run(x[:2], batch(2), torch.zeros(2, dtype=torch.int32))
    assert not calls
    b.run(x, batch(), torch.zeros(ROWS, dtype=torch.int32))
    assert calls[:2] == ["qmatvec_x", "lora_add"]


@pytest.mark.parametrize("kw,status", [
    (dict(W_qkv=weights(WIDTH - 1, HIDDEN)), "SHAPE"), (dict(W_qkv=weights(WIDTH, HIDDEN - 256)), "SHAPE"),
    (dict(W_o=weights(HIDDEN, HEADS * D - 256)), "SHAPE"), (dict(W_o=weights(HIDDEN + 8, HEADS * D)), "SHAPE"),
    (dict(W_o=weights(HIDDEN, HEADS * D).float()), "FORMAT"), (dict(hidden=HIDDEN + 64), "K_NOT_MULTIPLE"),
    (dict(W_qkv=weights(WIDTH, HIDDEN).t().contiguous().t()), "SHAPE"),
])
def test_weights_that_do_not_fit(calls, kw, status):
    with pytest.raises(q.QmdError, match=status):
        block(**kw)
