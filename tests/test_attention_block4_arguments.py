"""What AttentionBlock is given besides its rows (positions, weights of a 4-bit cache's tokens, adapters' choices, the batch)
is refused before anything is launched: by then the projection would have run, or the cache would hold the rows (no GPU
needed: the calls are replaced)."""
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from quantised_decode_mat_gb300 import step as S  # noqa: E402
from tests.test_attention_block4_checks import calls  # noqa: E402, F401
from tests.test_attention_block_checks import D, HIDDEN, KV, ROWS, batch, block  # noqa: E402


def four():
    return q.KV4Cache.empty(4, KV, 16, D, "cpu")


@pytest.mark.parametrize("positions,status", [
    (torch.zeros(2 * ROWS, dtype=torch.int32)[::2], "SHAPE"),               # every second one
    (torch.zeros((ROWS, 2), dtype=torch.int32)[:, 0], "SHAPE"),             # a column of a table
    (torch.zeros(1, dtype=torch.int32).expand(ROWS), "SHAPE"),
    (torch.zeros((1, ROWS), dtype=torch.int32), "SHAPE"), (torch.zeros(ROWS, dtype=torch.int64), "SHAPE"),
    (torch.zeros(ROWS, dtype=torch.int32, device="meta"), "DEVICE")])
def test_positions(calls, positions, status):  # noqa: F811
    b = block(cache=four())
    with pytest.raises(q.QmdError, match=status):
        b.run(torch.zeros((ROWS, HIDDEN)), batch(), positions=positions)
    assert calls == []
    b.run(torch.zeros((ROWS, HIDDEN)), batch(), positions=torch.zeros(2 * ROWS, dtype=torch.int32)[ROWS:])
    assert calls == ["qmatvec_x", "kv4_append", "kv4_attention", "qmatvec_x"]


@pytest.mark.parametrize("weights,status", [
    (torch.zeros((5, KV, 16)), "SHAPE"), (torch.zeros((4, KV + 1, 16)), "SHAPE"), (torch.zeros((4, KV, 32)), "SHAPE"),
    (torch.zeros((4, KV * 16)), "SHAPE"), (torch.zeros((4, 16, KV)).transpose(1, 2), "SHAPE"),
    (torch.zeros((4, KV, 16), dtype=torch.float64), "FORMAT"), (torch.zeros((4, KV, 16)).half(), "FORMAT"),
    (torch.zeros((4, KV, 16), device="meta"), "DEVICE"),
    (torch.zeros(4 * KV * 16 + 4)[1:-3].view(4, KV, 16), "MISALIGNED")])
def test_weights_of_another_pool(calls, weights, status):  # noqa: F811
    with pytest.raises(q.QmdError, match=status):
        block(cache=four(), weights=weights)
    assert calls == []


def adapters(**kw):
    f = dict(A=torch.zeros((2, 8, HIDDEN)).half(), B=torch.zeros((2, (4 + 2 * KV) * D, 8)).half(), scale=torch.ones(2))
    f.update(kw)
    return S.Adapters(**f)


@pytest.mark.parametrize("adapter,status", [
    (torch.zeros(ROWS, dtype=torch.int64), "FORMAT"), (torch.zeros(ROWS), "FORMAT"),
    (torch.zeros(2 * ROWS, dtype=torch.int32)[::2], "SHAPE"), (torch.zeros(ROWS, dtype=torch.int32, device="meta"), "DEVICE")])
@pytest.mark.parametrize("which", ["qkv_adapters", "o_adapters"])
def test_adapters_choices(calls, adapter, status, which):  # noqa: F811
    a = adapters() if which == "qkv_adapters" else adapters(A=torch.zeros((2, 8, 4 * D)).half(), B=torch.zeros((2, HIDDEN, 8)).half())
    b = block(cache=four(), **{which: a})
    with pytest.raises(q.QmdError, match=status):
        b.run(torch.zeros((ROWS, HIDDEN)), batch(), adapter)
    assert calls == []
    b.run(torch.zeros((ROWS, HIDDEN)), batch(), torch.zeros(ROWS, dtype=torch.int32))


@pytest.mark.parametrize("kw,status", [
    (dict(A=torch.zeros((2, 8, HIDDEN))), "FORMAT"), (dict(B=torch.zeros((2, (4 + 2 * KV) * D, 8)).bfloat16()), "FORMAT"),
    (dict(scale=torch.ones(2).double()), "FORMAT"), (dict(A=torch.zeros((2, 8, 2 * HIDDEN)).half()), "SHAPE"),
    (dict(B=torch.zeros((2, 4 * D, 8)).half()), "SHAPE"), (dict(B=torch.zeros((3, (4 + 2 * KV) * D, 8)).half()), "SHAPE"),
    (dict(scale=torch.ones(3)), "SHAPE"), (dict(A=torch.zeros((8, HIDDEN)).half()), "SHAPE"),
    (dict(A=torch.zeros((2, 12, HIDDEN)).half(), B=torch.zeros((2, (4 + 2 * KV) * D, 12)).half()), "SHAPE"),
    (dict(A=torch.zeros((2, 136, HIDDEN)).half(), B=torch.zeros((2, (4 + 2 * KV) * D, 136)).half()), "SHAPE"),
    (dict(A=torch.zeros((2, 8, 2 * HIDDEN)).half()[..., ::2]), "SHAPE"), (dict(scale=torch.ones(2, device="meta")), "DEVICE")])
def test_adapters_of_another_projection(calls, kw, status):  # noqa: F811
    with pytest.raises(q.QmdError, match=status):
        block(cache=four(), qkv_adapters=adapters(**kw))
    assert calls == []


@pytest.mark.parametrize("kw,status", [
    (dict(rope=torch.zeros((9, D)).double()), "FORMAT"), (dict(rope=torch.zeros(9 * D)), "SHAPE"),
    (dict(rope=torch.zeros((9, D + 32))), "SHAPE"), (dict(rope=torch.zeros((9, 48))), "SHAPE"),
    (dict(rope=torch.zeros((0, D))), "SHAPE"), (dict(rope=torch.zeros((9, 2 * D))[:, ::2]), "SHAPE"),
    (dict(rope=torch.zeros((9, D), device="meta")), "DEVICE"),
    (dict(rope=torch.zeros(9 * D + 4)[1:-3].view(9, D)), "MISALIGNED"),
    (dict(pairs=2), "VALUE"), (dict(window=-1), "VALUE"), (dict(window=1 << 63), "VALUE"),
    (dict(heads=3, W_qkv=torch.zeros(((3 + 2 * KV) * D, HIDDEN // 256 * 144), dtype=torch.uint8),
          cache=q.KV4Cache.empty(4, KV, 16, 256, "cpu")), "SHAPE")])
def test_rotation_window_and_heads(calls, kw, status):  # noqa: F811
    f = dict(cache=four())
    f.update(kw)
    with pytest.raises(q.QmdError, match=status):
        block(**f)
    assert calls == []


def test_heads_that_do_not_share_evenly(calls):  # noqa: F811
    """12 query heads over 8 of 128: found out by attention, when the cache holds the rows."""
    W_qkv = torch.zeros((28 * 128, HIDDEN // 256 * 144), dtype=torch.uint8)
    W_o = torch.zeros((HIDDEN, 12 * 128 // 256 * 144), dtype=torch.uint8)
    with pytest.raises(q.QmdError, match="SHAPE"):
        block(heads=12, W_qkv=W_qkv, W_o=W_o, cache=q.KV4Cache.empty(2, 8, 16, 128, "cpu"))
    for cache in (q.KV4Cache.empty(2, 2, 24, 128, "cpu"), q.KVCache.empty(2, 2, 16, 32, "cpu")):
        with pytest.raises(q.QmdError, match="SHAPE"):
            W_qkv = torch.zeros(((8 + 4) * cache.head_dim, HIDDEN // 256 * 144), dtype=torch.uint8)
            W_o = torch.zeros((HIDDEN, 8 * cache.head_dim // 256 * 144), dtype=torch.uint8)
            block(heads=8, W_qkv=W_qkv, W_o=W_o, cache=cache)
    assert calls == []


@pytest.mark.parametrize("seqs,columns,start,max_q,rows", [
    (ROWS, 2, True, 1, 0), (ROWS, 2, True, 0, ROWS), (ROWS, 2, True, (1 << 20) + 1, ROWS), (ROWS, 0, True, 1, ROWS),
    (2, 2, False, 2, 3), (2049, 1, True, 1, ROWS), (0, 2, True, 1, 1)])
def test_batches_that_no_call_takes(calls, seqs, columns, start, max_q, rows):  # noqa: F811
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    b = q.KVBatch(i32(seqs, columns), i32(seqs), i32(seqs + 1) if start else None, max_q, rows)
    for cache in (four(), q.KVCache.empty(4, KV, 16, D, "cpu")):
        with pytest.raises(q.QmdError, match="SHAPE"):
            block(cache=cache).run(torch.zeros((ROWS, HIDDEN)), b)
    assert calls == []


def test_another_device_than_the_current_one(calls, monkeypatch):  # noqa: F811
    b, rows = block(cache=four()), batch()
    b.cache.index = rows.index = 0
    monkeypatch.setattr(q, "_device_now", lambda: 1)
    with pytest.raises(q.QmdError, match="DEVICE"):
        b.run(torch.zeros((ROWS, HIDDEN)), rows)
    assert calls == []


@pytest.mark.parametrize("kw", [dict(weigh=True), dict(weigh=True, kv_bits=8), dict(kv_bits=3), dict(kv_bits=16, weigh=True)])
def test_a_block_of_a_kind_that_is_not_there(calls, monkeypatch, kw):  # noqa: F811
    """... is refused before its weights are made."""
    monkeypatch.setattr(S.synth, "weights", lambda *a: pytest.fail("weights were made"))
    with pytest.raises(q.QmdError, match="VALUE"):
        S.make_attention_block(1, 1, 16, 4, 2, 64, 256, device="cpu", **kw)
    assert calls == []
