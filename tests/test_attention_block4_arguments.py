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
