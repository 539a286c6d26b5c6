"""Eviction's outputs over its inputs: the page table is checked once and looked up again for every token that
moves, so an output that lies over it would turn a checked page into any address; refused before the device is
touched (no GPU needed: what is accepted ends at the device check)."""
import pytest

import quantised_decode_mat_gb300 as q
from quantised_decode_mat_gb300 import build as qbuild

FAR = 1 << 30
TABLE, LEN, WEIGHT, OUT, KEPT = (n * FAR for n in range(5, 10))
VALUE = 10
SEQS, STRIDE, HEADS, KEEP, PAGES, TOKENS = 3, 7, 2, 40, 10, 32
TABLE_BYTES, LEN_BYTES = SEQS * STRIDE * 4, SEQS * 4
WEIGHT_BYTES, KEPT_BYTES = PAGES * HEADS * TOKENS * 4, SEQS * HEADS * KEEP * 4


@pytest.fixture(scope="module")
def L():
    import torch
    if torch.cuda.is_available():
        pytest.skip("GPU present: the addresses are made up")
    qbuild.build()
    return q.lib()


def evict(L, table=TABLE, kv_len=LEN, weight=WEIGHT, out=OUT, kept=KEPT):
    cache = q.KV4CachePtrs(FAR, 2 * FAR, 3 * FAR, 4 * FAR, PAGES, HEADS, TOKENS, 128)
    batch = q.KVBatchPtrs(table, kv_len, None, STRIDE, 0, SEQS, 0)
    return L.qmd_kv4_evict(cache, batch, weight, KEEP, 4, 8, out, kept, None)


def test_side_by_side_is_taken(L):
    assert evict(L) == 9 and evict(L, kept=None) == 9
    assert evict(L, out=TABLE + TABLE_BYTES) == 9 and evict(L, out=TABLE - LEN_BYTES) == 9
    assert evict(L, kept=TABLE + TABLE_BYTES) == 9 and evict(L, kept=TABLE - KEPT_BYTES) == 9
    assert evict(L, out=WEIGHT + WEIGHT_BYTES) == 9 and evict(L, kept=WEIGHT - KEPT_BYTES) == 9
    assert evict(L, kept=OUT + LEN_BYTES) == 9 and evict(L, kv_len=TABLE + TABLE_BYTES) == 9


@pytest.mark.parametrize("kw", [
    dict(out=TABLE), dict(out=TABLE + TABLE_BYTES - 4), dict(out=TABLE - LEN_BYTES + 4), dict(out=TABLE, kept=None),
    dict(kept=TABLE), dict(kept=TABLE + TABLE_BYTES - 4), dict(kept=TABLE - KEPT_BYTES + 4),
    dict(out=WEIGHT), dict(out=WEIGHT + WEIGHT_BYTES - 4), dict(out=WEIGHT - LEN_BYTES + 4),
    dict(kept=WEIGHT + 64), dict(kept=WEIGHT + WEIGHT_BYTES - 4), dict(kept=WEIGHT - KEPT_BYTES + 4),
    dict(weight=TABLE), dict(weight=TABLE + 16), dict(table=WEIGHT + WEIGHT_BYTES - 4), dict(weight=LEN),
    dict(out=LEN), dict(kept=LEN), dict(kept=OUT), dict(kept=OUT + LEN_BYTES - 4)])
def test_outputs_over_inputs_are_refused(L, kw):
    assert evict(L, **kw) == VALUE
