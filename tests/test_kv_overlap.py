"""Which row buffers overlap: parts of one wider buffer do not, whatever their extents; q_out in place of
q is still checked against k, v and the table (no GPU needed: refused before the device is touched, and
what is accepted ends at the device check)."""
import pytest

import quantised_decode_mat_gb300 as q
from quantised_decode_mat_gb300 import build as qbuild

A = 0x10000
FAR = 1 << 30
VALUE = 10
KW, QW, T = 256, 512, 5  # f32 values of a row of keys, of queries; rows


@pytest.fixture(scope="module")
def L():
    import torch
    if torch.cuda.is_available():
        pytest.skip("GPU present: the addresses are made up")
    qbuild.build()
    return q.lib()


def structs(rows=T):
    return (q.KVCachePtrs(4 * FAR, 5 * FAR, 6 * FAR, 7 * FAR, 10, 2, 32, 128),
            q.KVBatchPtrs(8 * FAR, 9 * FAR, 10 * FAR, 4, rows, 3, 2))


def at(value):  # the address of an f32 value of the buffer
    return A + 4 * value


def append(L, k, v, x, o, ks=1024, vs=1024, xs=1024, os_=1024, rope=11 * FAR, rows=T, n=100):
    return L.qmd_kv_append(*structs(rows), k, ks, v, vs, x, xs, 4, o, os_, rope, n, 128, 0, None)


def read(L, k, v, ks=512, vs=512, rows=T):
    return L.qmd_kv_read(*structs(rows), k, ks, v, vs, None)


def attention(L, x, o, xs=1024, os_=1024, rows=T):
    return L.qmd_kv_attention(*structs(rows), x, xs, 4, 0.1, 0, o, os_, 12 * FAR, None)


def test_parts_of_one_buffer_are_apart(L):
    assert read(L, at(0), at(KW)) == 9 and read(L, at(KW), at(0)) == 9
    assert read(L, at(0), at(512 * 2 + KW)) == 9                     # ... from a later row on
    assert read(L, at(0), at(KW), 1024, 512) == 9 and read(L, at(0), at(KW), 1024, 1536) == 9
    assert read(L, at(0), at(KW), 1024, 768) == VALUE                 # (row 1 of v_out begins where k_out's does)
    assert attention(L, at(0), at(QW)) == 9 and attention(L, at(QW), at(0)) == 9
    # a fused row q | k | v: in place, from elsewhere into its q part, and into a part of its own
    assert append(L, at(512), at(768), at(0), at(0)) == 9
    assert append(L, at(512), at(768), FAR, at(0)) == 9
    assert append(L, at(512), at(768), at(0), at(1024), 1536, 1536, 1536, 1536) == 9


def test_rows_that_meet_are_refused(L):
    assert read(L, at(0), at(KW - 4)) == VALUE and read(L, at(KW - 4), at(0)) == VALUE
    assert read(L, at(0), at(512 * 4 + KW - 4)) == VALUE              # the last row's end
    assert read(L, at(0), at(512 * 4 + KW)) == 9
    assert read(L, at(4), at(KW)) == VALUE and read(L, at(4), at(KW), rows=1) == VALUE
    assert read(L, at(0), at(KW), rows=1) == 9
    assert read(L, at(0), at(KW + 4), 512, 512) == VALUE              # runs into the next row's keys
    assert attention(L, at(0), at(QW + 4)) == VALUE and attention(L, at(0), at(QW - 4)) == VALUE
    assert attention(L, at(0), at(0)) == VALUE


def test_in_place_queries_that_run_into_keys_or_values(L):
    assert append(L, at(508), FAR, at(0), at(0)) == VALUE
    assert append(L, FAR, at(0), at(0), at(0)) == VALUE
    assert append(L, at(512), at(896), at(0), at(0)) == VALUE         # values run into the next row's queries
    assert append(L, at(0), at(0), at(0), at(0), rows=1) == VALUE
    assert append(L, at(512), at(1024 - 256), at(0), at(0), rows=1) == 9


def test_rotated_queries_over_the_table(L):
    assert append(L, FAR, 2 * FAR, at(0), at(0), rope=at(1024 * 4 + 508)) == VALUE
    assert append(L, FAR, 2 * FAR, at(0), at(0), rope=at(1024 * 4 + 512)) == 9
    assert append(L, FAR, 2 * FAR, at(12800), at(12800), rope=at(0)) == 9
    assert append(L, FAR, 2 * FAR, at(12796), at(12796), rope=at(0)) == VALUE


def test_every_offset_and_stride_against_the_bytes(L):
    """Small strides and every offset of three rows: refused where a value is in both, and accepted for
    equal strides wherever none is."""
    import itertools
    w = 64
    def st(sk, sv, off, rows):
        c, b = structs(rows)
        c.kv_heads, c.head_dim = 1, 64
        return L.qmd_kv_read(c, b, at(4096), sk, at(4096 + off), sv, None)
    for sk, sv in itertools.product((64, 80, 128, 192), repeat=2):
        for off in range(-512, 513, 16):
            a = {i * sk + j for i in range(3) for j in range(w)}
            meet = any(off + i * sv + j in a for i in range(3) for j in range(w))
            got = st(sk, sv, off, 3)
            assert got in (9, VALUE) and (got == VALUE or not meet), (sk, sv, off)
            if sk == sv:
                assert (got == VALUE) == meet, (sk, off)
