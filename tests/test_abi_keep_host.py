"""Refusals of qlin_kv_keep, on the host (no GPU needed), and its oracle by hand."""

import numpy as np
import pytest

from test_abi_attn_host import BAD_CACHE, A, batch, cache, p


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    return qlin


def keep(q, caches=None, n=None, b="", path=A, width=4, kept=A, lengths=2 * A):
    caches = [cache(q)] if caches is None else caches
    arr = (q._KVCache * max(len(caches), 1))(*caches)
    return q.lib().qlin_kv_keep(arr, len(caches) if n is None else n, batch(q) if b == "" else b, p(path), width,
                                p(kept), p(lengths), None)


def test_refusals(q):
    assert keep(q, b=batch(q, batch=0, q_start=None, kv_len=None, page_table=None), path=None, kept=None) == q.OK
    for over, status in BAD_CACHE:
        assert keep(q, caches=[cache(q, **over)]) == getattr(q, status), over
    assert q.lib().qlin_kv_keep(None, 1, batch(q), p(A), 1, p(A), p(A), None) == q.ERR_ARG
    for bad in (dict(n=0), dict(n=65536), dict(width=-1), dict(width=1 << 31), dict(b=batch(q, table_cols=0)),
                dict(b=batch(q, batch=1 << 16)), dict(b=batch(q, batch=-1)), dict(caches=[cache(q), cache(q, pages=9)]),
                dict(caches=[cache(q), cache(q, kv_heads=1)]), dict(caches=[cache(q), cache(q, head_dim=128)]),
                dict(caches=[cache(q), cache(q, page_size=32)]),
                dict(caches=[cache(q), cache(q, fmt=q.KV_E4M3, k_scale=A, v_scale=A)])):
        assert keep(q, **bad) == q.ERR_SHAPE, bad
    for bad in (dict(b=None), dict(path=None), dict(kept=None), dict(lengths=None), dict(lengths=A),
                dict(b=batch(q, q_start=None)), dict(b=batch(q, page_table=None)), dict(caches=[cache(q), cache(q, v=None)])):
        assert keep(q, **bad) == q.ERR_ARG, bad
    for bad in (dict(path=A + 2), dict(kept=A + 1), dict(lengths=2 * A + 2), dict(b=batch(q, kv_len=A + 2))):
        assert keep(q, **bad) == q.ERR_ALIGN, bad


def test_lengths_that_overlap(q):
    """Every workgroup reads the batch, the path and its counts; one of them writes lengths."""
    B, F = 8 * A, q.OK
    far = dict(path=2 * B, kept=3 * B, lengths=4 * B, width=5)
    b = batch(q, batch=6, q_start=5 * B, kv_len=6 * B, page_table=7 * B, table_cols=3)
    for lengths in (2 * B, 2 * B + 4 * 29, 2 * B - 4 * 5, 3 * B, 3 * B + 20, 5 * B + 24, 6 * B - 4, 6 * B, 7 * B + 4 * 17):
        assert keep(q, b=b, **{**far, "lengths": lengths}) == q.ERR_ARG, lengths
    for lengths in (2 * B + 4 * 30, 2 * B - 4 * 6, 3 * B + 24, 5 * B + 28, 6 * B - 24, 7 * B + 4 * 18):
        assert keep(q, b=b, **{**far, "lengths": lengths}) not in (q.ERR_ARG, F), lengths  # (no GPU here)


def test_oracle_keep(oracle):
    pool = np.arange(3 * 16, dtype=np.int32).reshape(3, 1, 16, 1)  # three pages of one head
    table = np.array([[2, 0], [1, 1]], np.int32)
    lengths = oracle.kv_keep([pool], [0, 6, 8], [20, 5], table, [[1, 3, 5], [1, 0, 0]], [3, 1])
    assert lengths.tolist() == [17, 4]
    # the first sequence's new tokens are its tokens 14 .. 19: page 2 rows 14, 15, page 0 rows 0 .. 3
    assert pool[2, 0, 12:, 0].tolist() == [44, 45, 47, 1] and pool[0, 0, :5, 0].tolist() == [3, 1, 2, 3, 4]
    assert pool[1, 0, :6, 0].tolist() == [16, 17, 18, 20, 20, 21]
