"""Refusals of the tables' entry points, on the host (no GPU needed), and the oracle's
tables by hand."""

import numpy as np
import pytest

from test_abi_attn_host import A, p


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    return qlin


def pool(q, **over):
    f = dict(free_pages=A, count=A, pages=8, page_size=16)
    f.update(over)
    return q._KVPool(**f)


def tables(q, **over):
    f = dict(page_table=A, q_start=A, kv_len=A, slots=A, positions=A, batch=2, table_cols=4)
    f.update(over)
    return q._KVTables(**f)


BAD = [(dict(page_size=8), {}, "ERR_SHAPE"), (dict(page_size=48), {}, "ERR_SHAPE"), (dict(page_size=512), {}, "ERR_SHAPE"),
       (dict(pages=0), {}, "ERR_SHAPE"), (dict(pages=1 << 27), {}, "ERR_SHAPE"), ({}, dict(batch=-1), "ERR_SHAPE"),
       ({}, dict(batch=1 << 16), "ERR_SHAPE"), ({}, dict(table_cols=0), "ERR_SHAPE"),
       ({}, dict(table_cols=1 << 27), "ERR_SHAPE"), (dict(free_pages=None), {}, "ERR_ARG"),
       (dict(count=None), {}, "ERR_ARG"), ({}, dict(page_table=None), "ERR_ARG"), ({}, dict(kv_len=None), "ERR_ARG"),
       (dict(free_pages=A + 2), {}, "ERR_ALIGN"), (dict(count=A + 1), {}, "ERR_ALIGN"),
       ({}, dict(page_table=A + 2), "ERR_ALIGN"), ({}, dict(slots=A + 2), "ERR_ALIGN"),
       ({}, dict(positions=A + 3), "ERR_ALIGN"), ({}, dict(q_start=A + 2), "ERR_ALIGN")]


def reserve(q, pl="", t="", T=4, lengths=A, new=A):
    return q.lib().qlin_kv_reserve(pool(q) if pl == "" else pl, tables(q) if t == "" else t, T, p(lengths), p(new), None)


def release(q, pl="", t="", lengths=A):
    return q.lib().qlin_kv_release(pool(q) if pl == "" else pl, tables(q) if t == "" else t, p(lengths), None)


def test_refusals(q):
    none = tables(q, batch=0, page_table=None, q_start=None, kv_len=None)
    assert reserve(q, t=none) == q.OK and release(q, t=none) == q.OK
    for over, more, status in BAD:
        assert reserve(q, pl=pool(q, **over), t=tables(q, **more)) == getattr(q, status), (over, more)
        assert release(q, pl=pool(q, **over), t=tables(q, **more)) == getattr(q, status), (over, more)
    for bad in (dict(pl=None), dict(t=None), dict(lengths=None)):
        assert reserve(q, **bad) == q.ERR_ARG and release(q, **bad) == q.ERR_ARG
    assert reserve(q, new=None) == q.ERR_ARG and reserve(q, t=tables(q, q_start=None)) == q.ERR_ARG
    assert reserve(q, T=-1) == q.ERR_SHAPE and reserve(q, T=1 << 31) == q.ERR_SHAPE
    assert reserve(q, lengths=A + 2) == q.ERR_ALIGN and reserve(q, new=A + 2) == q.ERR_ALIGN
    assert release(q, lengths=A + 2) == q.ERR_ALIGN


def test_arrays_that_overlap(q):
    """What a call writes must not be what it reads or writes elsewhere, but for lengths in
    place; what a release only reads may be one array."""
    B = 8 * A
    pl = dict(free_pages=2 * B, count=3 * B, pages=40)
    t = dict(page_table=4 * B, q_start=5 * B, kv_len=6 * B, slots=7 * B, positions=8 * B, batch=6, table_cols=3)

    def calls(pl, t, lengths=9 * B, new=10 * B):
        return (reserve(q, pool(q, **pl), tables(q, **t), 11, lengths, new), release(q, pool(q, **pl), tables(q, **t), lengths))

    apart = calls(pl, t)
    assert q.ERR_ARG not in apart and calls(pl, t, lengths=6 * B) == apart and calls(pl, t, lengths=10 * B) == apart
    assert calls(pl, {**t, "slots": None, "positions": None}) == apart
    for pl2, t2, kw in (({"count": 2 * B + 4 * 39}, {}, {}), ({}, {"page_table": 2 * B - 4 * 17}, {}),
                        ({}, {"kv_len": 3 * B + 4}, {}), ({}, {}, {"lengths": 2 * B + 4 * 39}), ({"count": 4 * B + 4 * 17}, {}, {})):
        assert calls({**pl, **pl2}, {**t, **t2}, **kw) == (q.ERR_ARG, q.ERR_ARG), (pl2, t2, kw)
    for t2, kw in (({"kv_len": 5 * B + 24}, {}), ({"q_start": 6 * B - 24}, {}), ({"slots": 8 * B - 40}, {}),
                   ({"positions": 5 * B}, {}), ({}, {"lengths": 6 * B + 4}), ({}, {"new": 6 * B}), ({}, {"new": 5 * B + 24}),
                   ({}, {"lengths": 4 * B + 4 * 17}), ({}, {"lengths": 10 * B + 4})):
        got = calls(pl, {**t, **t2}, **kw)
        assert got == (q.ERR_ARG, apart[1]), (t2, kw)
    near = {**t, "q_start": 6 * B - 28, "slots": 8 * B - 44}
    assert calls({**pl, "count": 2 * B + 160}, near) == apart


def test_oracle_tables(oracle):
    table = np.full((3, 3), -5, np.int32)
    table[0, 0] = 4
    free, count = np.array([9, 8, 7, 6, 5, 0, 0, 0, 0, 0], np.int32), np.array([5, 0], np.int32)
    slots, positions = np.full(60, -9, np.int32), np.full(60, -9, np.int32)
    q_start, kv_len = oracle.kv_reserve([10, 0, 16], [7, 0, 33], table, free, count, 16, slots, positions)
    assert q_start.tolist() == [0, 7, 7, 40] and kv_len.tolist() == [17, 0, 49]
    assert table.tolist() == [[4, 5, -5], [-5, -5, -5], [-5, 6, 7]] and count.tolist() == [2, 0]
    assert slots[:7].tolist() == [74, 75, 76, 77, 78, 79, 80] and positions[:8].tolist() == [*range(10, 17), 16]
    assert slots[7:39].tolist() == [*range(96, 112), *range(112, 128)] and slots[39] == -1 and slots[40] == -9
    oracle.kv_release([16, 0, 40], kv_len, table, free, count, 16)
    assert count.tolist() == [3, 0] and free[:3].tolist() == [9, 8, 5]
    oracle.kv_release([0, 0, 16], kv_len, table, free, count, 16)
    assert count.tolist() == [7, 0] and free[:7].tolist() == [9, 8, 5, 7, 6, 5, 4]
