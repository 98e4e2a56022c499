"""The tables of a step, reserved and released on the GPU, against the oracle: integers,
equal."""

import numpy as np
import pytest
import torch

from helpers import dev, host
from test_gpu_attn import projections, stale_pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    assert torch.cuda.is_available()
    return qlin


class Both:
    """The same pool and tables on the GPU and for the oracle."""

    def __init__(self, q, rng, B, cols, page, pages, free, T, max_q=1):
        self.free = rng.permutation(pages).astype(np.int32)
        self.count = np.array([free, 0], np.int32)
        self.table = rng.integers(0, pages, (B, cols)).astype(np.int32)
        self.slots, self.positions = np.full(T, -9, np.int32), np.full(T, -9, np.int32)
        self.page = page
        self.pool = q.PagePool(dev(self.free), dev(self.count), page)
        self.tables = q.PageTables(self.pool, dev(self.table), T, max_q)
        self.tables.slots.fill_(-9)
        self.tables.positions.fill_(-9)

    def reserve(self, oracle, lengths, new):
        got = self.tables.reserve(dev(np.asarray(lengths, np.int32)), dev(np.asarray(new, np.int32)))
        assert got is self.tables.batch
        self.q_start, self.kv_len = oracle.kv_reserve(lengths, new, self.table, self.free, self.count, self.page,
                                                      self.slots, self.positions)
        self.same()

    def release(self, oracle, lengths):
        self.tables.release(dev(np.asarray(lengths, np.int32)))
        oracle.kv_release(lengths, self.kv_len, self.table, self.free, self.count, self.page)
        self.same()

    def same(self):
        for name in ("q_start", "kv_len", "slots", "positions"):
            assert np.array_equal(host(getattr(self.tables, name)), getattr(self, name)), name
        assert np.array_equal(host(self.tables.page_table), self.table)
        assert np.array_equal(host(self.pool.free), self.free)
        assert np.array_equal(host(self.pool.count), self.count)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("B,most,room", [(1, 1, 4), (1, 9000, 600), (5, 40, 9), (64, 16, 70), (64, 1300, 90), (300, 3, 30),
                                         (1023, 5, 12), (1024, 5, 12), (1025, 5, 12), (2500, 30, 8), (65535, 2, 3)])
def test_steps(q, oracle, B, most, room, page):
    """Reservations and releases in turn, as requests grow, are cut back and end."""
    rng = np.random.default_rng(B + most + page)
    T = max(1, B * most * 3 // 4)
    both = Both(q, rng, B, room, page, B * room + 7, B * room + 3, T)
    lengths = rng.integers(0, room * page // 2 + 1, B)
    for turn in range(4):
        new = rng.integers(0, most + 1, B)
        both.reserve(oracle, lengths, new)
        kept = lengths + rng.integers(0, most + 1, B) % (new + 1)
        if turn == 2:
            kept[rng.random(B) < 0.3] = 0  # requests that end
        both.release(oracle, kept)
        lengths = kept


@pytest.mark.parametrize("B,T", [(3, 5000), (3, 4096), (3, 4097), (70, 4096), (70, 4200), (1500, 4096), (1500, 9000)])
def test_rows_beyond_the_tokens(q, oracle, B, T):
    """More rows than tokens (left as they are) and fewer (the others not written), in
    one launch and in two; idle requests at both ends and in runs."""
    rng = np.random.default_rng(B + T)
    both = Both(q, rng, B, 200, 16, B * 200, B * 200, T)
    for total in (T - 1, T, T + 40, 7, 0):
        new = np.zeros(B, int)
        at = rng.choice(np.arange(1, B - 1), min(B - 2, 40), replace=False)
        new[at] = total // len(at)
        new[at[0]] += total - new.sum()
        both.slots[:] = both.positions[:] = -9
        both.tables.slots.fill_(-9)
        both.tables.positions.fill_(-9)
        both.reserve(oracle, rng.integers(0, 40, B), new)
        assert (both.slots[total:] == -9).all()


@pytest.mark.parametrize("B", [6, 1300])
def test_pools_that_run_short(q, oracle, B):
    """Pages that are lacking, a list of none, tables too narrow for their requests, and
    state of any value: counts, lengths and pages outside their ranges."""
    rng = np.random.default_rng(B)
    both = Both(q, rng, B, 4, 16, B * 3, B, 64 * B)
    both.reserve(oracle, rng.integers(0, 20, B), rng.integers(0, 60, B))
    assert both.count[0] == 0 and both.count[1] > 0 and (both.slots == -1).any()
    both.release(oracle, np.zeros(B, int))
    lengths, new = rng.integers(0, 90, B), rng.integers(0, 50, B)  # past the table's 64 tokens
    lengths[0], new[1], lengths[2], new[3] = -2 ** 31, -5, 2 ** 31 - 1, 0
    both.reserve(oracle, lengths, np.where(np.arange(B) == 2, 0, new))
    both.release(oracle, np.where(np.arange(B) % 2, -7, 2 ** 31 - 1))
    for count in (-3, 2 ** 31 - 1, -2 ** 31):
        both.count[0] = count
        both.pool.count.copy_(dev(both.count))
        both.table[0] = [-1, 2 ** 31 - 1, -2 ** 31, B * 3]
        both.tables.page_table.copy_(dev(both.table))
        both.reserve(oracle, np.full(B, 64), np.full(B, 3))
        both.release(oracle, np.zeros(B, int))
        both.release(oracle, np.zeros(B, int))  # twice: the list is full, not passed


def test_a_dropped_step_restores_the_pool(q, oracle):
    rng = np.random.default_rng(3)
    both = Both(q, rng, 200, 64, 16, 20000, 14000, 30000)
    before = both.free.copy()
    lengths = rng.integers(0, 300, 200)
    both.reserve(oracle, lengths, rng.integers(0, 200, 200))
    assert both.count[0] < 14000
    both.release(oracle, lengths)
    assert both.count[0] == 14000 and np.array_equal(host(both.pool.free), before)


def test_lengths_in_place(q, oracle):
    """kv_len as the lengths that it replaces (the call that the interface allows)."""
    rng = np.random.default_rng(4)
    for B, T in ((5, 100), (1100, 3000), (90, 9000)):
        both = Both(q, rng, B, 40, 16, B * 40, B * 40, T)
        lengths = rng.integers(0, 100, B).astype(np.int32)
        both.tables.kv_len.copy_(dev(lengths))
        for _ in range(3):
            new = rng.integers(0, 2 * T // B, B).astype(np.int32)
            both.tables.reserve(both.tables.kv_len, dev(new))
            both.q_start, both.kv_len = oracle.kv_reserve(lengths, new, both.table, both.free, both.count, 16,
                                                          both.slots, both.positions)
            both.same()
            lengths = both.kv_len


def test_graph_replays(q, oracle):
    """A captured reservation and release, replayed over growing requests with eager work
    between: the pool and the tables are state that stays in place."""
    rng = np.random.default_rng(5)
    for B, T in ((40, 400), (40, 9000)):
        both = Both(q, rng, B, 90, 16, B * 90, B * 90, T)
        ln, nw, kp = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                both.tables.reserve(ln, nw)
                both.tables.release(kp)
        lengths = rng.integers(0, 60, B)
        for _ in range(4):
            new = rng.integers(0, T // B, B)
            kept = lengths + new // 2
            for t, x in ((ln, lengths), (nw, new), (kp, kept)):
                t.copy_(dev(x.astype(np.int32)))
            graph.replay()
            torch.cuda.synchronize()
            both.q_start, both.kv_len = oracle.kv_reserve(lengths, new, both.table, both.free, both.count, 16,
                                                          both.slots, both.positions)
            oracle.kv_release(kept, both.kv_len, both.table, both.free, both.count, 16)
            both.same()
            lengths = kept


def test_slots_are_where_the_append_writes(q):
    rng = np.random.default_rng(6)
    pool = q.PagePool.full(40, 16)
    tables = q.PageTables(pool, torch.full((3, 12), -1, dtype=torch.int32, device="cuda"), 60, 50)
    batch = tables.reserve(dev(np.zeros(3, np.int32)), dev(np.array([33, 0, 16], np.int32)))
    assert host(pool.count).tolist() == [36, 0]
    cache = stale_pool(q, 40, 2, 16, 64, "bf16")
    k, v = (dev(projections(rng, (60, 2, 64))) for _ in range(2))
    q.kv_append(cache, batch, k, v)
    flat = cache.k.transpose(1, 2).reshape(40 * 16, 2, 64)
    rows = tables.slots[:49].long()
    assert torch.equal(flat[rows].view(torch.int16), k[:49].view(torch.int16))
    assert flat.isnan().all(-1).all(-1).sum() == 640 - 49
    assert host(tables.positions)[:49].tolist() == list(range(33)) + list(range(16))


def test_tables_binding_refusals(q):
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = q.PagePool.full(8, 16)
    assert host(pool.free).tolist() == list(range(7, -1, -1)) and host(pool.count).tolist() == [8, 0]
    table = torch.zeros((2, 3), **i32)
    tables = q.PageTables(pool, table, 8, 4)
    good = torch.zeros(2, **i32)
    for bad in (torch.zeros(3, **i32), torch.zeros(2, dtype=torch.int32)):
        for call in (lambda: tables.reserve(bad, good), lambda: tables.reserve(good, bad), lambda: tables.release(bad)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(TypeError):
        tables.reserve(good.long(), good)
    for args in ((torch.zeros(4, **i32), torch.zeros(1, **i32), 16), (torch.zeros(4, **i32), torch.zeros(2, **i32), 8),
                 (torch.zeros(4, dtype=torch.int32), torch.zeros(2, **i32), 16)):
        with pytest.raises(ValueError):
            q.PagePool(*args)
    with pytest.raises(ValueError):
        q.PageTables(pool, table.cpu(), 8, 4)
    empty = q.PageTables(pool, torch.zeros((0, 3), **i32), 8, 4)
    empty.reserve(torch.zeros(0, **i32), torch.zeros(0, **i32))
    empty.release(torch.zeros(0, **i32))
    assert host(pool.count).tolist() == [8, 0]


@pytest.mark.parametrize("T", [0, 300, 5000])
@pytest.mark.parametrize("B", [1, 40, 400])
def test_tables_without_slots_or_positions(q, oracle, B, T):
    """The C interface's tables may have no slots, no positions or neither, in one launch and
    in two: all other arrays are as with them."""
    import ctypes as C

    rng = np.random.default_rng(B + T)
    lib, stream = q.lib(), torch.cuda.current_stream().cuda_stream
    for absent in (("slots",), ("positions",), ("slots", "positions")):
        both = Both(q, rng, B, 30, 16, B * 30, B * 20, T)
        t = q._KVTables.from_buffer_copy(both.tables._c)
        for name in absent:
            setattr(t, name, None)
            setattr(both, name, np.full(T, -9, np.int32))
        lengths = rng.integers(0, 200, B).astype(np.int32)
        new = rng.integers(0, max(2 * T // B, 60), B).astype(np.int32)
        ld, nd = dev(lengths), dev(new)
        assert lib.qlin_kv_reserve(both.pool._ref, C.byref(t), T, ld.data_ptr(), nd.data_ptr(), stream) == q.OK
        slots, positions = both.slots.copy(), both.positions.copy()
        both.q_start, both.kv_len = oracle.kv_reserve(lengths, new, both.table, both.free, both.count, 16, slots, positions)
        for name, full in (("slots", slots), ("positions", positions)):
            if name not in absent:
                setattr(both, name, full)
        both.same()
        assert lib.qlin_kv_release(both.pool._ref, C.byref(t), ld.data_ptr(), stream) == q.OK
        oracle.kv_release(lengths, both.kv_len, both.table, both.free, both.count, 16)
        both.same()


def test_tokens_behind_the_table_are_not_lacking(q, oracle):
    """A request that outgrows its table: no page is taken or counted for those tokens."""
    both = Both(q, np.random.default_rng(8), 2, 3, 16, 6, 6, 60)
    both.reserve(oracle, [40, 0], [30, 20])
    assert both.count.tolist() == [4, 0]
    assert (both.slots[8:30] == -1).all() and (both.slots[:8] >= 0).all() and (both.slots[30:50] >= 0).all()
