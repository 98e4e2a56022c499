"""Steps of drafted tokens as a server runs them, on the GPU: tables reserved, heads
normalised, turned and cached, trees planned, attention, the accepted tokens' rows moved
together and the other pages given back; against the same tokens decoded in order."""

import numpy as np
import pytest
import torch

from helpers import dev, host
from test_gpu_attn import attn_check, projections, stale_pool
from test_gpu_tree import trees

pytestmark = pytest.mark.gpu

LAYERS, HKV, GROUP = 2, 2, 4


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    assert torch.cuda.is_available()
    return qlin


class Server:
    """The layers' caches and the tables of B requests; `tokens` rows a step at most."""

    def __init__(self, q, B, D, page, fmt, cols, tokens, max_q, rope, norms, window):
        self.q, self.rope, self.norms, self.window = q, rope, norms, window
        self.caches = [stale_pool(q, B * cols, HKV, page, D, fmt) for _ in range(LAYERS)]
        self.layers = q.PagedLayers(self.caches)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pool = q.PagePool.full(B * cols, page)
        self.tables = q.PageTables(self.pool, torch.full((B, cols), -1, **i32), tokens, max_q)
        self.lengths, self.new, self.kept = (torch.zeros(B, **i32) for _ in range(3))
        self.path = torch.zeros((B, max_q), **i32)
        self.parents = torch.zeros(tokens, **i32)
        self.tree = q.Tree.empty(tokens, 2)
        # a fused projection's rows: queries, keys and values
        self.qkv = torch.zeros((LAYERS, tokens, (GROUP + 2) * HKV, D), dtype=torch.bfloat16, device="cuda")
        self.turned = torch.zeros((LAYERS, tokens, GROUP * HKV, D), dtype=torch.bfloat16, device="cuda")
        self.out = torch.full_like(self.turned, 7.0)
        self.lse = [None] * LAYERS

    def parts(self, layer):
        x, n = self.qkv[layer], GROUP * HKV
        return x[:, :n], x[:, n:n + HKV], x[:, n + HKV:]

    def step(self, drafted=True):
        """A step of `new` tokens behind `lengths`; drafted ones are trees of which `path`
        is accepted."""
        q, b = self.q, self.tables.reserve(self.lengths, self.new)
        if drafted:
            q.tree_plan(b, self.parents, self.tree)
        for i, cache in enumerate(self.caches):
            x, k, v = self.parts(i)
            q.kv_append(cache, b, k, v, self.rope, x, self.turned[i], self.tree.positions if drafted else None,
                        self.norms[i])
            _, self.lse[i] = q.attn_paged(cache, b, self.turned[i], out=self.out[i], window=self.window,
                                          return_lse=True, tree=self.tree if drafted else None)
        if drafted:
            q.kv_keep(self.layers, b, self.path, self.kept, self.lengths)
            self.tables.release(self.lengths)
        else:
            self.lengths.copy_(self.tables.kv_len)


def rows_of(server, layer, b, n):
    """The first n cached tokens of request b: keys and values, and scales."""
    c, page = server.caches[layer], server.caches[layer].page_size
    table = host(server.tables.page_table)[b]
    at = [(table[t // page], t % page) for t in range(n)]
    parts = [host(t.view(torch.uint8) if t.dtype == torch.bfloat16 else t) for t in (c.k, c.v, c.k_scale, c.v_scale)
             if t is not None]
    return [np.array([p[g, :, s] for g, s in at]).view(np.uint8) for p in parts]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("D,page,fmt,window", [(128, 16, "bf16", 0), (64, 32, "e4m3", 0), (256, 64, "e4m3", 80),
                                               (128, 256, "bf16", 100)])
def test_drafted_steps_equal_decoding_in_order(q, oracle, D, page, fmt, window, graph):
    rng = np.random.default_rng(D + page)
    B, max_q, cols = 5, 70, -(-1100 // page)
    rope = q.Rope(D, base=5e5)
    norms = [q.HeadNorm(dev(projections(rng, (D,))), dev(projections(rng, (D,))), eps=1e-5) for _ in range(LAYERS)]
    tokens = B * max_q
    drafts = Server(q, B, D, page, fmt, cols, tokens, max_q, rope, norms, window)
    plain = Server(q, B, D, page, fmt, cols, 1000, 500, rope, norms, window)
    prompts = np.array([500, 0, 3, 130, 64], np.int32)  # prompts of both, the same rows
    text = projections(rng, (LAYERS, int(prompts.sum()), (GROUP + 2) * HKV, D))
    plain.qkv[:, :text.shape[1]].copy_(dev(text))
    plain.new.copy_(dev(prompts))
    plain.step(drafted=False)
    lengths = np.zeros(B, np.int32)
    while (lengths < prompts).any():  # (the drafting server's in chunks)
        new = np.minimum(prompts - lengths, max_q)
        starts = np.concatenate([[0], np.cumsum(prompts)])
        pick = np.concatenate([np.arange(starts[b] + lengths[b], starts[b] + lengths[b] + new[b]) for b in range(B)])
        drafts.qkv[:, :len(pick)].copy_(dev(text[:, pick]))
        drafts.new.copy_(dev(new.astype(np.int32)))
        drafts.step(drafted=False)
        lengths = lengths + new
    if graph:
        side, recorded = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(recorded, stream=side):
            drafts.step()
    moved = 0
    for turn in range(5):
        new = rng.integers(1, [9, 17, 33, 65, 71][turn], B)
        new[turn] = 0 if turn < 4 else new[turn]  # one request idles
        start = np.concatenate([[0], np.cumsum(new)])
        T = int(start[-1])
        parents = trees(rng, new, "random")
        path, kept, picked = np.full((B, max_q), -7, np.int32), np.zeros(B, np.int32), []
        for b in range(B):  # a token and those that it follows
            at, chain = int(rng.integers(-1, new[b])) if new[b] else -1, []
            while at >= 0:
                chain.append(at)
                at = int(parents[start[b] + at])
            kept[b] = len(chain)
            path[b, :kept[b]] = chain[::-1]
            moved += int((path[b, :kept[b]] != np.arange(kept[b])).sum())
            picked += [int(start[b]) + i for i in chain[::-1]]
        x = projections(rng, (LAYERS, T, (GROUP + 2) * HKV, D))
        drafts.qkv[:, :T].copy_(dev(x))
        drafts.out.fill_(7.0)
        drafts.new.copy_(dev(new.astype(np.int32)))
        drafts.parents[:T].copy_(dev(parents))
        drafts.path.copy_(dev(path))
        drafts.kept.copy_(dev(kept))
        torch.cuda.synchronize()
        recorded.replay() if graph else drafts.step()
        torch.cuda.synchronize()
        assert (drafts.out[:, T:] == 7.0).all()

        plain.qkv[:, :len(picked)].copy_(dev(x[:, picked]))
        plain.new.copy_(dev(kept))
        before = host(plain.lengths).copy()
        plain.step(drafted=False)
        lengths = host(drafts.lengths)
        assert np.array_equal(lengths, host(plain.lengths)) and np.array_equal(lengths, before + kept)
        assert host(drafts.pool.count).tolist() == [B * cols - int(sum(-(-n // page) for n in lengths)), 0]
        first = np.concatenate([[0], np.cumsum(kept)]).astype(np.int32)
        table = host(plain.tables.page_table)
        for i in range(LAYERS):
            for b in range(B):  # what is cached: the same bits
                for g, w in zip(rows_of(drafts, i, b, lengths[b]), rows_of(plain, i, b, lengths[b])):
                    assert np.array_equal(g, w)
            if not picked:
                continue
            assert torch.equal(drafts.turned[i, picked].view(torch.int16), plain.turned[i, :len(picked)].view(torch.int16))
            c = plain.caches[i]
            e4 = (host(c.k_scale), host(c.v_scale)) if fmt == "e4m3" else (None, None)
            want = oracle.attn_paged(host(drafts.turned[i, picked]), host(c.k), host(c.v), *e4, first, lengths, table,
                                     D ** -0.5, True, window)
            attn_check(want, host(drafts.out[i, picked]), host(drafts.lse[i][picked]), D, f"turn {turn} layer {i}")
    assert moved > 10
    drafts.new.zero_()  # all requests end
    drafts.tables.reserve(drafts.lengths, drafts.new)
    drafts.lengths.zero_()
    drafts.tables.release(drafts.lengths)
    assert host(drafts.pool.count).tolist() == [B * cols, 0]
    assert np.array_equal(np.sort(host(drafts.pool.free)), np.arange(B * cols))


def test_requests_that_end_and_start(q, oracle):
    """Pages of ended requests serve new ones; a step that the pool cannot hold whole says so
    and the rows that it lacked are neither cached nor seen."""
    rng = np.random.default_rng(11)
    D, page, B = 64, 16, 3
    s = Server(q, B, D, page, "bf16", 8, 200, 64, q.Rope(D), [q.HeadNorm(head_dim=D)] * LAYERS, 0)
    s.pool.count.copy_(dev(np.array([10, 0], np.int32)))  # ten pages
    for lengths, new, lacked in (([0, 0, 0], [40, 40, 40], 0), ([40, 40, 40], [9, 2, 0], 0), ([49, 42, 40], [9, 9, 9], 2),
                                 ([49, 0, 40], [3, 60, 9], 2), ([0, 0, 0], [60, 60, 20], 0)):
        s.lengths.copy_(dev(np.array(lengths, np.int32)))
        s.tables.release(s.lengths)  # (the last step's)
        s.new.copy_(dev(np.array(new, np.int32)))
        T = sum(new)
        s.qkv[:, :T].copy_(dev(projections(rng, (LAYERS, T, (GROUP + 2) * HKV, D))))
        s.parents[:T].copy_(dev(trees(rng, new)))
        b = s.tables.reserve(s.lengths, s.new)
        torch.cuda.synchronize()
        assert int(s.pool.count[1]) == lacked
        q.tree_plan(b, s.parents, s.tree)
        start, kv = host(b.q_start), host(b.kv_len)
        assert kv.tolist() == [n + m for n, m in zip(lengths, new)]
        for i, c in enumerate(s.caches):
            x, k, v = s.parts(i)
            q.kv_append(c, b, k, v, s.rope, x, s.turned[i], s.tree.positions, s.norms[i])
            got, lse = q.attn_paged(c, b, s.turned[i], tree=s.tree, return_lse=True)
            want = oracle.attn_paged(host(s.turned[i]), host(c.k), host(c.v), None, None, start, kv,
                                     host(s.tables.page_table), D ** -0.5, True, 0, host(s.tree.mask).view(np.uint64),
                                     host(s.tree.positions))
            attn_check(want, host(got), host(lse), D, f"{lengths} {new} layer {i}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_queries_in_place(q, fmt):
    """A fused projection's queries normalised and turned where they lie."""
    rng = np.random.default_rng(5)
    start, table = torch.tensor([0, 7, 40], dtype=torch.int32, device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda")
    b = q.PagedBatch(start, torch.tensor([20, 33], dtype=torch.int32, device="cuda"), table.view(2, 4), 33)
    norm, rope = q.HeadNorm(dev(projections(rng, (64,))), head_dim=64), q.Rope(64)
    for T in (40, 43):
        qkv = dev(projections(rng, (T, 8, 64)))
        other = qkv.clone()
        one, two = stale_pool(q, 8, 2, 16, 64, fmt), stale_pool(q, 8, 2, 16, 64, fmt)
        want = q.kv_append(one, b, qkv[:, 4:6], qkv[:, 6:], rope, qkv[:, :4], norm=norm)
        got = q.kv_append(two, b, other[:, 4:6], other[:, 6:], rope, other[:, :4], other[:, :4], norm=norm)
        assert torch.equal(got[:40].view(torch.int16), want[:40].view(torch.int16)) and torch.equal(
            other[:, 4:].view(torch.int16), qkv[:, 4:].view(torch.int16))
        assert torch.equal(other[40:].view(torch.int16), qkv[40:].view(torch.int16))
        assert torch.equal(one.k.view(torch.uint8), two.k.view(torch.uint8)) and torch.equal(one.v.view(torch.uint8), two.v.view(torch.uint8))
        x = qkv[:, :4].contiguous()
        want = q.norm_rope(x, norm, table[:1].expand(T).contiguous(), rope)
        assert q.norm_rope(x, norm, table[:1].expand(T).contiguous(), rope, out=x) is x
        assert torch.equal(x.view(torch.int16), want.view(torch.int16))


def test_empty_calls(q):
    """No tokens, no requests, requests without tokens: nothing is written and nothing fails."""
    i32 = dict(dtype=torch.int32, device="cuda")
    cache, rope, norm = stale_pool(q, 4, 2, 16, 64, "bf16"), q.Rope(64), q.HeadNorm(head_dim=64)
    before = cache.k.clone()
    none = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    for B in (0, 3):
        pool = q.PagePool.full(4, 16)
        tables = q.PageTables(pool, torch.full((B, 2), -1, **i32), 0, 1)
        zeros = torch.zeros(B, **i32)
        b = tables.reserve(zeros, zeros)
        tree = q.tree_plan(b, torch.empty(0, **i32))
        assert tree.mask.shape == (0, 1)
        out = q.kv_append(cache, b, none[:, :2], none[:, :2], rope, none, positions=tree.positions, norm=norm)
        assert out.shape == none.shape and q.norm_rope(none, norm, tree.positions, rope).shape == none.shape
        out, lse = q.attn_paged(cache, b, none, tree=tree, return_lse=True)
        assert out.shape == none.shape and lse.shape == (0, 4)
        assert q.kv_keep(cache, b, torch.zeros((B, 5), **i32), zeros).tolist() == [0] * B
        assert q.kv_keep(cache, b, torch.zeros((B, 0), **i32), zeros).tolist() == [0] * B
        tables.release(zeros)
        assert host(pool.count).tolist() == [4, 0] and host(b.q_start).tolist() == [0] * (B + 1)
    # rows that belong to no request
    x = torch.full((5, 8, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    b = q.PagedBatch(torch.zeros(4, **i32), torch.zeros(3, **i32), torch.zeros((3, 2), **i32), 1)
    tree = q.Tree(torch.full((5, 1), 7, dtype=torch.int64, device="cuda"), torch.full((5,), 7, **i32))
    q.tree_plan(b, torch.zeros(5, **i32), tree)
    assert (tree.mask == 7).all() and (tree.positions == 7).all()
    out = torch.full((5, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    q.kv_append(cache, b, x[:, 4:6], x[:, 6:], rope, x[:, :4], out, norm=norm)
    q.attn_paged(cache, b, x[:, :4], out=out, tree=tree)
    assert (out == 3.0).all() and torch.equal(cache.k.view(torch.int16), before.view(torch.int16))


def drafted_step(rng, s, new):
    """Rows, trees and an accepted chain of each request for a step of `new` tokens."""
    start, T = np.concatenate([[0], np.cumsum(new)]), int(sum(new))
    parents = trees(rng, new, "random")
    path, kept = np.zeros(s.path.shape, np.int32), np.zeros(len(new), np.int32)
    for b, n in enumerate(new):
        at, chain = n - 1, []
        while at >= 0:
            chain.append(at)
            at = int(parents[start[b] + at])
        kept[b] = len(chain)
        path[b, :kept[b]] = chain[::-1]
    return projections(rng, (LAYERS, T, (GROUP + 2) * HKV, s.qkv.shape[-1])), parents, path, kept


def load_step(s, new, x, parents, path, kept):
    s.qkv[:, :x.shape[1]].copy_(dev(x))
    s.parents[:len(parents)].copy_(dev(parents))
    for t, a in ((s.new, np.array(new, np.int32)), (s.path, path), (s.kept, kept)):
        t.copy_(dev(a))


@pytest.mark.parametrize("graph", [False, True])
def test_steps_that_lack_pages_are_dropped_and_tried_again(q, graph):
    """A pool that runs short tells so in count[1]. The step is dropped, before anything is
    kept (a release with the old lengths) or, where one graph holds it whole, after (a
    reservation of no tokens behind the new lengths, released to the old ones): the pool has
    its pages again, and once another request has ended the step gives what it gives with a
    pool that never runs short."""
    rng = np.random.default_rng(21)
    D, page, B, cols = 64, 16, 3, 12
    args = (q, B, D, page, "e4m3", cols, 200, 64, q.Rope(D), [q.HeadNorm(head_dim=D)] * LAYERS, 0)
    short, ample = Server(*args), Server(*args)
    short.pool.count.copy_(dev(np.array([10, 0], np.int32)))  # ten pages
    none = torch.zeros_like(short.lengths)
    if graph:
        side, recorded = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(recorded, stream=side):
            short.step()

    def held(lengths):
        return sum(-(-n // page) for n in lengths.tolist())

    drops = 0
    for new in ([20, 20, 20], [50, 50, 50], [30, 40, 30]):  # (the second needs twelve pages at least)
        while True:
            what = drafted_step(rng, short, new)
            for s in (short, ample):
                load_step(s, new, *what)
            before = short.lengths.clone()
            torch.cuda.synchronize()
            if graph:
                recorded.replay()
                torch.cuda.synchronize()
                lacking = int(short.pool.count[1])
                if lacking:
                    short.tables.reserve(short.lengths, none)
                    short.tables.release(before)
                    short.lengths.copy_(before)
            else:
                short.tables.reserve(short.lengths, short.new)
                lacking = int(short.pool.count[1])
                short.tables.release(short.lengths)  # (whole steps reserve for themselves)
                if not lacking:
                    short.step()
            if not lacking:
                break
            drops += 1
            assert host(short.pool.count)[0] == 10 - held(before)
            ends = int(np.argmax(new))
            new = [0 if b == ends else n for b, n in enumerate(new)]
            for s in (short, ample):
                s.tables.reserve(s.lengths, none)
                s.lengths[ends] = 0
                s.tables.release(s.lengths)
        ample.step()
        lengths = short.lengths
        assert torch.equal(lengths, ample.lengths)
        assert host(short.pool.count).tolist() == [10 - held(lengths), 0]
        for i in range(LAYERS):
            for b in range(B):
                for g, w in zip(rows_of(short, i, b, int(lengths[b])), rows_of(ample, i, b, int(lengths[b]))):
                    assert np.array_equal(g, w)
            assert torch.equal(short.out[i, :sum(new)].view(torch.int16), ample.out[i, :sum(new)].view(torch.int16))
    assert drops
    assert np.unique(host(short.pool.free)[:int(short.pool.count[0])]).size == int(short.pool.count[0])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_tables_of_prompts_serve_trees(q, oracle, fmt):
    """Tables with room for prompts, whose own batch is too long for trees, and a second batch
    over the same tensors for the steps of drafted tokens."""
    rng = np.random.default_rng(31)
    D, page, B, cols = 128, 32, 3, 70
    s = Server(q, B, D, page, fmt, cols, 4500, 2000, q.Rope(D), [q.HeadNorm(head_dim=D)] * LAYERS, 0)
    prompts = [2000, 7, 600]
    T = sum(prompts)
    s.qkv[:, :T].copy_(dev(projections(rng, (LAYERS, T, (GROUP + 2) * HKV, D))))
    s.new.copy_(dev(np.array(prompts, np.int32)))
    s.step(drafted=False)
    with pytest.raises(q.QlinError):
        q.tree_plan(s.tables.batch, s.parents, s.tree)
    steps = q.PagedBatch(s.tables.q_start, s.tables.kv_len, s.tables.page_table, 64)
    lengths = prompts
    for new in ([64, 1, 33], [5, 64, 0]):
        x, parents, path, kept = drafted_step(rng, s, new)
        load_step(s, new, x, parents, path, kept)
        T = sum(new)
        assert s.tables.reserve(s.lengths, s.new) is s.tables.batch
        parents, rows = s.parents[:T], [s.qkv[i, :T] for i in range(LAYERS)]
        tree = q.tree_plan(steps, parents)
        start, kv, table = host(steps.q_start), host(steps.kv_len), host(steps.page_table)
        assert kv.tolist() == [n + m for n, m in zip(lengths, new)]
        for i, c in enumerate(s.caches):
            n = GROUP * HKV
            turned = q.kv_append(c, steps, rows[i][:, n:n + HKV], rows[i][:, n + HKV:], s.rope, rows[i][:, :n],
                                 positions=tree.positions, norm=s.norms[i])
            got, lse = q.attn_paged(c, steps, turned, tree=tree, return_lse=True)
            e4 = (host(c.k_scale), host(c.v_scale)) if fmt == "e4m3" else (None, None)
            want = oracle.attn_paged(host(turned), host(c.k), host(c.v), *e4, start, kv, table, D ** -0.5, True, 0,
                                     host(tree.mask).view(np.uint64), host(tree.positions))
            attn_check(want, host(got), host(lse), D, f"{new} layer {i}")
        q.kv_keep(s.layers, steps, s.path, s.kept, s.lengths)
        s.tables.release(s.lengths)
        lengths = [n + int(k) for n, k in zip(lengths, kept)]
        assert s.lengths.tolist() == lengths
        assert host(s.pool.count).tolist() == [B * cols - sum(-(-n // page) for n in lengths), 0]
