"""Accepted tokens' rows moved together on the GPU against the oracle: copies, equal."""

import numpy as np
import pytest
import torch

from helpers import dev, host
from test_gpu_attn import make_batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    assert torch.cuda.is_available()
    return qlin


def random_cache(q, rng, pages, Hkv, page, D, fmt):
    c = q.PagedKV.empty(pages, Hkv, D, page, fmt)
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(dev(rng.integers(0, 256, t.view(torch.uint8).shape, dtype=np.uint8)))
    if fmt == "e4m3":
        for t in (c.k_scale, c.v_scale):
            t.copy_(dev(rng.random(t.shape, dtype=np.float32)))
    return c


def pools(c):
    return [host(t.view(torch.uint8) if t.dtype == torch.bfloat16 else t) for t in (c.k, c.v, c.k_scale, c.v_scale)
            if t is not None]


def paths(rng, new, width):
    """Ascending numbers of each sequence's new tokens, and how many of them are kept."""
    path, kept = rng.integers(-9, 9, (len(new), width)).astype(np.int32), np.zeros(len(new), np.int32)
    for b, n in enumerate(new):
        kept[b] = rng.integers(0, min(n, width) + 1)
        path[b, :kept[b]] = np.sort(rng.choice(n, kept[b], replace=False)) if n else 0
    return path, kept


def run_keep(q, oracle, rng, caches, start, kv, table, path, kept, layers=None):
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), 1)
    want = [pools(c) for c in caches]
    got = q.kv_keep(layers or q.PagedLayers(caches), b, dev(path), dev(kept))
    for c, w in zip(caches, want):
        lengths = oracle.kv_keep(w, start, kv, table, path, kept)
        assert np.array_equal(host(got), lengths)
        for g, x in zip(pools(c), w):
            assert np.array_equal(g.view(np.uint8), x.view(np.uint8))  # (the bytes: bf16 NaNs and scales too)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page,Hkv,layers", [(64, 16, 1, 1), (128, 64, 8, 3), (128, 16, 2, 35), (256, 32, 5, 2),
                                               (256, 256, 40, 1), (64, 32, 130, 1)])
def test_keep(q, oracle, D, page, Hkv, layers, fmt):
    rng = np.random.default_rng(D + page + Hkv)
    new, kv = [1, 0, 8, 40, 3, 17], [page, 9, 8, 3 * page + 41, 30, 2 * page + 5]
    start, table, pages = make_batch(rng, new, kv, page)
    caches = [random_cache(q, rng, pages, Hkv, page, D, fmt) for _ in range(layers)]
    for width in (40, 3, 1):
        path, kept = paths(rng, new, width)
        run_keep(q, oracle, rng, caches, start, kv, table, path, kept)
    path = np.tile(np.arange(40, dtype=np.int32), (6, 1))  # all kept: nothing moves
    run_keep(q, oracle, rng, caches, start, kv, table, path, np.full(6, 2 ** 31 - 1, np.int32))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (8, 128), (24, 256)])
def test_long_paths(q, oracle, Hkv, D, fmt):
    """Paths of many passes, each of whose places are sources of later ones."""
    rng = np.random.default_rng(Hkv)
    new, kv = [500, 1100, 60], [700, 1100, 300]
    start, table, pages = make_batch(rng, new, kv, 16)
    cache = random_cache(q, rng, pages, Hkv, 16, D, fmt)
    path = np.zeros((3, 1024), np.int32)
    kept = np.array([499, 1024, 30], np.int32)
    for b, n in enumerate(new):
        path[b, :kept[b]] = np.sort(rng.choice(n, kept[b], replace=False))
    run_keep(q, oracle, rng, [cache], start, kv, table, path, kept, layers=cache)
    path[0, :499] = np.arange(1, 500)  # everything one place down
    run_keep(q, oracle, rng, [cache], start, kv, table, path, kept)


def test_state_of_any_value(q, oracle):
    """Numbers outside the new tokens, pages outside the pool, lengths below the new tokens
    and behind the table, counts of any size: those rows stay."""
    rng = np.random.default_rng(7)
    new, kv = [8, 8, 8, 8, 8, 0], [100, 40, 5, 2 ** 31 - 1, -3, 2 ** 31 - 1]
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    table = rng.permutation(48)[:42].reshape(6, 7).astype(np.int32)
    table[0, 5], table[1, 2] = 48, -1
    cache = random_cache(q, rng, 48, 2, 16, 64, "e4m3")
    path = np.array([[0, 2, 5, 7], [1, 4, 6, 7], [4, 5, 6, 7], [1, 2, 3, 4], [1, 2, 3, 4], [0, 0, 0, 0]], np.int32)
    for kept in ([4, 4, 4, 4, 4, 4], [2 ** 31 - 1, -2 ** 31, 3, 0, 9, -1]):
        run_keep(q, oracle, rng, [cache], start, kv, table, path, np.array(kept, np.int32))
    path[0, 1], path[1, 0], path[2, 3] = 8, -1, 2 ** 31 - 1
    run_keep(q, oracle, rng, [cache], start, kv, table, path, np.full(6, 4, np.int32))
    run_keep(q, oracle, rng, [cache], start, kv, table, path[:, :0], np.full(6, 4, np.int32))


def test_pool_beyond_32_bit_offsets(q, oracle):
    D, Hkv, page = 256, 8, 256
    pages = (1 << 32) // (Hkv * page * D * 2) + 40
    rng = np.random.default_rng(8)
    cache = q.PagedKV.empty(pages, Hkv, D, page)
    used = [pages - 1, 3, pages - 7]
    rows = dev(rng.integers(0, 30000, (3, Hkv, page, D)).astype(np.int16)).view(torch.bfloat16)
    for c in (cache.k, cache.v):
        c[used] = rows
    small = [host(rows) for _ in range(2)]
    start, kv, path, kept = [0, 300], [700], np.arange(1, 300, 3, dtype=np.int32)[None], np.array([100], np.int32)
    b = q.PagedBatch(dev(np.array(start, np.int32)), dev(np.array(kv, np.int32)), dev(np.array([used], np.int32)), 300)
    got = q.kv_keep(cache, b, dev(path), dev(kept))
    assert host(got).tolist() == oracle.kv_keep(small, start, kv, np.array([[0, 1, 2]]), path, kept).tolist() == [500]
    for c, w in zip((cache.k, cache.v), small):
        assert np.array_equal(host(c[used]), w)


def test_graph_replays(q, oracle):
    rng = np.random.default_rng(9)
    new, kv = [30, 12, 25], [90, 12, 300]
    start, table, pages = make_batch(rng, new, kv, 16)
    cache = random_cache(q, rng, pages, 4, 16, 128, "e4m3")
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), 30)
    path, kept = torch.zeros((3, 9), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    lengths, layers = torch.zeros_like(kept), q.PagedLayers([cache])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            assert q.kv_keep(layers, b, path, kept, lengths) is lengths
    for _ in range(4):
        pa, kp = paths(rng, new, 9)
        path.copy_(dev(pa))
        kept.copy_(dev(kp))
        want = pools(cache)
        graph.replay()
        torch.cuda.synchronize()
        assert host(lengths).tolist() == oracle.kv_keep(want, start, kv, table, pa, kp).tolist()
        for g, x in zip(pools(cache), want):
            assert np.array_equal(g.view(np.uint8), x.view(np.uint8))


def test_keep_binding_refusals(q):
    i32 = dict(dtype=torch.int32, device="cuda")
    one, two = q.PagedKV.empty(4, 2, 64, 16), q.PagedKV.empty(4, 2, 64, 16, "e4m3")
    b = q.PagedBatch(torch.tensor([0, 8], **i32), torch.tensor([8], **i32), torch.zeros((1, 2), **i32), 8)
    path, kept = torch.zeros((1, 4), **i32), torch.zeros(1, **i32)
    for bad in ((one, two), (one, q.PagedKV.empty(5, 2, 64, 16)), ()):
        with pytest.raises(ValueError):
            q.PagedLayers(bad)
    for args in ((path[:0], kept), (path, torch.zeros(2, **i32)), (path.cpu(), kept), (path, kept, torch.zeros(2, **i32))):
        with pytest.raises(ValueError):
            q.kv_keep(one, b, *args)
    with pytest.raises(TypeError):
        q.kv_keep(one, b, path.long(), kept)
    with pytest.raises(q.QlinError):
        q.kv_keep(one, b, path, kept, b.kv_len)


def test_caches_that_share_memory(q):
    c = q.PagedKV.empty(8, 2, 64, 16)
    for caches in ([c, c], [c, q.PagedKV(c.v, torch.empty_like(c.v))], [q.PagedKV(c.k, c.k)]):
        with pytest.raises(ValueError):
            q.PagedLayers(caches)
    whole = torch.empty(17, 2, 16, 64, dtype=torch.bfloat16, device="cuda")  # neighbours in one allocation
    q.PagedLayers([q.PagedKV(whole[:8], c.v), q.PagedKV(whole[8:16], c.k)])
    with pytest.raises(ValueError):
        q.PagedLayers([q.PagedKV(whole[:8], c.v), q.PagedKV(whole[7:15], c.k)])
    e = [q.PagedKV.empty(4, 2, 64, 16, "e4m3") for _ in range(2)]
    q.PagedLayers(e)
    with pytest.raises(ValueError):
        q.PagedLayers([e[0], q.PagedKV(e[1].k, e[1].v, e[0].v_scale, e[1].v_scale)])
