"""Attention of trees of new tokens over the paged cache, and the trees' masks, on the GPU
against the fp64 oracle. Bounds as in the tests of attention (attn_check)."""

import numpy as np
import pytest
import torch

from helpers import dev, host
from test_abi_tree_host import KERNELS
from test_gpu_attn import attn_check, bits, fill_cache, long_table, make_batch, projections, stale_pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    assert torch.cuda.is_available()
    return qlin


def trees(rng, new, shape="any"):
    """Parents of every sequence's tokens: chains, wide trees, random ones, forests."""
    out = []
    for n in new:
        kind = shape if shape != "any" else rng.choice(["chain", "wide", "random", "forest"])
        for i in range(n):
            at = i - 1
            if kind == "wide":
                at = (i - 1) // 3 if i else -1
            elif kind == "random" and i:
                at = int(rng.integers(0, i))
            elif kind == "forest":
                at = -1 if rng.random() < 0.4 else int(rng.integers(-1, i)) if i else -1
            out.append(at)
    return np.array(out, np.int32)


def planned(oracle, start, kv, parents, words, T):
    mask, pos = np.zeros((T, words), np.uint64), np.zeros(T, np.int32)
    oracle.tree_plan(start, kv, parents, words, mask[:len(parents)], pos[:len(parents)])
    return mask, pos


def run_tree(q, oracle, seed, new, kv, Hkv, G, D, page, fmt, words=1, window=0, pad=0, extra_cols=0, shape="any",
             edit=None, table_edit=None, scale=None, max_q=None, use_positions=True):
    rng = np.random.default_rng(seed)
    start, table, pages = make_batch(rng, new, kv, page)
    if extra_cols:
        table = np.concatenate([table, np.full((len(kv), extra_cols), -1, np.int32)], 1)
    cache = stale_pool(q, pages, Hkv, page, D, fmt)
    fill_cache(q, rng, cache, start, np.array(kv), table)
    if table_edit is not None:
        table_edit(table)
    T = int(start[-1]) + pad
    x = projections(rng, (T, Hkv * G, D))
    mask, pos = planned(oracle, start, kv, trees(rng, new, shape), words, T)
    if edit is not None:
        edit(rng, mask, pos)
    sc = D ** -0.5 if scale is None else scale
    batch = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), max(new) if max_q is None else max_q)
    tree = q.Tree(dev(mask.view(np.int64)), dev(pos) if use_positions else None)
    out = torch.full((T, Hkv * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got, lse = q.attn_paged(cache, batch, dev(x), scale=sc, window=window, out=out, return_lse=True, tree=tree)
    assert got is out
    torch.cuda.synchronize()
    e4 = fmt == "e4m3"
    r = oracle.attn_paged(x, host(cache.k), host(cache.v), host(cache.k_scale) if e4 else None,
                          host(cache.v_scale) if e4 else None, start, kv, table, sc, True, window, mask, pos)
    attn_check(r, host(got), host(lse), D, f"new={new} kv={kv} D={D} page={page} {fmt}")
    assert (host(got)[int(start[-1]):] == 0x40E0).all(), "padding rows were written"
    return r


# ------------------------------------------------------------------ masks
@pytest.mark.parametrize("new,words", [([1], 1), ([8], 1), ([64, 0, 3, 1, 63], 1), ([65, 128, 1], 2), ([70, 200, 0, 192], 4),
                                       ([512, 1, 300], 8), ([5] * 700, 1), ([33, 2], 8)])
def test_plan(q, oracle, new, words):
    rng = np.random.default_rng(len(new) + words)
    for shape in ("chain", "wide", "random", "forest", "any"):
        parents = trees(rng, new, shape)
        parents[rng.random(len(parents)) < 0.02] = 2 ** 31 - 1  # no earlier token: from the tokens before
        parents[rng.random(len(parents)) < 0.02] = -2 ** 31
        kv = [n + int(rng.integers(0, 9000)) for n in new]
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T, pad = int(start[-1]), 3
        mask, pos = np.full((T + pad, words), 77, np.uint64), np.full(T + pad, 77, np.int32)
        tree = q.Tree(dev(mask.view(np.int64)), dev(pos))
        oracle.tree_plan(start, kv, np.concatenate([parents, np.zeros(pad, np.int32)]), words, mask, pos)
        batch = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(np.zeros((len(new), 1), np.int32)), max(new))
        got = q.tree_plan(batch, dev(np.concatenate([parents, np.zeros(pad, np.int32)])), tree)
        assert got is tree
        assert np.array_equal(host(tree.mask).view(np.uint64), mask)
        assert np.array_equal(host(tree.positions), pos)
        # positions left out; a tree of its own
        bare = q.Tree(torch.full_like(tree.mask, 77))
        q.tree_plan(batch, dev(np.concatenate([parents, np.zeros(pad, np.int32)])), bare)
        assert torch.equal(bare.mask, tree.mask)
        same = dev(np.concatenate([parents, np.full(pad, 77, np.int32)]))  # positions in the parents' place
        q.tree_plan(batch, same, q.Tree(bare.mask, same))
        assert torch.equal(same, tree.positions) and torch.equal(bare.mask, tree.mask)
        own = q.tree_plan(batch, dev(parents))
        wide = own.mask.shape[1]
        assert wide == -(-max(new) // 64) and torch.equal(own.mask, tree.mask[:T, :wide])


def test_plan_of_more_tokens_than_bits(q, oracle):
    """A sequence longer than max_q says (device data): its first tokens are right, the
    others' rows are not written."""
    parents = np.array([-1, 0, 1] + list(range(2, 99)) + [-1, 0], np.int32)
    start, kv = np.array([0, 100, 102], np.int32), [130, 2]
    mask, pos = np.full((102, 1), 5, np.uint64), np.full(102, 5, np.int32)
    tree = q.Tree(dev(mask.view(np.int64)), dev(pos))
    oracle.tree_plan(start, kv, parents, 1, mask, pos)
    q.tree_plan(q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(np.zeros((2, 1), np.int32)), 8), dev(parents), tree)
    assert np.array_equal(host(tree.mask).view(np.uint64), mask) and np.array_equal(host(tree.positions), pos)
    assert (mask[64:100] == 5).all()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page,Hkv,G", [(64, 16, 2, 4), (64, 64, 1, 8), (128, 16, 2, 4), (128, 128, 1, 5), (128, 32, 3, 1),
                                          (256, 16, 1, 2), (256, 256, 2, 2)])
def test_tree(q, oracle, D, page, Hkv, G, fmt):
    # lengths around the tiles of 32 keys: the trees' first tokens at every place in one
    new = [1, 8, 3, 0, 7, 16, 5, 12, 16, 9]
    kv = [1, 8, 35, 9, 39, 47, 69, 143, 200, 321]
    run_tree(q, oracle, D + page, new, kv, Hkv, G, D, page, fmt, pad=3)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,Hkv", [(64, 1), (128, 1), (256, 1), (64, 40), (128, 24), (256, 24)])
def test_tree_long_table(q, oracle, D, Hkv, fmt):
    """The chunks' kernels, whole and in parts."""
    run_tree(q, oracle, D, [64, 33, 0, 50, 1], [64, 133, 9, 1050, 90], Hkv, 4, D, 16, fmt, pad=2,
             extra_cols=long_table(16))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", KERNELS)
def test_tree_kernels(q, oracle, name, D, fmt):
    """Every variant of the kernels; which one a case runs is pinned beside the plans."""
    new, words, Hkv, G, keys, _ = KERNELS[name]
    keys = keys[(64, 128, 256).index(D)][fmt == "e4m3"]
    rng = np.random.default_rng(D)
    kv = [n + int(rng.integers(0, min(keys, 500) - 16 * words)) for n in new]
    if keys > 1024:
        kv[0] = new[0] + 1000
    cols = max(-(-k // 16) for k in kv)
    run_tree(q, oracle, D, new, kv, Hkv, G, D, 16, fmt, words=words, extra_cols=keys // 16 - cols, pad=1)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("more", [0, long_table(16)])
@pytest.mark.parametrize("words,new", [(2, [65, 128, 100]), (4, [256, 7, 129]), (8, [512, 449]), (8, [3, 60])])
def test_tree_words(q, oracle, words, new, more, fmt):
    run_tree(q, oracle, words, new, [n + m for n, m in zip(new, (77, 0, 450))], 1, 3, 128, 16, fmt, words=words,
             extra_cols=more, shape="random")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_split_over_keys(q, oracle, D, fmt):
    run_tree(q, oracle, 7, [8, 5, 16], [1500, 5, 700], 2, 2, D, 64, fmt, extra_cols=40)
    run_tree(q, oracle, 8, [16], [2500], 1, 4, D, 64, fmt, extra_cols=9)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("more", [0, long_table(16)])
@pytest.mark.parametrize("window", [64, 65, 100, 333, 2 ** 40])
def test_tree_window(q, oracle, window, more, fmt):
    def edit(rng, mask, pos):  # positions before the first and behind the last token: the nearest of those
        pos[3], pos[10], pos[70] = -5, 2 ** 31 - 1, 0

    run_tree(q, oracle, 3, [64, 30, 5, 1], [300, 33, 200, 500], 2, 2, 128, 16, fmt, window=window, extra_cols=more)
    run_tree(q, oracle, 4, [64, 30, 5, 1], [300, 133, 200, 500], 1, 1, 64, 16, fmt, window=window, extra_cols=more,
             edit=edit)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("more", [0, long_table(16)])
def test_any_mask(q, oracle, more, fmt):
    """Masks that are no trees: random bits, bits of later tokens and behind the last
    one, none at all (rows that see only the earlier tokens, or nothing)."""
    def edit(rng, mask, pos):
        mask[:] = rng.integers(0, 2 ** 64, mask.shape, dtype=np.uint64)
        mask[5] = mask[41] = mask[42] = 0
        mask[6] = np.uint64(2 ** 64 - 1)

    r = run_tree(q, oracle, 5, [40, 40, 20], [90, 40, 500], 2, 4, 128, 16, fmt, extra_cols=more, edit=edit)
    assert (r["seen"][41] == 0).all() and (r["seen"][5] == 50).all() and (r["seen"][6] == 90).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("more", [0, long_table(16)])
def test_tree_shorter_sequences_and_missing_pages(q, oracle, more, fmt):
    """Fewer cached keys than new tokens (the first lie before the sequence), none, and
    pages that do not exist among earlier and new tokens."""
    def edit(t):
        t[0, 1] = -1
        t[0, 5] = 10 ** 9
        t[3, :] = 2 ** 31 - 1

    run_tree(q, oracle, 6, [40, 9, 7, 5], [130, 3, 0, 33], 2, 3, 128, 16, fmt, extra_cols=more, table_edit=edit)


def test_tree_longer_than_its_table(q, oracle):
    """Tokens behind the table's reach are not seen, whatever the mask says."""
    rng = np.random.default_rng(4)
    start, table, pages = make_batch(rng, [8], [64], 16)
    cache = stale_pool(q, pages, 1, 16, 64, "bf16")
    fill_cache(q, rng, cache, start, np.array([64]), table)
    x = projections(rng, (8, 2, 64))
    for length in (64, 66, 71, 72, 90, 2 ** 31 - 1):
        mask, pos = planned(oracle, start, [length], trees(rng, [8], "chain"), 1, 8)
        b = q.PagedBatch(dev(start), dev(np.array([length], np.int32)), dev(table), 8)
        got, lse = q.attn_paged(cache, b, dev(x), return_lse=True, tree=q.Tree(dev(mask.view(np.int64))))
        r = oracle.attn_paged(x, host(cache.k), host(cache.v), None, None, start, [length], table, 0.125, mask=mask)
        attn_check(r, host(got), host(lse), 64, f"length {length}")


@pytest.mark.parametrize("new,kv,more", [([8, 5], [300, 40], 0), ([60, 33], [300, 100], 0), ([60, 33], [300, 100], long_table(16))])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_chain_is_causal(q, oracle, new, kv, more, fmt):
    """A tree that is a chain sees what a causal call sees (both are within the bounds;
    here of each other, two roundings to bf16 and the weights' apart)."""
    rng = np.random.default_rng(8)
    start, table, pages = make_batch(rng, new, kv, 16)
    table = np.concatenate([table, np.full((2, more), -1, np.int32)], 1)
    cache = stale_pool(q, pages, 2, 16, 128, fmt)
    fill_cache(q, rng, cache, start, np.array(kv), table)
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), max(new))
    x = dev(projections(rng, (int(start[-1]), 8, 128)))
    tree = q.tree_plan(b, dev(trees(rng, new, "chain")))
    for window in (0, 80):
        got, l1 = q.attn_paged(cache, b, x, return_lse=True, tree=tree, window=window)
        want, l2 = q.attn_paged(cache, b, x, return_lse=True, window=window)
        top = cache.v.float().nan_to_num().abs().max() if fmt == "bf16" else 448 * cache.v_scale.nan_to_num().max()
        assert (got.float() - want.float()).abs().max() <= 4 * 2.0 ** -8 * top
        assert (l1 - l2).abs().max() <= 1e-4


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_tree_strides_and_scales(q, oracle, fmt):
    run_tree(q, oracle, 51, [8, 6], [90, 61], 1, 4, 128, 16, fmt, scale=-0.09)
    run_tree(q, oracle, 52, [60, 40], [90, 61], 1, 2, 128, 16, fmt, scale=0.0, extra_cols=long_table(16))
    run_tree(q, oracle, 53, [8, 6], [90, 61], 1, 4, 128, 16, fmt, max_q=64, use_positions=False)
    rng = np.random.default_rng(54)
    start, table, pages = make_batch(rng, [9, 20], [70, 33], 16)
    cache = stale_pool(q, pages, 2, 16, 64, fmt)
    fill_cache(q, rng, cache, start, np.array([70, 33]), table)
    b = q.PagedBatch(dev(start), dev(np.array([70, 33], np.int32)), dev(table), 20)
    qkv = dev(projections(rng, (29, 12, 64)))
    tree = q.tree_plan(b, dev(trees(rng, [9, 20])))
    want = q.attn_paged(cache, b, qkv[:, 2:8].contiguous(), tree=tree)
    out = torch.full((29, 9, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q.attn_paged(cache, b, qkv[:, 2:8], out=out[:, 3:], tree=tree)
    assert torch.equal(out[:, 3:].contiguous().view(torch.int16), want.view(torch.int16))
    assert (out[:, :3] == 7).all()


def test_queries_that_are_not_finite_stay_in_their_rows(q):
    """And keys that are not finite in the rows that see them: a masked score is never
    looked at."""
    rng = np.random.default_rng(55)
    for new, kv, more in (([8, 8], [40, 70], 0), ([60, 40], [300, 100], long_table(16))):
        start, table, pages = make_batch(rng, new, kv, 16)
        table = np.concatenate([table, np.full((2, more), -1, np.int32)], 1)
        cache = stale_pool(q, pages, 1, 16, 128, "bf16")
        fill_cache(q, rng, cache, start, np.array(kv), table)
        b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), max(new))
        x = dev(projections(rng, (int(start[-1]), 4, 128)))
        tree = q.tree_plan(b, dev(trees(rng, new, "wide")))
        want, wl = q.attn_paged(cache, b, x, tree=tree, return_lse=True)
        node = 3  # of the first sequence: it and its descendants (10 to 12, of 60 tokens) see it
        at = kv[0] - new[0] + node
        cache.k[int(table[0, at // 16]), :, at % 16] = float("nan")
        got, gl = q.attn_paged(cache, b, x, tree=tree, return_lse=True)
        sees = ((tree.mask[:, 0] >> node) & 1).bool()
        sees[new[0]:] = False
        assert got[sees].isnan().all() and sees.any()
        assert torch.equal(got[~sees].view(torch.int16), want[~sees].view(torch.int16)) and torch.equal(gl[~sees], wl[~sees])


def test_tree_graph_and_streams(q):
    """Captured plan and attention on a stream of its own, replayed with other parents,
    keys and queries, with eager calls between."""
    rng = np.random.default_rng(56)
    for new, kv, cols in (([8] * 5, [800, 30, 8, 500, 61], 60), ([64] * 3, [900, 64, 301], long_table(16))):
        start, table, pages = make_batch(rng, new, kv, 16)
        table = np.concatenate([table, np.full((len(new), cols), -1, np.int32)], 1)
        cache = stale_pool(q, pages, 2, 16, 128, "e4m3")
        fill_cache(q, rng, cache, start, np.array(kv), table)
        b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), max(new))
        T = int(start[-1])
        x, parents = dev(projections(rng, (T, 8, 128))), dev(trees(rng, new))
        tree = q.Tree.empty(T)
        side = torch.cuda.Stream()

        def step():
            q.tree_plan(b, parents, tree)
            return q.attn_paged(cache, b, x, tree=tree, return_lse=True)

        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out, lse = step()
        for turn in range(4):
            x.copy_(dev(projections(rng, (T, 8, 128))))
            parents.copy_(dev(trees(rng, new)))
            b.kv_len.copy_(dev(np.array([max(n, m - turn) for n, m in zip(new, kv)], np.int32)))
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone(), lse.clone()
            want = step()
            assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])


def test_tree_binding_refusals(q):
    cache = q.PagedKV.empty(4, 2, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    b = q.PagedBatch(torch.tensor([0, 8], **i32), torch.tensor([8], **i32), torch.zeros((1, 2), **i32), 8)
    x = torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda")
    tree = q.Tree.empty(8)
    for bad, kw in ((q.Tree.empty(7), {}), (tree, dict(causal=False))):
        with pytest.raises(ValueError):
            q.attn_paged(cache, b, x, tree=bad, **kw)
    with pytest.raises(q.QlinError):  # a window below max_q
        q.attn_paged(cache, b, x, tree=tree, window=7)
    with pytest.raises(q.QlinError):  # a window without positions
        q.attn_paged(cache, b, x, tree=q.Tree(tree.mask), window=8)
    wide = q.PagedBatch(b.q_start, b.kv_len, b.page_table, 65)
    for call in (lambda: q.attn_paged(cache, wide, x, tree=tree), lambda: q.tree_plan(wide, torch.zeros(8, **i32), tree),
                 lambda: q.tree_plan(b, torch.zeros(8, **i32), q.Tree.empty(8, 9))):
        with pytest.raises(q.QlinError):
            call()
    with pytest.raises(TypeError):
        q.Tree(tree.mask.int())
    with pytest.raises(ValueError):
        q.Tree(tree.mask, torch.zeros(7, **i32))
    with pytest.raises(ValueError):
        q.tree_plan(b, torch.zeros(7, **i32), tree)
    with pytest.raises(ValueError):
        q.tree_plan(b, torch.zeros(8, dtype=torch.int32), tree)
    assert q.tree_plan(b, torch.zeros(0, **i32)).mask.shape == (0, 1)
