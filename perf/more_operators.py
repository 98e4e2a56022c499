"""What the operators of a step that verifies drafted tokens are measured on.

A served model may let a cheaper one draft several next tokens of each request, as
a tree (a token's parent is the drafted token that it follows), and verify all of
them in one step over the paged key/value cache:

  tables  the step's tables from the requests' lengths: where each request's
          tokens start, its new pages, every token's slot and position; and the
          pages back to the pool when the step is dropped
  plan    the tree's masks (a token's ancestors) and positions from the parents
  norm    queries, keys and values normalised for each head, rotated, and the
          keys and values appended to the cache; or queries alone
  tree    attention of a tree's tokens: the cached tokens and their own ancestors
  keep    the accepted tokens' keys and values moved together, in every layer

Each case is one call of one of them (``tables``: the two calls of a step that
is dropped). ``run`` computes it in plain torch operations, or, where ``own`` is set,
with the library's entry points.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def _tables(name, batch, new, context, page, **more):
    return dict(name=name, op="tables", batch=batch, new=new, context=context, page=page, ragged=True,
                mix=1, **more)


def _plan(name, batch, new, **more):
    return dict(name=name, op="plan", batch=batch, new=new, context=4096, page=64, ragged=True, mix=1, **more)


def _heads_case(name, op, batch, new, context, q_heads, kv_heads, dim, page, fmt, **more):
    c = dict(name=name, op=op, batch=batch, new=new, context=context, q_heads=q_heads, kv_heads=kv_heads,
             dim=dim, page=page, fmt=fmt, ragged=True, mix=1)
    if op == "norm":
        c.update(rot=dim, interleaved=False, offset=0.0, eps=1e-6, values=False, tree=False)
    elif op == "tree":
        c.update(window=0)
    elif op == "keep":
        c.update(layers=1)
    c.update(more)
    return c


def listed():
    return [
        # the tables of a step of 64 requests with up to 16 drafted tokens each
        _tables("tables_step", 64, 16, 4096, 64),
        # 64 new prompts of up to 8192 tokens, the smallest pages
        _tables("tables_prompts", 64, 8192, 8192, 16),
        # one request's tree of 8 drafted tokens: latency
        _plan("plan_one", 1, 8),
        # 256 requests with trees of up to 256 tokens
        _plan("plan_many", 256, 256),
        # 8 requests that verify trees of 8 tokens: the smallest append
        _heads_case("norm_step_bf16", "norm", 8, 8, 1536, 32, 8, 128, 64, "bf16", tree=True),
        # three odd chunks, wide heads, values normalised too, weights stored less
        # one, half of each head turning, FP8 in the smallest pages
        _heads_case("norm_chunk_fp8", "norm", 3, 1111, 4099, 16, 4, 256, 16, "e4m3", rot=128,
                    offset=1.0, values=True),
        # the queries of a prompt batch of 8192 tokens in a layer that reads another
        # layer's cache
        _heads_case("norm_queries", "norm", 1, 8192, 8192, 32, 0, 128, 64, "none", interleaved=True),
        # one request with a tree of 8 after a 1024-token prompt: latency
        _heads_case("tree_one", "tree", 1, 8, 1025, 32, 8, 128, 16, "bf16"),
        # 64 requests of many lengths with trees of up to 16 over an FP8 cache
        _heads_case("tree_fp8", "tree", 64, 16, 4096, 32, 8, 128, 64, "e4m3"),
        # 8 long contexts with trees of 64: 1 GB of cache
        _heads_case("tree_long", "tree", 8, 64, 32768, 32, 8, 128, 64, "bf16", ragged=False),
        # one request's accepted tokens in 16 layers: latency
        _heads_case("keep_one", "keep", 1, 16, 128, 0, 8, 128, 64, "bf16", layers=16),
        # 64 requests' accepted tokens of trees of up to 48 in 16 layers, FP8
        _heads_case("keep_many", "keep", 64, 48, 160, 0, 8, 128, 32, "e4m3", layers=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "plan", "norm", "norm", "tree", "tree", "tree", "keep"])
    ragged, mix = rng.random() < 0.8, rng.randint(1, 1 << 20)
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "tables":
        new = rng.choice([1, 1, 4, 16, 61]) if rng.random() < 0.5 else _log(rng, 16, 8192)
        c = _tables("", _log(rng, 1, 4096), new, max(new, _log(rng, 16, 32768)), page)
        while c["batch"] * c["new"] > 64 * 8192 or c["batch"] * c["context"] > 64 * 8192 * page // 16:
            c["batch"] = c["batch"] // 2 or 1
            c["new"] = max(1, c["new"] * 3 // 4)
            c["context"] = max(c["new"], c["context"] * 3 // 4)
    elif op == "plan":
        c = _plan("", _log(rng, 1, 2048), _log(rng, 1, 512))
        while c["batch"] * c["new"] * -(-c["new"] // 64) > 170 * 256 * 4:
            c["batch"] //= 2
    else:
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
        q_heads = kv_heads * rng.choice([1, 2, 4, 4, 5, 8])
        fmt = rng.choice(["bf16", "e4m3"])
        if op == "norm":
            step = rng.random() < 0.5
            new = rng.choice([1, 1, 2, 8, 33]) if step else _log(rng, 16, 8192)
            c = _heads_case("", op, _log(rng, 1, 256 if step else 16), new, max(new, _log(rng, 16, 16384)),
                            q_heads, kv_heads, dim, page, fmt, rot=rng.choice([dim, dim, dim // 2, dim // 4]),
                            interleaved=rng.random() < 0.5, offset=rng.choice([0.0, 1.0]),
                            eps=rng.choice([1e-6, 1e-5, 1e-3]), values=rng.random() < 0.5,
                            tree=step and rng.random() < 0.5)
            if rng.random() < 0.25:
                c.update(kv_heads=0, fmt="none", values=False)
            while _too_large(c):
                _shrink(c)
        elif op == "tree":
            c = _heads_case("", op, _log(rng, 1, 256), _log(rng, 1, 256), 1, q_heads, kv_heads, dim, page, fmt)
            c["context"] = max(c["new"], _log(rng, 16, 65536))
            if rng.random() < 0.25:
                c["window"] = _log(rng, 256, 8192)
            while _too_large(c):
                _shrink(c)
        else:
            c = _heads_case("", op, _log(rng, 1, 128), _log(rng, 1, 256), 1, 0, kv_heads, dim, page, fmt,
                            layers=_log(rng, 1, 64))
            c["context"] = c["new"] + rng.randint(0, 200)
            while _too_large(c):
                c["layers"] = max(1, c["layers"] // 2)
                c["batch"] = max(1, c["batch"] // 2)
    c.update(ragged=ragged, mix=mix)
    del c["name"]
    return c


def _shrink(c):
    if c["batch"] > 1:
        c["batch"] //= 2
    elif c["context"] > 2 * c["new"]:
        c["context"] //= 2
    else:
        c["new"] = c["new"] * 2 // 3
        c["context"] = max(c["new"], c["context"] * 3 // 4)


def _too_large(c):
    """Whether a drawn case costs more than the largest listed one of its kind (in
    cached bytes, moved bytes or products, also as padded rectangles)."""
    if c["op"] == "norm":
        cached = 2 * c["batch"] * (c["context"] + c["page"]) * c["kv_heads"] * c["dim"]
        return cached > 2 * 8 * 8192 * 8 * 128 or (
            c["batch"] * c["new"] * (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"] > 8192 * 32 * 128)
    if c["op"] == "keep":
        pool = c["batch"] * (c["context"] + c["page"]) * c["kv_heads"] * c["dim"] * c["layers"]
        return pool > 64 * 192 * 8 * 128 * 16
    if 2 * c["batch"] * (c["context"] + c["page"]) * c["kv_heads"] * c["dim"] > 2 * 8 * 33000 * 8 * 128:
        return True
    pairs = c["batch"] * c["new"] * c["context"] * c["q_heads"]
    return pairs > 8 * 64 * 32768 * 32 or pairs * c["dim"] > 8 * 64 * 32768 * 32 * 128


def _lengths(c):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    r = random.Random(c["mix"])
    new, kv = [c["new"]], [c["context"]]
    for _ in range(c["batch"] - 1):
        n = r.randint(max(1, c["new"] // 3), c["new"]) if c["ragged"] else c["new"]
        most = c["context"] - c["new"]
        new.append(n)
        kv.append(n + (r.randint(most // 4, most) if c["ragged"] else most))
    return new, kv


def _parents(c):
    """Each sequence's tree: every token's parent among the tokens before it, -1 for
    one that follows the cached tokens. Level by level with one to four children, a
    chain at one end and a wide tree at the other, some tokens elsewhere."""
    r = random.Random(c["mix"] + 1)
    trees = []
    for n in _lengths(c)[0]:
        width = r.randint(1, 4)
        tree = []
        for i in range(n):
            at = (i - 1) // width if i else -1
            if i and r.random() < 0.2:
                at = r.randint(-1, i - 1)
            tree.append(at)
        trees.append(tree)
    return trees


def _ancestors(tree):
    """For each token the numbers of its ancestors and itself."""
    seen = []
    for i, at in enumerate(tree):
        seen.append((seen[at] if at >= 0 else []) + [i])
    return seen


def _accepted(c):
    """The accepted tokens of each sequence, numbers among its new ones, ascending.
    (Those that move come from behind the places that are written, as in a tree whose
    first levels are wide: the call can be made again on what it left.)"""
    r = random.Random(c["mix"] + 2)
    paths = []
    for n in _lengths(c)[0]:
        kept = r.randint(1, max(1, min(n // 2, 12)))
        stay = r.randint(1, kept) if r.random() < 0.2 else 1
        paths.append(list(range(stay)) + sorted(r.sample(range(kept, n), kept - stay)))
    return paths


# ------------------------------------------------------------------ inputs
BASE = 10000.0


def _heads(shape, gen, gain=1.0):
    """bf16 projections: normal values, one channel in a hundred large."""
    x = torch.randn(shape, generator=gen, device=DEV)
    big = torch.rand(shape[-1], generator=gen, device=DEV) < 0.01
    return (x * torch.where(big, 6.0 * gain, gain)).to(torch.bfloat16)


def _pool(shape, fmt, gen):
    """A cache's pages, filled as earlier tokens leave them: bf16 rows, or E4M3
    codes of rows over their largest magnitude / 448."""
    if fmt == "bf16":
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16), None
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).float()
    scale = x.abs().amax(-1) / 448.0
    return (x / scale[..., None]).to(F8).view(torch.uint8), scale


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _page_table(kv, page, gen, spare=3):
    """Pages of the sequences in random order over a pool: [B, cols], the pool's size
    and the pages that no sequence has."""
    counts = [-(-n // page) for n in kv]
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).cpu()
    table = torch.zeros((len(kv), max(counts)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table.to(DEV), pages, order[at:].to(DEV)


def _starts(new):
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return start


def _tree_masks(c):
    """The trees' masks [T, words] (bit u of a token: it sees its sequence's new
    token u) and the tokens' positions."""
    new, kv = _lengths(c)
    words = -(-c["new"] // 64)
    masks, positions = [], []
    for tree, n, m in zip(_parents(c), new, kv):
        for seen in _ancestors(tree):
            row = [0] * words
            for u in seen:
                row[u // 64] |= 1 << (u % 64)
            masks.append([w - (1 << 64) if w >> 63 else w for w in row])
            positions.append(m - n + len(seen) - 1)
    return torch.tensor(masks, dtype=torch.int64, device=DEV), _ints(positions)


def _prepare_tables(s, c, gen):
    new, kv = _lengths(c)
    old = [m - n for n, m in zip(new, kv)]
    cols = -(-max(kv) // c["page"])
    table, _, _ = _page_table([max(m, 1) for m in old], c["page"], gen)
    full = torch.zeros((len(kv), cols), dtype=torch.int32, device=DEV)
    full[:, :table.shape[1]] = table
    used = sum(-(-max(m, 1) // c["page"]) for m in old)
    need = sum(-(-m // c["page"]) + 1 for m in kv)
    pages = used + need + 5
    free = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    # (pages beyond those in use; the order in which a pool's life has left them)
    free[:need] = (torch.randperm(need, generator=gen, device=DEV) + used + 3).to(torch.int32)
    s.update(lengths=_ints(old), new=_ints(new), table=full, free=free, count=_ints([need, 0]),
             tokens=sum(new))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    c = case
    s = {"case": c}
    new, kv = _lengths(c)
    start = _starts(new)
    if c["op"] == "tables":
        _prepare_tables(s, c, gen)
    else:
        s["q_start"], s["kv_len"] = _ints(start), _ints(kv)
    if c["op"] == "plan":
        # (other trees for another seed)
        shift = torch.randint(0, 1 << 20, (1,), generator=gen, device=DEV).item()
        trees = _plan_trees(c, shift)
        s["parents"] = _ints([p for tree in trees for p in tree])
        s["table"] = torch.zeros((len(kv), -(-max(kv) // c["page"])), dtype=torch.int32, device=DEV)
        s["words"] = -(-c["new"] // 64)
    if c["op"] in ("norm", "tree", "keep") and c["kv_heads"]:
        s["table"], pages, _ = _page_table(kv, c["page"], gen)
        # (all layers' caches in one allocation)
        shape = (c.get("layers", 1), pages, c["kv_heads"], c["page"], c["dim"])
        s["k"], s["k_scale"] = _pool(shape, c["fmt"], gen)
        s["v"], s["v_scale"] = _pool(shape, c["fmt"], gen)
    if c["op"] == "norm":
        qkv = _heads((start[-1], c["q_heads"] + 2 * c["kv_heads"], c["dim"]), gen)
        s["q"] = qkv[:, :c["q_heads"]]
        s["k_new"] = qkv[:, c["q_heads"]:c["q_heads"] + c["kv_heads"]]
        s["v_new"] = qkv[:, c["q_heads"] + c["kv_heads"]:]
        for name in "qkv":
            w = torch.randn((c["dim"],), generator=gen, device=DEV) * 0.2 + 1.0 - c["offset"]
            s[name + "_weight"] = w.to(torch.bfloat16)
        positions = []
        for tree, n, m in zip(_parents(c), new, kv):
            depth = [len(seen) - 1 for seen in _ancestors(tree)] if c["tree"] else list(range(n))
            positions += [m - n + d for d in depth]
        s["positions"] = _ints(positions)
    if c["op"] == "tree":
        s["q"] = _heads((start[-1], c["q_heads"], c["dim"]), gen, 1.5)
        s["mask"], s["positions"] = _tree_masks(c)
    if c["op"] == "keep":
        paths = _accepted(c)
        wide = max(len(p) for p in paths)
        s["path"] = _ints([p + [0] * (wide - len(p)) for p in paths])
        s["kept"] = _ints([len(p) for p in paths])
    if own:
        _handles(s, c, new)
    return s


def _plan_trees(c, shift):
    """The trees of a plan's case: its sizes, other shapes for each seed."""
    r = random.Random(shift)
    trees = []
    for n in _lengths(c)[0]:
        wide = r.randint(1, 4)
        trees.append([-1 if i == 0 or r.random() < 0.02 else
                      (r.randint(0, i - 1) if r.random() < 0.2 else (i - 1) // wide) for i in range(n)])
    return trees


def _handles(s, c, new):
    """What a program that uses the library keeps beside its tensors."""
    import quantized_linear_layers_amd as qlin

    if c["op"] == "tables":
        s["pool"] = qlin.PagePool(s["free"], s["count"], c["page"])
        s["tables"] = qlin.PageTables(s["pool"], s["table"], s["tokens"], max(new))
        return
    if "k" in s:
        s["caches"] = [qlin.PagedKV(*(None if x is None else x[i] for x in _pools(s).values()))
                       for i in range(s["k"].shape[0])]
    if "table" in s:
        s["batch"] = qlin.PagedBatch(s["q_start"], s["kv_len"], s["table"], max_q=max(new))
    if c["op"] == "plan":
        s["tree"] = qlin.Tree.empty(s["parents"].numel(), s["words"])
    if c["op"] == "tree":
        s["tree"] = qlin.Tree(s["mask"], s["positions"])
    if c["op"] == "norm":
        s["rope"] = qlin.Rope(c["dim"], rot_dim=c["rot"], base=BASE, interleaved=c["interleaved"], device=DEV)
        s["norm"] = qlin.HeadNorm(s["q_weight"], s["k_weight"], s["v_weight"] if c["values"] else None,
                                  eps=c["eps"], offset=c["offset"])
    if c["op"] == "keep":
        s["layers"] = qlin.PagedLayers(s["caches"])


# ------------------------------------------------------------------ plain forms
def _plain_tables(s, c):
    """Pages from the end of the free list, in the order of the requests; the same pages
    back, so that the list is what it was."""
    page, cols = c["page"], s["table"].shape[1]
    old, new = s["lengths"].long(), s["new"].long()
    total = old + new
    q_start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    c0, c1 = (old + page - 1) // page, ((total + page - 1) // page).clamp(max=cols)
    need = (c1 - c0).clamp(min=0)
    first = need.cumsum(0) - need
    count = s["count"][0].long()
    j = torch.arange(cols, device=DEV)
    fresh = (j >= c0[:, None]) & (j < c1[:, None])
    at = count - 1 - (first[:, None] + j - c0[:, None])
    taken = s["free"][at.clamp(min=0, max=s["free"].numel() - 1)]
    taken = torch.where(at >= 0, taken, -1)
    table = torch.where(fresh, taken, s["table"])
    s["table"].copy_(table)
    t = torch.arange(s["tokens"], device=DEV)
    seq = torch.searchsorted(q_start, t, right=True) - 1
    pos = old[seq] + t - q_start[seq]
    entry = table[seq, (pos // page).clamp(max=cols - 1)].long()
    slots = torch.where((entry >= 0) & (pos // page < cols), entry * page + pos % page, -1)
    left = (count - need.sum()).clamp(min=0)
    # the way back
    fresh = fresh & (table >= 0)
    rank = fresh.flatten().flip(0).cumsum(0).flip(0) - 1  # pages behind this one
    end = s["free"].numel()
    where = torch.where(fresh.flatten(), left + rank, end)
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free[where] = table.flatten()
    s["free"].copy_(free[:end])
    short = (need.sum() - count).clamp(min=0)
    s["count"].copy_(torch.stack([left + fresh.sum(), short]))
    return {"q_start": q_start.to(torch.int32), "kv_len": total.to(torch.int32), "table": s["table"],
            "slots": slots.to(torch.int32), "positions": pos.to(torch.int32), "free": s["free"],
            "count": s["count"]}


def _plain_plan(s, c):
    """Ancestors by jumps of twice the distance each time, as truth values [B, n, n]."""
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    B, n, T = c["batch"], c["new"], s["parents"].numel()
    i = torch.arange(n, device=DEV)
    rows = (s["q_start"][:-1, None].long() + i).clamp(max=T - 1)
    jump = s["parents"].long()[rows]
    jump = torch.where((i < new[:, None]) & (jump < i) & (jump >= 0), jump, n)  # n: none
    seen = torch.zeros((B, n + 1, n), dtype=torch.bool, device=DEV)
    seen[:, :n] = i[:, None] == i[None]
    jump = torch.cat([jump, jump.new_full((B, 1), n)], 1)
    reach = 1
    while reach < n:
        seen = seen | seen.gather(1, jump[:, :, None].expand(B, n + 1, n))
        jump = jump.gather(1, jump)
        reach *= 2
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["q_start"], t.to(torch.int32), right=True) - 1
    mine = seen[seq, t - s["q_start"][seq]]
    depth = mine.sum(1) - 1
    words = s["words"]
    bits = torch.zeros((T, words * 64), dtype=torch.int64, device=DEV)
    bits[:, :n] = mine
    mask = (bits.view(T, words, 64) << torch.arange(64, device=DEV)).sum(2)
    first = (s["kv_len"].long() - new)[seq]
    return {"mask": mask, "positions": (first + depth).to(torch.int32)}


def _turn(x, positions, c):
    """x [T, H, D] (32 bits) with the first `rot` values of each head turned (angles
    in 64)."""
    rot = c["rot"]
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot
    angle = positions.double()[:, None] * BASE ** -i
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y = x.clone()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    return y


def _normed(x, weight, c):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + c["eps"])
    return x * (weight.float() + c["offset"])


def _store(pool, scale, rows, page, slot):
    """Rows [T, H, D] in 32 bits into a cache's pages."""
    if scale is None:
        pool[page, :, slot] = rows.to(torch.bfloat16)
        return
    sc = rows.abs().amax(-1) / 448.0
    pool[page, :, slot] = (rows / sc[..., None]).to(F8).view(torch.uint8)
    scale[page, :, slot] = sc


def _plain_norm(s, c):
    q = _turn(_normed(s["q"], s["q_weight"], c), s["positions"], c).to(torch.bfloat16)
    if not c["kv_heads"]:
        return q
    t = torch.arange(q.shape[0], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"], t, right=True) - 1
    new = s["q_start"][1:] - s["q_start"][:-1]
    place = (s["kv_len"] - new)[seq] + t - s["q_start"][seq]
    page, slot = s["table"][seq, place // c["page"]].long(), (place % c["page"]).long()
    k, v, ks, vs = (None if x is None else x[0] for x in _pools(s).values())
    _store(k, ks, _turn(_normed(s["k_new"], s["k_weight"], c), s["positions"], c), page, slot)
    value = _normed(s["v_new"], s["v_weight"], c) if c["values"] else s["v_new"].float()
    _store(v, vs, value, page, slot)
    return q


def _gather(pool, scale, table):
    """A cache's pages as [B, H, L, D] in 32 bits."""
    x = pool.view(F8).float() * scale[..., None] if scale is not None else pool.float()
    x = x[table.long()]  # [B, P, H, page, D]
    B, P, H, page, D = x.shape
    return x.transpose(1, 2).reshape(B, H, P * page, D)


def _plain_tree(s, c):
    G, D, H = c["q_heads"] // c["kv_heads"], c["dim"], c["kv_heads"]
    T, n, L, B = s["q"].shape[0], c["new"], c["context"], c["batch"]
    pk, pv, ks, vs = (None if x is None else x[0] for x in _pools(s).values())
    k = _gather(pk, ks, s["table"])[:, :, :L]
    v = _gather(pv, vs, s["table"])[:, :, :L]
    i = torch.arange(n, device=DEV)
    rows = (s["q_start"][:-1, None] + i).clamp(max=T - 1).long()
    q = s["q"].float()[rows].view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * D ** -0.5
    del k
    first = s["kv_len"] - (s["q_start"][1:] - s["q_start"][:-1])
    j = torch.arange(L, device=DEV)
    u = j - first[:, None]  # [B, L]: a key's number among the new tokens
    word = s["mask"][rows]  # [B, n, words]
    at = u.clamp(min=0, max=64 * word.shape[2] - 1)
    bit = word.gather(2, (at // 64)[:, None].expand(B, n, L)) >> (at % 64)[:, None] & 1
    seen = (bit == 1) & (j < s["kv_len"][:, None])[:, None] | (u < 0)[:, None]
    if c["window"]:
        seen = seen & (j > (s["positions"][rows] - c["window"])[..., None])
    score = score.view(B, H, G, n, L)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1)
    out = torch.matmul(p.view(B, H, G * n, L), v).view(B, H, G, n, D)
    out = out / torch.where(total == 0, 1.0, total)[..., None]
    lse = top[..., 0] + total.log()
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"], t, right=True) - 1
    i = t - s["q_start"][seq]
    out = out.reshape(B, c["q_heads"], n, D)[seq, :, i].to(torch.bfloat16)
    return out, lse.reshape(B, c["q_heads"], n)[seq, :, i]


def _plain_keep(s, c):
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    first = s["kv_len"].long() - new
    i = torch.arange(s["path"].shape[1], device=DEV)
    real = i < s["kept"][:, None]
    last = new[:, None] - 1  # (what is no move copies the last new token to itself)
    place = {"from": torch.where(real, s["path"].long(), last), "to": torch.where(real, i, last)}
    at = {}
    for name, u in place.items():
        p = (first[:, None] + u).flatten()
        row = torch.arange(c["batch"], device=DEV).repeat_interleave(i.numel())
        at[name] = s["table"][row, p // c["page"]].long(), p % c["page"]
    for pool in _pools(s).values():
        if pool is not None:
            pool[:, at["to"][0], :, at["to"][1]] = pool[:, at["from"][0], :, at["from"][1]]
    return (first + s["kept"]).to(torch.int32)


def _values(pool):
    """A cache's pages as what they hold."""
    return pool.view(F8) if pool.dtype == torch.uint8 else pool


def _pools(s):
    """All layers' caches: [layers, pages, heads, page(, values)], scales with FP8."""
    return {name: s[name] for name in ("k", "v", "k_scale", "v_scale")}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "tables":
            return _plain_tables(s, c)
        if op == "plan":
            return _plain_plan(s, c)
        if op == "tree":
            return _plain_tree(s, c)
        y = _plain_norm(s, c) if op == "norm" else _plain_keep(s, c)
    else:
        import quantized_linear_layers_amd as qlin

        if op == "tables":
            t = s["tables"]
            t.reserve(s["lengths"], s["new"])
            t.release(s["lengths"])
            return {"q_start": t.q_start, "kv_len": t.kv_len, "table": s["table"], "slots": t.slots,
                    "positions": t.positions, "free": s["free"], "count": s["count"]}
        if op == "plan":
            tree = qlin.tree_plan(s["batch"], s["parents"], s["tree"])
            return {"mask": tree.mask, "positions": tree.positions}
        if op == "tree":
            return qlin.attn_paged(s["caches"][0], s["batch"], s["q"], window=c["window"], tree=s["tree"],
                                   return_lse=True)
        if op == "keep":
            y = qlin.kv_keep(s["layers"], s["batch"], s["path"], s["kept"])
        elif c["kv_heads"]:
            y = qlin.kv_append(s["caches"][0], s["batch"], s["k_new"], s["v_new"], rope=s["rope"], q=s["q"],
                               positions=s["positions"], norm=s["norm"])
        else:
            y = qlin.norm_rope(s["q"], s["norm"], s["positions"], s["rope"])
    if "k" not in s:
        return y
    return {"y": y, **{name: x if x is None else _values(x) for name, x in _pools(s).items()}}


# ------------------------------------------------------------------ work
def work(case):
    c = case
    new, kv = _lengths(c)
    T, B = sum(new), len(new)
    if c["op"] == "tables":
        pages = sum(-(-m // c["page"]) - -(-(m - n) // c["page"]) for n, m in zip(new, kv))
        # lengths and counts, starts; each page from the free list to the table and back
        return {"bytes": 4 * (4 * B + 2) + 8 * T + 16 * pages, "flops": 2 * T}
    if c["op"] == "plan":
        words = -(-c["new"] // 64)
        return {"bytes": 4 * (2 * B + 1) + T * (8 + 8 * words), "flops": 2 * T * words}
    D = c["dim"]
    one, scale = (1, 4) if c["fmt"] == "e4m3" else (2, 0)
    if c["op"] == "norm":
        row = c["q_heads"] * 4 * D + c["kv_heads"] * 2 * ((2 + one) * D + scale) + 4
        normed = c["q_heads"] + c["kv_heads"] * (2 if c["values"] else 1)
        return {"bytes": T * row, "flops": T * (4 * normed * D + 3 * (c["q_heads"] + c["kv_heads"]) * c["rot"])}
    if c["op"] == "keep":
        moved = sum(sum(u != i for i, u in enumerate(p)) for p in _accepted(c))
        rows = moved * c["layers"] * 2 * c["kv_heads"]
        return {"bytes": 2 * rows * (one * D + scale) + 4 * (T + 3 * B), "flops": rows}
    rows = pairs = 0
    for tree, n, m in zip(_parents(c), new, kv):
        first = m - n
        lo = first
        for seen in _ancestors(tree):
            least = max(0, first + len(seen) - c["window"]) if c["window"] else 0
            lo = min(lo, least)
            pairs += max(0, first - least) + len(seen)
        rows += first - lo + n
    return {"bytes": rows * c["kv_heads"] * 2 * (one * D + scale)
            + T * (c["q_heads"] * (4 * D + 4) + 8 * -(-c["new"] // 64)),
            "flops": 4 * D * c["q_heads"] * pairs}


# ------------------------------------------------------------------ 64 bits
def _exact_tables(s, c):
    """The same tables by going through the requests and their tokens."""
    page = c["page"]
    table, free = s["table"].tolist(), s["free"].tolist()
    left = s["count"].tolist()[0]
    q_start, kv_len, slots, positions = [0], [], [], []
    taken = []
    for b, (m, n) in enumerate(zip(s["lengths"].tolist(), s["new"].tolist())):
        for col in range(-(-m // page), -(-(m + n) // page)):
            left -= 1
            table[b][col] = free[left]
            taken.append(free[left])
        for p in range(m, m + n):
            slots.append(table[b][p // page] * page + p % page)
            positions.append(p)
        q_start.append(q_start[-1] + n)
        kv_len.append(m + n)
    return {"q_start": _ints(q_start), "kv_len": _ints(kv_len), "table": _ints(table), "slots": _ints(slots),
            "positions": _ints(positions), "free": s["free"].clone(), "count": s["count"].clone()}


def _exact_plan(s, c):
    new, kv = _lengths(c)
    parents = s["parents"].tolist()
    masks, positions, at = [], [], 0
    for n, m in zip(new, kv):
        for i in range(n):
            row, u, depth = 0, i, -1
            while u >= 0:
                row |= 1 << u
                depth += 1
                u = parents[at + u]
            masks.append([((row >> (64 * w)) + (1 << 63)) % (1 << 64) - (1 << 63) for w in range(s["words"])])
            positions.append(m - n + depth)
        at += n
    return {"mask": torch.tensor(masks, dtype=torch.int64, device=DEV), "positions": _ints(positions)}


def _exact_turn(y, positions, c):
    """The rotation as a product of complex numbers."""
    rot = c["rot"]
    step = torch.tensor([BASE ** (-2.0 * k / rot) for k in range(rot // 2)], dtype=torch.float64, device=DEV)
    angle = torch.outer(positions.double(), step)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    if c["interleaved"]:
        pair = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous())
        head = torch.view_as_real(pair * turn).reshape(*y.shape[:-1], rot)
    else:
        got = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        head = torch.cat([got.real, got.imag], -1)
    return torch.cat([head, y[..., rot:]], -1)


def _exact_normed(x, weight, c):
    x = x.double()
    return x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / c["dim"] + c["eps"]) * (c["offset"] + weight.double())


def _exact_norm(s, c):
    q = _exact_turn(_exact_normed(s["q"], s["q_weight"], c), s["positions"], c)
    if not c["kv_heads"]:
        return q
    new, kv = _lengths(c)
    place = torch.tensor([m - n + i for n, m in zip(new, kv) for i in range(n)], device=DEV)
    seq = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], device=DEV)
    page, slot = s["table"][seq, place // c["page"]].long(), place % c["page"]
    rows = {"k": _exact_turn(_exact_normed(s["k_new"], s["k_weight"], c), s["positions"], c),
            "v": _exact_normed(s["v_new"], s["v_weight"], c) if c["values"] else s["v_new"].double()}
    out = {"y": q}
    for name in ("k", "v"):
        x, scale = rows[name], s[name + "_scale"]
        out[name], out[name + "_scale"] = _values(s[name]).double(), None
        if scale is not None:
            sc = x.abs().max(-1).values / 448.0
            out[name + "_scale"] = scale.double()
            out[name + "_scale"][0, page, :, slot] = sc
            x = x / sc[..., None]
            # nearest value of the format: 3 fraction bits, steps of 2^-9 at least
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(x / step) * step
        out[name][0, page, :, slot] = x
    return out


def _exact_tree(s, c):
    new, kv = _lengths(c)
    G, D, H = c["q_heads"] // c["kv_heads"], c["dim"], c["kv_heads"]
    outs, lses, at = [], [], 0
    pk, pv, ks, vs = (None if x is None else x[0] for x in _pools(s).values())
    for b, (tree, n, m) in enumerate(zip(_parents(c), new, kv)):
        used = s["table"][b, :-(-m // c["page"])].long()

        def rows(pool, scale):
            x = _values(pool)[used].to(torch.float64)
            if scale is not None:
                x = x * scale[used].double()[..., None]
            return torch.cat(list(x), 1)[:, :m]

        k, v = rows(pk, ks), rows(pv, vs)
        see = torch.zeros((n, m), dtype=torch.bool)
        for i, seen in enumerate(_ancestors(tree)):
            p = m - n + len(seen) - 1
            see[i, max(0, p - c["window"] + 1) if c["window"] else 0:m - n] = True
            see[i, [m - n + u for u in seen]] = True
        hide = ~see.to(DEV)
        q = s["q"][at:at + n].double().transpose(0, 1)
        o, l = [], []
        for h in range(H):
            z = (q[h * G:h * G + G] @ k[h].T.contiguous() / math.sqrt(D)).masked_fill(hide, -math.inf)
            l.append(torch.logsumexp(z, 2))
            o.append(torch.softmax(z, 2) @ v[h])
        outs.append(torch.cat(o).transpose(0, 1))
        lses.append(torch.cat(l).transpose(0, 1))
        at += n
    return torch.cat(outs), torch.cat(lses)


def _exact_keep(s, c):
    new, kv = _lengths(c)
    to, source, lengths = ([], []), ([], []), []
    table = s["table"].tolist()
    for b, (path, n, m) in enumerate(zip(_accepted(c), new, kv)):
        for i, u in enumerate(path):
            for at, p in ((to, m - n + i), (source, m - n + u)):
                at[0].append(table[b][p // c["page"]])
                at[1].append(p % c["page"])
        lengths.append(m - n + len(path))
    to, source = [torch.tensor(x, device=DEV) for x in to], [torch.tensor(x, device=DEV) for x in source]
    out = {"y": _ints(lengths)}
    for name, pool in _pools(s).items():
        out[name] = None
        if pool is not None:
            out[name] = _values(pool).double()
            for layer in out[name]:
                layer[to[0], :, to[1]] = layer[source[0], :, source[1]]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "plan": _exact_plan, "norm": _exact_norm, "tree": _exact_tree,
            "keep": _exact_keep}[case["op"]](s, case)
