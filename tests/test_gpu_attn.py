"""Rotary positions, the paged cache's append and paged attention on the GPU
against the fp64 oracle.

Bounds (a rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24):
  rotation  bf16 rounding, and fp32 sums of two products: the part of a turn is
            rounded to fp32 (2^-25 turns, 2 pi 2^-25 rad), sine and cosine are
            within 2 units in the last place, the products and the sum round
            three times: together under 2^-20 of magnitude * (|a| + |b|);
  scores    fp32 sums over D: dz = (D + 8) 2^-24 of the sum of |q k| * scale;
  weights   exp2 of (z - max) in fp32: relative 2 dz + 2^-20, and bf16: 2^-8;
  sums      over n keys in fp32: n 2^-24 of the sum of magnitudes;
  output    weights and both sums, then one bf16 rounding.
"""

import numpy as np
import pytest
import torch

from helpers import bf16_to_f32, dev, host, tol_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    assert torch.cuda.is_available()
    return qlin


def bits(x):
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def projections(rng, shape):
    x = rng.standard_normal(shape)
    x[..., rng.random(shape[-1]) < 0.02] *= 6
    return bits(x)


# ------------------------------------------------------------------ rotation
def rope_check(got, y, mag, what):
    g = bf16_to_f32(got).astype(np.float64)
    err = np.abs(g - y)
    tol = 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * mag
    assert (err <= tol).all(), f"{what}: worst {np.max(err / np.maximum(tol, 1e-300)):.3f}"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 16, 16), (3, 5, 48, 32), (8, 32, 128, 128), (7, 3, 256, 64),
                                       (70, 2, 64, 16), (5, 9, 1024, 512), (9, 33, 64, 64), (2, 1, 512, 512)])
def test_rope(q, oracle, T, H, D, rot, inter):
    rng = np.random.default_rng(T * 1000 + D)
    x = projections(rng, (T, H, D))
    pos = rng.integers(-5, 1 << 20, T).astype(np.int32)
    pos[0] = 0
    pos[-1] = 2 ** 31 - 1
    plan = q.Rope(D, rot_dim=rot, interleaved=inter, scaling=("ramp", 16.0, 8192, 1.0, 32.0), magnitude=1.25)
    turns = oracle.rope_turns(rot, 10000.0, 3, 16.0, 8192.0, 1.0, 32.0)
    xd, pd = dev(x), dev(pos)
    for inverse in (False, True):
        y, mag = oracle.rope(x, pos, host(plan.turns), rot, inter, 1.25, inverse)
        got = q.rope(xd, pd, plan, inverse=inverse)
        rope_check(host(got), y, mag, f"inverse={inverse}")
        assert np.array_equal(host(got)[..., rot:], x[..., rot:])
    np.testing.assert_allclose(host(plan.turns), turns, rtol=1e-13)


def test_rope_large_folds_heads_and_strides(q, oracle):
    """Enough tokens that a thread handles several heads; rows of a fused
    projection; in place; equal to the same rows called one by one."""
    rng = np.random.default_rng(1)
    T, H, D = 8195, 18, 64
    qkv = dev(projections(rng, (T, H + 4, D)))
    x = qkv[:, :H]
    pos = torch.from_numpy(rng.integers(0, 70000, T).astype(np.int32)).cuda()
    plan = q.Rope(D, base=500000.0)
    y = q.rope(x, pos, plan)
    for lo in (0, 4097, 8190):
        part = q.rope(x[lo:lo + 5], pos[lo:lo + 5], plan)
        assert torch.equal(part.view(torch.int16), y[lo:lo + 5].view(torch.int16))
    want, mag = oracle.rope(host(x[8000:8010]), host(pos[8000:8010]), host(plan.turns), D)
    rope_check(host(y[8000:8010]), want, mag, "rows")
    tail = qkv[:, H:].clone()
    got = q.rope(x, pos, plan, out=x)
    assert got.data_ptr() == qkv.data_ptr()
    assert torch.equal(qkv[:, :H].view(torch.int16), y.view(torch.int16))
    assert torch.equal(qkv[:, H:].view(torch.int16), tail.view(torch.int16))


@pytest.mark.parametrize("as_tensor", [False, True])
@pytest.mark.parametrize("rot", [64, 32])
def test_rope_given_turns(q, oracle, rot, as_tensor):
    """Frequencies of one's own: a blend that is linear in the pair's index, which
    the ramp rule (linear in turns) does not give."""
    rng = np.random.default_rng(rot)
    i = np.arange(rot // 2)
    f = 10000.0 ** (-2.0 * i / rot) / (2 * np.pi)
    keep = 1.0 - np.clip((i - 3) / (rot // 2 - 8), 0.0, 1.0)
    turns = f * keep + f / 8.0 * (1.0 - keep)
    given = torch.from_numpy(turns).float().cuda().double() if as_tensor else turns.tolist()
    plan = q.Rope(64, rot_dim=rot, turns=given, magnitude=1.1)
    want = host(given) if as_tensor else turns
    assert np.array_equal(host(plan.turns), want)
    if as_tensor:
        given.zero_()  # the plan has its own
    x, pos = projections(rng, (9, 3, 64)), rng.integers(0, 100000, 9).astype(np.int32)
    y, mag = oracle.rope(x, pos, want, rot, False, 1.1)
    rope_check(host(q.rope(dev(x), dev(pos), plan)), y, mag, "own turns")


def test_rope_gradient(q):
    """The inverse rotation is the gradient: <R x, g> differenced in every
    direction of a small x, in exact arithmetic of its linear map."""
    rng = np.random.default_rng(2)
    T, H, D = 2, 1, 16
    pos = torch.tensor([3, 71], dtype=torch.int32, device="cuda")
    plan = q.Rope(D, magnitude=1.5)
    g = dev(projections(rng, (T, H, D)))
    grad = q.rope(g, pos, plan, inverse=True).float()
    # the map is linear: the difference along unit vector e is R e itself
    for t in range(T):
        for d in range(D):
            e = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
            e[t, 0, d] = 1.0
            diff = (q.rope(e, pos, plan).float() * g.float()).sum().item()
            # R e rounds to bf16 (2^-8 of each of two values up to 1.5), the gradient once more
            tol = 2.0 ** -8 * (1.5 * 2 * g.float().abs().max().item() + abs(diff)) + 1e-5
            assert abs(diff - grad[t, 0, d].item()) <= tol


# ------------------------------------------------------------------ batches
def make_batch(rng, new, kv, page, extra_pages=2, pad=0, order=None):
    """q_start, table and the number of pages; pages in random order."""
    counts = [-(-max(n, 0) // page) for n in kv]
    pages = sum(counts) + extra_pages
    perm = rng.permutation(pages) if order is None else order
    table = np.zeros((len(kv), max(max(counts), 1)), np.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = perm[at:at + n]
        at += n
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32), table, pages


def stale_pool(q, pages, Hkv, page, D, fmt):
    """A cache of NaN: whatever no token wrote must reach no result."""
    c = q.PagedKV.empty(pages, Hkv, D, page, fmt)
    if fmt == "bf16":
        c.k.fill_(float("nan"))
        c.v.fill_(float("nan"))
    else:
        c.k.fill_(0x7F)
        c.v.fill_(0x7F)
        c.k_scale.fill_(float("nan"))
        c.v_scale.fill_(float("nan"))
    return c


def fill_cache(q, rng, cache, start, kv, table, gain=1.0):
    """Random keys and values for every sequence's whole length, appended as
    one prompt each (no rotation)."""
    kv = np.minimum(np.maximum(kv, 0), table.shape[1] * cache.page_size)
    T = int(kv.sum())
    k = dev(bits(rng.standard_normal((max(T, 1), cache.kv_heads, cache.head_dim)) * gain))
    v = dev(projections(rng, (max(T, 1), cache.kv_heads, cache.head_dim)))
    if T:
        b = q.PagedBatch(dev(np.concatenate([[0], np.cumsum(kv)]).astype(np.int32)), dev(kv.astype(np.int32)),
                         dev(table), max(int(kv.max()), 1))
        q.kv_append(cache, b, k, v)


def attn_check(r, got, lse, D, what):
    seen = r["seen"]
    rows = ~np.isnan(r["lse"])
    dz = r["zmag"] * (D + 8) * 2.0 ** -24
    rel = (2.0 ** -8 + 4 * dz + 2.0 ** -19 + 2 * seen * 2.0 ** -24)[..., None]
    tol = r["mag"] * rel * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(r["out"]) + 1e-30
    err = np.abs(bf16_to_f32(got).astype(np.float64) - r["out"])
    bad = ~(err <= tol) & rows[..., None]
    if bad.any():
        i = np.argwhere(bad)
        raise AssertionError(f"{what}: {bad.sum()}/{bad.size} outside, first {i[:3].tolist()} got "
                             f"{bf16_to_f32(got)[bad][:3]} want {r['out'][bad][:3]}; worst "
                             f"{np.nanmax(np.where(bad, err / tol, 0)):.2f}")
    if lse is not None:
        with np.errstate(invalid="ignore"):
            e = np.abs(lse - r["lse"])
        ltol = dz + seen * 2.0 ** -24 + 2.0 ** -19 + np.abs(r["lse"]) * 2.0 ** -21
        ok = (e <= ltol) | ((seen == 0) & (lse == -np.inf)) | ~rows
        assert ok.all(), f"{what}: lse {np.argwhere(~ok)[:3].tolist()} {lse[~ok][:3]} {r['lse'][~ok][:3]}"


def run_attn(q, oracle, seed, new, kv, Hkv, G, D, page, fmt, causal=True, window=0, scale=None, pad=0, max_q=None,
             table_edit=None, extra_cols=0):
    rng = np.random.default_rng(seed)
    start, table, pages = make_batch(rng, new, kv, page)
    if extra_cols:  # a table with room for longer sequences
        table = np.concatenate([table, np.full((len(kv), extra_cols), -1, np.int32)], 1)
    cache = stale_pool(q, pages, Hkv, page, D, fmt)
    fill_cache(q, rng, cache, start, np.array(kv), table)
    if table_edit is not None:
        table_edit(table)
    T = int(start[-1]) + pad
    x = projections(rng, (T, Hkv * G, D))
    sc = D ** -0.5 if scale is None else scale
    batch = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), max(new) if max_q is None else max_q)
    out = torch.full((T, Hkv * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got, lse = q.attn_paged(cache, batch, dev(x), scale=sc, causal=causal, window=window, out=out, return_lse=True)
    assert got is out
    torch.cuda.synchronize()
    e4 = fmt == "e4m3"
    r = oracle.attn_paged(x, host(cache.k), host(cache.v), host(cache.k_scale) if e4 else None,
                          host(cache.v_scale) if e4 else None, start, kv, table, sc, causal, window)
    attn_check(r, host(got), host(lse), D, f"new={new} kv={kv} D={D} page={page} {fmt}")
    assert (host(got)[int(start[-1]):] == 0x40E0).all(), "padding rows were written"
    return cache, batch, x, host(got), host(lse)


# one decode step (up to 32 rows), every head size, cache type and page size
STEP_LENGTHS = [1, 15, 16, 17, 31, 32, 33, 64, 65, 127, 200, 0, 321]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page,Hkv,G", [(64, 16, 2, 4), (64, 64, 1, 32), (128, 16, 2, 4), (128, 128, 1, 5),
                                          (128, 32, 3, 1), (256, 16, 1, 8), (256, 256, 2, 2)])
def test_step(q, oracle, D, page, Hkv, G, fmt):
    run_attn(q, oracle, D + page, [1] * len(STEP_LENGTHS), STEP_LENGTHS, Hkv, G, D, page, fmt, pad=3)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 37), (True, 200)])
def test_step_masks_and_several_tokens(q, oracle, causal, window, fmt):
    # 4 new tokens x 4 heads; idle slots; fewer keys than new tokens (rows
    # that see nothing); a long sequence alone: the key axis is split
    run_attn(q, oracle, 5, [4, 0, 1, 3, 4, 2], [130, 50, 1, 1, 0, 77], 2, 4, 128, 16, fmt, causal, window, pad=1)
    run_attn(q, oracle, 6, [3], [2049], 1, 4, 128, 32, fmt, causal, window, extra_cols=5)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_step_split_over_keys(q, oracle, D, fmt):
    run_attn(q, oracle, 7, [1, 1, 1], [1500, 3, 700], 2, 4, D, 64, fmt, extra_cols=40)


# chunks: rows that fill tiles, pass them, end inside them
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page,Hkv,G", [(64, 16, 2, 2), (128, 16, 1, 4), (128, 64, 2, 1), (128, 256, 1, 3),
                                          (256, 32, 1, 2), (64, 128, 1, 8), (256, 16, 1, 4)])
def test_chunk(q, oracle, D, page, Hkv, G, fmt):
    run_attn(q, oracle, 20 + D + page, [33, 0, 64, 129, 1], [33, 17, 200, 150, 90], Hkv, G, D, page, fmt, pad=2)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 50), (True, 128), (True, 10 ** 15)])
@pytest.mark.parametrize("D", [128, 256])
def test_chunk_masks(q, oracle, causal, window, fmt, D):
    # the second has fewer keys than new tokens, the third none at all
    run_attn(q, oracle, 31, [100, 40, 35, 70], [260, 7, 0, 70], 1, 4, D, 16, fmt, causal, window, pad=1)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_chunk_split_over_keys(q, oracle, fmt):
    run_attn(q, oracle, 41, [40], [1333], 2, 4, 128, 64, fmt, extra_cols=9)
    run_attn(q, oracle, 42, [40, 9], [1333, 600], 1, 4, 64, 16, fmt, causal=False)
    run_attn(q, oracle, 43, [150], [900], 1, 2, 256, 32, fmt, window=300)


# Chunks over tables of 2^18 tokens, which have workgroups of 128 rows, E4M3 256 (the
# shorter ones above: of 32): the key axis in parts, and with many heads whole.
def long_table(page):
    return (1 << 18) // page


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page,Hkv,G", [(64, 16, 2, 2), (128, 16, 1, 4), (128, 64, 2, 1), (128, 256, 1, 3),
                                          (256, 32, 1, 2), (64, 128, 1, 8), (256, 16, 1, 4), (64, 32, 70, 2),
                                          (128, 32, 40, 2), (256, 64, 40, 2)])
def test_chunk_long_table(q, oracle, D, page, Hkv, G, fmt):
    run_attn(q, oracle, 20 + D + page, [33, 0, 64, 129, 1], [33, 17, 200, 150, 90], Hkv, G, D, page, fmt, pad=2,
             extra_cols=long_table(page))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 10 ** 15)])
@pytest.mark.parametrize("D,Hkv", [(64, 1), (128, 1), (256, 1), (64, 40), (128, 24), (256, 24)])
def test_chunk_masks_long_table(q, oracle, causal, window, fmt, D, Hkv):
    run_attn(q, oracle, 31, [100, 40, 35, 70], [260, 7, 0, 70], Hkv, 4, D, 16, fmt, causal, window, pad=1,
             extra_cols=long_table(16))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_chunk_window_in_parts(q, oracle, fmt):
    """A window of so many keys that the chunk's axis is split all the same."""
    run_attn(q, oracle, 33, [131], [4700], 90, 1, 128, 128, fmt, True, 4600, extra_cols=2)


def test_chunk_window_inside(q, oracle):
    """A window in chunks of so many rows that they have workgroups of 256."""
    run_attn(q, oracle, 34, [700, 300], [900, 300], 20, 4, 64, 32, "bf16", window=77)
    run_attn(q, oracle, 35, [700, 300], [900, 300], 16, 4, 128, 32, "e4m3", window=130)
    run_attn(q, oracle, 36, [500, 600], [900, 600], 16, 4, 256, 64, "bf16", window=33)


def test_chunk_split_over_keys_long_table(q, oracle):
    run_attn(q, oracle, 41, [40], [1333], 2, 4, 128, 64, "bf16", extra_cols=long_table(64))
    run_attn(q, oracle, 42, [70, 9], [1333, 600], 2, 4, 64, 16, "e4m3", causal=False, extra_cols=long_table(16))
    run_attn(q, oracle, 43, [150], [4900], 1, 2, 256, 32, "bf16", extra_cols=long_table(32))


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-6, 1.5])
def test_scales_long_table(q, oracle, scale):
    run_attn(q, oracle, 51, [100, 40], [190, 61], 1, 2, 128, 16, "bf16", scale=scale, extra_cols=long_table(16))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_pages_that_do_not_exist_long_table(q, oracle, fmt):
    def edit(t):
        t[0, 1] = -1
        t[0, 3] = 10 ** 9
        t[1, :] = 2 ** 31 - 1

    run_attn(q, oracle, 61, [80, 70], [90, 71], 2, 2, 128, 16, fmt, table_edit=edit, extra_cols=long_table(16))


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-6, 1.5])
@pytest.mark.parametrize("new,G", [([1, 1], 4), ([60, 40], 2)])
def test_scales(q, oracle, scale, new, G):
    run_attn(q, oracle, 51, new, [90, 61], 1, G, 128, 16, "bf16", scale=scale)


@pytest.mark.parametrize("scale,gain", [(0.0, 60), (1e-38, 60), (-1e-38, 60), (1e-40, 60), (2.3e38, -62), (-2.3e38, -62)])
@pytest.mark.parametrize("new,G,more", [([1, 3], 4, 0), ([60, 40], 2, 0), ([60, 40], 2, long_table(16))])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_scales_at_the_ends_of_fp32(q, oracle, scale, gain, new, G, more, fmt):
    """Scores up to 2^126 under scales of 0 and of about their inverse, and scores of
    2^-121 (and of 0) under the largest scales: queries and keys are signs times
    2^gain, so that products are exact and within fp32's normal range."""
    rng = np.random.default_rng(52)
    D, page, kv = 64, 16, [90, 61]
    start, table, pages = make_batch(rng, new, kv, page)
    table = np.concatenate([table, np.full((2, more), -1, np.int32)], 1)
    cache = stale_pool(q, pages, 1, page, D, fmt)
    b = q.PagedBatch(dev(np.array([0, 90, 151], np.int32)), dev(np.array(kv, np.int32)), dev(table), 90)

    def signs(*shape):
        return bits(np.where(rng.random(shape) < 0.5, 1.0, -1.0) * 2.0 ** gain)

    q.kv_append(cache, b, dev(signs(151, 1, D)), dev(projections(rng, (151, 1, D))))
    T = int(start[-1])
    x = signs(T, G, D)
    x[T - 1, 0] = 0  # a row of scores 0
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), max(new))
    got, lse = q.attn_paged(cache, b, dev(x), scale=scale, return_lse=True)
    e4 = fmt == "e4m3"
    r = oracle.attn_paged(x, host(cache.k), host(cache.v), host(cache.k_scale) if e4 else None,
                          host(cache.v_scale) if e4 else None, start, kv, table, scale)
    attn_check(r, host(got), host(lse), D, f"scale {scale}")


@pytest.mark.parametrize("new,G", [([1, 1], 4), ([60, 70], 2)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_pages_that_do_not_exist(q, oracle, new, G, fmt):
    """Keys of a page outside the pool are not seen (also a row that then sees
    nothing): ids are device data, no error and no access."""
    def edit(t):
        t[0, 1] = -1
        t[0, 3] = 10 ** 9
        t[1, :] = 2 ** 31 - 1

    run_attn(q, oracle, 61, new, [90, 71], 2, G, 128, 16, fmt, table_edit=edit)


def test_max_q_may_exceed(q, oracle):
    a = run_attn(q, oracle, 71, [1, 2], [70, 200], 2, 4, 128, 16, "bf16")
    b = run_attn(q, oracle, 71, [1, 2], [70, 200], 2, 4, 128, 16, "bf16", max_q=4096)
    np.testing.assert_allclose(a[4], b[4], rtol=1e-5)


def test_many_sequences(q, oracle):
    """More than one pass of 64 in the sequence searches, idle ones among them."""
    rng = np.random.default_rng(9)
    new = rng.integers(0, 3, 150).tolist()
    kv = [n + int(x) for n, x in zip(new, rng.integers(0, 60, 150))]
    run_attn(q, oracle, 81, new, kv, 1, 2, 64, 16, "bf16", pad=2)
    new[70] = 40
    kv[70] = 95
    run_attn(q, oracle, 82, new, kv, 1, 2, 64, 16, "bf16", pad=2)


@pytest.mark.parametrize("B", [70, 150])
def test_chunk_of_many_sequences(q, oracle, B):
    """The same in workgroups of 256 rows, with the key axis split (70) and whole."""
    rng = np.random.default_rng(B)
    new = rng.integers(0, 3, B).tolist()
    kv = [n + int(x) for n, x in zip(new, rng.integers(0, 60, B))]
    for b, n, more in ((2, 300, 40), (66, 200, 500), (B - 1, 140, 0)):
        new[b], kv[b] = n, n + more
    run_attn(q, oracle, 83, new, kv, 1, 2, 128, 16, "bf16", pad=2, extra_cols=long_table(16))
    run_attn(q, oracle, 84, new, kv, 1, 2, 64, 32, "e4m3", window=90, extra_cols=long_table(16))


def test_length_over_the_table(q, oracle):
    rng = np.random.default_rng(4)
    start, table, pages = make_batch(rng, [1], [64], 16)
    cache = stale_pool(q, pages, 1, 16, 64, "bf16")
    fill_cache(q, rng, cache, start, np.array([64]), table)
    x = projections(rng, (1, 2, 64))
    for length in (64, 65, 2 ** 31 - 1):
        b = q.PagedBatch(dev(start), dev(np.array([length], np.int32)), dev(table), 1)
        got, lse = q.attn_paged(cache, b, dev(x), return_lse=True)
        r = oracle.attn_paged(x, host(cache.k), host(cache.v), None, None, start, [length], table, 0.125)
        attn_check(r, host(got), host(lse), 64, f"length {length}")
    b = q.PagedBatch(dev(start), dev(np.array([-3], np.int32)), dev(table), 1)
    got, lse = q.attn_paged(cache, b, dev(x), return_lse=True)
    assert (host(got) == 0).all() and (host(lse) == -np.inf).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,G,window,cols", [(3, 4, 0, 8), (3, 4, 2, 8), (3, 4, 40, 8), (90, 2, 0, 8), (90, 2, 25, 8),
                                               (5, 16, 3, 8)])
def test_sequences_longer_than_their_tables(q, oracle, new, G, window, cols, fmt):
    """The tokens behind the table's reach are not stored and not seen; the others
    keep their places."""
    rng = np.random.default_rng(new + window)
    D, Hkv, page = 128, 2, 16
    kv = [cols * page + 2, cols * page + new + 40, 100]
    table = rng.permutation(3 * cols).reshape(3, cols).astype(np.int32)
    start = (np.arange(4) * new).astype(np.int32)
    pages, T, Hq = 3 * cols, 3 * new, Hkv * G
    cache = q.PagedKV.empty(pages, Hkv, D, page, fmt)
    fill_cache(q, rng, cache, None, np.array([cols * page] * 3), table)
    before = [host(t) for t in (cache.k, cache.v)]
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), new)
    qkv = projections(rng, (T, Hq + 2 * Hkv, D))
    d, plan = dev(qkv), q.Rope(D)
    qq = q.kv_append(cache, b, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], rope=plan, q=d[:, :Hq])
    slot, place = oracle.kv_slots(start, kv, table, page, pages, T)
    assert (slot >= 0).sum() == (new - 2) + new and place[new - 1] == cols * page + 1
    y, mag = oracle.rope(qkv, place, host(plan.turns), D)
    rope_check(host(qq), y[:, :Hq], mag[:, :Hq], "queries")
    kept = np.ones((pages, page), bool)
    kept[slot[slot >= 0] // page, slot[slot >= 0] % page] = False
    for t, o in zip((cache.k, cache.v), before):
        assert np.array_equal(host(t).transpose(0, 2, 1, 3)[kept], o.transpose(0, 2, 1, 3)[kept])
    got, lse = q.attn_paged(cache, b, qq, window=window, return_lse=True)
    e4 = fmt == "e4m3"
    r = oracle.attn_paged(host(qq), host(cache.k), host(cache.v), host(cache.k_scale) if e4 else None,
                          host(cache.v_scale) if e4 else None, start, kv, table, D ** -0.5, True, window)
    attn_check(r, host(got), host(lse), D, f"longer than the table {fmt}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,G,cols", [(1, 4, 64), (40, 2, 64), (90, 2, 4000)])
def test_no_key_at_all_and_the_next_call(q, oracle, new, G, cols, fmt):
    """A batch of empty sequences over tables that split the key axis: zeros, and
    the workspace serves the next call."""
    rng = np.random.default_rng(new)
    B, Hkv, D, page = 3, 2, 128, 16
    T, Hq = B * new, Hkv * G
    cache = q.PagedKV.empty(B * 64, Hkv, D, page, fmt)
    table = rng.permutation(B * 64).reshape(B, 64).astype(np.int32)
    fill_cache(q, rng, cache, None, np.array([64 * page] * B), table)
    table = np.concatenate([table, np.full((B, cols - 64), -1, np.int32)], 1)
    start = (np.arange(B + 1) * new).astype(np.int32)
    x = projections(rng, (T, Hq, D))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    b = q.PagedBatch(dev(start), lens, dev(table), new)
    nbytes = q.lib().qlin_attn_workspace_bytes(cache._c, b._c, T, Hq)
    assert nbytes > 0
    e4 = fmt == "e4m3"
    for kv in ([0, 0, 0], [0, 900, 3], [-5, 0, 0], [1000, 1, 400]):
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        got, lse = q.attn_paged(cache, b, dev(x), return_lse=True)
        r = oracle.attn_paged(x, host(cache.k), host(cache.v), host(cache.k_scale) if e4 else None,
                              host(cache.v_scale) if e4 else None, start, kv, table, D ** -0.5)
        attn_check(r, host(got), host(lse), D, f"{kv} {fmt}")
        assert not q.workspace(nbytes, got.device)[:65536].any().item(), "counters"


@pytest.mark.parametrize("new,G,cols", [(2, 4, 64), (40, 2, 64), (40, 8, 16384)])
def test_window_of_any_size(q, new, G, cols):
    rng = np.random.default_rng(3)
    cache = q.PagedKV.empty(cols, 1, 128, 16)
    table = rng.permutation(cols)[None].astype(np.int32)
    fill_cache(q, rng, cache, None, np.array([1000]), table)
    b = q.PagedBatch(dev(np.array([0, new], np.int32)), dev(np.array([1000], np.int32)), dev(table), new)
    x = dev(projections(rng, (new, G, 128)))
    ref = q.attn_paged(cache, b, x)
    # (the same kernel with and without a window of at least the table's tokens)
    for window in (16 * cols, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1):
        assert torch.equal(q.attn_paged(cache, b, x, window=window), ref), window


@pytest.mark.parametrize("new,G,more", [(1, 4, 0), (80, 2, 0), (80, 2, 300)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_pool_beyond_32_bit_offsets(q, oracle, fmt, new, G, more):
    """Pages whose byte offsets pass 2^32."""
    D, Hkv, page = 256, 8, 256
    one = Hkv * page * D * (2 if fmt == "bf16" else 1)
    pages = (1 << 32) // one + 40
    rng = np.random.default_rng(12)
    cache = q.PagedKV.empty(pages, Hkv, D, page, fmt)
    table = np.array([[pages - 1, pages - 7, 3] + [-1] * more], np.int32)
    kv = np.array([600])
    start = np.array([0, new], np.int32)
    fill_cache(q, rng, cache, start, kv, table)
    x = projections(rng, (new, Hkv * G, D))
    b = q.PagedBatch(dev(start), dev(kv.astype(np.int32)), dev(table), new)
    got, lse = q.attn_paged(cache, b, dev(x), return_lse=True)
    e4 = fmt == "e4m3"
    small = [host(t[table[0, :3].tolist()]) if t is not None else None
             for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    r = oracle.attn_paged(x, small[0], small[1], small[2] if e4 else None, small[3] if e4 else None, start, kv,
                          np.array([[0, 1, 2]]), D ** -0.5)
    attn_check(r, host(got), host(lse), D, f"{fmt}")


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page,Hkv,Hq,rot,inter", [(64, 16, 1, 3, 64, False), (128, 64, 2, 8, 128, False),
                                                     (128, 16, 3, 0, 32, True), (256, 32, 2, 4, 128, True),
                                                     (256, 256, 1, 1, 256, False), (64, 128, 5, 5, 16, False),
                                                     (128, 32, 2, 4, 0, False)])
def test_append(q, oracle, D, page, Hkv, Hq, rot, inter, fmt):
    rng = np.random.default_rng(D + page + Hq)
    new, kv = [1, 0, 5, 40, 3, 2], [page, 9, 5, 3 * page + 1, 1, 30]  # the fifth: only its last token fits
    start, table, pages = make_batch(rng, new, kv, page)
    table[5, :] = pages  # its tokens have no page
    T, pad = int(start[-1]), 2
    cache = stale_pool(q, pages, Hkv, page, D, fmt)
    before = [t.clone() for t in (cache.k, cache.v)]
    qkv = projections(rng, (T + pad, Hq + 2 * Hkv, D))
    qkv[3, Hq:] = 0  # a zero row: scale 0
    d = dev(qkv)
    plan = q.Rope(D, rot_dim=rot, interleaved=inter, scaling=("linear", 4.0)) if rot else None
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), max(new))
    slot, place = oracle.kv_slots(start, kv, table, page, pages, T + pad)
    custom = rng.integers(0, 1 << 18, T + pad).astype(np.int32)
    for positions in (None, custom):
        for t, o in zip((cache.k, cache.v), before):
            t.copy_(o)
        q_out = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda") if Hq else None
        r = q.kv_append(cache, b, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], rope=plan, q=d[:, :Hq] if Hq else None,
                        q_out=q_out, positions=None if positions is None else dev(positions))
        assert r is q_out
        pos = place if positions is None else positions
        turns = host(plan.turns) if rot else np.zeros(8)
        y, mag = oracle.rope(qkv, pos, turns, rot, inter)
        if Hq:
            rope_check(host(q_out)[:T], y[:T, :Hq], mag[:T, :Hq], "queries")
            assert (host(q_out)[T:] == 0x40E0).all()
        stored = np.flatnonzero(slot >= 0)
        assert len(stored) == 1 + 5 + 40 + 1
        page_of, row = slot[stored] // page, slot[stored] % page
        for name, y_part, m_part, x_part in (("k", y[:, Hq:Hq + Hkv], mag[:, Hq:Hq + Hkv], qkv[:, Hq:Hq + Hkv]),
                                             ("v", None, None, qkv[:, Hq + Hkv:])):
            got = host(getattr(cache, name))[page_of, :, row]
            xs = x_part[stored]
            if fmt == "bf16":
                if name == "v":
                    assert np.array_equal(got, xs)
                else:
                    rope_check(got, y_part[stored], m_part[stored], "keys")
                continue
            sc = host(getattr(cache, name + "_scale"))[page_of, :, row]
            if name == "v" or not rot:  # as the per-token quantiser, bit for bit
                want, ws = oracle.quant_act(xs.reshape(-1, D), oracle.OCP)
                assert np.array_equal(got.reshape(-1, D), want) and np.array_equal(sc.ravel(), ws)
                continue
            yy, mm = y_part[stored], m_part[stored]
            top = np.abs(yy).max(-1)
            eps = 2.0 ** -20 * mm.max(-1)  # of the fp32 rotated values
            assert (np.abs(sc - top / 448) <= (eps + top * 2.0 ** -23) / 448).all()
            val = oracle.fp8_decode_table(oracle.OCP)[got] * np.where(sc > 0, sc, 0)[..., None].astype(np.float64)
            # half a step of the format (2^-4 of the value, 2^-10 below its
            # normal range) and the fp32 errors of row and scale
            tol = np.maximum(2.0 ** -4 * np.abs(yy), 2.0 ** -10 * (top / 448)[..., None]) + 3 * eps[..., None]
            assert (np.abs(val - yy) <= tol).all()
        # nothing else was written
        for t, o in zip((cache.k, cache.v), before):
            keep = np.ones((pages, page), bool)
            keep[page_of, row] = False
            a, bb = host(t).transpose(0, 2, 1, 3)[keep], host(o).transpose(0, 2, 1, 3)[keep]
            assert np.array_equal(a, bb)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_codes_of_any_magnitude(q, oracle, D):
    """E4M3 rows from the smallest to the largest magnitudes, ties among their
    quotients: the per-token quantiser's scales and codes, bit for bit."""
    rng = np.random.default_rng(D)
    T, Hkv, page = 4096, 2, 64
    x = rng.standard_normal((T, Hkv, D)) * 2.0 ** rng.integers(-126, 127, (T, Hkv, 1))
    x[:512] = 2.0 ** rng.integers(-100, 100, (512, Hkv, 1)) * rng.integers(-448, 449, (512, Hkv, D)) / 16  # exact quotients
    k = bits(np.clip(x, -3e38, 3e38))
    cache = q.PagedKV.empty(T // page, Hkv, D, page, "e4m3")
    table = rng.permutation(T // page)[None].astype(np.int32)
    b = q.PagedBatch(dev(np.array([0, T], np.int32)), dev(np.array([T], np.int32)), dev(table), T)
    q.kv_append(cache, b, dev(k), dev(k[::-1].copy()))
    slot, _ = oracle.kv_slots([0, T], [T], table, page, T // page, T)
    for name, rows in (("k", k), ("v", k[::-1])):
        want, ws = oracle.quant_act(np.ascontiguousarray(rows).reshape(-1, D), oracle.OCP)
        got = host(getattr(cache, name))[slot // page, :, slot % page].reshape(-1, D)
        sc = host(getattr(cache, name + "_scale"))[slot // page, :, slot % page].ravel()
        assert np.array_equal(sc, ws), name
        assert np.array_equal(got, want), name


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_codes_of_negative_zeros(q, oracle, D):
    """A zero keeps its sign in its E4M3 code at every scale, as in the per-token
    quantiser: rows of any magnitude with zeros of both signs among them, and values
    so small that their codes are zeros."""
    rng = np.random.default_rng(D + 1)
    T, Hkv, page = 509, 3, 16
    x = rng.standard_normal((T, Hkv, D)) * 2.0 ** rng.integers(-126, 127, (T, Hkv, 1))
    x *= np.where(rng.random(x.shape) < 0.2, 2.0 ** -30, 1.0)
    k = bits(np.clip(x, -3e38, 3e38))
    k[rng.random(k.shape) < 0.2] = 0x8000
    k[rng.random(k.shape) < 0.1] = 0x0000
    k[7] = 0x8000  # rows of nothing else: scale 0, codes 0
    pages = -(-T // page)
    cache = q.PagedKV.empty(pages, Hkv, D, page, "e4m3")
    table = rng.permutation(pages)[None].astype(np.int32)
    b = q.PagedBatch(dev(np.array([0, T], np.int32)), dev(np.array([T], np.int32)), dev(table), T)
    q.kv_append(cache, b, dev(k), dev(k[::-1].copy()))
    slot, _ = oracle.kv_slots([0, T], [T], table, page, pages, T)
    for name, rows in (("k", k), ("v", k[::-1])):
        want, ws = oracle.quant_act(np.ascontiguousarray(rows).reshape(-1, D), oracle.OCP)
        assert (want == 0x80).sum() > T * Hkv * D // 8
        got = host(getattr(cache, name))[slot // page, :, slot % page].reshape(-1, D)
        assert np.array_equal(host(getattr(cache, name + "_scale"))[slot // page, :, slot % page].ravel(), ws), name
        assert np.array_equal(got, want), name


def test_append_in_place_queries(q):
    rng = np.random.default_rng(8)
    start, table, pages = make_batch(rng, [20], [60], 16)
    cache = stale_pool(q, pages, 2, 16, 64, "bf16")
    qkv = dev(projections(rng, (20, 8, 64)))
    b = q.PagedBatch(dev(start), dev(np.array([60], np.int32)), dev(table), 20)
    plan = q.Rope(64)
    want = q.kv_append(cache, b, qkv[:, 4:6], qkv[:, 6:], rope=plan, q=qkv[:, :4])
    k, v = cache.k.clone(), cache.v.clone()
    got = q.kv_append(cache, b, qkv[:, 4:6], qkv[:, 6:], rope=plan, q=qkv[:, :4], q_out=qkv[:, :4])
    assert torch.equal(want.view(torch.int16), got.contiguous().view(torch.int16))
    assert torch.equal(k.view(torch.int16), cache.k.view(torch.int16))
    assert torch.equal(v.view(torch.int16), cache.v.view(torch.int16))


# ------------------------------------------------------------------ together
def layer_weights(q, rng, H, heads, D):
    w = (rng.standard_normal((heads * D, H)) * 0.05).astype(np.float32)
    return q.quant_weight(dev(bits(w)))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_layer_prompt_then_steps(q, oracle, fmt):
    """A layer's attention path (FP8 QKV linear, append with rotation,
    attention, FP8 output linear): a prompt as two chunks and three single steps
    gives what one chunk over everything gives, row by row."""
    rng = np.random.default_rng(77)
    H, Hq, Hkv, D, page, n = 512, 8, 2, 128, 16, 150
    wqkv, sqkv = layer_weights(q, rng, H, Hq + 2 * Hkv, D)
    wo, so = q.quant_weight(dev(bits(rng.standard_normal((H, Hq * D)) * 0.05)))
    x = dev(bits(rng.standard_normal((n, H))))
    qkv_all = q.linear_fp8(x, wqkv, sqkv).view(n, Hq + 2 * Hkv, D)
    plan = q.Rope(D)
    table = torch.from_numpy(rng.permutation(12)[None].astype(np.int32)).cuda()

    def step(cache, qkv, done):
        T = qkv.shape[0]
        b = q.PagedBatch(torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                         torch.tensor([done + T], dtype=torch.int32, device="cuda"), table, T)
        qq = q.kv_append(cache, b, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], rope=plan, q=qkv[:, :Hq])
        a = q.attn_paged(cache, b, qq)
        return a, q.linear_fp8(a.view(T, Hq * D), wo, so)

    whole = step(stale_pool(q, 12, Hkv, page, D, fmt), qkv_all, 0)
    cache, at, parts = stale_pool(q, 12, Hkv, page, D, fmt), 0, []
    for m in (100, 47, 1, 1, 1):
        parts.append(step(cache, qkv_all[at:at + m], at))
        at += m
    a = torch.cat([p[0] for p in parts])
    # the same queries over the same cached values: both are within 2^-8 (weights)
    # of the largest cached value (E4M3: 2^-4 above what was stored) and 2^-8
    # (output) of their own value from the exact result, and fp32 sums
    vmax = qkv_all[:, Hq + Hkv:].abs().max().item() * (1 + 2.0 ** -4)
    assert (a.float() - whole[0].float()).abs().max().item() <= 4 * 2.0 ** -8 * vmax * 1.01
    for got, y in ((a, torch.cat([p[1] for p in parts])), whole):
        aq, sa = oracle.quant_act(host(got).reshape(n, Hq * D), oracle.OCP)
        y32, _ = oracle.gemm_fp8(aq, sa, host(wo), host(so))
        tol_check(bf16_to_f32(host(y)), y32, "output linear")


# ------------------------------------------------------------------ streams, graphs
def decode_setup(q, seed, fmt="bf16", B=5, cap=40, Hkv=2, G=4, D=128, page=16):
    rng = np.random.default_rng(seed)
    table = rng.permutation(B * cap).reshape(B, cap).astype(np.int32)
    kv = rng.integers(20, 300, B).astype(np.int32)
    cache = stale_pool(q, B * cap, Hkv, page, D, fmt)
    fill_cache(q, rng, cache, None, kv, table)
    batch = q.PagedBatch(torch.arange(B + 1, dtype=torch.int32, device="cuda"), dev(kv), dev(table), 1)
    qkv = dev(projections(rng, (B, (G + 2) * Hkv, D)))
    return cache, batch, qkv, q.Rope(D), G * Hkv


def decode_step(q, cache, batch, qkv, plan, Hq):
    Hkv = cache.kv_heads
    qq = q.kv_append(cache, batch, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], rope=plan, q=qkv[:, :Hq])
    return q.attn_paged(cache, batch, qq, return_lse=True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_graph_replays(q, fmt):
    """A captured step (key axis split: workspace and join) replayed with new
    lengths and inputs, eager work between the replays, equals the eager step."""
    s = decode_setup(q, 1, fmt)
    cache, batch, qkv, plan, Hq = s
    assert q.lib().qlin_attn_workspace_bytes(cache._c, batch._c, 5, Hq) > 0
    for _ in range(2):
        decode_step(q, *s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = decode_step(q, *s)
    rng = np.random.default_rng(2)
    for rep in range(4):
        batch.kv_len.add_(1)
        qkv.copy_(dev(projections(rng, tuple(qkv.shape))))
        pools = [t.clone() for t in (cache.k, cache.v)]
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = (host(out), host(lse), host(cache.k), host(cache.v))
        for t, o in zip((cache.k, cache.v), pools):
            t.copy_(o)
        ref = decode_step(q, *s)
        torch.cuda.synchronize()
        assert np.array_equal(got[0], host(ref[0])), rep
        assert np.array_equal(got[1], host(ref[1])), rep
        assert np.array_equal(got[2], host(cache.k)) and np.array_equal(got[3], host(cache.v)), rep


def test_two_streams_and_two_graphs(q):
    """Steps on two streams at once, eager and as two graphs, equal the serial
    results: nothing is shared between the calls."""
    sets = [decode_setup(q, 3), decode_setup(q, 4, cap=30)]
    refs = [tuple(host(t) for t in decode_step(q, *s)) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [[], []]
        for _ in range(5):
            for i, s in enumerate(sets):
                with torch.cuda.stream(streams[i]):
                    got[i].append(decode_step(q, *s))
        torch.cuda.synchronize()
        for i in range(2):
            for o, l in got[i]:
                assert np.array_equal(host(o), refs[i][0]) and np.array_equal(host(l), refs[i][1])
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(decode_step(q, *s))
        graphs.append(g)
    for _ in range(4):
        for o, l in outs:
            o.zero_()
            l.zero_()
        torch.cuda.synchronize()
        for i, g in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                g.replay()
        torch.cuda.synchronize()
        for i, (o, l) in enumerate(outs):
            assert np.array_equal(host(o), refs[i][0]) and np.array_equal(host(l), refs[i][1])


def chunk_setup(q, seed, fmt, cols):
    rng = np.random.default_rng(seed)
    Hkv, G, D, page = 2, 4, 128, 16
    new, kv = [70, 0, 33], [1100, 5, 700]
    table = rng.permutation(240).reshape(3, 80).astype(np.int32)
    cache = stale_pool(q, 240, Hkv, page, D, fmt)
    fill_cache(q, rng, cache, None, np.array(kv), table)
    table = np.concatenate([table, np.full((3, cols - 80), -1, np.int32)], 1)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    batch = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), 70)
    qkv = dev(projections(rng, (sum(new), (G + 2) * Hkv, D)))
    assert q.lib().qlin_attn_workspace_bytes(cache._c, batch._c, sum(new), G * Hkv) > 0
    return cache, batch, qkv, q.Rope(D), G * Hkv


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("cols", [80, 5000])
def test_chunks_in_graphs_on_two_streams(q, fmt, cols):
    """Chunks whose key axis is split (parts in a workspace, joined by the last
    workgroup or by a second launch), eager on two streams and as two graphs
    replayed at once."""
    sets = [chunk_setup(q, 21, fmt, cols), chunk_setup(q, 22, fmt, cols)]
    refs = [tuple(host(t) for t in decode_step(q, *s)) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(decode_step(q, *s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(np.array_equal(host(o), refs[i][0]) and np.array_equal(host(z), refs[i][1]) for o, z in got[i])
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(decode_step(q, *s))
        graphs.append(g)
    for _ in range(4):
        for o, z in outs:
            o.zero_()
            z.zero_()
        decode_step(q, *sets[0])
        torch.cuda.synchronize()
        for i, g in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                g.replay()
        torch.cuda.synchronize()
        for i, (o, z) in enumerate(outs):
            assert np.array_equal(host(o), refs[i][0]) and np.array_equal(host(z), refs[i][1])


@pytest.mark.parametrize("cols", [80, 5000])
def test_one_workspace_with_the_products(q, cols):
    """Attention (split steps and chunks) and split-K products take turns in one
    stream's workspace."""
    rng = np.random.default_rng(8)
    step, chunk = decode_setup(q, 23), chunk_setup(q, 24, "bf16", cols)
    M, N, K = 8, 512, 8192
    assert q.workspace_bytes(q.OP_GEMM_FP8, M, N, K) > 0
    w, ws = q.quant_weight(dev(bits(rng.standard_normal((N, K)))))
    a, sa = q.quant_act(dev(bits(rng.standard_normal((M, K)))))

    def turn():
        return [*decode_step(q, *step), q.gemm_fp8(a, sa, w, ws), *decode_step(q, *chunk), q.gemm_fp8(a, sa, w, ws)]

    ref = [host(t) for t in turn()]
    for _ in range(4):
        assert all(np.array_equal(host(x), y) for x, y in zip(turn(), ref))
    r = q.linear_fp8(dev(bits(rng.standard_normal((M, K)))), w, ws)
    assert torch.isfinite(r.float()).all()


@pytest.mark.parametrize("first", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,new", [([20000], [64]), ([8192, 700, 64, 3000], [100, 100, 64, 99])])
def test_one_batch_over_caches_of_both_types(q, oracle, lens, new, first):
    """Layers of one model may keep their caches in different types: a batch serves
    both, in either order, although the calls' workspaces differ in size."""
    rng = np.random.default_rng(len(lens))
    Hkv, G, D, page = 8, 4, 128, 16
    start, table, pages = make_batch(rng, new, lens, page)
    T = int(start[-1])
    batch = q.PagedBatch(dev(start), dev(np.array(lens, np.int32)), dev(table), max(new))
    x = projections(rng, (T, Hkv * G, D))
    caches = {f: stale_pool(q, pages, Hkv, page, D, f) for f in ("bf16", "e4m3")}
    sizes = {f: q.lib().qlin_attn_workspace_bytes(c._c, batch._c, T, Hkv * G) for f, c in caches.items()}
    assert sizes["bf16"] != sizes["e4m3"]
    rows = [0, T // 2, T - 1]  # checked against the oracle, as sequences of one token of their own
    b = np.searchsorted(start, rows, side="right") - 1
    upto = [lens[i] - new[i] + r - start[i] + 1 for i, r in zip(b, rows)]
    for f in sorted(caches, key=lambda f: f != first):
        c = caches[f]
        fill_cache(q, rng, c, None, np.array(lens), table)
        got, lse = q.attn_paged(c, batch, dev(x), return_lse=True)
        e4 = f == "e4m3"
        r = oracle.attn_paged(x[rows], host(c.k), host(c.v), host(c.k_scale) if e4 else None,
                              host(c.v_scale) if e4 else None, np.arange(4), upto, table[b], D ** -0.5)
        attn_check(r, host(got)[rows], host(lse)[rows], D, f"{f} after {first}")


def test_same_result_every_time(q):
    """No atomics: repeated calls agree bit for bit, with and without other
    work on the device."""
    s = decode_setup(q, 5, "e4m3")
    ref = [host(t) for t in decode_step(q, *s)]
    a = torch.randn(2048, 2048, device="cuda")
    for _ in range(5):
        a = a @ a * 1e-3
        got = [host(t) for t in decode_step(q, *s)]
        assert all(np.array_equal(x, y) for x, y in zip(got, ref))


def test_binding_refusals(q):
    cache, batch, qkv, plan, Hq = decode_setup(q, 6)
    k, v, x = qkv[:, 8:10], qkv[:, 10:], qkv[:, :8]
    with pytest.raises(TypeError):
        q.attn_paged(cache, batch, x.float())
    with pytest.raises(ValueError):
        q.attn_paged(cache, batch, x[:, :, :64])  # head size
    with pytest.raises(ValueError):
        q.attn_paged(cache, batch, x.transpose(0, 1))
    with pytest.raises(ValueError):
        q.attn_paged(cache, batch, x[0])
    with pytest.raises(q.QlinError):
        q.attn_paged(cache, batch, x[:, :3])  # no multiple of the cache's heads
    with pytest.raises(q.QlinError):
        q.attn_paged(cache, batch, x, window=4, causal=False)
    with pytest.raises(q.QlinError):
        q.attn_paged(cache, batch, x, scale=float("nan"))
    with pytest.raises(ValueError):
        q.attn_paged(cache, batch, x, out=torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        q.kv_append(cache, batch, k[:2], v)
    with pytest.raises(ValueError):
        q.kv_append(cache, batch, k, v, q_out=x)
    with pytest.raises(ValueError):
        q.kv_append(cache, batch, k[:, :1], v)
    with pytest.raises(ValueError):
        q.kv_append(cache, batch, k, v, rope=q.Rope(64))
    with pytest.raises(TypeError):
        q.kv_append(cache, batch, k, v, positions=torch.zeros(5, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        q.rope(x, torch.zeros(4, dtype=torch.int32, device="cuda"), plan)
    with pytest.raises(ValueError):
        q.rope(x, torch.zeros(5, dtype=torch.int32), plan)
    with pytest.raises(ValueError):
        q.PagedKV.empty(4, 2, 96)
    with pytest.raises(ValueError):
        q.PagedKV.empty(4, 2, 64, 48)
    with pytest.raises(ValueError):
        q.PagedKV.empty(4, 2, 64, 16, "int8")
    with pytest.raises(ValueError):
        q.PagedKV(cache.k, cache.v[:, :, :, :64].contiguous())
    with pytest.raises(ValueError):
        q.PagedKV(cache.k, cache.v, k_scale=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        q.PagedBatch(batch.q_start, batch.kv_len[:2], batch.page_table, 1)
    # empty calls
    none = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    assert q.attn_paged(cache, batch, none).shape == (0, 8, 128)
    assert q.rope(none, torch.zeros(0, dtype=torch.int32, device="cuda"), plan).shape == (0, 8, 128)


def test_integers_beyond_64_bits_are_refused(q):
    """Not taken modulo 2^64: a window of 2^64 + 5 is not one of 5."""
    cache, batch, qkv, plan, Hq = decode_setup(q, 6)
    for window in (1 << 63, (1 << 64) + 5, -(1 << 63) - 1):
        with pytest.raises(ValueError):
            q.attn_paged(cache, batch, qkv[:, :Hq], window=window)
    with pytest.raises(q.QlinError):
        q.attn_paged(cache, batch, qkv[:, :Hq], window=-(1 << 63))
    with pytest.raises(ValueError):
        q.PagedBatch(batch.q_start, batch.kv_len, batch.page_table, (1 << 64) + 1)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,kv,G,D,more,window", [
    ([1, 2, 0, 1], [300, 70, 5, 1], 4, 128, 0, 0), ([1], [2000], 4, 128, 100, 0), ([60, 3, 40], [90, 3, 400], 5, 128, 0, 0),
    ([60, 3, 40], [90, 3, 400], 3, 64, long_table(16), 0), ([130, 7], [1130, 7], 2, 256, long_table(16), 90),
    ([1], [777], 71, 64, 0, 0), ([1, 1], [777, 30], 71, 128, long_table(16), 0), ([3, 1], [400, 400], 40, 256, 0, 17)])
def test_strided_rows_and_rows_before_the_first_sequence(q, oracle, new, kv, G, D, more, window, fmt):
    """Queries and outputs inside wider rows, groups of heads of any size, padding on
    both sides of the sequences: nothing else is written."""
    rng = np.random.default_rng(G + D)
    Hkv, page, lead, pad = 2, 16, 3, 2
    start, table, pages = make_batch(rng, new, kv, page)
    cache = stale_pool(q, pages, Hkv, page, D, fmt)
    fill_cache(q, rng, cache, start, np.array(kv), table)
    table = np.concatenate([table, np.full((len(kv), more), -1, np.int32)], 1)
    start = (start + lead).astype(np.int32)
    T, Hq, e4 = int(start[-1]) + pad, Hkv * G, fmt == "e4m3"
    wide = projections(rng, (T, Hq + 2 * Hkv, D))
    d = dev(wide)
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), max(new))
    buf = torch.full((T, Hq + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")

    def untouched():
        h = host(buf)
        return (h[:, 0] == 0x40E0).all() and (h[:lead] == 0x40E0).all() and (h[T - pad:] == 0x40E0).all()

    out, lse = q.attn_paged(cache, b, d[:, Hkv:Hkv + Hq], window=window, out=buf[:, 1:], return_lse=True)
    x = np.ascontiguousarray(wide[:, Hkv:Hkv + Hq])
    r = oracle.attn_paged(x, host(cache.k), host(cache.v), host(cache.k_scale) if e4 else None,
                          host(cache.v_scale) if e4 else None, start, kv, table, D ** -0.5, True, window)
    attn_check(r, host(out), host(lse), D, "strided")
    assert untouched()
    before, plan = [host(t) for t in (cache.k, cache.v)], q.Rope(D)
    buf.fill_(7.0)
    q.kv_append(cache, b, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], rope=plan, q=d[:, :Hq], q_out=buf[:, 1:])
    slot, place = oracle.kv_slots(start, kv, table, page, pages, T)
    y, mag = oracle.rope(wide, place, host(plan.turns), D)
    rope_check(host(buf)[lead:T - pad, 1:], y[lead:T - pad, :Hq], mag[lead:T - pad, :Hq], "queries")
    assert untouched()
    kept = np.ones((pages, page), bool)
    kept[slot[slot >= 0] // page, slot[slot >= 0] % page] = False
    for t, o in zip((cache.k, cache.v), before):
        assert np.array_equal(host(t).transpose(0, 2, 1, 3)[kept], o.transpose(0, 2, 1, 3)[kept])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,G,more", [([3, 1], 4, 0), ([60, 40], 2, 0), ([60, 40], 2, long_table(16))])
def test_queries_and_keys_that_are_not_finite(q, new, G, more, fmt):
    """They reach their own rows, or the rows that see them, and no other, by a bit."""
    rng = np.random.default_rng(5)
    D, Hkv, page, kv = 128, 1, 16, [90, 61]
    start, table, pages = make_batch(rng, new, kv, page)
    cache = stale_pool(q, pages, Hkv, page, D, fmt)
    fill_cache(q, rng, cache, start, np.array(kv), table)
    T, last = int(start[-1]), new[0] - 1
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)),
                     dev(np.concatenate([table, np.full((2, more), -1, np.int32)], 1)), max(new))

    def run(x, rows):  # rows: what must differ from the finite call
        got, lse = (host(t) for t in q.attn_paged(cache, b, dev(x), return_lse=True))
        keep = np.ones((T, G), bool)
        for i in rows:
            keep[i] = False
            assert np.isnan(bf16_to_f32(got[i])).all() and np.isnan(lse[i]).all()
        return got[keep], lse[keep], keep

    x = projections(rng, (T, G, D))
    out, lse, _ = run(x, [])
    out, lse = out.reshape(T, G, D), lse.reshape(T, G)
    bad = x.copy()
    bad[1, 0, 5] = 0x7FC0  # NaN
    got, gl, keep = run(bad, [(1, 0)])
    assert np.array_equal(got, out[keep]) and np.array_equal(gl, lse[keep])
    page_of, row = table[0, 89 // page], 89 % page  # the first sequence's last key: its last token's own
    if fmt == "bf16":
        cache.k[page_of, 0, row, 3] = float("nan")
    else:
        cache.k_scale[page_of, 0, row] = float("nan")
    got, gl, keep = run(x, [last])
    assert np.array_equal(got, out[keep]) and np.array_equal(gl, lse[keep])
