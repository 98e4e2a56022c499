"""Norms of single heads with the rotation and the cache's append in the same pass, on the
GPU against the fp64 oracle.

Bounds (fp32 2^-24 a rounding): the sum of D squares, all positive, 16 in a row and then
up to six pairwise, is off by 23 * 2^-24 of itself, the reciprocal root by half of that
and its own 2^-23; three products and offset + w round once each: under 18 * 2^-24, which
is below 2^-19 of the value. The rotation adds 2^-20 of the magnitudes that it sums
(tests of the rotation), so that a value is within 3 * 2^-20 of its magnitude, and bf16
rounds by 2^-8 of it."""

import numpy as np
import pytest
import torch

from helpers import bf16_to_f32, dev, host
from test_gpu_attn import bits, make_batch, projections, stale_pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    assert torch.cuda.is_available()
    return qlin


def norm_check(got, y, mag, what):
    err = np.abs(bf16_to_f32(got).astype(np.float64) - y)
    tol = 2.0 ** -8 * np.abs(y) + 3 * 2.0 ** -20 * mag + 2.0 ** -133  # (bf16's smallest step)
    assert (err <= tol).all(), f"{what}: worst {np.max(err / tol):.3f}"


def weight(rng, D, offset):
    return bits(rng.standard_normal(D) * 0.3 + 1.0 - offset)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 16, 16), (3, 5, 32, 32), (8, 32, 128, 128), (7, 3, 256, 64), (70, 2, 64, 16),
                                       (5, 9, 1024, 512), (9, 33, 64, 0), (2, 1, 512, 512), (8195, 6, 128, 64),
                                       (1031, 4, 256, 0)])
def test_norm_rope(q, oracle, T, H, D, rot, inter):
    rng = np.random.default_rng(T * 1000 + D)
    x = projections(rng, (T, H, D))
    x[0, 0] = 0  # a zero head stays zero
    pos = rng.integers(-5, 1 << 20, T).astype(np.int32)
    pos[-1] = 2 ** 31 - 1
    plan = q.Rope(D, rot_dim=rot, interleaved=inter, magnitude=1.25) if rot else None
    turns = host(plan.turns) if rot else np.zeros(1)
    xd, pd = dev(x), dev(pos)
    for offset, eps, weighted in ((0.0, 1e-6, True), (1.0, 0.5, True), (0.0, 1e-5, False)):
        w = weight(rng, D, offset) if weighted else None
        norm = q.HeadNorm(dev(w), eps=eps, offset=offset) if weighted else q.HeadNorm(eps=eps, offset=7.0, head_dim=D)
        rows = slice(None) if T < 100 else np.r_[0:40, T - 40:T]
        y, mag = oracle.norm_rope(x[rows], w, norm._c.eps, offset, pos[rows], turns, rot, inter, 1.25)
        got = q.norm_rope(xd, norm, pd if rot else None, plan)
        norm_check(host(got)[rows], y, mag, f"offset {offset} weighted {weighted}")
        assert (host(got)[0, 0] & 0x7FFF == 0).all()
        if T >= 100:  # heads folded over a thread: the same as row by row
            part = q.norm_rope(xd[4097 % T:4097 % T + 5], norm, pd[4097 % T:4097 % T + 5] if rot else None, plan)
            assert torch.equal(part.view(torch.int16), got[4097 % T:4097 % T + 5].view(torch.int16))


def test_norm_rope_strides_and_in_place(q):
    rng = np.random.default_rng(4)
    qkv = dev(projections(rng, (37, 10, 128)))
    x, tail = qkv[:, 2:8], qkv[:, 8:].clone()
    pos = dev(rng.integers(0, 9000, 37).astype(np.int32))
    plan, norm = q.Rope(128), q.HeadNorm(dev(weight(rng, 128, 0.0)))
    want = q.norm_rope(x.contiguous(), norm, pos, plan)
    out = torch.full((37, 9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q.norm_rope(x, norm, pos, plan, out=out[:, 1:7])
    assert torch.equal(out[:, 1:7].view(torch.int16), want.view(torch.int16))
    assert (out[:, 0] == 7).all() and (out[:, 7:] == 7).all()
    assert q.norm_rope(x, norm, pos, plan, out=x) is x
    assert torch.equal(x.contiguous().view(torch.int16), want.view(torch.int16))
    assert torch.equal(qkv[:, 8:].view(torch.int16), tail.view(torch.int16))


@pytest.mark.parametrize("D", [16, 64, 128, 256, 1024])
def test_norm_of_any_magnitude(q, oracle, D):
    """Heads from bf16's smallest to its largest values: squares pass fp32's range on both
    sides, and one large value stands among small ones."""
    rng = np.random.default_rng(D)
    x = rng.standard_normal((256, 3, D)) * 2.0 ** rng.integers(-130, 127, (256, 3, 1))
    x[0] = 3e38
    x[1, :, 1:] = 0
    x[2, :, 0] = 3e38
    x = bits(np.clip(x, -3.3e38, 3.3e38))
    for eps in (2.0 ** -100, 1e-6, 2.0 ** 100):
        norm = q.HeadNorm(eps=eps, head_dim=D)
        y, mag = oracle.norm_rope(x, None, eps, 0.0, np.zeros(256), np.zeros(1), 0)
        got = host(q.norm_rope(dev(x), norm))
        # (a square below 2^-149 is lost: D of them, beside eps)
        norm_check(got, y, mag + np.abs(y) * 2.0 ** 20 * min(1.0, 2.0 ** -149 / eps), f"eps {eps}")
        assert np.isfinite(bf16_to_f32(got)).all()


def test_norm_of_values_that_are_not_finite(q):
    """NaN makes its head NaN, an infinity itself NaN and the head's finite values zero
    (what the formula gives); no other head sees them."""
    rng = np.random.default_rng(6)
    x = dev(projections(rng, (9, 4, 64)))
    norm = q.HeadNorm(dev(weight(rng, 64, 0.0)))
    want = q.norm_rope(x, norm)
    x[2, 1, 5] = float("nan")
    x[4, 3, 60] = float("-inf")
    got = q.norm_rope(x, norm)
    assert got[2, 1].isnan().all()
    assert got[4, 3, 60].isnan() and (got[4, 3, :60] == 0).all()
    got[2, 1], got[4, 3] = want[2, 1], want[4, 3]
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("values", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page,Hkv,Hq,rot,inter", [(64, 16, 1, 3, 64, False), (128, 64, 2, 8, 128, False),
                                                     (128, 16, 3, 0, 32, True), (256, 32, 2, 4, 128, True),
                                                     (256, 256, 1, 1, 256, False), (128, 32, 2, 4, 0, False)])
def test_append_norm(q, oracle, D, page, Hkv, Hq, rot, inter, fmt, values):
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
    plan = q.Rope(D, rot_dim=rot, interleaved=inter) if rot else None
    turns = host(plan.turns) if rot else np.zeros(1)
    w = [weight(rng, D, 1.0) for _ in range(3)]
    norm = q.HeadNorm(dev(w[0]), dev(w[1]), dev(w[2]) if values else None, eps=1e-5, offset=1.0)
    eps = norm._c.eps
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), max(new))
    slot, place = oracle.kv_slots(start, kv, table, page, pages, T + pad)
    custom = rng.integers(0, 1 << 18, T + pad).astype(np.int32)
    for positions in (None, custom):
        for t, o in zip((cache.k, cache.v), before):
            t.copy_(o)
        q_out = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda") if Hq else None
        r = q.kv_append(cache, b, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], rope=plan, q=d[:, :Hq] if Hq else None,
                        q_out=q_out, positions=None if positions is None else dev(positions), norm=norm)
        assert r is q_out
        pos = place if positions is None else positions
        if Hq:
            y, mag = oracle.norm_rope(qkv[:T, :Hq], w[0], eps, 1.0, pos[:T], turns, rot, inter)
            norm_check(host(q_out)[:T], y, mag, "queries")
            assert (host(q_out)[T:] == 0x40E0).all()
        stored = np.flatnonzero(slot >= 0)
        assert len(stored) == 1 + 5 + 40 + 1
        page_of, row = slot[stored] // page, slot[stored] % page
        for name, at in (("k", Hq), ("v", Hq + Hkv)):
            xs = np.ascontiguousarray(qkv[stored, at:at + Hkv])
            got = host(getattr(cache, name))[page_of, :, row]
            if name == "k":
                y, mag = oracle.norm_rope(xs, w[1], eps, 1.0, pos[stored], turns, rot, inter)
            elif values:
                y, mag = oracle.norm_rope(xs, w[2], eps, 1.0, pos[stored], turns, 0)
            elif fmt == "bf16":
                assert np.array_equal(got, xs)
                continue
            if fmt == "bf16":
                norm_check(got, y, mag, name)
                continue
            sc = host(getattr(cache, name + "_scale"))[page_of, :, row]
            if name == "v" and not values:  # as the per-token quantiser, bit for bit
                want, ws = oracle.quant_act(xs.reshape(-1, D), oracle.OCP)
                assert np.array_equal(got.reshape(-1, D), want) and np.array_equal(sc.ravel(), ws)
                continue
            top = np.abs(y).max(-1)
            off = 3 * 2.0 ** -20 * mag.max(-1)  # of the fp32 normalised and rotated values
            assert (np.abs(sc - top / 448) <= (off + top * 2.0 ** -23) / 448).all()
            val = oracle.fp8_decode_table(oracle.OCP)[got] * np.where(sc > 0, sc, 0)[..., None].astype(np.float64)
            # half a step of the format (2^-4 of the value, 2^-10 below its normal
            # range) and the fp32 errors of row and scale
            tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * (top / 448)[..., None]) + 3 * off[..., None]
            assert (np.abs(val - y) <= tol).all()
            assert (sc[stored == 3] == 0).all() and (got[stored == 3] == 0).all()
        # nothing else was written
        for t, o in zip((cache.k, cache.v), before):
            keep = np.ones((pages, page), bool)
            keep[page_of, row] = False
            a, bb = host(t).transpose(0, 2, 1, 3)[keep], host(o).transpose(0, 2, 1, 3)[keep]
            assert np.array_equal(a, bb)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_append_norm_is_the_norm_and_the_append(q, fmt):
    """Without a rotation, and with one in bf16's exact cases, the pass equals the two
    steps: keys normalised by norm_rope, then appended (bf16: rounded once, equal bits)."""
    rng = np.random.default_rng(9)
    start, table, pages = make_batch(rng, [20, 700], [60, 900], 16)
    one, two = stale_pool(q, pages, 4, 16, 128, fmt), stale_pool(q, pages, 4, 16, 128, fmt)
    qkv = dev(projections(rng, (720, 24, 128)))
    b = q.PagedBatch(dev(start), dev(np.array([60, 900], np.int32)), dev(table), 700)
    w = [dev(weight(rng, 128, 0.0)) for _ in range(3)]
    norm = q.HeadNorm(w[0], w[1], w[2])
    qn = q.kv_append(one, b, qkv[:, 16:20], qkv[:, 20:], q=qkv[:, :16], norm=norm)
    k = q.norm_rope(qkv[:, 16:20], q.HeadNorm(w[1]))
    v = q.norm_rope(qkv[:, 20:], q.HeadNorm(w[2]))
    assert torch.equal(qn.view(torch.int16), q.norm_rope(qkv[:, :16], norm).view(torch.int16))
    if fmt == "bf16":
        q.kv_append(two, b, k, v)
        assert torch.equal(one.k.view(torch.int16), two.k.view(torch.int16))
        assert torch.equal(one.v.view(torch.int16), two.v.view(torch.int16))


def test_norm_binding_refusals(q):
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    norm = q.HeadNorm(w)
    for bad in (dict(q_weight=w, k_weight=torch.ones(32, dtype=torch.bfloat16, device="cuda")), dict(),
                dict(q_weight=w, v_weight=w, values=False), dict(q_weight=w.cpu()), dict(q_weight=w, head_dim=128)):
        with pytest.raises(ValueError):
            q.HeadNorm(**bad)
    with pytest.raises(TypeError):
        q.HeadNorm(w.float())
    with pytest.raises(ValueError):
        q.norm_rope(x, norm, None, q.Rope(64))
    with pytest.raises(ValueError):
        q.norm_rope(x, norm, pos, q.Rope(128))
    with pytest.raises(ValueError):
        q.norm_rope(x, norm, pos[:3], q.Rope(64))
    with pytest.raises(ValueError):
        q.norm_rope(x, q.HeadNorm(head_dim=128))
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-38):
        with pytest.raises(q.QlinError):
            q.norm_rope(x, q.HeadNorm(w, eps=eps))
    with pytest.raises(q.QlinError):
        q.norm_rope(x, q.HeadNorm(w, offset=float("inf")))
    with pytest.raises(q.QlinError):
        q.norm_rope(torch.zeros(4, 2, 48, dtype=torch.bfloat16, device="cuda"), q.HeadNorm(head_dim=48))
    cache = q.PagedKV.empty(3, 2, 128, 16)
    b = q.PagedBatch(torch.tensor([0, 4], dtype=torch.int32, device="cuda"),
                     torch.tensor([4], dtype=torch.int32, device="cuda"),
                     torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 4)
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        q.kv_append(cache, b, k, k, norm=norm)
    assert q.norm_rope(x[:0], norm).shape == (0, 2, 64)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("rot,inter", [(0, False), (128, False), (64, True)])
def test_append_norm_e4m3_of_many_tokens(q, oracle, rot, inter, page):
    """Enough tokens that a thread handles several heads: every stored row's codes and scale
    against the oracle (bounds as in test_append_norm), values that are not normalised bit
    for bit, and queries against norm_rope."""
    rng = np.random.default_rng(rot + page)
    new, kv = [20, 0, 700], [60, 9, 900]
    start, table, pages = make_batch(rng, new, kv, page)
    T, Hq, Hkv, D = 720, 16, 4, 128
    qkv = projections(rng, (T, Hq + 2 * Hkv, D))
    qkv[5, Hq:] = 0
    d = dev(qkv)
    b = q.PagedBatch(dev(start), dev(np.array(kv, np.int32)), dev(table), 700)
    plan = q.Rope(D, rot_dim=rot, interleaved=inter) if rot else None
    turns = host(plan.turns) if rot else np.zeros(1)
    w = [weight(rng, D, 0.0) for _ in range(3)]
    slot, place = oracle.kv_slots(start, kv, table, page, pages, T)
    assert (slot >= 0).all()
    page_of, row = slot // page, slot % page
    decode = oracle.fp8_decode_table(oracle.OCP)
    for values in (False, True):
        cache = stale_pool(q, pages, Hkv, page, D, "e4m3")
        norm = q.HeadNorm(dev(w[0]), dev(w[1]), dev(w[2]) if values else None, eps=1e-5)
        qn = q.kv_append(cache, b, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], rope=plan, q=d[:, :Hq], norm=norm)
        alone = q.norm_rope(d[:, :Hq], norm, dev(place.astype(np.int32)) if rot else None, plan)
        assert torch.equal(qn.view(torch.int16), alone.view(torch.int16))
        for name, at in (("k", Hq), ("v", Hq + Hkv)):
            x = np.ascontiguousarray(qkv[:, at:at + Hkv])
            got, sc = (host(getattr(cache, name + s))[page_of, :, row] for s in ("", "_scale"))
            if name == "v" and not values:
                want, ws = oracle.quant_act(x.reshape(-1, D), oracle.OCP)
                assert np.array_equal(got.reshape(-1, D), want) and np.array_equal(sc.ravel(), ws)
                continue
            turned = (place.astype(np.int32), turns, rot, inter) if name == "k" else (place.astype(np.int32), turns, 0)
            y, mag = oracle.norm_rope(x, w[1 if name == "k" else 2], norm._c.eps, 0.0, *turned)
            top = np.abs(y).max(-1)
            off = 3 * 2.0 ** -20 * mag.max(-1)
            assert (np.abs(sc - top / 448) <= (off + top * 2.0 ** -23) / 448).all()
            val = decode[got] * sc[..., None].astype(np.float64)
            tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * (top / 448)[..., None]) + 3 * off[..., None]
            assert (np.abs(val - y) <= tol).all()
            assert (sc[5] == 0).all() and (got[5] == 0).all()
