"""Pins of the attention oracle: rotation, cache slots and paged attention
against numpy written another way (complex products, dense softmax)."""

import math

import numpy as np
import pytest

from helpers import bf16_to_f32


def bits(x):
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


@pytest.mark.parametrize("rule,args", [(0, {}), (1, dict(factor=4.0)), (2, dict(factor=8.0)),
                                       (3, dict(factor=16.0, trained_len=8192.0, low=1.0, high=32.0))])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_turns(oracle, rule, args, rot):
    got = oracle.rope_turns(rot, 10000.0, rule, **args)
    plain = np.array([10000.0 ** (-2 * i / rot) for i in range(rot // 2)]) / (2 * math.pi)
    if rule == 0:
        want = plain
    elif rule == 1:
        want = plain / 4.0
    elif rule == 2:
        want = np.array([(10000.0 * 8.0 ** (rot / (rot - 2))) ** (-2 * i / rot) for i in range(rot // 2)]) / \
            (2 * math.pi)
        # the slowest pair turns `factor` times slower, the first as before
        assert abs(got[-1] / plain[-1] - 1 / 8.0) < 1e-12 and got[0] == plain[0]
    else:
        n = 8192.0 * plain
        keep = np.clip((n - 1.0) / 31.0, 0, 1)
        want = plain * keep + plain / 16.0 * (1 - keep)
        np.testing.assert_allclose(got[n >= 32], plain[n >= 32], rtol=1e-15)
        np.testing.assert_allclose(got[n <= 1], plain[n <= 1] / 16, rtol=1e-15)
    np.testing.assert_allclose(got, want, rtol=1e-13)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_is_a_complex_product(oracle, inter):
    rng = np.random.default_rng(3)
    T, H, D, rot = 7, 3, 64, 32
    x = bits(rng.standard_normal((T, H, D)))
    pos = np.array([0, 1, 5, 4099, 1 << 20, -3, 2 ** 31 - 1], np.int32)
    turns = oracle.rope_turns(rot)
    y, mag = oracle.rope(x, pos, turns, rot, inter, 1.25)
    f = bf16_to_f32(x).astype(np.float64)
    a, b = (f[..., 0:rot:2], f[..., 1:rot:2]) if inter else (f[..., :rot // 2], f[..., rot // 2:rot])
    w = pos.astype(np.float64)[:, None] * turns
    z = 1.25 * (a + 1j * b) * np.exp(2j * math.pi * (w - np.rint(w)))[:, None]
    ya, yb = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    np.testing.assert_allclose(ya, z.real, atol=1e-12)
    np.testing.assert_allclose(yb, z.imag, atol=1e-12)
    assert (y[..., rot:] == f[..., rot:]).all()
    assert (mag >= np.abs(y) - 1e-12).all()


def test_slots(oracle):
    # sequence 0: 2 new of 5 (pages of 16: page 4), 1: idle, 2: 3 new ending at 18
    # (positions 15, 16, 17: a page border; the second page does not exist), one
    # padding row behind
    slot, place = oracle.kv_slots([0, 2, 2, 5], [5, 9, 18], [[4, 0], [1, 1], [2, 7]], 16, 7, 6)
    assert slot.tolist() == [4 * 16 + 3, 4 * 16 + 4, 2 * 16 + 15, -1, -1, -1]
    assert place.tolist() == [3, 4, 15, 16, 17, 0]
    # fewer keys than new tokens: the first lie before the sequence
    slot, _ = oracle.kv_slots([0, 3], [1], [[0]], 16, 1, 3)
    assert slot.tolist() == [-1, -1, 0]
    # what lies behind the table's reach is not stored
    slot, place = oracle.kv_slots([0, 3], [17], [[0]], 16, 1, 3)
    assert slot.tolist() == [14, 15, -1] and place.tolist() == [14, 15, 16]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 5)])
def test_attn_is_a_dense_softmax(oracle, fp8, causal, window):
    rng = np.random.default_rng(11)
    new, kv = [3, 1, 0, 4], [20, 33, 7, 2]
    T, Hq, Hkv, D, page, pages = sum(new), 6, 2, 64, 16, 9
    q = bits(rng.standard_normal((T, Hq, D)))
    if fp8:
        k, v = (rng.integers(0, 0x7F, (pages, Hkv, page, D)).astype(np.uint8) for _ in range(2))
        ks, vs = (rng.random((pages, Hkv, page)).astype(np.float32) * 0.01 for _ in range(2))
        dec = oracle.fp8_decode_table(oracle.OCP)
        kf, vf = dec[k] * ks[..., None].astype(np.float64), dec[v] * vs[..., None].astype(np.float64)
    else:
        k, v = (bits(rng.standard_normal((pages, Hkv, page, D))) for _ in range(2))
        ks = vs = None
        kf, vf = bf16_to_f32(k).astype(np.float64), bf16_to_f32(v).astype(np.float64)
    start = np.concatenate([[0], np.cumsum(new)])
    table = np.array([[3, 1, 0], [0, 8, 5], [2, 2, 2], [7, 0, 0]])
    r = oracle.attn_paged(q, k, v, ks, vs, start, kv, table, 0.2, causal, window)
    qf = bf16_to_f32(q).astype(np.float64)
    for b in range(4):
        kk = np.concatenate([kf[p] for p in table[b]], 1)[:, :kv[b]]
        vv = np.concatenate([vf[p] for p in table[b]], 1)[:, :kv[b]]
        for i in range(new[b]):
            p = kv[b] - new[b] + i
            j = np.arange(kv[b])
            see = (j <= p if causal else j >= 0) & ((j > p - window) if window else True)
            for h in range(Hq):
                t = start[b] + i
                assert r["seen"][t, h] == see.sum()
                if not see.any():
                    assert (r["out"][t, h] == 0).all() and r["lse"][t, h] == -np.inf
                    continue
                z = kk[h // 3][see] @ qf[t, h] * 0.2
                e = np.exp(z)
                np.testing.assert_allclose(r["out"][t, h], e @ vv[h // 3][see] / e.sum(), rtol=1e-10, atol=1e-12)
                np.testing.assert_allclose(r["lse"][t, h], np.log(e.sum()), rtol=1e-12)
    # the last sequence has more new tokens than keys: its first two see nothing when causal
    assert (r["seen"][4:6] == 0).all() == causal


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_norm_then_rotation(oracle, inter, weighted):
    """Normalised heads have a root mean square of 1 (without eps and weight), and the
    rotation of the normalised values is the rotation that is pinned above."""
    rng = np.random.default_rng(12)
    T, H, D, rot = 6, 3, 64, 48
    x = bits(rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-60, 60, (T, H, 1)))
    w = bits(rng.standard_normal(D)) if weighted else None
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    turns = oracle.rope_turns(rot)
    f = bf16_to_f32(x).astype(np.float64)
    n, _ = oracle.norm_rope(x, None, 0.0, 3.0, pos, turns, 0)
    np.testing.assert_allclose((n ** 2).mean(-1), 1.0, rtol=1e-12)
    np.testing.assert_allclose(n * np.sqrt((f ** 2).mean(-1, keepdims=True)), f, rtol=1e-12)
    g, mag = oracle.norm_rope(x, w, 0.25, 1.0, pos, turns, rot, inter, 1.5)
    m = f / np.sqrt((f * f).sum(-1, keepdims=True) / D + 0.25)
    if weighted:
        m = m * (1.0 + bf16_to_f32(w).astype(np.float64))
    a, b = (m[..., 0:rot:2], m[..., 1:rot:2]) if inter else (m[..., :rot // 2], m[..., rot // 2:rot])
    part = pos.astype(np.float64)[:, None] * turns
    z = 1.5 * (a + 1j * b) * np.exp(2j * math.pi * (part - np.rint(part)))[:, None]
    ya, yb = (g[..., 0:rot:2], g[..., 1:rot:2]) if inter else (g[..., :rot // 2], g[..., rot // 2:rot])
    np.testing.assert_allclose(ya, z.real, atol=1e-11)
    np.testing.assert_allclose(yb, z.imag, atol=1e-11)
    np.testing.assert_allclose(g[..., rot:], m[..., rot:], rtol=1e-12)
    assert (mag >= np.abs(g) - 1e-12).all()


def test_tree_masks_and_attention(oracle):
    """Masks and positions by hand, and attention under them as a dense softmax over
    the keys that a set of ancestors names."""
    start, kv = np.array([0, 5, 5, 8], np.int32), np.array([9, 4, 3], np.int32)
    parents = np.array([-1, 0, 0, 1, 7, -1, -1, 1], np.int32)  # (7 is no earlier token)
    mask, pos = np.zeros((8, 2), np.uint64), np.zeros(8, np.int32)
    oracle.tree_plan(start, kv, parents, 2, mask, pos)
    assert mask[:, 0].tolist() == [1, 3, 5, 11, 16, 1, 2, 6] and (mask[:, 1] == 0).all()
    assert pos.tolist() == [4, 5, 5, 6, 4, 0, 0, 1]
    rng = np.random.default_rng(13)
    D, page = 64, 16
    k, v = (bits(rng.standard_normal((4, 1, page, D))) for _ in range(2))
    x = bits(rng.standard_normal((8, 2, D)))
    table = np.array([[2], [1], [0]], np.int32)
    for window in (0, 5):
        r = oracle.attn_paged(x, k, v, None, None, start, kv, table, 0.3, True, window, mask, pos)
        kf, vf, xf = (bf16_to_f32(a).astype(np.float64) for a in (k, v, x))
        for b, (s0, s1) in enumerate(zip(start[:-1], start[1:])):
            first = kv[b] - (s1 - s0)
            for t in range(s0, s1):
                keys = [j for j in range(first) if not window or j > pos[t] - window]
                keys += [first + u for u in range(s1 - s0) if (int(mask[t, 0]) >> u) & 1]
                z = xf[t] @ kf[table[b, 0], 0, keys].T * 0.3
                w = np.exp(z - z.max(-1, keepdims=True))
                np.testing.assert_allclose(r["out"][t], w @ vf[table[b, 0], 0, keys] / w.sum(-1, keepdims=True), rtol=1e-9, atol=1e-12)
                np.testing.assert_allclose(r["lse"][t], z.max(-1) + np.log(w.sum(-1)), rtol=1e-12)
                assert (r["seen"][t] == len(keys)).all()
