"""Refusals of the trees' entry points, on the host (no GPU needed)."""

import ctypes as C
import math

import pytest

from test_abi_attn_host import BAD_BATCH, BAD_CACHE, LONG, A, any_cache, batch, cache, p


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    return qlin


def tree(q, **over):
    f = dict(mask=A, positions=A, words=1)
    f.update(over)
    return q._Tree(**f)


def attn_call(q, c=None, b=None, T=4, qq=A, ldq=256, heads=4, scale=0.1, t="", window=0, out=2 * A, ldo=256,
              lse=None, ws=1 << 20, nb=1 << 40):
    t = tree(q) if t == "" else t
    return q.lib().qlin_attn_tree(cache(q) if c is None else c, batch(q) if b is None else b, T, p(qq), ldq, heads,
                                  scale, t, window, p(out), ldo, p(lse), p(ws), nb, None)


def test_attn_tree_refusals(q):
    assert attn_call(q, T=0) == q.OK
    assert attn_call(q, b=batch(q, batch=0)) == q.OK
    for over, status in BAD_CACHE:
        assert attn_call(q, c=cache(q, **over)) == getattr(q, status), over
    for over, status in BAD_BATCH:
        assert attn_call(q, b=batch(q, **over)) == getattr(q, status), over
    for over, status in [(dict(t=None), "ERR_ARG"), (dict(t=tree(q, mask=None)), "ERR_ARG"),
                         (dict(t=tree(q, words=0)), "ERR_SHAPE"), (dict(t=tree(q, words=9)), "ERR_SHAPE"),
                         (dict(t=tree(q, words=-1)), "ERR_SHAPE"), (dict(b=batch(q, max_q=65)), "ERR_SHAPE"),
                         (dict(b=batch(q, max_q=513), t=tree(q, words=8)), "ERR_SHAPE"),
                         (dict(t=tree(q, mask=A + 4)), "ERR_ALIGN"), (dict(t=tree(q, positions=A + 2)), "ERR_ALIGN"),
                         (dict(window=-1), "ERR_ARG"), (dict(window=7, b=batch(q, max_q=8)), "ERR_ARG"),
                         (dict(window=8, t=tree(q, positions=None)), "ERR_ARG"), (dict(heads=3), "ERR_SHAPE"),
                         (dict(scale=math.nan), "ERR_ARG"), (dict(qq=None), "ERR_ARG"), (dict(out=None), "ERR_ARG"),
                         (dict(qq=A + 4), "ERR_ALIGN"), (dict(lse=A + 2), "ERR_ALIGN"), (dict(T=1 << 30), "ERR_SHAPE")]:
        assert attn_call(q, **over) == getattr(q, status), over
    assert q.lib().qlin_attn_tree(None, batch(q), 0, None, 0, 1, 0.1, tree(q), 0, None, 0, None, None, 0, None) == q.ERR_ARG


def test_attn_tree_workspace(q):
    c, b = cache(q), batch(q, batch=1, table_cols=4096, max_q=8)
    need = q.lib().qlin_attn_tree_workspace_bytes(c, b, 8, 4)
    assert need > 0 and need % 256 == 0
    kw = dict(c=c, b=b, T=8)
    assert attn_call(q, nb=need - 1, **kw) == q.ERR_WORKSPACE
    assert attn_call(q, ws=None, nb=need, **kw) == q.ERR_WORKSPACE
    assert attn_call(q, ws=(1 << 20) + 16, nb=need, **kw) == q.ERR_ALIGN


def attn_plan(q, c, b, T, heads, window=0):
    out = (C.c_int64 * 3)(-1, -1, -1)
    assert q.lib().qlin_attn_tree_plan(c, b, T, heads, window, out) == q.OK
    return tuple(out)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_no_window_needs_more_workspace_than_reported(q, fmt, D):
    """A call plans with its window, and its parts have to fit the workspace that is sized
    without one, whatever kind of workgroups the window turns it to."""
    page, calls, kinds = 64, 0, set()
    for Hkv in (1, 2, 8, 40):
        for G in (1, 4, 8):
            c = any_cache(q, fmt, D, Hkv, page)
            for B in (1, 2, 5, 64, 700):
                for mq in (1, 3, 16, 17, 40, 129, 512):
                    for cols in (1, 9, 31, 32, 64, 65, 128, 513, 4096):
                        b = batch(q, batch=B, max_q=mq, table_cols=cols)
                        for T in {mq, B * mq, B * (mq // 2 + 1)}:
                            have = q.lib().qlin_attn_tree_workspace_bytes(c, b, T, Hkv * G)
                            for w in (0, mq, 512, 1000, 2047, 2048, 4000, 8192, 16384, 70000, 2 ** 62):
                                rows, parts, used = attn_plan(q, c, b, T, Hkv * G, w)
                                assert used <= have, (Hkv, G, B, mq, cols, T, w)
                                assert (parts > 1) == (used > 0) and (rows > 32 or parts <= 16)
                                kinds.add((rows, parts > 1))
                                calls += 1
    step = (16,) if fmt == "e4m3" and D == 256 else (16, 32)
    assert calls > 100000 and kinds == {(r, s) for r in step + (128 if fmt == "bf16" else 256,) for s in (False, True)}


# The kernels' variants, for the GPU tests: new tokens, words of the mask, key/value heads,
# query heads of one, keys of the table for (bf16, E4M3) and heads of 64, 128 and 256, rows of a
# workgroup and whether the key axis may be in parts.
KERNELS = {
    "16 rows, eight waves": ([8, 3], 1, 2, 2, [(400, 400)] * 3, [(16, 16)] * 3),
    "16 rows, eight waves, parts": ([16, 0, 9], 1, 1, 4, [(2048, 2048)] * 3, [(16, 16)] * 3),
    "16 rows, four waves": ([8, 1, 0, 5, 7] * 14, 1, 8, 2, [(320, 320)] * 3, [(16, 16)] * 3),
    "32 rows, eight waves": ([16, 9, 0, 13], 1, 8, 2, [(2 ** 15, 2 ** 17), (2 ** 14, 2 ** 16), (2 ** 13, 2 ** 16)],
                             [(32, 32), (32, 32), (32, 16)]),
    "32 rows, four waves": ([16, 9, 0, 13] * 10, 1, 8, 2, [(1536, 1536), (1536, 1536), (800, 1536)],
                            [(32, 32), (32, 32), (32, 16)]),
    "chunk": ([200, 0, 65], 4, 64, 4, [(720, 720)] * 3, [(128, 256)] * 3),
    "chunk, parts": ([200, 0, 65, 128], 4, 1, 5, [(2 ** 18, 2 ** 18)] * 3, [(128, 256)] * 3),
}


@pytest.mark.parametrize("name", KERNELS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_kernels_that_the_gpu_tests_are_for(q, fmt, D, name):
    new, words, Hkv, G, keys, rows = KERNELS[name]
    i, f = (64, 128, 256).index(D), fmt == "e4m3"
    b = batch(q, batch=len(new), max_q=max(new), table_cols=keys[i][f] // 16)
    got = attn_plan(q, any_cache(q, fmt, D, Hkv, 16), b, sum(new), Hkv * G)
    assert got[0] == rows[i][f] and (got[1] > 1) == ("parts" in name or keys[i][f] >= 8192)


def test_attn_tree_plan_refusals(q):
    out = (C.c_int64 * 3)()
    c, b, f = cache(q), batch(q), q.lib().qlin_attn_tree_plan
    assert f(None, b, 1, 4, 0, out) == q.ERR_ARG and f(c, None, 1, 4, 0, out) == q.ERR_ARG
    assert f(c, b, 1, 4, -1, out) == q.ERR_ARG and f(c, b, 1, 4, 0, None) == q.ERR_ARG
    assert f(c, batch(q, max_q=513), 1, 4, 0, out) == q.ERR_SHAPE and f(c, b, 1, 3, 0, out) == q.ERR_SHAPE
    assert attn_plan(q, c, b, 0, 4) == (0, 0, 0)


def plan_call(q, b="", T=4, parents=A, words=1, mask=A, positions=A):
    b = batch(q) if b == "" else b
    return q.lib().qlin_tree_plan(b, T, p(parents), words, p(mask), p(positions), None)


def test_tree_plan_refusals(q):
    assert plan_call(q, T=0, parents=None, mask=None) == q.OK
    assert plan_call(q, b=batch(q, batch=0)) == q.OK
    for over, status in [(dict(b=None), "ERR_ARG"), (dict(parents=None), "ERR_ARG"), (dict(mask=None), "ERR_ARG"),
                         (dict(words=0), "ERR_SHAPE"), (dict(words=9), "ERR_SHAPE"), (dict(T=-1), "ERR_SHAPE"),
                         (dict(T=1 << 31), "ERR_SHAPE"), (dict(b=batch(q, max_q=65)), "ERR_SHAPE"),
                         (dict(b=batch(q, max_q=0)), "ERR_SHAPE"), (dict(b=batch(q, batch=-1)), "ERR_SHAPE"),
                         (dict(b=batch(q, batch=1 << 16)), "ERR_SHAPE"), (dict(b=batch(q, q_start=None)), "ERR_ARG"),
                         (dict(b=batch(q, kv_len=None)), "ERR_ARG"), (dict(mask=A + 4), "ERR_ALIGN"),
                         (dict(parents=A + 2), "ERR_ALIGN"), (dict(positions=A + 1), "ERR_ALIGN")]:
        assert plan_call(q, **over) == getattr(q, status), over


def test_tree_plan_arrays_that_overlap(q):
    B = 8 * A
    far = dict(b=batch(q, q_start=B, kv_len=2 * B, batch=6), parents=3 * B, mask=4 * B, positions=5 * B, T=11, words=2)
    apart = plan_call(q, **far)
    assert apart not in (q.OK, q.ERR_ARG)  # (no GPU here)
    assert plan_call(q, **{**far, "positions": 3 * B}) == apart and plan_call(q, **{**far, "positions": None}) == apart
    for at in (dict(mask=5 * B - 8 * 22 + 8), dict(mask=3 * B + 40), dict(mask=B + 24), dict(positions=2 * B + 20),
               dict(positions=3 * B + 4), dict(positions=B - 40), dict(positions=4 * B + 8 * 22 - 4)):
        assert plan_call(q, **{**far, **at}) == q.ERR_ARG, at
    for at in (dict(mask=5 * B - 8 * 22), dict(mask=3 * B + 48), dict(positions=2 * B + 24), dict(positions=3 * B - 44)):
        assert plan_call(q, **{**far, **at}) == apart, at
