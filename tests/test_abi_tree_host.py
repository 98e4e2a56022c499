"""Refusals of the trees' entry points, on the host (no GPU needed)."""

import math

import pytest

from test_abi_attn_host import BAD_BATCH, BAD_CACHE, A, batch, cache, p


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
    need = q.lib().qlin_attn_workspace_bytes(c, b, 8, 4)
    assert need > 0
    kw = dict(c=c, b=b, T=8)
    assert attn_call(q, nb=need - 1, **kw) == q.ERR_WORKSPACE
    assert attn_call(q, ws=None, nb=need, **kw) == q.ERR_WORKSPACE
    assert attn_call(q, ws=(1 << 20) + 16, nb=need, **kw) == q.ERR_ALIGN


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
