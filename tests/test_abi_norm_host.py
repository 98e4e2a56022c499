"""Refusals of the head norms' entry points, on the host (no GPU needed)."""

import math

import pytest
import torch

from test_abi_attn_host import BAD_BATCH, BAD_CACHE, A, batch, cache, p, plan


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    return qlin


def norm(q, **over):
    f = dict(q_weight=A, k_weight=A, v_weight=None, eps=1e-6, offset=0.0, values=0)
    f.update(over)
    return q._HeadNorm(**f)


BAD_NORM = [(dict(eps=0.0), "ERR_ARG"), (dict(eps=-1e-6), "ERR_ARG"), (dict(eps=math.nan), "ERR_ARG"),
            (dict(eps=math.inf), "ERR_ARG"), (dict(eps=1e-31), "ERR_ARG"), (dict(eps=1e31), "ERR_ARG"),
            (dict(offset=math.inf), "ERR_ARG"), (dict(offset=math.nan), "ERR_ARG"), (dict(q_weight=A + 2), "ERR_ALIGN"),
            (dict(k_weight=A + 8), "ERR_ALIGN"), (dict(v_weight=A + 4), "ERR_ALIGN")]


def norm_call(q, x=A, ldx=128, T=4, H=2, D=64, n="", pos=A, pl="", y=2 * A, ldy=128):
    n = norm(q) if n == "" else n
    pl = plan(q) if pl == "" else pl
    return q.lib().qlin_norm_rope(p(x), ldx, T, H, D, n, p(pos), pl, p(y), ldy, None)


def test_norm_rope_refusals(q):
    assert norm_call(q, T=0) == q.OK and norm_call(q, H=0) == q.OK
    assert norm_call(q, T=0, pl=None, pos=None) == q.OK
    for over, status in BAD_NORM:
        assert norm_call(q, n=norm(q, **over)) == getattr(q, status), over
    for bad in (dict(T=-1), dict(H=-1), dict(D=48), dict(D=8), dict(D=2048, ldx=4096, ldy=4096), dict(ldx=120),
                dict(ldy=120), dict(y=A, ldy=136), dict(T=1 << 31), dict(pl=plan(q, rot=80)),
                dict(T=1 << 30, H=16, ldx=1024, ldy=1024)):
        assert norm_call(q, **bad) == q.ERR_SHAPE, bad
    for bad in (dict(n=None), dict(x=None), dict(y=None), dict(pos=None), dict(pl=plan(q, turns=None))):
        assert norm_call(q, **bad) == q.ERR_ARG, bad
    for bad in (dict(x=A + 2), dict(y=A + 8), dict(pos=A + 2), dict(ldx=132), dict(ldy=132)):
        assert norm_call(q, **bad) == q.ERR_ALIGN, bad


def append_call(q, c=None, b=None, T=4, k=A, ldk=128, v=A, ldv=128, n="", pl=None, pos=None, qq=None, ldq=0, heads=0,
                out=None, ldo=0):
    n = norm(q) if n == "" else n
    return q.lib().qlin_kv_append_norm(cache(q) if c is None else c, batch(q) if b is None else b, T, p(k), ldk, p(v),
                                       ldv, n, pl, p(pos), p(qq), ldq, heads, p(out), ldo, None)


def test_append_norm_refusals(q):
    assert append_call(q, T=0) == q.OK
    assert append_call(q, b=batch(q, batch=0)) == q.OK
    assert append_call(q, n=None) == q.ERR_ARG
    for over, status in BAD_NORM:
        assert append_call(q, n=norm(q, **over)) == getattr(q, status), over
    for over, status in BAD_CACHE:
        assert append_call(q, c=cache(q, **over)) == getattr(q, status), over
    for over, status in BAD_BATCH:
        assert append_call(q, b=batch(q, **over)) == getattr(q, status), over
    for over, status in [(dict(T=-1), "ERR_SHAPE"), (dict(ldk=120), "ERR_SHAPE"), (dict(k=None), "ERR_ARG"),
                         (dict(v=A + 4), "ERR_ALIGN"), (dict(pl=plan(q, rot=128)), "ERR_SHAPE"), (dict(qq=A), "ERR_ARG")]:
        assert append_call(q, **over) == getattr(q, status), over


def test_binding_refuses_host_weights(q):
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.HeadNorm(w)
    with pytest.raises(ValueError):
        q.HeadNorm(head_dim=64, device="cpu")
    with pytest.raises(ValueError):
        q.HeadNorm(device="cpu")
