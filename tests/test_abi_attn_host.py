"""Refusals of the attention entry points, on the host (no GPU needed)."""

import ctypes as C
import math

import pytest
import torch


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    return qlin


A = 0x10000  # fake (never dereferenced) addresses: validation fails before use


def cache(q, **over):
    f = dict(k=A, v=A, k_scale=None, v_scale=None, pages=8, kv_heads=2, page_size=16, head_dim=64, fmt=q.KV_BF16)
    f.update(over)
    return q._KVCache(**f)


def batch(q, **over):
    f = dict(q_start=A, kv_len=A, page_table=A, batch=2, table_cols=4, max_q=1)
    f.update(over)
    return q._KVBatch(**f)


def plan(q, **over):
    f = dict(turns=A, rot=64, interleaved=0, magnitude=1.0)
    f.update(over)
    return q._RopePlan(**f)


def p(x):
    return None if x is None else C.c_void_p(x)


def test_turns_on_the_host(q, oracle):
    for rot in (16, 48, 128):
        for rule, args in ((0, (1, 1, 0, 1)), (1, (4, 1, 0, 1)), (2, (8, 1, 0, 1)), (3, (16, 8192, 1, 32))):
            out = (C.c_double * (rot // 2))()
            assert q.lib().qlin_rope_turns(rot, 10000.0, rule, *map(float, args), out) == q.OK
            want = oracle.rope_turns(rot, 10000.0, rule, *map(float, args))
            assert all(abs(g - w) <= 1e-13 * w for g, w in zip(out, want))


@pytest.mark.parametrize("args,status", [
    ((16, 1e4, 4, 1, 1, 0, 1), "ERR_ARG"), ((16, 1e4, -1, 1, 1, 0, 1), "ERR_ARG"),
    ((8, 1e4, 0, 1, 1, 0, 1), "ERR_SHAPE"), ((40, 1e4, 0, 1, 1, 0, 1), "ERR_SHAPE"),
    ((1040, 1e4, 0, 1, 1, 0, 1), "ERR_SHAPE"), ((16, 1.0, 0, 1, 1, 0, 1), "ERR_ARG"),
    ((16, math.inf, 0, 1, 1, 0, 1), "ERR_ARG"), ((16, 1e4, 1, 0, 1, 0, 1), "ERR_ARG"),
    ((16, 1e4, 2, math.nan, 1, 0, 1), "ERR_ARG"), ((16, 1e4, 3, 2, 0, 1, 2), "ERR_ARG"),
    ((16, 1e4, 3, 2, 8, 2, 2), "ERR_ARG"), ((16, 1e4, 3, 2, 8, -1, 2), "ERR_ARG"),
    ((16, 1e4, 3, 2, 8, 1, math.inf), "ERR_ARG")])
def test_turns_refusals(q, args, status):
    out = (C.c_double * 512)()
    rot, base, rule, *rest = args
    assert q.lib().qlin_rope_turns(rot, base, rule, *map(float, rest), out) == getattr(q, status)
    assert q.lib().qlin_rope_turns(16, 1e4, 0, 1.0, 1.0, 0.0, 1.0, None) == q.ERR_ARG


@pytest.mark.parametrize("args", [(1e4, 1, 5e-324, 1, 0, 1), (1e4, 2, 1e-308, 1, 0, 1), (1e4, 3, 1e-313, 8192, 1, 32)])
def test_turns_that_overflow(q, args):
    """Parameters within their ranges whose frequencies are infinite: no NaN angles."""
    base, rule, *rest = args
    out = (C.c_double * 8)()
    assert q.lib().qlin_rope_turns(16, base, rule, *map(float, rest), out) == q.ERR_ARG
    assert q.lib().qlin_rope_turns(16, base, rule, 1e-30, *map(float, rest[1:]), out) == q.OK
    assert all(math.isfinite(x) for x in out)


def rope_call(q, x=A, ldx=128, T=4, H=2, D=64, pos=A, pl="", inverse=0, y=2 * A, ldy=128):
    pl = plan(q) if pl == "" else pl
    return q.lib().qlin_rope(p(x), ldx, T, H, D, p(pos), pl, inverse, p(y), ldy, None)


def test_rope_refusals(q):
    assert rope_call(q, T=0) == q.OK
    assert rope_call(q, H=0) == q.OK
    for bad in (dict(T=-1), dict(H=-1), dict(D=56), dict(D=0), dict(D=1040, ldx=4096, ldy=4096), dict(ldx=120),
                dict(ldy=120), dict(y=A, ldy=136), dict(T=1 << 31), dict(pl=plan(q, rot=72)),
                dict(pl=plan(q, rot=80)), dict(pl=plan(q, rot=0)), dict(H=1 << 16, ldx=1 << 23, ldy=1 << 23)):
        assert rope_call(q, **bad) == q.ERR_SHAPE, bad
    for bad in (dict(x=None), dict(y=None), dict(pos=None), dict(pl=None), dict(pl=plan(q, turns=None)),
                dict(pl=plan(q, magnitude=math.nan))):
        assert rope_call(q, **bad) == q.ERR_ARG, bad
    for bad in (dict(x=A + 2), dict(y=A + 8), dict(pos=A + 2), dict(ldx=132), dict(ldy=132),
                dict(pl=plan(q, turns=A + 4))):
        assert rope_call(q, **bad) == q.ERR_ALIGN, bad


def append_call(q, c=None, b=None, T=4, k=A, ldk=128, v=A, ldv=128, pl=None, pos=None, qq=None, ldq=0, heads=0,
                out=None, ldo=0):
    return q.lib().qlin_kv_append(cache(q) if c is None else c, batch(q) if b is None else b, T, p(k), ldk, p(v),
                                  ldv, pl, p(pos), p(qq), ldq, heads, p(out), ldo, None)


BAD_CACHE = [(dict(head_dim=96), "ERR_SHAPE"), (dict(head_dim=512), "ERR_SHAPE"), (dict(page_size=8), "ERR_SHAPE"),
             (dict(page_size=48), "ERR_SHAPE"), (dict(page_size=512), "ERR_SHAPE"), (dict(pages=0), "ERR_SHAPE"),
             (dict(pages=1 << 31), "ERR_SHAPE"), (dict(kv_heads=0), "ERR_SHAPE"), (dict(fmt=2), "ERR_ARG"),
             (dict(k=None), "ERR_ARG"), (dict(v=None), "ERR_ARG"), (dict(k_scale=A), "ERR_ARG"),
             (dict(fmt=1), "ERR_ARG"), (dict(fmt=1, k_scale=A), "ERR_ARG"), (dict(k=A + 8), "ERR_ALIGN"),
             (dict(fmt=1, k_scale=A, v_scale=A + 2), "ERR_ALIGN")]
BAD_BATCH = [(dict(batch=-1), "ERR_SHAPE"), (dict(table_cols=0), "ERR_SHAPE"), (dict(max_q=0), "ERR_SHAPE"),
             (dict(table_cols=1 << 28), "ERR_SHAPE"), (dict(batch=1 << 16), "ERR_SHAPE"), (dict(q_start=None), "ERR_ARG"),
             (dict(kv_len=None), "ERR_ARG"), (dict(page_table=None), "ERR_ARG"), (dict(kv_len=A + 2), "ERR_ALIGN")]


def test_append_refusals(q):
    assert append_call(q, T=0) == q.OK
    assert append_call(q, b=batch(q, batch=0)) == q.OK
    for over, status in BAD_CACHE:
        assert append_call(q, c=cache(q, **over)) == getattr(q, status), over
    for over, status in BAD_BATCH:
        assert append_call(q, b=batch(q, **over)) == getattr(q, status), over
    ok_q = dict(qq=A, ldq=256, heads=4, out=2 * A, ldo=256)
    for over, status in [(dict(T=-1), "ERR_SHAPE"), (dict(ldk=120), "ERR_SHAPE"), (dict(ldv=64), "ERR_SHAPE"),
                         (dict(ldk=132), "ERR_ALIGN"), (dict(k=None), "ERR_ARG"), (dict(v=None), "ERR_ARG"),
                         (dict(v=A + 4), "ERR_ALIGN"), (dict(pos=A + 1), "ERR_ALIGN"),
                         (dict(pl=plan(q, rot=128)), "ERR_SHAPE"), (dict(pl=plan(q, turns=None)), "ERR_ARG"),
                         (dict(qq=A), "ERR_ARG"), (dict(out=A), "ERR_ARG"), ({**ok_q, "heads": 0}, "ERR_SHAPE"),
                         ({**ok_q, "ldq": 248}, "ERR_SHAPE"), ({**ok_q, "out": A, "ldo": 264}, "ERR_SHAPE"),
                         ({**ok_q, "ldo": 260}, "ERR_ALIGN"), ({**ok_q, "qq": A + 2}, "ERR_ALIGN")]:
        assert append_call(q, **over) == getattr(q, status), over


def attn_call(q, c=None, b=None, T=4, qq=A, ldq=256, heads=4, scale=0.1, causal=1, window=0, out=2 * A, ldo=256,
              lse=None, ws=1 << 20, nb=1 << 40):
    return q.lib().qlin_attn_paged(cache(q) if c is None else c, batch(q) if b is None else b, T, p(qq), ldq, heads,
                                   scale, causal, window, p(out), ldo, p(lse), p(ws), nb, None)


def test_attn_refusals(q):
    assert attn_call(q, T=0) == q.OK
    assert attn_call(q, b=batch(q, batch=0)) == q.OK
    for over, status in BAD_CACHE:
        assert attn_call(q, c=cache(q, **over)) == getattr(q, status), over
    for over, status in BAD_BATCH:
        assert attn_call(q, b=batch(q, **over)) == getattr(q, status), over
    for over, status in [(dict(heads=0), "ERR_SHAPE"), (dict(heads=3), "ERR_SHAPE"), (dict(ldq=248), "ERR_SHAPE"),
                         (dict(ldo=192), "ERR_SHAPE"), (dict(scale=math.nan), "ERR_ARG"),
                         (dict(scale=math.inf), "ERR_ARG"), (dict(window=-1), "ERR_ARG"),
                         (dict(window=4, causal=0), "ERR_ARG"), (dict(qq=None), "ERR_ARG"), (dict(out=None), "ERR_ARG"),
                         (dict(qq=A + 4), "ERR_ALIGN"), (dict(lse=A + 2), "ERR_ALIGN"), (dict(ldq=260), "ERR_ALIGN"),
                         (dict(T=1 << 30), "ERR_SHAPE")]:
        assert attn_call(q, **over) == getattr(q, status), over


def test_attn_workspace(q):
    # one sequence, long table: the key axis is split, and the call checks it
    c, b = cache(q), batch(q, batch=1, table_cols=4096)
    need = q.lib().qlin_attn_workspace_bytes(c, b, 1, 4)
    assert need > 0 and need % 256 == 0
    kw = dict(c=c, b=b, T=1)
    assert attn_call(q, nb=need - 1, **kw) == q.ERR_WORKSPACE
    assert attn_call(q, ws=None, nb=need, **kw) == q.ERR_WORKSPACE
    assert attn_call(q, ws=(1 << 20) + 16, nb=need, **kw) == q.ERR_ALIGN
    # a window never needs more than the call without one
    for cols in (1, 7, 300, 4096):
        for B, mq in ((1, 1), (3, 2), (1, 700), (40, 1)):
            bb = batch(q, batch=B, table_cols=cols, max_q=mq)
            assert q.lib().qlin_attn_workspace_bytes(c, bb, B * mq, 4) >= 0
    assert q.lib().qlin_attn_workspace_bytes(c, b, 0, 4) == 0
    assert q.lib().qlin_attn_workspace_bytes(None, b, 1, 4) == 0
    # sizes that the call refuses need none
    for over, _ in BAD_CACHE:
        if set(over) & {"head_dim", "page_size", "pages", "kv_heads"}:
            assert q.lib().qlin_attn_workspace_bytes(cache(q, **over), b, 1, 4) == 0, over
    assert q.lib().qlin_attn_workspace_bytes(c, b, 1 << 62, 4) == 0
    assert q.lib().qlin_attn_workspace_bytes(c, batch(q, batch=1, table_cols=1 << 60), 1, 4) == 0
    assert q.lib().qlin_attn_workspace_bytes(c, b, 1, 3) == 0


def test_binding_refuses_host_tensors(q):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.PagedKV(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        q.PagedBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                     torch.zeros(1, 1, dtype=torch.int32), 1)
    with pytest.raises(ValueError):
        q.Rope(64, device="cpu")
    with pytest.raises(ValueError):
        q.Rope(64, rot_dim=128)
    with pytest.raises(q.QlinError):
        q.Rope(64, rot_dim=24, device="cpu")
    with pytest.raises(ValueError):
        q.Rope(64, scaling=("linear",), device="cpu")
    with pytest.raises(ValueError):
        q.Rope(64, scaling=("other", 2.0), device="cpu")

    class P:
        head_dim = 64
        device = torch.device("cuda", 0)

    with pytest.raises(ValueError):
        q.rope(x, torch.zeros(4, dtype=torch.int32), P)


def test_attn_scales_whose_factor_overflows(q):
    """Scores are multiplied by |scale| * log2(e) in fp32: a scale for which that is
    infinite would turn a score of 0 into NaN."""
    assert attn_call(q, T=0, scale=2.3e38) == q.OK
    assert attn_call(q, T=0, scale=-2.3e38) == q.OK
    for scale in (2.4e38, -2.4e38, 3.4e38, math.nan, -math.inf):
        assert attn_call(q, T=0, scale=scale) == q.ERR_ARG, scale
        assert attn_call(q, scale=scale) == q.ERR_ARG, scale


def attn_plan(q, c, b, T, heads, window=0):
    out = (C.c_int64 * 3)(-1, -1, -1)
    assert q.lib().qlin_attn_plan(c, b, T, heads, window, out) == q.OK
    return tuple(out)


def any_cache(q, fmt, D, Hkv, page):
    e4 = fmt == "e4m3"
    return cache(q, head_dim=D, kv_heads=Hkv, page_size=page, pages=1 << 20, fmt=q.KV_E4M3 if e4 else q.KV_BF16,
                 k_scale=A if e4 else None, v_scale=A if e4 else None)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_no_window_needs_more_workspace_than_reported(q, fmt, D):
    """A call plans with its window, and its parts have to fit the workspace that is
    sized without one, also where the window turns a chunk's kernel into a step's."""
    page, turned, calls = 64, 0, 0
    windows = (1, 33, 500, 511, 512, 1500, 2048, 4000, 8191, 20000, 65536, 10 ** 6, 2 ** 62)
    for Hkv in (1, 2, 8, 40):
        for G in (1, 4, 8):
            c = any_cache(q, fmt, D, Hkv, page)
            for B in (1, 2, 5, 64, 700):
                for mq in (1, 3, 16, 17, 40, 129, 1024, 5000):
                    for cols in (1, 9, 64, 65, 128, 513, 4096):
                        b = batch(q, batch=B, max_q=mq, table_cols=cols)
                        for T in {mq, B * mq, B * (mq // 2 + 1)}:
                            if T * Hkv * G >= 1 << 30:  # (the call's limit)
                                continue
                            have = q.lib().qlin_attn_workspace_bytes(c, b, T, Hkv * G)
                            whole = attn_plan(q, c, b, T, Hkv * G)
                            assert whole[2] <= have
                            for w in windows:
                                rows, parts, used = attn_plan(q, c, b, T, Hkv * G, w)
                                assert used <= have, (Hkv, G, B, mq, cols, T, w)
                                assert (parts > 1) == (used > 0)
                                calls += 1
                                turned += whole[0] > 32 and rows == 32 and parts > 1
    assert turned > 0 and calls > 100000


def test_attn_plan_refusals(q):
    out = (C.c_int64 * 3)()
    c, b = cache(q), batch(q)
    f = q.lib().qlin_attn_plan
    assert f(None, b, 1, 4, 0, out) == q.ERR_ARG and f(c, None, 1, 4, 0, out) == q.ERR_ARG
    assert f(c, b, 1, 4, -1, out) == q.ERR_ARG and f(c, b, 1, 4, 0, None) == q.ERR_ARG
    assert f(cache(q, fmt=2), b, 1, 4, 0, out) == q.ERR_ARG
    for cc, bb, T, heads in ((cache(q, head_dim=96), b, 1, 4), (c, batch(q, max_q=0), 1, 4), (c, b, -1, 4), (c, b, 1, 3),
                             (c, batch(q, table_cols=0), 1, 4), (c, batch(q, table_cols=1 << 60), 1, 4),
                             (c, b, 1 << 30, 4), (c, b, 1, 0)):
        assert f(cc, bb, T, heads, 0, out) == q.ERR_SHAPE
    assert attn_plan(q, c, b, 0, 4) == (0, 0, 0) and attn_plan(q, c, batch(q, batch=0), 1, 4) == (0, 0, 0)
    # no array is looked at
    assert attn_plan(q, cache(q, k=None, v=None), batch(q, q_start=None, kv_len=None, page_table=None), 1, 4)[0] == 32


# Which kernel runs in the GPU tests that are meant for one of them, and whether the key
# axis is in parts: (rows of a workgroup in bf16, in E4M3, parts), for batches of `new`
# tokens over tables of `keys`.
LONG = 1 << 18
PLANS = [
    # decode steps, whole (2304 keys: two tokens a head beyond a table of 2049) and in parts
    (64, 2, 4, 16, [1] * 13, 321 + 15, (32, 32, True)), (128, 1, 4, 32, [3], 2049 + 31 + 160, (32, 32, True)),
    (64, 1, 2, 16, [2] * 150, 64, (32, 32, False)),
    # chunks over their own tables: 32 rows
    (128, 1, 4, 16, [33, 0, 64, 129, 1], 208, (32, 32, False)), (128, 2, 4, 64, [40], 1344 + 576, (32, 32, True)),
    # over long tables: the chunks' kernels, with few heads in parts, with many whole
    (64, 2, 2, 16, [33, 0, 64, 129, 1], LONG + 208, (128, 256, True)),
    (128, 1, 4, 16, [33, 0, 64, 129, 1], LONG + 208, (128, 256, True)),
    (256, 1, 2, 32, [33, 0, 64, 129, 1], LONG + 224, (128, 256, True)),
    (64, 70, 2, 32, [33, 0, 64, 129, 1], LONG + 224, (128, 256, False)),
    (128, 40, 2, 32, [33, 0, 64, 129, 1], LONG + 224, (128, 256, False)),
    (256, 40, 2, 64, [33, 0, 64, 129, 1], LONG + 256, (128, 256, False)),
    (128, 24, 4, 16, [100, 40, 35, 70], LONG + 272, (128, 256, False)),
    (128, 1, 2, 16, [300] + [1] * 69, LONG + 352, (128, 256, True)),
    # whole prompts with windows
    (64, 20, 4, 32, [700, 300], 928, (128, 256, False)), (256, 16, 4, 64, [500, 600], 960, (128, 256, False)),
]


@pytest.mark.parametrize("D,Hkv,G,page,new,keys,want", PLANS)
def test_kernels_that_the_gpu_tests_are_for(q, D, Hkv, G, page, new, keys, want):
    for fmt, rows in (("bf16", want[0]), ("e4m3", want[1])):
        b = batch(q, batch=len(new), max_q=max(new), table_cols=keys // page)
        got = attn_plan(q, any_cache(q, fmt, D, Hkv, page), b, sum(new), Hkv * G)
        assert (got[0], got[1] > 1) == (rows, want[2]), (fmt, got)


def test_given_turns_refusals(q):
    for turns in ([0.1] * 31, [0.1] * 33, [[0.1] * 32], 0.1, [math.nan] * 32, [0.1] * 31 + [math.inf]):
        with pytest.raises(ValueError):
            q.Rope(64, turns=turns, device="cpu")
    with pytest.raises(ValueError):
        q.Rope(64, turns=[0.1] * 32, scaling=("linear", 2.0), device="cpu")
    with pytest.raises(q.QlinError):
        q.Rope(64, rot_dim=24, turns=[0.1] * 12, device="cpu")


def test_grids_that_would_pass_32_bits(q):
    """Threads of a grid are counted in 32 bits: calls beyond are refused, not cut."""
    # rotation: pieces of 16 values, eight heads a thread
    assert rope_call(q, T=(1 << 31) - 1, H=1, D=64, ldx=64, ldy=64) == q.ERR_SHAPE
    assert rope_call(q, T=1 << 30, H=16, D=64, ldx=1024, ldy=1024) == q.ERR_SHAPE
    assert rope_call(q, T=1 << 27, H=9, D=1024, ldx=9216, ldy=9216, pl=plan(q)) == q.ERR_SHAPE
    # (the largest sizes that fit get as far as the next check)
    assert rope_call(q, T=(1 << 30) - 64, H=1, D=64, ldx=64, ldy=64, x=A + 2) == q.ERR_ALIGN
    big = cache(q, kv_heads=8, head_dim=256)
    assert append_call(q, c=big, T=1 << 28, ldk=2048, ldv=2048) == q.ERR_SHAPE
    assert append_call(q, c=big, T=1 << 25, ldk=2048, ldv=2048, k=A + 2) == q.ERR_ALIGN
    # chunks: 256 (E4M3 512) threads for 128 (256) rows, and a workgroup for every
    # (sequence, head) that ends inside one
    for fmt, most in (("bf16", 1 << 24), ("e4m3", 1 << 23)):
        c = any_cache(q, fmt, 64, 255, 16)
        out = (C.c_int64 * 3)()
        for B, T, rows, ok in ((65535, 65535, 100, (65535 * 255 + 65535 * 255 // 128) < most), (65535, 65535, 64, True),
                               (32000, 65535, 100, True), (65535, 4000000, 100, False)):
            b = batch(q, batch=B, max_q=rows)
            status = q.lib().qlin_attn_plan(c, b, T, 255, 0, out)
            assert status == (q.OK if ok else q.ERR_SHAPE), (fmt, B, T, rows)
            if not ok:
                assert attn_call(q, c=c, b=b, T=T, heads=255, ldq=255 * 64, ldo=255 * 64) == q.ERR_SHAPE
                assert q.lib().qlin_attn_workspace_bytes(c, b, T, 255) == 0
