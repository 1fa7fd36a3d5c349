"""Host-side checks of the rotary, cache and attention calls (no GPU needed):
sizes, refusals before any launch, the plan's contents, the layout's sizes."""
import ctypes as C
import math

import numpy as np
import pytest

import attn_ref as ref
import gemm_q4_q8_gb300 as qg
from gemm_q4_q8_gb300 import build as qbuild

A = 0x100000  # fake, aligned, far apart; never dereferenced
NULL, SHAPE, ALIGN, TYPE, WORKSPACE, CUDA, ALIAS = 1, 2, 3, 4, 5, 6, 7


def at(i):
    return A + i * (1 << 36)


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qg.load()


def cache(**kw):
    c = dict(pool=at(1), page_table=at(2), type=8, n_kv_heads=8, head_dim=128, page_size=64, n_pages=10,
             max_pages=5, n_seq=2)
    c.update(kw)
    return qg.QGKVCache(*[c[f[0]] for f in qg.QGKVCache._fields_])


def done(st):
    """A call whose arguments are all right fails for want of a GPU."""
    from conftest import gpu_available
    return st == CUDA or gpu_available()


def test_plan_steps_are_turns(lib):
    for rot, base, factor, orig in ((64, 1e7, 1.0, 0), (128, 5e5, 8.0, 8192), (20, 1e4, 4.0, 0), (256, 1e6, 1.0, 0)):
        plan = qg.qrope_plan(rot, base=base, factor=factor, orig_ctx=orig, mscale=1.25)
        want = ref.thetas(rot, base, factor, orig) / (2 * math.pi)
        got = np.array([plan.step[i] for i in range(rot // 2)], np.float64) / 2.0 ** 64
        # pow and the division in f64 on both sides, and the fixed point's step
        np.testing.assert_allclose(got, want, rtol=1e-14, atol=2.0 ** -64)
        assert all(plan.step[i] == 0 for i in range(rot // 2, 128))
        assert plan.rot_dim == rot and plan.interleaved == 0 and plan.mscale == 1.25
    assert qg.qrope_plan(64, interleaved=True).interleaved == 1


def test_plan_takes_whole_turns_off(lib):
    """base < 1: frequencies above a turn a position keep their fraction."""
    plan = qg.qrope_plan(8, base=1e-4)
    for i in range(4):
        turns = 1e-4 ** (-2 * i / 8) / (2 * math.pi)
        assert plan.step[i] / 2.0 ** 64 == pytest.approx(turns - math.floor(turns), abs=1e-12)


def test_plan_refusals(lib):
    bad = [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=258), dict(base=0.0), dict(base=-1.0), dict(base=math.inf),
           dict(base=math.nan), dict(factor=0.0), dict(factor=math.nan), dict(orig_ctx=-1), dict(mscale=math.inf),
           dict(mscale=1e300), dict(orig_ctx=10, low_turns=3.0, high_turns=3.0), dict(orig_ctx=10, high_turns=math.nan)]
    for kw in bad:
        with pytest.raises(qg.QGError) as e:
            qg.qrope_plan(kw.pop("rot_dim", 64), **kw)
        assert e.value.status == SHAPE
    assert lib.qrope_plan(None, 64, 0, 1e4, 1.0, 0, 1.0, 32.0, 1.0) == NULL


def rope(lib, **kw):
    a = dict(plan=qg.qrope_plan(64), xt=0, x=at(1), xs=1024, pos=at(2), ntok=3, heads=8, d=128, yt=1, y=at(3), ys=1024)
    a.update(kw)
    return lib.qrope(a["plan"], a["xt"], a["x"], a["xs"], a["pos"], a["ntok"], a["heads"], a["d"], a["yt"], a["y"],
                     a["ys"], None)


def test_rope_refusals(lib):
    assert rope(lib, xt=8) == TYPE and rope(lib, yt=2) == TYPE
    assert rope(lib, plan=None) == NULL and rope(lib, x=None) == NULL and rope(lib, y=None) == NULL
    assert rope(lib, pos=None) == NULL
    assert rope(lib, d=60) == SHAPE and rope(lib, d=264) == SHAPE and rope(lib, d=32) == SHAPE  # rot_dim 64 > 32
    assert rope(lib, heads=0) == SHAPE and rope(lib, ntok=-1) == SHAPE
    assert rope(lib, xs=1016) == SHAPE and rope(lib, ys=8) == SHAPE
    assert rope(lib, xs=1028) == ALIGN and rope(lib, x=at(1) + 8) == ALIGN and rope(lib, y=at(3) + 4) == ALIGN
    assert rope(lib, pos=at(2) + 2) == ALIGN
    assert rope(lib, y=at(1), yt=0, ys=1032) == ALIAS  # same start, other stride
    assert rope(lib, y=at(1)) == ALIAS                 # same start, other type
    assert rope(lib, y=at(1) + 1024, yt=0) == ALIAS
    assert rope(lib, y=at(2)) == ALIAS                 # over the positions
    empty = qg.QGRope()
    assert rope(lib, plan=empty) == SHAPE
    assert rope(lib, ntok=0, x=None, y=None, pos=None) == 0
    assert done(rope(lib)) and done(rope(lib, ntok=1, xs=0, ys=3)) and done(rope(lib, y=at(1), yt=0))


def test_page_bytes(lib):
    for t in (1, 8):
        for d in (64, 128, 256):
            for ps in (16, 32, 64, 128, 256):
                for kv in (1, 3, 8):
                    assert qg.qkv_page_bytes(t, kv, d, ps) == kv * (ps // 16) * ref.record_sizes(t, d)[1]
    for t, kv, d, ps in ((2, 1, 64, 16), (0, 1, 64, 16), (8, 0, 64, 16), (8, 257, 64, 16), (8, 1, 96, 16),
                         (8, 1, 64, 8), (8, 1, 64, 48), (8, 1, 64, 512)):
        assert qg.qkv_page_bytes(t, kv, d, ps) == 0


def append(lib, c=None, **kw):
    a = dict(rope=None, xt=0, k=at(3), ks=1024, v=at(4), vs=1024, q=None, qs=0, nq=0, qo=None, seq=at(5), pos=at(6),
             ntok=4, err=None)
    a.update(kw)
    return lib.qkv_append(c or cache(), a["rope"], a["xt"], a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"],
                          a["nq"], a["qo"], a["seq"], a["pos"], a["ntok"], a["err"], None)


def read(lib, c=None, **kw):
    a = dict(seq=at(5), pos=at(6), ntok=4, yt=1, k=at(3), v=at(4), err=None)
    a.update(kw)
    return lib.qkv_read(c or cache(), a["seq"], a["pos"], a["ntok"], a["yt"], a["k"], a["v"], a["err"], None)


def attn(lib, c=None, **kw):
    a = dict(q=at(3), heads=40, ncols=2, lens=at(5), window=0, scale=0.1, y=at(4), ws=at(6), wsb=1 << 32, err=None)
    a.update(kw)
    return lib.qattn_paged(c or cache(), a["q"], a["heads"], a["ncols"], a["lens"], a["window"], a["scale"], a["y"],
                           a["ws"], a["wsb"], a["err"], None)


CACHES = [(dict(type=2), TYPE), (dict(type=0), TYPE), (dict(n_kv_heads=0), SHAPE), (dict(head_dim=80), SHAPE),
          (dict(page_size=24), SHAPE), (dict(n_pages=0), SHAPE), (dict(n_seq=0), SHAPE), (dict(n_seq=1025), SHAPE),
          (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 25, page_size=64), SHAPE), (dict(pool=None), NULL),
          (dict(page_table=None), NULL), (dict(pool=at(1) + 8), ALIGN), (dict(page_table=at(2) + 2), ALIGN)]


@pytest.mark.parametrize("kw,status", CACHES)
def test_cache_refusals(lib, kw, status):
    c = cache(**kw)
    assert append(lib, c) == status and read(lib, c) == status and attn(lib, c) == status


def test_null_cache(lib):
    assert lib.qkv_append(None, None, 0, at(3), 1024, at(4), 1024, None, 0, 0, None, at(5), at(6), 4, None, None) == NULL
    assert lib.qkv_read(None, at(5), at(6), 4, 1, at(3), at(4), None, None) == NULL
    assert lib.qattn_paged(None, at(3), 40, 2, at(5), 0, 0.1, at(4), at(6), 1 << 32, None, None) == NULL


def test_append_refusals(lib):
    assert append(lib, xt=8) == TYPE
    assert append(lib, ntok=-1) == SHAPE and append(lib, seq=None, ntok=3) == SHAPE
    assert append(lib, ks=1016) == SHAPE and append(lib, vs=512) == SHAPE
    assert append(lib, rope=qg.qrope_plan(256)) == SHAPE
    q = dict(q=at(7), qs=5120, nq=40, qo=at(8))
    assert append(lib, **dict(q, nq=0)) == SHAPE and append(lib, **dict(q, qs=5112)) == SHAPE
    assert append(lib, **dict(q, qo=None)) == NULL
    assert append(lib, k=None) == NULL and append(lib, v=None) == NULL and append(lib, pos=None) == NULL
    assert append(lib, k=at(3) + 8) == ALIGN and append(lib, vs=1028) == ALIGN and append(lib, pos=at(6) + 1) == ALIGN
    assert append(lib, seq=at(5) + 2) == ALIGN and append(lib, err=at(9) + 2) == ALIGN
    assert append(lib, **dict(q, qo=at(8) + 8)) == ALIGN and append(lib, **dict(q, qs=5124)) == ALIGN
    assert append(lib, **dict(q, qo=at(7))) == ALIAS and append(lib, **dict(q, qo=at(1))) == ALIAS
    assert append(lib, k=at(1) + 1024) == ALIAS and append(lib, pos=at(1)) == ALIAS
    assert append(lib, ntok=0, k=None, v=None, pos=None) == 0
    assert done(append(lib)) and done(append(lib, rope=qg.qrope_plan(128), **q)) and done(append(lib, seq=None))


def test_read_refusals(lib):
    assert read(lib, yt=8) == TYPE
    assert read(lib, ntok=-2) == SHAPE and read(lib, seq=None, ntok=5) == SHAPE
    assert read(lib, pos=None) == NULL
    assert read(lib, k=at(3) + 8) == ALIGN and read(lib, v=at(4) + 2) == ALIGN and read(lib, pos=at(6) + 2) == ALIGN
    assert read(lib, v=at(3)) == ALIAS and read(lib, k=at(1)) == ALIAS and read(lib, k=at(6)) == ALIAS
    assert read(lib, v=at(2)) == ALIAS
    assert read(lib, ntok=0, pos=None) == 0 and read(lib, k=None, v=None) == 0
    assert done(read(lib)) and done(read(lib, k=None)) and done(read(lib, v=None))


def test_attention_refusals(lib):
    need = lib.qattn_workspace_bytes(2, 40, 8, 128, 2)
    assert need > 0
    for bad in ((0, 40, 8, 128, 2), (1025, 40, 8, 128, 2), (2, 41, 8, 128, 2), (2, 4, 8, 128, 2), (2, 8 * 65, 8, 128, 2),
                (2, 40, 8, 96, 2), (2, 40, 8, 128, 0), (2, 40, 8, 128, 17), (2, 40, 0, 128, 1)):
        assert lib.qattn_workspace_bytes(*bad) == 0
    assert attn(lib, heads=41) == SHAPE and attn(lib, heads=0) == SHAPE and attn(lib, heads=8 * 65) == SHAPE
    assert attn(lib, ncols=0) == SHAPE and attn(lib, ncols=17) == SHAPE and attn(lib, window=-1) == SHAPE
    assert attn(lib, scale=math.nan) == SHAPE and attn(lib, scale=math.inf) == SHAPE
    assert attn(lib, cache(max_pages=1 << 24, n_kv_heads=256, n_seq=1024), heads=256, wsb=1 << 35) == SHAPE
    assert attn(lib, q=None) == NULL and attn(lib, lens=None) == NULL and attn(lib, y=None) == NULL
    assert attn(lib, q=at(3) + 2) == ALIGN and attn(lib, y=at(4) + 8) == ALIGN and attn(lib, lens=at(5) + 2) == ALIGN
    assert attn(lib, ws=None) == WORKSPACE and attn(lib, wsb=need - 1) == WORKSPACE
    assert attn(lib, ws=at(6) + 8) == ALIGN
    assert attn(lib, y=at(3)) == ALIAS and attn(lib, ws=at(4)) == ALIAS and attn(lib, y=at(1)) == ALIAS
    assert attn(lib, ws=at(2)) == ALIAS
    assert done(attn(lib)) and done(attn(lib, wsb=need))


def test_binding_refusals():
    """The binding's own checks: types, shapes and strides that the C side cannot see."""
    torch = pytest.importorskip("torch")
    table = torch.zeros((2, 5), dtype=torch.int32)
    pool = torch.zeros(10 * qg.qkv_page_bytes(8, 2, 64, 16), dtype=torch.uint8)
    c = qg.qkv_cache(qg.Q8_0, pool, table, 2, 64, 16)
    assert (c.n_pages, c.max_pages, c.n_seq) == (10, 5, 2)
    with pytest.raises(ValueError):
        qg.qkv_cache(qg.Q8_0, pool[:-1], table, 2, 64, 16)
    with pytest.raises(ValueError):
        qg.qkv_cache(qg.Q8_0, pool, table.long(), 2, 64, 16)
    with pytest.raises(ValueError):
        qg.qkv_cache(qg.Q4_0, pool, table, 2, 64, 16)
    k = torch.zeros(4, 2, 64)
    pos, seq = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    calls = [lambda: qg.qkv_append(c, k.double(), k.double(), pos, seq, stream=0),
             lambda: qg.qkv_append(c, k, k.half(), pos, seq, stream=0),
             lambda: qg.qkv_append(c, k, k[:, :1], pos, seq, stream=0),
             lambda: qg.qkv_append(c, k.transpose(0, 1).contiguous().transpose(0, 1), k, pos, seq, stream=0),
             lambda: qg.qkv_append(c, k, k, pos.long(), seq, stream=0),
             lambda: qg.qkv_append(c, k, k, pos[:3], seq, stream=0),
             lambda: qg.qkv_append(c, k, k, pos, seq, q=k, stream=0),
             lambda: qg.qkv_read(c, pos, k[:3], k, seq, stream=0),
             lambda: qg.qkv_read(c, pos, k, k.half(), seq, stream=0),
             lambda: qg.qrope(qg.qrope_plan(64), k, pos, k[:3], stream=0),
             lambda: qg.qrope(qg.qrope_plan(64), k, pos.float(), k, stream=0),
             lambda: qg.qattn_paged(c, torch.zeros(2, 1, 4, 64), pos[:2], torch.zeros(2, 1, 4, 64), pool, stream=0),
             lambda: qg.qattn_paged(c, torch.zeros(3, 1, 4, 64).half(), pos[:3], torch.zeros(3, 1, 4, 64).half(), pool,
                                    stream=0)]
    for f in calls:
        with pytest.raises(ValueError):
            f()
