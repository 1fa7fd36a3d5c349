"""Host-side checks of the norm, the lookup and the routing (no GPU needed): refusals before any launch, plans, the binding's own
checks, and the plain forms on worked values."""
import math

import numpy as np
import pytest

import gemm_q4_q8_gb300 as qg
import layer_ref as ref
from gemm_q4_q8_gb300 import build as qbuild

NULL, SHAPE, ALIGN, TYPE, CUDA, ALIAS = 1, 2, 3, 4, 6, 7


def at(i):
    return 0x100000 + i * (1 << 36)


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qg.load()


def done(f):
    """A call whose arguments are all right fails for want of a GPU; with one it is not made."""
    from conftest import gpu_available
    return gpu_available() or f() == CUDA


# ----------------------------------------------------------------------- norm
def norm(lib, **kw):
    a = dict(xt=0, x=at(1), xs=512, add=at(2), adds=520, sum=at(3), sums=528, w=at(4), w_add=0.0, eps=1e-6, ntok=4, heads=2, n=256,
             yt=1, y=at(5), ys=536, scl=None)
    a.update(kw)
    return lib.qrms_norm(*[a[k] for k in ("xt", "x", "xs", "add", "adds", "sum", "sums", "w", "w_add", "eps", "ntok", "heads", "n",
                                          "yt", "y", "ys", "scl")], None)


def test_norm_refusals(lib):
    assert norm(lib, xt=8) == TYPE and norm(lib, yt=2) == TYPE and norm(lib, yt=3) == TYPE and norm(lib, xt=5) == TYPE
    for kw in (dict(ntok=-1), dict(heads=0), dict(n=0), dict(n=32769, heads=1), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf),
               dict(w_add=math.inf), dict(xs=511), dict(adds=511), dict(sums=504), dict(ys=0), dict(ntok=1 << 30, heads=2),
               dict(yt=8, n=248, scl=at(6)), dict(xs=-512)):
        assert norm(lib, **kw) == SHAPE, kw
    assert norm(lib, x=None) == NULL and norm(lib, y=None) == NULL and norm(lib, yt=8) == NULL
    for kw in (dict(x=at(1) + 2), dict(add=at(2) + 1), dict(sum=at(3) + 2), dict(w=at(4) + 2), dict(y=at(5) + 1), dict(xt=1, x=at(1) + 1),
               dict(yt=8, scl=at(6) + 8), dict(yt=8, scl=at(6), y=at(5) + 8), dict(yt=8, scl=at(6), x=at(1) + 4),
               dict(yt=8, scl=at(6), xs=513), dict(yt=8, scl=at(6), w=at(4) + 4)):
        assert norm(lib, **kw) == ALIGN, kw
    for kw in (dict(y=at(1)), dict(y=at(3)), dict(y=at(2) + 64), dict(sum=at(1)), dict(sum=at(4)), dict(y=at(4)),
               dict(sum=at(1) + 4, sums=512), dict(yt=0, y=at(1), ys=528), dict(yt=0, y=at(3), ys=528), dict(yt=8, y=at(1), scl=at(6)),
               dict(yt=8, scl=at(1)), dict(yt=8, scl=at(5)), dict(yt=8, scl=at(3)), dict(yt=8, scl=at(4))):
        assert norm(lib, **kw) == ALIAS, kw
    assert norm(lib, ntok=0, x=None, y=None) == 0


def test_norm_accepted(lib):
    for kw in (dict(), dict(add=None, sum=None, w=None), dict(sum=at(1), sums=512), dict(sum=at(2), sums=520),
               dict(yt=0, y=at(1), ys=512), dict(yt=0, y=at(2), ys=520, sum=None), dict(ntok=1, xs=0, ys=3, adds=-1, sums=5),
               dict(n=1, heads=1), dict(n=32768, heads=1, xs=32768, adds=32768, sums=32768, ys=32768), dict(yt=8, scl=at(6)),
               dict(n=77, x=at(1) + 4, w=at(4) + 4, y=at(5) + 2), dict(ntok=1, yt=0, y=at(1), ys=7, xs=9, sum=None)):
        assert done(lambda: norm(lib, **kw)), kw


def test_norm_plain_form():
    y, _ = ref.norm(np.array([3.0, 4.0]), np.array([1.0, 2.0]), 0.0, 0.0)
    np.testing.assert_allclose(y, [3 / math.sqrt(12.5), 8 / math.sqrt(12.5)], rtol=1e-15)
    y, _ = ref.norm(np.array([[1.0, -1.0]] * 2), None, 1.0, 3.0)
    np.testing.assert_allclose(y, [[1.0, -1.0]] * 2, rtol=1e-15)


# --------------------------------------------------------------------- lookup
def embed(lib, **kw):
    a = dict(t=8, q=at(1), scl=at(2), rows=100, k=64, ids=at(3), ntok=5, scale=1.0, yt=0, y=at(4), ys=72, err=None)
    a.update(kw)
    return lib.qembed(*[a[k] for k in ("t", "q", "scl", "rows", "k", "ids", "ntok", "scale", "yt", "y", "ys", "err")], None)


def test_embed_refusals(lib):
    assert embed(lib, t=0) == TYPE and embed(lib, t=3) == TYPE and embed(lib, yt=8) == TYPE
    for kw in (dict(rows=0), dict(k=0), dict(k=48), dict(ntok=-1), dict(scale=math.nan), dict(scale=math.inf), dict(ys=63)):
        assert embed(lib, **kw) == SHAPE, kw
    assert embed(lib, q=None) == NULL and embed(lib, scl=None) == NULL and embed(lib, ids=None) == NULL and embed(lib, y=None) == NULL
    for kw in (dict(q=at(1) + 8), dict(scl=at(2) + 8), dict(ids=at(3) + 2), dict(y=at(4) + 8), dict(ys=68), dict(err=at(5) + 2)):
        assert embed(lib, **kw) == ALIGN, kw
    for kw in (dict(y=at(1)), dict(y=at(1) + 6384), dict(y=at(2)), dict(y=at(3) + 16)):
        assert embed(lib, **kw) == ALIAS, kw
    assert embed(lib, ntok=0, q=None, y=None) == 0
    assert done(lambda: embed(lib)) and done(lambda: embed(lib, t=1, scl=None, yt=1)) and done(lambda: embed(lib, t=2, ntok=1, ys=0))


# -------------------------------------------------------------------- routing
def test_plan(lib):
    p = qg.qroute_plan("sigmoid", n_group=8, top_group=4, group_top=2, renorm=True, scale=2.5)
    assert [getattr(p, f[0]) for f in qg.QGRoute._fields_] == [1, 8, 4, 2, 1, 2.5]
    p = qg.qroute_plan()
    assert [getattr(p, f[0]) for f in qg.QGRoute._fields_] == [0, 1, 1, 1, 1, 1.0]
    for kw in (dict(n_group=0), dict(n_group=33), dict(n_group=4, top_group=5), dict(top_group=0), dict(group_top=0),
               dict(group_top=3), dict(scale=math.nan), dict(scale=1e300)):
        with pytest.raises(qg.QGError) as e:
            qg.qroute_plan(**kw)
        assert e.value.status == SHAPE
    with pytest.raises(ValueError):
        qg.qroute_plan("tanh")
    assert lib.qroute_plan(None, 0, 1, 1, 1, 1, 1.0) == NULL and lib.qroute_plan(qg.QGRoute(), 2, 1, 1, 1, 1, 1.0) == SHAPE


def route(lib, plan=None, **kw):
    a = dict(logits=at(1), stride=64, bias=at(2), ntok=3, e=64, k=8, ids=at(3), rw=at(4))
    a.update(kw)
    return lib.qmoe_route(plan or qg.qroute_plan(), *[a[k] for k in ("logits", "stride", "bias", "ntok", "e", "k", "ids", "rw")], None)


def planned(lib, plan=None, **kw):
    a = dict(w=at(1), x=at(2), bias=at(3), e=64, hidden=128, ncols=4, k=8, logits=at(4), ids=at(5), rw=at(6))
    a.update(kw)
    return lib.qmoe_router_planned(plan or qg.qroute_plan(),
                                   *[a[k] for k in ("w", "x", "bias", "e", "hidden", "ncols", "k", "logits", "ids", "rw")], None)


def test_route_refusals(lib):
    grouped = qg.qroute_plan("sigmoid", n_group=8, top_group=2, group_top=2)
    assert lib.qmoe_route(None, at(1), 64, None, 3, 64, 8, at(3), at(4), None) == NULL
    for kw in (dict(e=0), dict(e=1025, stride=2000), dict(k=0), dict(k=33), dict(e=7, k=8), dict(ntok=-1), dict(stride=63)):
        assert route(lib, **kw) == SHAPE, kw
    for kw in (dict(e=63), dict(k=17), dict(e=8, k=2)):  # not a multiple; more than the open groups hold; one expert a group
        assert route(lib, grouped, **kw) == SHAPE, kw
    assert route(lib, qg.QGRoute()) == SHAPE
    assert route(lib, logits=None) == NULL and route(lib, ids=None) == NULL and route(lib, rw=None) == NULL
    for kw in (dict(logits=at(1) + 2), dict(bias=at(2) + 1), dict(ids=at(3) + 2), dict(rw=at(4) + 2)):
        assert route(lib, **kw) == ALIGN, kw
    for kw in (dict(ids=at(4)), dict(ids=at(1)), dict(rw=at(2)), dict(rw=at(1) + 64), dict(ids=at(4) + 92)):
        assert route(lib, **kw) == ALIAS, kw
    assert route(lib, ntok=0, logits=None) == 0
    assert done(lambda: route(lib)) and done(lambda: route(lib, grouped, bias=None, ntok=1, stride=0, k=16))


def test_router_planned_refusals(lib):
    assert lib.qmoe_router_planned(None, at(1), at(2), None, 64, 128, 1, 8, None, at(5), at(6), None) == NULL
    for kw in (dict(e=0), dict(e=1025), dict(hidden=0), dict(ncols=0), dict(ncols=17), dict(k=0), dict(k=33), dict(e=4)):
        assert planned(lib, **kw) == SHAPE, kw
    assert planned(lib, qg.qroute_plan(n_group=7)) == SHAPE and planned(lib, qg.QGRoute()) == SHAPE
    assert planned(lib, w=None) == NULL and planned(lib, x=None) == NULL and planned(lib, ids=None) == NULL and planned(lib, rw=None) == NULL
    for kw in (dict(w=at(1) + 8), dict(x=at(2) + 1), dict(bias=at(3) + 2), dict(logits=at(4) + 2), dict(ids=at(5) + 1), dict(rw=at(6) + 2)):
        assert planned(lib, **kw) == ALIGN, kw
    for kw in (dict(ids=at(6)), dict(ids=at(4)), dict(rw=at(1)), dict(rw=at(2)), dict(ids=at(3)), dict(logits=at(1)), dict(logits=at(2)),
               dict(logits=at(3)), dict(logits=at(5))):
        assert planned(lib, **kw) == ALIAS, kw
    assert done(lambda: planned(lib)) and done(lambda: planned(lib, logits=None, bias=None))


def test_route_plain_form():
    """Worked by hand: sigmoid of 0 is 1/2, of log 3 it is 3/4."""
    l3 = np.float32(math.log(3))
    ids, w, _ = ref.route(np.array([0, l3, 0, -100], np.float32), None, 3, "sigmoid", renorm=False)
    assert ids.tolist() == [1, 0, 2]
    np.testing.assert_allclose(w, [0.75, 0.5, 0.5], rtol=1e-7)
    ids, w, _ = ref.route(np.array([0, l3, 0, -100], np.float32), np.array([0, -0.5, 0.1, 0.7], np.float32), 2, "sigmoid", scale=2.0)
    assert ids.tolist() == [3, 2]  # 0.7, 0.6, 0.5, 0.25
    np.testing.assert_allclose(w, [0, 2], atol=1e-30)
    # groups (0, 1), (2, 3): sums of two 1.25 and 1.2, best one 0.75 and 0.9
    x = np.array([0, l3, math.log(9), math.log(3 / 7)], np.float32)
    assert ref.route(x, None, 1, "sigmoid", 2, 1, 2)[0].tolist() == [1]
    assert ref.route(x, None, 1, "sigmoid", 2, 1, 1)[0].tolist() == [2]
    p = ref.scores(np.array([0, 0, np.nan, -np.inf], np.float32), "softmax")
    assert p[:2].tolist() == [0.5, 0.5] and np.isnan(p[2]) and p[3] == 0
    assert ref.route(np.array([np.nan, 1, np.inf, 2], np.float32), None, 4)[0].tolist() == [2, 3, 1, 0]


# -------------------------------------------------------------------- binding
def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 64), torch.zeros(64)
    ids, rw = torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8)
    plan = qg.qroute_plan()
    q8, s8 = torch.zeros(10, 64, dtype=torch.int8), torch.zeros(10, 2, dtype=torch.float16)
    y8, ys = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.float16)
    calls = [lambda: qg.qrms_norm(x.double(), w, x, stream=0),
             lambda: qg.qrms_norm(x[0], w, x, stream=0),
             lambda: qg.qrms_norm(x, w[:32], x, stream=0),
             lambda: qg.qrms_norm(x, w.half(), x, stream=0),
             lambda: qg.qrms_norm(x, w, x[:3], stream=0),
             lambda: qg.qrms_norm(x, w, x, add=x.half(), stream=0),
             lambda: qg.qrms_norm(x, w, x, add=x[:2], stream=0),
             lambda: qg.qrms_norm(x, w, x, sum_out=x.half(), stream=0),
             lambda: qg.qrms_norm(x.t(), torch.zeros(4), x.t(), stream=0),
             lambda: qg.qrms_norm(x, w, y8, stream=0),
             lambda: qg.qrms_norm(x, w, y8, y_scl=ys[:3], stream=0),
             lambda: qg.qrms_norm(x, w, x, y_scl=ys, stream=0),
             lambda: qg.qrms_norm(x.view(4, 2, 32), w[:32], x, stream=0),
             lambda: qg.qembed(qg.Q8_0, q8, s8, ids[0].long(), x[:8], stream=0),
             lambda: qg.qembed(qg.Q8_0, q8, s8, ids[0], x, stream=0),
             lambda: qg.qembed(qg.Q8_0, q8, s8[:9], ids[0, :4], x, stream=0),
             lambda: qg.qembed(qg.QG_F16, q8, None, ids[0, :4], x, stream=0),
             lambda: qg.qembed(qg.Q8_0, q8.t(), s8, ids[0, :4], x, stream=0),
             lambda: qg.qmoe_route(plan, x.half(), 8, ids, rw, stream=0),
             lambda: qg.qmoe_route(plan, x.t(), 8, ids, rw, stream=0),
             lambda: qg.qmoe_route(plan, x, 8, ids.long(), rw, stream=0),
             lambda: qg.qmoe_route(plan, x, 4, ids, rw, stream=0),
             lambda: qg.qmoe_route(plan, x, 8, ids, rw, bias=w[:8], stream=0),
             lambda: qg.qmoe_router_planned(plan, x, x, 4, ids, rw, stream=0),
             lambda: qg.qmoe_router_planned(plan, x, x.half(), 4, ids, rw, stream=0),
             lambda: qg.qmoe_router_planned(plan, x.half(), x.half(), 8, ids, rw, stream=0)]
    for i, f in enumerate(calls):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i}")


def test_binding_refuses_rows_with_gaps():
    """Rows whose elements are not neighbours, though their stride is that of contiguous ones."""
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 64), torch.zeros(64)
    gap = torch.zeros(400).as_strided((4, 64), (64, 2))
    heads = torch.zeros(600).as_strided((4, 2, 32), (64, 40, 1))
    ids, rw = torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8)
    plan = qg.qroute_plan()
    q8, s8 = torch.zeros(10, 64, dtype=torch.int8), torch.zeros(10, 2, dtype=torch.float16)
    calls = [lambda: qg.qrms_norm(gap, w, x, stream=0), lambda: qg.qrms_norm(x, w, gap, stream=0),
             lambda: qg.qrms_norm(x, w, x, add=gap, stream=0), lambda: qg.qrms_norm(x, w, x, add=x, sum_out=gap, stream=0),
             lambda: qg.qrms_norm(heads, w[:32], x.view(4, 2, 32), stream=0),
             lambda: qg.qrms_norm(x.view(4, 2, 32), w[:32], heads, stream=0),
             lambda: qg.qembed(qg.Q8_0, q8, s8, ids[0, :4], gap, stream=0),
             lambda: qg.qmoe_route(plan, gap, 8, ids, rw, stream=0)]
    for i, f in enumerate(calls):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i}")
