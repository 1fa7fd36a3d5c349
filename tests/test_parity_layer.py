"""GPU parity of the norm, the embedding lookup and the routing by a plan against plain 64-bit forms (layer_ref.py)."""
import math

import numpy as np
import pytest

import attn_ref
import layer_ref as ref
from helpers import assert_within, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gemm_q4_q8_gb300 as qg  # noqa: E402

NP = {torch.float32: np.float32, torch.float16: np.float16}
BAND = 1 << 14


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_q4_q8_gb300 import build
    build.build()


def rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def banded(shape, dtype):
    """(a tensor of this shape between two guard bands, whether the bands still are as they were); bytes all ones."""
    n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((BAND + n + BAND,), 0xFF, dtype=torch.uint8, device="cuda")
    return buf[BAND:BAND + n].view(dtype).view(shape), lambda: bool((buf[:BAND] == 0xFF).all() and (buf[BAND + n:] == 0xFF).all())


# ----------------------------------------------------------------------- norm
def check_norm(x, add, w, w_add, eps, out, in_place=None, heads=None):
    dx, da = cuda(x), None if add is None else cuda(add)
    kept = dx.clone(), None if da is None else da.clone()
    s_out, s_ok = (None, lambda: True) if add is None else banded(x.shape, dx.dtype)
    y, y_ok = banded(x.shape, out)
    qg.qrms_norm(dx, None if w is None else cuda(w), y, eps=eps, add=da, sum_out=s_out, w_add=w_add)
    s = ref.add_up(x, add)
    if add is not None:
        np.testing.assert_array_equal(host(s_out), s)
        assert torch.equal(da, kept[1])
    want, bound = ref.norm(s, w, w_add, eps)
    if out == torch.float16:
        bound = bound * (1 + ref.HALF) + ref.HALF * np.abs(want) + ref.SUB
    assert_within(host(y), want, bound, f"{x.shape} {x.dtype} to {out}")
    assert y_ok() and s_ok() and torch.equal(dx, kept[0])
    return y


@pytest.mark.parametrize("out", [torch.float32, torch.float16])
@pytest.mark.parametrize("src", [torch.float32, torch.float16])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 31, 33, 64, 100, 128, 255, 256, 257, 264, 1000, 1024, 1032, 2048, 2049, 5120, 8192, 8200,
                               16385, 32760, 32768])
def test_norm(n, src, out):
    """One row, a few, and more than take the other form; with and without the residual."""
    for rows in (1, 5, 160) if n <= 8200 else (1, 3):
        g = rng(1, n, rows)
        x = (g.standard_normal((rows, n)) * np.exp(g.standard_normal((rows, 1)))).astype(NP[src])
        add = g.standard_normal((rows, n)).astype(NP[src])
        w = (1 + 0.2 * g.standard_normal(n)).astype(np.float32)
        check_norm(x, None, w, 0.0, 1e-6, out)
        check_norm(x, add, w - 1, 1.0, 1e-5, out)
    check_norm(x, add, None, 0.0, 0.25, out)


@pytest.mark.parametrize("src", [torch.float32, torch.float16])
@pytest.mark.parametrize("heads,n", [(1, 128), (3, 64), (40, 128), (5, 80), (2, 256), (7, 33), (2, 5120)])
def test_norm_heads_in_wider_rows(heads, n, src):
    """The queries' heads inside the rows of a fused projection, in place and out of place; the rest of the rows keeps its bytes."""
    g = rng(2, heads, n)
    tok = 37
    rows = cuda(g.standard_normal((tok, (heads + 4) * n)).astype(NP[src]))
    keep = rows.clone()
    w = cuda((1 + 0.1 * g.standard_normal(n)).astype(np.float32))
    x = rows[:, 2 * n:(2 + heads) * n].view(tok, heads, n)
    y = torch.empty((tok, heads, n), dtype=src, device="cuda")
    qg.qrms_norm(x, w, y)
    qg.qrms_norm(x, w, x)
    assert torch.equal(x, y)
    assert torch.equal(rows[:, :2 * n], keep[:, :2 * n]) and torch.equal(rows[:, (2 + heads) * n:], keep[:, (2 + heads) * n:])
    s = host(keep)[:, 2 * n:(2 + heads) * n].reshape(tok, heads, n)
    want, bound = ref.norm(s, host(w), 0.0, 1e-6)
    if src == torch.float16:
        bound = bound * (1 + ref.HALF) + ref.HALF * np.abs(want) + ref.SUB
    assert_within(host(y), want, bound, "heads")


@pytest.mark.parametrize("src", [torch.float32, torch.float16])
@pytest.mark.parametrize("n", [256, 5120, 333])
def test_norm_sum_in_place(n, src):
    """The sum over x or over add, and y over add or x: the same bits as with outputs of their own."""
    g = rng(3, n)
    x, add = (cuda(g.standard_normal((9, n)).astype(NP[src])) for _ in range(2))
    w = cuda((1 + 0.1 * g.standard_normal(n)).astype(np.float32))
    s, y = torch.empty_like(x), torch.empty_like(x)
    qg.qrms_norm(x, w, y, add=add, sum_out=s)
    for sum_at, y_at in ((0, None), (1, None), (None, 0), (None, 1), (0, 1), (1, 0)):
        a, b = x.clone(), add.clone()
        own = torch.empty_like(x)
        both = [a, b]
        qg.qrms_norm(a, w, own if y_at is None else both[y_at], add=b, sum_out=None if sum_at is None else both[sum_at])
        assert torch.equal(own if y_at is None else both[y_at], y)
        if sum_at is not None:
            assert torch.equal(both[sum_at], s)


@pytest.mark.parametrize("n", [128, 512, 5120])
def test_norm_wide_and_narrow_rows_agree(n):
    """Rows that begin at odd places are read element by element: the same within the bound, and strides of their own for each."""
    g = rng(4, n)
    big = cuda(g.standard_normal((6, n + 5)).astype(np.float32))
    w = cuda((1 + 0.1 * g.standard_normal(n + 1)).astype(np.float32))
    x = big[:, 3:3 + n]
    add, s = torch.randn(6, 2 * n, device="cuda")[:, 1:1 + n], torch.zeros(6, n + 8, device="cuda")
    y = torch.full((6, n + 3), 7.0, dtype=torch.float16, device="cuda")
    qg.qrms_norm(x, w[1:], y[:, 1:1 + n], add=add, sum_out=s[:, :n])
    want, bound = ref.norm(ref.add_up(host(x), host(add)), host(w)[1:], 0.0, 1e-6)
    assert_within(host(y)[:, 1:1 + n], want, bound * (1 + ref.HALF) + ref.HALF * np.abs(want) + ref.SUB, "narrow")
    assert (y[:, 0] == 7).all() and (y[:, 1 + n:] == 7).all() and (s[:, n:] == 0).all()


@pytest.mark.parametrize("n", [64, 1000, 5120])
@pytest.mark.parametrize("size,eps", [(1e30, 1e-6), (3e38, 0.0), (1e-30, 0.0), (1e-38, 1e-40), (1e-25, 1e-6), (1e18, 1e-6), (1e-44, 0.0)])
def test_norm_out_of_range_squares(n, size, eps):
    """Rows whose squares leave the range of f32, next to ordinary ones, which keep their bits."""
    g = rng(5, n)
    x = g.standard_normal((8, n)).astype(np.float32)
    plain = torch.empty((8, n), device="cuda")
    qg.qrms_norm(cuda(x), None, plain, eps=eps)
    x[3] = np.clip(x[3].astype(np.float64) / 4 * size, -3.4e38, 3.4e38).astype(np.float32)
    y = torch.empty((8, n), device="cuda")
    qg.qrms_norm(cuda(x), None, y, eps=eps)
    want, bound = ref.norm(x, None, 0.0, float(np.float32(eps)))
    assert_within(host(y)[3], want[3], bound[3], f"rows of {size}")
    rest = [i for i in range(8) if i != 3]
    assert torch.equal(y[rest], plain[rest])


def test_norm_not_finite_and_zero_rows():
    """A NaN reaches its own row; an infinite element makes its row NaN there and 0 elsewhere; zeros stay zeros."""
    for n in (100, 640, 5120):
        x = rng(6, n).standard_normal((6, n)).astype(np.float32)
        x[1, n // 2], x[3, 1], x[4] = np.nan, np.inf, 0
        y = torch.empty((6, n), device="cuda")
        qg.qrms_norm(cuda(x), None, y, eps=1e-6)
        y = host(y)
        assert np.isnan(y[1]).all() and np.isnan(y[3, 1]) and (np.delete(y[3], 1) == 0).all() and (y[4] == 0).all()
        assert np.isfinite(y[[0, 2, 5]]).all()


@pytest.mark.parametrize("src", [torch.float32, torch.float16])
@pytest.mark.parametrize("tok,heads,n", [(1, 1, 32), (5, 1, 64), (300, 1, 96), (3, 2, 256), (2, 1, 1056), (9, 1, 2048), (160, 1, 5120),
                                         (1, 1, 8224), (2, 1, 32768), (70, 3, 128)])
def test_norm_to_q8_rows(tok, heads, n, src):
    """Every scale is the smallest that holds its block, every quant the nearest; the rows in the layout of the weights."""
    g = rng(7, n, heads)
    x = (g.standard_normal((tok, heads, n)) * np.exp(g.standard_normal(n))).astype(NP[src])
    add = g.standard_normal(x.shape).astype(NP[src])
    w = (1 + 0.2 * g.standard_normal(n)).astype(np.float32)
    q, q_ok = banded(x.shape, torch.int8)
    scl, s_ok = banded((tok, heads, n // 32), torch.float16)
    qg.qrms_norm(cuda(x), cuda(w), q, add=cuda(add), y_scl=scl, eps=1e-5)
    assert q_ok() and s_ok()
    want, err = ref.norm(ref.add_up(x, add), w, 0.0, 1e-5)
    d = host(scl).astype(np.float64)
    top, off = (a.reshape(tok, heads, -1, 32).max(-1) for a in (np.abs(want), err))
    assert (d >= (top - off) / 127).all() and (np.nextafter(host(scl), np.float16(0)).astype(np.float64) <= (top + off) / 127).all()
    got = ref.weights(8, host(q).view(np.uint8).reshape(-1, n), host(scl).reshape(-1, n // 32).view(np.uint16)).reshape(x.shape)
    # half a step, err, and the division's rounding (2 half steps of f32 of 127)
    assert_within(got, want, err + np.repeat(d, 32, -1) * (0.5 + 127 * 2 * ref.SINGLE), "values")
    back = torch.empty((tok * heads, n), dtype=torch.float32, device="cuda")
    qg.qembed(qg.Q8_0, q.view(-1, n), scl.view(-1, n // 32), torch.arange(tok * heads, dtype=torch.int32, device="cuda"), back)
    np.testing.assert_array_equal(host(back), got.reshape(-1, n).astype(np.float32))


def test_norm_to_q8_blocks_where_the_last_bit_decides():
    """A row of ones is normed to the weights, exactly: blocks with halves, zeros, subnormals, outliers, NaN and infinities, byte for
    byte."""
    g = rng(8)
    n = 32 * 600
    w = g.standard_normal((600, 32)).astype(np.float32)
    for i in range(600):
        d = np.float32(np.float16(2.0 ** g.uniform(-20, 3)))
        if i % 6 == 0:
            w[i] = d * (g.integers(-126, 126, 32) + np.float32(0.5))
            w[i, 0] = 127 * d
        elif i % 6 == 1:
            w[i] = np.nextafter(d * (g.integers(-126, 126, 32) + np.float32(0.5)), np.float32(np.inf if i % 4 else -np.inf))
            w[i, 31] = -127 * d
        elif i % 6 == 2:
            w[i] *= np.float32(10.0 ** g.uniform(-12, 6))
        elif i % 6 == 3:
            w[i] = 0 if i % 4 else 1e-9
    w[7, 3], w[11, 0], w[13, 31] = np.nan, np.inf, -3e38
    q = torch.empty((1, n), dtype=torch.int8, device="cuda")
    scl = torch.empty((1, n // 32), dtype=torch.float16, device="cuda")
    qg.qrms_norm(torch.ones(1, n, device="cuda"), cuda(w.reshape(-1)), q, y_scl=scl, eps=0.0)
    with np.errstate(invalid="ignore", over="ignore"):
        wq, wd = attn_ref.quantise(w)
    np.testing.assert_array_equal(host(scl).reshape(-1), wd)
    np.testing.assert_array_equal(ref.unstored(host(q).view(np.uint8)).view(np.int8).reshape(-1, 32), wq)


@pytest.mark.parametrize("n", [32, 96, 256, 2048, 5120])
@pytest.mark.parametrize("rows", [7, 1600])
def test_norm_to_q8_rows_next_to_odd_ones(n, rows):
    """Rows with a NaN, an infinity, nothing at all or blocks that saturate leave the others' bytes as they are."""
    g = rng(18, n)
    x = g.standard_normal((rows, n)).astype(np.float32)
    w = (1 + 0.2 * g.standard_normal(n)).astype(np.float32)
    w[n - 1] = 1e12  # times 0, but in one row
    x[:, n - 1] = 0

    def run():
        q = torch.empty((rows, n), dtype=torch.int8, device="cuda")
        scl = torch.empty((rows, n // 32), dtype=torch.float16, device="cuda")
        qg.qrms_norm(cuda(x), cuda(w), q, y_scl=scl, eps=0.0)
        return host(q), host(scl)

    q0, s0 = run()
    assert np.isfinite(s0).all()
    x[1, 3], x[2, n // 2], x[4], x[5, n - 1] = np.nan, np.inf, 0, 2.0
    q1, s1 = run()
    rest = [i for i in range(rows) if i not in (1, 2, 4, 5)]
    np.testing.assert_array_equal(q1[rest], q0[rest])
    np.testing.assert_array_equal(s1[rest], s0[rest])
    assert np.isnan(s1[1]).all() and np.isnan(s1[4]).all()
    assert [bool(b) for b in np.isnan(s1[2])] == [i == n // 2 // 32 for i in range(n // 32)]
    assert s1[5, -1] == 65504 and ref.unstored(q1.view(np.uint8)).view(np.int8)[5, n - 1] == 127


def test_norm_rows_score_as_an_index():
    """Normed rows as a Q8_0 matrix: qgemv_q8_0 scores a query against them."""
    import oracle
    oracle.build()
    g = rng(9)
    rows, n = 515, 256
    x, query = g.standard_normal((rows, n)).astype(np.float16), g.standard_normal((1, n)).astype(np.float16)
    q, scl = torch.empty((rows, n), dtype=torch.int8, device="cuda"), torch.empty((rows, n // 32), dtype=torch.float16, device="cuda")
    qg.qrms_norm(cuda(x), None, q, y_scl=scl)
    y = torch.empty((1, rows), device="cuda")
    qg.qgemv_q8_0(q, scl, cuda(query), y)
    w = ref.weights(8, host(q).view(np.uint8), host(scl).view(np.uint16))
    want = query.astype(np.float64) @ w.T
    assert_within(host(y), want, 1e-3 * (np.abs(query.astype(np.float64)) @ np.abs(w).T) + 1e-6, "scores")


# --------------------------------------------------------------------- lookup
def table(qtype, rows, k, seed):
    g = rng(10, rows, k, seed)
    if qtype == qg.QG_F16:
        q = (g.standard_normal((rows, k)) * 0.1).astype(np.float16)
        return q, None, q.astype(np.float64)
    q = g.integers(0, 256, (rows, k if qtype == qg.Q8_0 else k // 2), dtype=np.uint8)
    scl = (np.abs(g.standard_normal((rows, k // 32))) * 0.01).astype(np.float16).view(np.uint16)
    return q, scl, ref.weights(qtype, q, scl)


@pytest.mark.parametrize("out", [torch.float32, torch.float16])
@pytest.mark.parametrize("qtype", [qg.Q4_0, qg.Q8_0, qg.QG_F16])
@pytest.mark.parametrize("rows,k,ntok", [(1, 32, 1), (50, 64, 7), (1000, 2048, 1), (300, 5120, 33), (77, 1056, 500), (20, 32, 3000),
                                         (9, 40960, 3)])
def test_embed(qtype, rows, k, ntok, out):
    q, scl, w = table(qtype, rows, k, ntok)
    ids = rng(11, ntok).integers(0, rows, ntok).astype(np.int32)
    if ntok > 2:
        ids[:3] = 0, rows - 1, rows - 1
    ds = None if scl is None else cuda(scl.view(np.float16))
    dq = cuda(q)
    for scale in (1.0, math.sqrt(k), -0.37):
        y, ok = banded((ntok, k), out)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        qg.qembed(qtype, dq, ds, cuda(ids), y, scale=scale, err_flag=err)
        s32 = np.float32(scale)
        want = (w[ids].astype(np.float32) * s32).astype(NP[out])  # (a weight is exact in f32)
        np.testing.assert_array_equal(host(y), want)
        assert ok() and int(err) == 0


def test_embed_matches_the_product():
    """Row i equals W^T e_i of the products: the layout is the GEMV's, and qrepack's."""
    import synth
    g = synth.rng(5)
    for qtype in (qg.Q4_0, qg.Q8_0):
        rows, k = 40, 512
        q, s = synth.draw_matrix(g, qtype, rows, k)
        blocks = cuda(synth.to_gguf_blocks(qtype, q, s))
        qd, sd = torch.empty(q.shape, dtype=torch.uint8, device="cuda"), torch.empty(s.shape, dtype=torch.int16, device="cuda")
        qg.qrepack(qtype, blocks, rows, k, qd, sd)
        got = torch.empty((rows, k), device="cuda")
        qg.qembed(qtype, qd, sd, torch.arange(rows, dtype=torch.int32, device="cuda"), got)
        for c in (0, 1, 15, 16, 17, 31, 32, 300, 511):
            e = torch.zeros((1, k), dtype=torch.float16, device="cuda")
            e[0, c] = 1
            y = torch.empty((1, rows), device="cuda")
            qg.qgemm_cols(qtype, qd, sd, e, y)
            assert torch.equal(y[0], got[:, c])


def test_embed_bad_ids_and_strides():
    """Ids outside the table: zeros, flagged; rows inside wider rows."""
    q, scl, w = table(qg.Q8_0, 10, 64, 0)
    ids = np.array([3, -1, 10, 2 ** 31 - 1, -2 ** 31, 9], np.int32)
    y = torch.full((6, 96), 5.0, device="cuda")
    for err in (torch.zeros(1, dtype=torch.int32, device="cuda"), None):
        y.fill_(5.0)
        qg.qembed(qg.Q8_0, cuda(q), cuda(scl.view(np.float16)), cuda(ids), y[:, 16:80], err_flag=err)
        if err is not None:
            assert int(err) == qg.QG_EMBED_BAD_ID
        got = host(y)
        assert (got[:, :16] == 5).all() and (got[:, 80:] == 5).all() and (got[1:5, 16:80] == 0).all()
        np.testing.assert_array_equal(got[[0, 5], 16:80], w[[3, 9]].astype(np.float32))


def test_embed_table_beyond_4_gib():
    rows, k = 900_000, 5120
    q = torch.empty((rows, k), dtype=torch.int8, device="cuda")
    scl = torch.empty((rows, k // 32), dtype=torch.float16, device="cuda")
    ids = torch.tensor([0, 419_500, rows - 1], dtype=torch.int32, device="cuda")
    part, ps, w = table(qg.Q8_0, 3, k, 1)
    q[ids.long()] = cuda(part).view(torch.int8)
    scl[ids.long()] = cuda(ps.view(np.float16))
    y = torch.empty((3, k), device="cuda")
    qg.qembed(qg.Q8_0, q, scl, ids, y)
    np.testing.assert_array_equal(host(y), w.astype(np.float32))


# -------------------------------------------------------------------- routing
def weights_within(got, want, what=""):
    """rw is within 2^-19 of itself (and f32's smallest number)."""
    ok = np.isnan(got) == np.isnan(want)
    assert ok.all(), what
    assert_within(np.nan_to_num(got), np.nan_to_num(want), 2.0 ** -19 * np.abs(np.nan_to_num(want)) + 2.0 ** -126, what)


def check_route(logits, bias, k, extra=0, **plan):
    n, e = logits.shape
    wide = np.full((n, e + extra), 99, np.float32)
    wide[:, :e] = logits
    ids, i_ok = banded((n, k), torch.int32)
    rw, r_ok = banded((n, k), torch.float32)
    qg.qmoe_route(qg.qroute_plan(**plan), cuda(wide)[:, :e], k, ids, rw, bias=None if bias is None else cuda(bias))
    ids, rw = host(ids), host(rw)
    assert i_ok() and r_ok()
    for t in range(n):
        want, w, near = ref.route(logits[t], bias, k, **plan)
        if near > 1e-14:  # (two exponentials in 64 bits may differ by less)
            assert np.array_equal(ids[t], want), (t, ids[t], want, near)
            weights_within(rw[t], w, f"token {t}")
    return ids, rw


PLANS = [dict(), dict(score="sigmoid"), dict(score="sigmoid", renorm=False, scale=2.5), dict(renorm=False),
         dict(score="sigmoid", n_group=8, top_group=4, group_top=2, scale=2.5), dict(n_group=4, top_group=1, group_top=1),
         dict(score="sigmoid", n_group=4, top_group=3, group_top=1), dict(n_group=8, top_group=8, group_top=2),
         dict(n_group=2, top_group=1, group_top=2, renorm=False)]


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("e,k", [(256, 8), (64, 6), (128, 1), (512, 10), (1024, 32), (16, 2), (40, 4)])
def test_route(e, k, plan, biased):
    g = rng(12, e, k)
    groups = plan.get("n_group", 1)
    if k > plan.get("top_group", 1) * (e // groups):
        k = plan["top_group"] * (e // groups)
    logits = (g.standard_normal((37, e)) * 1.5).astype(np.float32)
    check_route(logits, (g.standard_normal(e) * 0.1).astype(np.float32) if biased else None, k, extra=e % 3, **plan)


@pytest.mark.parametrize("e,k,groups,keep", [(1, 1, 1, 1), (2, 2, 1, 1), (7, 7, 1, 1), (31, 31, 1, 1), (33, 32, 1, 1), (96, 5, 32, 2),
                                             (1000, 20, 5, 3), (999, 9, 27, 1), (32, 1, 32, 1), (62, 2, 31, 30)])
def test_route_odd_sizes(e, k, groups, keep):
    g = rng(13, e, k)
    logits = g.standard_normal((11, e)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for bias in (None, (g.standard_normal(e) * 0.2).astype(np.float32)):
            check_route(logits, bias, k, score=score, n_group=groups, top_group=keep, group_top=1)
            if e // groups > 1:
                check_route(logits, bias, k, score=score, n_group=groups, top_group=keep, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_choice_is_that_of_64_bits(score):
    """Biases that make experts equal but for f32's rounding: thousands of neighbours at distances far below a step of f32."""
    g = rng(14)
    n, e, k = 60, 64, 8
    logits = (g.standard_normal((n, e)) * 2).astype(np.float32)
    seen = 0
    for t in range(n):
        p = ref.scores(logits[t], score)
        bias = (p.max() + 0.1 - p).astype(np.float32)  # all c within a rounding of each other
        bias[g.permutation(e)[:20]] -= np.float32(0.3)
        _, _, near = ref.route(logits[t], bias, k, score)
        seen += near < 2.0 ** -26
        check_route(logits[t:t + 1], bias, k, score=score)
        check_route(logits[t:t + 1], bias, k, score=score, n_group=8, top_group=2, group_top=2)
    assert seen > n // 2


@pytest.mark.parametrize("renorm", [True, False])
def test_route_weights_far_below_the_largest(renorm):
    """Logits 32 to 64 below the largest: their difference in f32 is off by up to 2^-19, which the weights must not be."""
    g = rng(43)
    logits = g.uniform(-33, 28, (100, 64)).astype(np.float32)
    logits[:, 0] = np.float32(30) + (np.float32(2.0) ** -19) * g.integers(0, 999, 100).astype(np.float32)
    logits[:, 1] = -20  # the difference has a half step left where the largest is an odd number of steps
    check_route(logits, None, 32, renorm=renorm)
    check_route(logits, (0.01 * g.standard_normal(64)).astype(np.float32), 32, renorm=renorm)


def test_route_saturated_sigmoids():
    """Sigmoids that f32 rounds to 1: still in order with a bias; without one in the order of the logits, past 64 bits' end."""
    x = np.linspace(12, 30, 64).astype(np.float32)[None]
    ids, _ = check_route(x, np.zeros(64, np.float32), 8, score="sigmoid")
    assert ids.tolist() == [list(range(63, 55, -1))]
    x = np.linspace(35, 90, 64).astype(np.float32)[None]
    ids, rw = check_route(x, None, 8, score="sigmoid")
    assert ids.tolist() == [list(range(63, 55, -1))] and (rw == 0.125).all()
    x = -np.linspace(80, 200, 64).astype(np.float32)[None]  # far below: weights that f32 does not hold are renormalised all the same
    check_route(x, None, 4, score="sigmoid")
    check_route(x, None, 4, score="softmax")


def test_route_ties_go_to_the_lowest_id():
    for e, k in ((256, 8), (1000, 32), (40, 40 // 2)):
        for bias in (None, np.zeros(e, np.float32)):
            for score in ("softmax", "sigmoid"):
                ids, rw = check_route(np.zeros((3, e), np.float32), bias, k, score=score)
                assert (ids == np.arange(k)).all() and np.allclose(rw, 1 / k, rtol=2e-6)
    x = np.tile(np.array([1, 3, 3, 2], np.float32), 16)[None]
    ids, _ = check_route(x, None, 4)
    assert ids.tolist() == [[1, 2, 5, 6]]
    ids, _ = check_route(np.zeros((2, 64), np.float32), None, 8, n_group=8, top_group=2, group_top=2)  # equal groups
    assert (ids == np.arange(8)).all()
    x = np.array([[0.0, -0.0, 0.0, -0.0, -1, -1, -1, -1]], np.float32)
    assert check_route(x, None, 4)[0].tolist() == [[0, 1, 2, 3]]


def test_route_nan_and_infinities():
    g = rng(15)
    x = g.standard_normal((9, 64)).astype(np.float32)
    x[0, 5], x[1, 7], x[2, 9] = np.nan, np.inf, -np.inf
    x[3] = np.nan
    x[4] = -np.inf
    x[5, ::2] = np.inf
    x[6, 3:] = np.nan
    x[7, :30], x[7, 30:] = -np.inf, np.nan
    bias = (g.standard_normal(64) * 0.1).astype(np.float32)
    odd = bias.copy()
    odd[3], odd[10], odd[20] = np.inf, -np.inf, np.nan
    for score in ("softmax", "sigmoid"):
        for b in (None, bias, odd):
            for more in ({}, dict(n_group=8, top_group=3, group_top=2), dict(renorm=False)):
                with np.errstate(invalid="ignore"):
                    check_route(x, b, 6, score=score, **more)


def test_route_many_tokens():
    """More tokens than warps in flight, against 64-bit torch."""
    n, e, k = 20011, 256, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(n, e, generator=g, device="cuda") * 1.5
    bias = torch.randn(e, generator=g, device="cuda") * 0.1
    ids = torch.empty((n, k), dtype=torch.int32, device="cuda")
    rw = torch.empty((n, k), device="cuda")
    qg.qmoe_route(qg.qroute_plan("sigmoid", n_group=8, top_group=4, group_top=2, scale=2.5), logits, k, ids, rw, bias=bias)
    p = torch.sigmoid(logits.double())
    c = p + bias.double()
    worth = c.view(n, 8, 32).topk(2, -1)[0].sum(-1)
    shut = torch.ones(n, 8, dtype=torch.bool, device="cuda").scatter_(1, worth.topk(4, -1)[1], False)
    want = c.masked_fill(shut.repeat_interleave(32, 1), -math.inf).topk(k, -1)[1]
    assert torch.equal(ids.long(), want)
    w = p.gather(1, want)
    w = w / w.sum(-1, keepdim=True) * 2.5
    assert ((rw.double() - w).abs() <= 2.0 ** -19 * w).all()


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("plan", range(len(PLANS)))
@pytest.mark.parametrize("e,k", [(256, 8), (128, 6), (512, 10), (256, 32), (64, 4), (40, 4), (250, 9), (100, 16), (1024, 8), (8, 2), (504, 3)])
def test_route_many_tokens_as_few(e, k, plan, biased):
    """A call of many tokens decides as calls of few do: ordinary tokens, equal and nearly equal experts, NaN and infinities; and a few
    of them as the plain form."""
    plan = dict(PLANS[plan])
    if e % plan.get("n_group", 1):
        plan["n_group"], plan["top_group"] = 2, 1
    if plan.get("group_top", 1) > e // plan.get("n_group", 1):
        plan["group_top"] = 1
    k = min(k, plan.get("top_group", 1) * (e // plan.get("n_group", 1)))
    n = 2600
    g = rng(17, e, k)
    x = (g.standard_normal((n, e)) * 1.5).astype(np.float32)
    x[::7] = np.round(x[::7])            # many equal ones
    x[1::50] = 0
    x[2::101, e // 2], x[3::103, 0], x[4::107, e - 1] = np.nan, np.inf, -np.inf
    x[5::109] *= 40                      # weights next to nothing
    bias = (g.standard_normal(e) * 0.1).astype(np.float32) if biased else None
    if biased:
        x[6::7, 1] = x[6::7, 0]
        bias[1] = np.nextafter(bias[0], np.float32(9))  # a pair that only 64 bits tell apart
    dx, db = cuda(x), None if bias is None else cuda(bias)
    ids, i_ok = banded((n, k), torch.int32)
    rw, r_ok = banded((n, k), torch.float32)
    made = qg.qroute_plan(**plan)
    qg.qmoe_route(made, dx, k, ids, rw, bias=db)
    assert i_ok() and r_ok()
    few, fw = torch.empty_like(ids), torch.empty_like(rw)
    for a in range(0, n, 1000):
        qg.qmoe_route(made, dx[a:a + 1000], k, few[a:a + 1000], fw[a:a + 1000], bias=db)
    assert torch.equal(ids, few)
    a, b = host(rw).astype(np.float64), host(fw).astype(np.float64)
    assert np.array_equal(np.isnan(a), np.isnan(b))
    assert (np.abs(np.nan_to_num(a - b)) <= 2.0 ** -18 * np.abs(np.nan_to_num(b)) + 2.0 ** -125).all()
    for t in (0, 1, 2, 3, 4, 5, 6, 13, 20, 51, 103, 2599):
        with np.errstate(invalid="ignore"):
            want, w, near = ref.route(x[t], bias, k, **plan)
        if near > 1e-14:
            assert np.array_equal(host(ids)[t], want), t
            weights_within(host(rw)[t], w, f"token {t}")


def test_route_biases_not_finite_for_many_tokens():
    """A bias that is not finite: every token in 64 bits."""
    n, e, k = 2100, 64, 4
    g = rng(18)
    x = g.standard_normal((n, e)).astype(np.float32)
    bias = (g.standard_normal(e) * 0.1).astype(np.float32)
    bias[3], bias[10], bias[20] = np.inf, -np.inf, np.nan
    ids, rw = torch.empty((n, k), dtype=torch.int32, device="cuda"), torch.empty((n, k), device="cuda")
    qg.qmoe_route(qg.qroute_plan("sigmoid"), cuda(x), k, ids, rw, bias=cuda(bias))
    for t in range(0, n, 191):
        want, w, _ = ref.route(x[t], bias, k, "sigmoid")
        assert np.array_equal(host(ids)[t], want)
        weights_within(host(rw)[t], w)


@pytest.mark.parametrize("e,hidden,ncols,k", [(256, 2048, 1, 8), (256, 2048, 16, 8), (1024, 768, 3, 32), (7, 33, 2, 7), (64, 8192, 16, 8),
                                              (64, 8190, 13, 8), (40, 128, 5, 4), (512, 5120, 2, 10)])
@pytest.mark.parametrize("plan", [0, 1, 4, 5])
def test_router_planned(e, hidden, ncols, k, plan):
    """The logits are qmoe_router's, bit for bit; the routing is qmoe_route's of those logits, bit for bit, and the plain form's."""
    plan = dict(PLANS[plan])
    if e % plan.get("n_group", 1) or k > plan.get("top_group", 1) * (e // plan.get("n_group", 1)):
        plan["n_group"] = plan["top_group"] = 1
    g = rng(16, e, hidden, ncols)
    w, x = (g.standard_normal((e, hidden)) * 0.02).astype(np.float32), g.standard_normal((ncols, hidden)).astype(np.float16)
    for bias in (None, cuda((g.standard_normal(e) * 0.1).astype(np.float32))):
        lg, l_ok = banded((ncols, e), torch.float32)
        ids, i_ok = banded((ncols, k), torch.int32)
        rw, r_ok = banded((ncols, k), torch.float32)
        made = qg.qroute_plan(**plan)
        qg.qmoe_router_planned(made, cuda(w), cuda(x), k, ids, rw, bias=bias, logits_out=lg)
        assert l_ok() and i_ok() and r_ok()
        lg0, ids0, rw0 = torch.empty_like(lg), torch.empty_like(ids), torch.empty_like(rw)
        qg.qmoe_router(cuda(w), cuda(x), k, ids0, rw0, logits_out=lg0)
        assert torch.equal(lg, lg0)
        qg.qmoe_route(made, lg, k, ids0, rw0, bias=bias)
        assert torch.equal(ids, ids0) and torch.equal(rw, rw0)
        qg.qmoe_router_planned(made, cuda(w), cuda(x), k, ids0.fill_(-1), rw0, bias=bias)
        assert torch.equal(ids, ids0) and torch.equal(rw, rw0)
        for t in range(ncols):
            want, wt, _ = ref.route(host(lg)[t], None if bias is None else host(bias), k, **plan)
            assert np.array_equal(host(ids)[t], want)
            weights_within(host(rw)[t], wt)


# ------------------------------------------------- streams, graphs, determinism
def test_all_calls_in_a_graph_and_on_another_stream():
    """Captured once and replayed with new inputs, and on a stream of its own, equal to eager calls bit for bit; a plan may be
    dropped after its capture."""
    n, k, e = 16, 512, 64
    q, scl, _ = table(qg.Q8_0, 200, k, 3)
    dq, ds = cuda(q), cuda(scl.view(np.float16))
    w = torch.rand(k, device="cuda") + 0.5
    wr = torch.randn(e, k, device="cuda") * 0.05
    bias = torch.randn(e, device="cuda") * 0.1
    ids_in = torch.zeros(n, dtype=torch.int32, device="cuda")
    add = torch.zeros(n, k, device="cuda")
    outs = dict(h=torch.zeros(n, k, device="cuda"), s=torch.zeros(n, k, device="cuda"), y=torch.zeros(n, k, dtype=torch.float16, device="cuda"),
                q=torch.zeros(n, k, dtype=torch.int8, device="cuda"), qs=torch.zeros(n, k // 32, dtype=torch.float16, device="cuda"),
                lg=torch.zeros(n, e, device="cuda"), ids=torch.zeros(n, 6, dtype=torch.int32, device="cuda"), rw=torch.zeros(n, 6, device="cuda"),
                ids2=torch.zeros(n, 6, dtype=torch.int32, device="cuda"), rw2=torch.zeros(n, 6, device="cuda"))

    def run():
        o = outs
        qg.qembed(qg.Q8_0, dq, ds, ids_in, o["h"], scale=3.0)
        qg.qrms_norm(o["h"], w, o["y"], add=add, sum_out=o["s"])
        qg.qrms_norm(o["s"], w, o["q"], y_scl=o["qs"])
        qg.qmoe_router_planned(qg.qroute_plan("sigmoid", n_group=4, top_group=2, group_top=2), wr, o["y"], 6, o["ids"], o["rw"],
                               bias=bias, logits_out=o["lg"])
        qg.qmoe_route(qg.qroute_plan(), o["lg"], 6, o["ids2"], o["rw2"])

    got = {}
    side = torch.cuda.Stream()
    for mode in ("eager", "graph", "stream"):
        if mode == "graph":
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
        for i in range(4):
            g = torch.Generator(device="cuda").manual_seed(i)
            ids_in.copy_(torch.randint(0, 200, (n,), generator=g, device="cuda"))
            add.copy_(torch.randn(n, k, generator=g, device="cuda"))
            for t in outs.values():
                t.zero_()
            if mode == "graph":
                graph.replay()
            elif mode == "stream":
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    run()
                torch.cuda.current_stream().wait_stream(side)
            else:
                run()
            for name, t in outs.items():
                got.setdefault((i, name), []).append(t.clone())
    for key, three in got.items():
        assert torch.equal(three[0], three[1]) and torch.equal(three[0], three[2]), key


def test_no_wait_was_given_up():
    torch.cuda.synchronize()
    assert qg.qg_device_error() == 0
