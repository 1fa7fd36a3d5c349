"""GPU parity of the routing by a plan at the ends of f32's range, through both of its calls, against the plain 64-bit form."""
import numpy as np
import pytest

import layer_ref as ref
from helpers import assert_within, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gemm_q4_q8_gb300 as qg  # noqa: E402

MOST = np.finfo(np.float32).max


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


def against(ids, rw, logits, bias, k, plan):
    """ids equal, weights within 2^-19 of themselves, as documented. (Where two c that decide differ by less than 1e-14, two
    exponentials in 64 bits may order them either way.)"""
    for t in range(len(logits)):
        with np.errstate(all="ignore"):
            want, w, near = ref.route(logits[t], bias, k, **plan)
        assert (ids[t] >= 0).all() and (ids[t] < logits.shape[1]).all(), (t, ids[t])
        if near > 1e-14:
            assert np.array_equal(ids[t], want), (t, ids[t], want)
            assert np.array_equal(np.isnan(rw[t]), np.isnan(w)), (t, rw[t], w)
            w = np.nan_to_num(w)
            assert_within(np.nan_to_num(rw[t]), w, 2.0 ** -19 * np.abs(w) + 2.0 ** -126, f"token {t}")


def check(logits, bias, k, **plan):
    """At most 16 tokens, by qmoe_route and by qmoe_router_planned, whose columns are one-hot: weights [experts, column] are the logits
    (of experts whose weights are finite: 0 times an infinity is NaN), and the routing is that of the logits it made."""
    n, e = logits.shape
    made, b = qg.qroute_plan(**plan), None if bias is None else cuda(bias)
    for fused in (False, True):
        ids = torch.full((n, k), -1, dtype=torch.int32, device="cuda")
        rw = torch.full((n, k), -1.0, device="cuda")
        if fused:
            w = np.zeros((e, 16), np.float32)
            w[:, :n] = logits.T
            lg = torch.empty((n, e), device="cuda")
            qg.qmoe_router_planned(made, cuda(w), torch.eye(16, dtype=torch.float16, device="cuda")[:n].contiguous(), k, ids, rw, bias=b,
                                   logits_out=lg)
            finite = np.isfinite(w).all(1)
            assert np.array_equal(host(lg)[:, finite], logits[:, finite])
            made_of = host(lg)
        else:
            qg.qmoe_route(made, cuda(logits), k, ids, rw, bias=b)
            made_of = logits
        against(host(ids), host(rw), made_of, bias, k, plan)


SIZES = [(64, 4), (50, 25), (256, 8), (300, 32), (512, 10), (1000, 6)]
SCORES = ["softmax", "sigmoid"]


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("e,k", SIZES)
def test_logits_whose_differences_leave_f32(e, k, score):
    """Finite logits up to the largest: a few of both signs, all of them, alike and not."""
    g = rng(1, e)
    x = g.standard_normal((9, e)).astype(np.float32)
    x[0, 3], x[0, 4] = 3e38, -3e38
    x[1, 7], x[1, e - 8] = MOST, -MOST
    x[2] = np.where(np.arange(e) % 2, MOST, -MOST)
    x[3, 1] = -MOST
    x[4, ::3] = 2e38
    with np.errstate(over="ignore"):
        x[5] *= 1e38  # (some of them infinite)
    x[6] = MOST
    x[7] = -MOST
    x[8, :] = np.linspace(-float(MOST), float(MOST), e).astype(np.float32)
    for bias in (None, (0.1 * g.standard_normal(e)).astype(np.float32)):
        for plan in ({}, dict(renorm=False), dict(n_group=2, top_group=1, group_top=2), dict(n_group=2, top_group=1, group_top=1, scale=2.5)):
            check(x, bias, k, score=score, **plan)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("e,k", SIZES + [(40, 4), (50, 3), (20, 2), (63, 6)])
def test_biases_at_the_least_number(e, k, score):
    """All experts but a few shut out by f32's least number, so that such ones are chosen, too; and all of them."""
    g = rng(2, e)
    x = g.standard_normal((5, e)).astype(np.float32)
    for n_open in (0, 1, k - 1, k):
        bias = np.full(e, -MOST, np.float32)
        bias[g.permutation(e)[:n_open]] = 0.1
        for plan in ({}, dict(renorm=False), dict(n_group=3 if e % 2 else 2, top_group=1, group_top=1)):
            check(x, bias, k, score=score, **plan)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("value", [2e38, MOST, 1e30, -1e30, -2e38, -MOST])
@pytest.mark.parametrize("e,k,groups", [(64, 4, 8), (256, 8, 8), (300, 10, 12), (40, 6, 5), (1000, 8, 4)])
def test_groups_whose_sums_leave_f32(e, k, groups, value, score):
    """Two experts of a group with biases of this size, one group kept; two such groups; all experts; and all below the least number
    in sum, one group above the others."""
    g = rng(3, e)
    x = g.standard_normal((5, e)).astype(np.float32)
    size = e // groups
    two, four, rest = ((0.1 * g.standard_normal(e)).astype(np.float32) for _ in range(3))
    two[2 * size:2 * size + 2] = value
    four[2 * size:2 * size + 2] = four[4 * size:4 * size + 2] = value
    rest[:] = value
    rest[3 * size:4 * size] = np.float32(value) * np.float32(0.9)
    for bias in (two, four, np.full(e, value, np.float32), rest):
        for keep in (1, 2):
            for best in (1, 2):
                check(x, bias, k, score=score, n_group=groups, top_group=keep, group_top=best)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("value", [-1e2, -1e4, -1e6, -1e9, -1e30, -MOST, -np.inf])
@pytest.mark.parametrize("e,k,groups", [(64, 4, 8), (256, 8, 8), (300, 10, 12), (40, 6, 5), (1000, 8, 4)])
def test_experts_shut_out(e, k, groups, value, score):
    """One expert, a group, all but one of a group, half of all and all but k shut out by their bias or by their logit, among experts that
    are equal or so near that only 64 bits tell them apart."""
    g = rng(4, e)
    x = g.standard_normal((8, e)).astype(np.float32)
    x[1] = np.round(x[1])
    x[2] = 0
    x[3:5, 1::2] = x[3:5, ::2]
    size, n = e // groups, np.arange(e)
    alive = g.permutation(e)
    kept = np.zeros(e, bool)
    kept[alive[:k]] = True
    for shut in (n == 5, n // size == 1, (n // size == 1) & (n != size), alive < e // 2, ~kept):
        bias = (0.1 * g.standard_normal(e)).astype(np.float32)
        bias[1::2] = np.nextafter(bias[::2], np.float32(9))  # pairs that f32 scores do not tell apart
        masked = np.where(shut, np.float32(value), bias)
        low = np.where(shut, np.float32(value), x)
        for plan in ({}, dict(renorm=False), dict(n_group=groups, top_group=2, group_top=2), dict(n_group=groups, top_group=2, group_top=1)):
            check(x, masked, k, score=score, **plan)
            check(low, bias, k, score=score, **plan)
            check(low, None, k, score=score, **plan)
