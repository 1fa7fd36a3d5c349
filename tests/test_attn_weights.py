"""Softmax weights of attention where a 16-bit or 32-bit exponent ends: scores of any size that finite f16 queries and keys
can give, and every finite scale."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref as ref  # noqa: E402
from test_parity_attn import F16, Q8, _lib, assert_within, attend, filled, rng  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def tops_of(c, q, n, kv, scale):
    """The tokens with the largest 64-bit score for each query row [heads, d] of one sequence, and whether every other token is
    so far below that its weight is 0 (by more than 200 powers of two and 2^-10 of the largest magnitude, many times what the
    f32 sums can be off)."""
    heads, d = q.shape
    out = []
    for h in range(heads):
        head = h // (heads // kv)
        k = np.stack([c.get(0, j, head)[0] for j in range(n)])
        s = k @ q[h].astype(np.float64) * scale * np.log2(np.e)
        mag = (np.abs(k) @ np.abs(q[h].astype(np.float64))).max() * abs(scale) * np.log2(np.e)
        top = s == s.max()
        assert (s[~top] < s.max() - max(200, mag * 2.0 ** -11)).all()
        out.append(top)
    return out


def check_tops(c, vs, q, n, kv, scale, what):
    """y is the mean of the top tokens' values. All weigh the same: one rounding of that weight to f16, f32 sums of three
    terms and a division, y's own rounding."""
    y, err = attend(c, q[None, None], [n], scale=scale)
    assert err == 0
    heads = q.shape[0]
    for h, top in enumerate(tops_of(c, q, n, kv, scale)):
        v = vs[0][top, h // (heads // kv)]
        want = v.mean(0)
        bound = (ref.HALF + 8 * ref.SINGLE) * np.abs(v).mean(0) + ref.HALF * np.abs(want) + ref.SUB
        assert_within(y[0, 0, h], want, bound, f"{what}, row {h}")


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("heads,d,n,wide", [(3, 64, 200, 0), (1, 128, 90, 300), (12, 256, 200, 300), (20, 64, 200, 300)])
@pytest.mark.parametrize("a,b", [(60000, 60000), (3000, 20000), (200, 60000)])
@pytest.mark.parametrize("order", ["ties", "rising", "falling"])
def test_scores_of_any_size(qtype, heads, d, n, wide, a, b, order):
    """Scores of 10^8 to 10^11 powers of two: a reference that is rounded in units of log 2 is off by many of them. Three tokens
    share the largest score, or the scores rise or fall from token to token."""
    c, _, vs = filled(qtype, 1, d, 16, [n], seed=a % 97 + b % 89, extra_pages=wide)
    g = rng(31, d, heads)
    sign = g.choice([-1.0, 1.0], d)
    for j in range(n):
        if order == "ties":
            k = b * sign if j in (5, 77, n - 1) else g.uniform(-0.4, 0.4, d) * b
        else:
            k = b * sign * (1 - (n - 1 - j if order == "rising" else j) * 2.0 ** -8)
        v = g.standard_normal(d)
        c.put(0, j, 0, k.astype(np.float32), v.astype(np.float32))
        vs[0][j, 0] = c.get(0, j, 0)[1]
    c.upload()
    q = np.tile(a * sign, (heads, 1)).astype(np.float16)
    check_tops(c, vs, q, n, 1, d ** -0.5, f"{order} {a} x {b}")


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("heads,d,wide", [(3, 64, 0), (12, 256, 0), (8, 128, 300), (33, 64, 300)])
@pytest.mark.parametrize("scale", [1e20, 1e30, 3e31, -1e34, 2.5e38, 3.4e38, -3.4e38])
def test_scale_up_to_the_end_of_f32(qtype, heads, d, wide, scale):
    """Every finite scale has an answer: one token takes all the weight."""
    n, kv = 70, heads // 4 or 1
    c, _, vs = filled(qtype, kv, d, 16, [n], seed=17, extra_pages=wide)
    q = rng(32, d).standard_normal((heads // kv * kv, d)).astype(np.float16)
    check_tops(c, vs, q, n, kv, scale, f"scale {scale}")


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("heads,d,wide", [(3, 64, 0), (12, 256, 300)])
@pytest.mark.parametrize("scale", [1e-37, -1e-40, 1e-45])
def test_scale_down_to_subnormals(qtype, heads, d, wide, scale):
    c, ks, vs = filled(qtype, 1, d, 16, [70], 19, extra_pages=wide)
    q = rng(33, heads).standard_normal((1, 1, heads, d)).astype(np.float16)
    y, err = attend(c, q, [70], scale=scale)
    want, bound = ref.attention(q, ks, vs, [70], 1, 0, scale)
    assert err == 0
    assert_within(y, want, bound, f"scale {scale}")
