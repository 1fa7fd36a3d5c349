"""Softmax weights of attention where a 16-bit or 32-bit exponent ends: scores of any size that finite f16 queries and keys
can give, every finite scale, and sums of weights far below the largest."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref as ref  # noqa: E402
import gemm_q4_q8_gb300 as qg  # noqa: E402
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


@pytest.mark.parametrize("qtype,heads,d,lift", [(F16, 1, 64, 7), (F16, 16, 128, 7), (F16, 32, 256, 7), (Q8, 1, 64, 5),
                                                (Q8, 16, 256, 5)])
@pytest.mark.parametrize("below", [20.5, 23.5, 24.40625, 25.125])
def test_many_tokens_far_below_the_first(qtype, heads, d, lift, below):
    """A first token that takes nearly all the weight, with a value of zero, before 30,000 tokens that weigh about 2^-below of it
    each: what they add up to is the answer. As many sequences as a call takes, all over the same pages, so that a warp has the
    first token and many of the others in one run. Scores are key element 0, in powers of two (scale = log 2).

    A weight in f16 has half a step of 2^-25 below the normals, and the largest is at least 2^lift (Q8_0: times the block's
    scale, which comes with 127 times it), so each weight is off by 2^-11 of itself and by 2^-(25 + lift) of the
    largest. Its exponent passes three f32 roundings of numbers up to 26 (as a factor: 3 x 26 half steps), exp2 and the sums as
    in attn_ref.attention: 16 half steps and those of at most 4,160 terms."""
    n, ps, n_seq = 30001, 64, 1024
    pages = -(-n // ps)
    g = rng(34, d, int(below * 32))
    k, v = np.zeros((n, 1, d), np.float32), np.abs(1 + 0.2 * g.standard_normal((n, 1, d))).astype(np.float32)
    k[1:, 0, 0] = -below + g.integers(-16, 17, n - 1) / 64
    v[0] = 0
    pool = torch.zeros(pages * qg.qkv_page_bytes(qtype, 1, d, ps), dtype=torch.uint8, device="cuda")
    table = torch.randperm(pages, device="cuda").to(torch.int32).view(1, pages)
    one = qg.qkv_cache(qtype, pool, table, 1, d, ps)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    qg.qkv_append(one, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), pos)
    kr, vr = (torch.empty((n, 1, d), dtype=torch.float32, device="cuda") for _ in range(2))
    qg.qkv_read(one, pos, kr, vr)
    c = qg.qkv_cache(qtype, pool, table.repeat(n_seq, 1), 1, d, ps)
    q = torch.zeros((n_seq, 1, heads, d), dtype=torch.float16, device="cuda")
    q[..., 0] = 1
    y = torch.empty_like(q)
    ws = torch.empty(qg.qattn_workspace_bytes(c, heads, 1), dtype=torch.uint8, device="cuda")
    qg.qattn_paged(c, q, torch.full((n_seq,), n, dtype=torch.int32, device="cuda"), y, ws, scale=float(np.log(2)))
    w, vr = torch.exp2(kr[:, 0, 0].double()), vr[:, 0].double()
    want = w @ vr / w.sum()
    rel = (16 + 2 * 3 * 26 + 2 * 4160) * ref.SINGLE + ref.HALF
    least = 2.0 ** -(25 + lift) * (vr.sum(0) if qtype == F16 else n * vr.max())
    bound = rel * want + least / w.sum() + ref.HALF * want + ref.SUB
    off = (y.double() - want).abs()
    assert (off <= bound).all(), float((off / want).max())
