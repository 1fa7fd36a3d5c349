"""GPU parity of the cache in 4 bits where the pool was written in another way than by qkv_append: blocks whose d is of either sign."""
import numpy as np
import pytest

import kv4_ref as ref
from attn_ref import HALF, SINGLE, SUB
from helpers import assert_within, host
from test_parity_kv4 import Cache, attend, cuda, rng

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gemm_q4_q8_gb300 as qg  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_q4_q8_gb300 import build
    build.build()


def put_block(c, s, j, h, is_v, b, q, d, m):
    """Block b of a token's row as it stands in the pool."""
    off, i = c.where(s, j, h, is_v)
    at = off + b * 256 + i * 16
    got = np.zeros(16, np.uint8)
    np.bitwise_or.at(got, ref.BYTES, (q << ref.SHIFTS).astype(np.uint8))
    c.host[at:at + 16] = got
    at = off + ref.scale_offset(c.d, i, b, is_v)
    for k, x in ((0, d), (c.d, m)):
        c.host[at + k:at + k + 2] = np.array([x], np.float16).view(np.uint8)


def attention(q, ks, vs, n, ncols, scale):
    """(y, bound) in f64 of one sequence: ref.attention's bound, with the magnitudes of what may be negative here: q d of keys in A, and
    d of values in the last term."""
    (kq, km, _), (vq, vm, vd) = ks, vs
    _, _, heads, d = q.shape
    y, bound = np.zeros(q.shape), np.zeros(q.shape)
    g = heads // kq.shape[1]
    for c in range(ncols):
        at = np.arange(n - ncols + c + 1)
        for h in range(heads):
            k1, k2, v1, v2, v3 = (a[at, h // g] for a in (kq, km, vq, vm, vd))
            qq = q[0, c, h].astype(np.float64)
            sc = (k1 + k2) @ qq * scale
            mag = ((np.abs(k1) + np.abs(k2)) @ np.abs(qq)).max() * abs(scale)
            w = np.exp(sc - sc.max())
            w /= w.sum()
            y[0, c, h] = w @ (v1 + v2)
            e_score = (d + 8) * SINGLE * mag + 4 * SINGLE * np.abs(sc).max()
            rel = 2 * e_score + 16 * SINGLE + 2 * len(at) * SINGLE
            a, c8 = np.abs(v1 - 8 * v3), np.abs(v2 + 8 * v3)
            bound[0, c, h] = rel * (w @ (a + c8)) + 1.01 * HALF * (w @ a) + 2.01 * HALF * (w @ c8) + HALF * np.abs(y[0, c, h]) + \
                SUB * (1 + w.sum()) + w.max() * (2.0 ** -32 * c8.sum(0) + 8 * len(at) * 2.0 ** -30 * np.abs(v3).max())
    return y, bound


@pytest.mark.parametrize("wide", [0, 2000])
@pytest.mark.parametrize("kind", ["negative", "either", "small and large", "large"])
@pytest.mark.parametrize("d,heads,ncols", [(64, 3, 1), (128, 5, 1), (128, 8, 2), (256, 6, 1), (64, 16, 2)])
def test_steps_of_either_sign(d, heads, ncols, kind, wide):
    """d negative, of both signs, tiny positive ones beside negative ones of 4, and negative ones near the largest that m + 8 d
    allows; read back and attended, by clusters and by runs."""
    n, kv, ps = 330, 1, 16
    g = rng(40, d, heads)
    c = Cache(kv, d, ps, 1, -(-n // ps) + wide, seed=3, fill=0xFF)
    parts = np.empty((2, 3, n, kv, d))
    for j in range(n):
        for b in range(d // 32):
            sign = -1 if kind == "negative" or (j + b) % 2 else 1
            key = sign * 0.2 * g.uniform(0.5, 1)
            val = dict(negative=-0.1, either=sign * 0.1, large=-7000.0)[kind] if kind != "small and large" else (-4.0 if sign < 0 else 2.0 ** -10)
            val *= g.uniform(0.5, 1)
            put_block(c, 0, j, 0, False, b, g.integers(0, 16, 32), key, -7.5 * key + 0.3)
            put_block(c, 0, j, 0, True, b, g.integers(0, 16, 32), val, -8 * val + g.standard_normal() * 0.1)
        parts[:, :, j, 0] = c.get(0, j, 0)
    c.upload()
    ko, vo = (torch.empty((n, kv, d), dtype=torch.float32, device="cuda") for _ in range(2))
    qg.qkv_read(c.c, cuda(np.arange(n, dtype=np.int32)), ko, vo)
    for got, (qd, m, _) in zip((ko, vo), parts):
        assert np.array_equal(host(got), (qd + m).astype(np.float32))
    q = g.standard_normal((1, ncols, heads, d)).astype(np.float16)
    y, err = attend(c, q, [n])
    assert err == 0
    want, bound = attention(q, parts[0], parts[1], n, ncols, d ** -0.5)
    assert np.isfinite(y).all()
    assert_within(y, want, bound, kind)
