"""The attention layer of examples/attention_layer.py, checked stage by stage on the GPU's own
intermediate values: projections against the oracle, rotation, cache and attention against the
plain 64-bit forms."""
import importlib.util
import os

import numpy as np
import pytest

import attn_ref as ref
import oracle
from helpers import assert_within, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_q4_q8_gb300 import build
    build.build()
    oracle.build()
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def cached(layer, seq, n):
    """(keys, values) f64 [n, kv, D] of a sequence, from the pool's bytes."""
    pool, table, ps = host(layer.pool), host(layer.table), layer.cache.page_size
    out = np.empty((2, n, layer.kv, layer.d))
    for j in range(n):
        for h in range(layer.kv):
            for v in (0, 1):
                off, i = ref.locate(layer.cache.type, layer.d, layer.kv, ps, int(table[seq, j // ps]), h, j % ps, bool(v))
                out[v, j, h] = ref.read_row(pool, layer.cache.type, layer.d, off, i)
    return out


@pytest.mark.parametrize("weights,cache_type", [(2, 8), (8, 1)])
def test_layer_stage_by_stage(example, weights, cache_type):
    hidden, heads, kv, d, n_seq, rot = 256, 6, 2, 64, 2, 32
    layer, ((wq, sq), (wo, so)) = example.random_layer(weights, hidden, heads, kv, d, n_seq=n_seq, tokens=96, page_size=16,
                                                       cache_type=cache_type, rot_dim=rot, seed=weights)
    g = np.random.Generator(np.random.PCG64(weights))
    theta = ref.thetas(rot, 1e6)
    done = 0
    for piece in (8, 8, 1, 4):
        n = n_seq * piece
        x = g.standard_normal((n, hidden)).astype(np.float16)
        res = g.standard_normal((n, hidden)).astype(np.float32)
        y, (rows, q, att) = layer.step(torch.from_numpy(x).cuda(), torch.from_numpy(res).cuda())
        rows, q, att = host(rows), host(q).astype(np.float64), host(att)
        want, S = oracle.matmul(weights, wq, sq, x.view(np.uint16))
        assert_within(rows.reshape(n, -1), want, 1e-3 * S + 1e-6, "QKV")
        pos = np.tile(np.arange(done, done + piece), n_seq)
        turned, size = ref.rotate(rows[:, :heads + kv], pos, theta, False)
        err = ref.ROT * size
        qw = turned[:, :heads]
        assert_within(q, qw, err[:, :heads] * (1 + ref.HALF) + ref.HALF * np.abs(qw) + ref.SUB, "queries")
        done += piece
        ks, vs = zip(*(cached(layer, s, done) for s in range(n_seq)))
        want, bound = ref.attention(q.reshape(n_seq, piece, heads, d), ks, vs, [done] * n_seq, piece, 0, d ** -0.5)
        assert_within(att, want, bound, "attention")
        want, S = oracle.matmul(weights, wo, so, att.reshape(n, -1).view(np.uint16), res)
        assert_within(host(y), want, 1e-3 * S + 1e-6, "output projection")
    assert int(layer.err) == 0


def test_shift_moves_tokens_to_the_front(example):
    """After a context shift the cache holds the same values, and keys turned back by the dropped positions."""
    import gemm_q4_q8_gb300 as qg
    hidden, heads, kv, d, rot, drop = 256, 4, 2, 64, 64, 5
    layer, _ = example.random_layer(8, hidden, heads, kv, d, n_seq=2, tokens=64, page_size=16, cache_type=qg.QG_F16, seed=3)
    for _ in range(3):
        x = torch.randn(16, hidden, device="cuda")
        layer.step(x.half(), x)
    k0, v0 = cached(layer, 0, 24)
    other = cached(layer, 1, 24)
    layer.shift(0, drop)
    assert layer.lens.tolist() == [24 - drop, 24]
    k1, v1 = cached(layer, 0, 24 - drop)
    want, size = ref.rotate(k0[drop:], np.full(24 - drop, -drop), ref.thetas(rot, 1e6), False)
    assert_within(k1, want, ref.ROT * size * (1 + ref.HALF) + ref.HALF * np.abs(want) + ref.SUB, "keys")
    assert np.array_equal(v1, v0[drop:])
    assert np.array_equal(cached(layer, 1, 24), other)
    x = torch.randn(2, hidden, device="cuda")
    y, _ = layer.step(x.half(), x)
    assert torch.isfinite(y).all() and int(layer.err) == 0
