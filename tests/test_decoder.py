"""The decoder of examples/decoder.py, checked stage by stage on the GPU's own intermediate values: lookup, norms and routing
against the plain 64-bit forms, products and experts against the oracle, the 4-bit cache and the attention over it against their
plain forms; and the whole step captured into a graph, on another stream, and with an f16 cache beside it."""
import importlib.util
import os

import numpy as np
import pytest

import attn_ref
import kv4_ref
import layer_ref as ref
import oracle
from helpers import NTHREADS, assert_within, check_moe_staged, host, workspace_h

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPE = dict(vocab=300, hidden=256, heads=6, kv_heads=2, head_dim=64, experts=16, ffn=64, n_layers=2, topk=4)


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_q4_q8_gb300 import build
    build.build()
    oracle.build()
    spec = importlib.util.spec_from_file_location("decoder", os.path.join(ROOT, "examples", "decoder.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def normed(got, s, w, what):
    want, bound = ref.norm(s, host(w), 0.0, 1e-6)
    if got.dtype == np.float16:
        bound = bound * (1 + ref.HALF) + ref.HALF * np.abs(want) + ref.SUB
    assert_within(got, want, bound, what)


def product(got, weights, plain, x, what):
    want, size = oracle.matmul(weights, *plain, np.ascontiguousarray(x).view(np.uint16))
    assert_within(got.reshape(want.shape), want, 1e-3 * size + 1e-6, what)


def cached(cache, seq, n):
    """(keys, values), each (q d, m, d) [n, kv, D] of a sequence, from the pool's bytes."""
    pool, table = (host(t) for t in cache.tensors)
    kv, d, ps = cache.n_kv_heads, cache.head_dim, cache.page_size
    out = np.empty((2, 3, n, kv, d))
    for j in range(n):
        for h in range(kv):
            for v in (0, 1):
                off, i = kv4_ref.offset(d, kv, ps, int(table[seq, j // ps]), h, j % ps, bool(v))
                out[v, :, j, h] = kv4_ref.read_row(pool, d, off, i, bool(v))
    return out


@pytest.mark.parametrize("weights", [2, 8])
def test_decoder_stage_by_stage(example, weights):
    n_seq, heads, kv, d, dim, experts, ffn, topk = 2, 6, 2, 64, 256, 16, 64, 4
    plan = dict(score="sigmoid", n_group=4, top_group=2, group_top=2, scale=2.0)
    model, plain = example.random_decoder(weights, **SHAPE, n_seq=n_seq, tokens=64, seed=weights, embed_scale=16.0)
    table = ref.weights(weights, host(model.table[0]), host(model.table[1]).view(np.uint16))
    g = np.random.Generator(np.random.PCG64(weights))
    done = 0
    for piece in (8, 5, 1, 3):
        ids = g.integers(0, 300, n_seq * piece).astype(np.int32)
        keep = []
        logits, token = model.step(torch.from_numpy(ids).cuda(), keep)
        done += piece
        x = table[ids].astype(np.float32) * np.float32(16)
        delta = None
        for i, (w, hidden, cache) in enumerate(zip(model.layers, plain[1:], model.caches)):
            k = {n: host(t) for n, t in keep[i].items()}
            np.testing.assert_array_equal(k["x"], x)
            np.testing.assert_array_equal(k["residual"], ref.add_up(x, delta))
            normed(k["a"], k["residual"], w.norm1, "first norm")
            product(k["projected"], weights, hidden["wqkv"], k["a"], "QKV")
            normed(k["rows"][:, :heads], k["projected"][:, :heads], w.norm_q, "queries' norm")
            normed(k["rows"][:, heads:heads + kv], k["projected"][:, heads:heads + kv], w.norm_k, "keys' norm")
            np.testing.assert_array_equal(k["rows"][:, heads + kv:], k["projected"][:, heads + kv:])
            turned, size = attn_ref.rotate(k["rows"][:, :heads + kv], k["pos"], attn_ref.thetas(d, 1e6), False)
            q = turned[:, :heads]
            assert_within(k["q"], q, attn_ref.ROT * size[:, :heads] * (1 + ref.HALF) + ref.HALF * np.abs(q) + ref.SUB, "queries")
            ks, vs = [], []
            for s in range(n_seq):
                both = cached(cache, s, done)
                ks.append(both[0])
                vs.append(both[1])
                for t in range(piece):  # the new tokens
                    n = s * piece + t
                    vq, vd, vm = kv4_ref.quantise(k["rows"][n, heads + kv:].reshape(kv, -1, 32))
                    np.testing.assert_array_equal(both[1, 0, done - piece + t].reshape(kv, -1, 32), vq * vd.astype(np.float64)[..., None])
                    np.testing.assert_array_equal(both[1, 1, done - piece + t].reshape(kv, -1, 32)[..., 0], vm.astype(np.float64))
                    off = (both[0, 0] + both[0, 1])[done - piece + t] - turned[n, heads:]
                    # half a step, of a block whose step is d
                    assert (np.abs(off) <= both[0, 2, done - piece + t] * (0.5 + 15 * 4 * ref.SINGLE) + attn_ref.ROT * size[n, heads:]).all()
            y, bound = kv4_ref.attention(k["q"].reshape(n_seq, piece, heads, d), ks, vs, [done] * n_seq, piece, 0, d ** -0.5)
            assert_within(k["att"], y, bound, "attention")
            product(k["out"], weights, hidden["wo"], k["att"].reshape(n_seq * piece, -1), "output projection")
            np.testing.assert_array_equal(k["middle"], ref.add_up(k["residual"], k["out"]))
            normed(k["b"], k["middle"], w.norm2, "second norm")
            want, size = oracle.router_logits(host(w.router), k["b"].view(np.uint16))
            assert_within(k["logits"], want, 1e-3 * size + 1e-6, "router")
            for t in range(n_seq * piece):
                want, rw, near = ref.route(k["logits"][t], host(w.bias), topk, **plan)
                assert near < 1e-14 or np.array_equal(k["chosen"][t], want)
                assert_within(k["rw"][t], rw, 2.0 ** -19 * np.abs(rw), "routing weights")
            case = dict(qtype=weights, qg=hidden["gate"][0], sg=hidden["gate"][1], qu=hidden["up"][0], su=hidden["up"][1],
                        qd=hidden["down"][0], sd=hidden["down"][1], n_expert=experts, ffn=ffn, hidden=dim, ids=k["chosen"], rw=k["rw"],
                        topk=topk, ncols=n_seq * piece, x=np.ascontiguousarray(k["b"]).view(np.uint16), y0=None, shared=None)
            check_moe_staged(case, k["delta"], workspace_h(keep[i]["ws"], case), what="experts")
            x, delta = k["middle"], k["delta"]
        k = {n: host(t) for n, t in keep[-1].items()}
        np.testing.assert_array_equal(k["final"], ref.add_up(x, delta))
        normed(k["c"], k["final"], model.last_norm, "last norm")
        product(k["logits"], weights, plain[0], k["c"], "logits")
        np.testing.assert_array_equal(host(token), host(logits).argmax(1))
    assert int(model.err) == 0 and example.qg.qg_device_error() == 0


def decode(model, how):
    """Logits of a prompt and of tokens decoded after it: eagerly, by one captured step replayed, on another stream."""
    prompt = torch.arange(16, dtype=torch.int32, device="cuda") * 7 % 300
    logits, token = model.step(prompt)
    got, token = [logits], token.view(2, 8)[:, -1].contiguous()
    if how == "graph":
        graph, static = torch.cuda.CUDAGraph(), token.clone()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out, nxt = model.step(static)
        for _ in range(6):
            static.copy_(token)
            graph.replay()
            got.append(out.clone())
            token = nxt.clone()
        return got
    stream = torch.cuda.Stream() if how == "stream" else torch.cuda.current_stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(6):
            logits, token = model.step(token)
            got.append(logits)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    return got


def test_decoder_in_a_graph_and_on_another_stream(example):
    outs = []
    for how in ("eager", "graph", "stream"):
        model, _ = example.random_decoder(8, **SHAPE, n_seq=2, tokens=64, seed=3)
        outs.append(decode(model, how))
        assert model.lens.tolist() == [14, 14] and int(model.err) == 0
    for a, b, c in zip(*outs):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_decoder_flags_an_id_outside_the_table(example):
    model, _ = example.random_decoder(8, **SHAPE, n_seq=2, tokens=64, seed=4)
    logits, _ = model.step(torch.tensor([5, 300], dtype=torch.int32, device="cuda"))
    assert int(model.err) == example.qg.QG_EMBED_BAD_ID and torch.isfinite(logits).all()


def test_example_runs(example, capsys):
    example.main()
    assert "[32, 32] tokens cached" in capsys.readouterr().out
