"""GPU parity of the cache in 4 bits (qkv_append, qkv_read, qattn_paged on QG_Q4_1) against plain forms (kv4_ref.py)."""
import numpy as np
import pytest

import attn_ref
import kv4_ref as ref
from helpers import assert_within, host
from test_parity_attn import append_random, cuda, odd_rows, rng, step

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gemm_q4_q8_gb300 as qg  # noqa: E402

Q4 = qg.Q4_1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_q4_q8_gb300 import build
    build.build()


class Cache:
    """A cache on the GPU with shuffled pages, every byte of its pool set at the start."""

    def __init__(self, kv, d, ps, n_seq, max_pages, seed=0, fill=0xFF, spare=2):
        g = rng(9, seed, d, ps)
        self.kv, self.d, self.ps = kv, d, ps
        n = n_seq * max_pages + spare
        self.table = g.permutation(n)[:n_seq * max_pages].reshape(n_seq, max_pages).astype(np.int32)
        self.host = np.full(n * qg.qkv_page_bytes(Q4, kv, d, ps), fill, np.uint8)
        self.upload()

    def upload(self):
        self.pool = cuda(self.host)
        self.c = qg.qkv_cache(Q4, self.pool, cuda(self.table), self.kv, self.d, self.ps)

    def where(self, seq, pos, head, is_v):
        return ref.offset(self.d, self.kv, self.ps, int(self.table[seq, pos // self.ps]), head, pos % self.ps, is_v)

    def put(self, seq, pos, head, k, v):
        for row, is_v in ((k, False), (v, True)):
            ref.write_row(self.host, self.d, *self.where(seq, pos, head, is_v), is_v, row)

    def get(self, seq, pos, head):
        """((q d, m, d) of the key, the same of the value)."""
        return [ref.read_row(self.host, self.d, *self.where(seq, pos, head, is_v), is_v) for is_v in (False, True)]


# -------------------------------------------------------------- written, read
@pytest.mark.parametrize("src", [torch.float32, torch.float16])
@pytest.mark.parametrize("d,kv,ps", [(64, 1, 16), (64, 5, 32), (128, 8, 64), (256, 2, 128), (256, 3, 16), (128, 3, 256)])
def test_append_bytes(d, kv, ps, src):
    """Without rotation every byte of the pool is known: the written slots, and all others unchanged."""
    g = rng(4, d, kv, ps)
    c = Cache(kv, d, ps, 3, 3, seed=ps, fill=0xA5)
    n = 23
    slots = g.permutation(3 * 3 * ps)[:n]
    seq, pos = (slots // (3 * ps)).astype(np.int32), (slots % (3 * ps)).astype(np.int32)
    pos[[3, 17]] = [-1, -2 ** 31]  # padding
    of = {torch.float32: np.float32, torch.float16: np.float16}[src]
    k, v = odd_rows(g, n, kv, d).astype(of), odd_rows(g, n, kv, d).astype(of)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qg.qkv_append(c.c, cuda(k), cuda(v), cuda(pos), seq=cuda(seq), err_flag=err)
    for t in range(n):
        if pos[t] >= 0:
            for h in range(kv):
                c.put(seq[t], pos[t], h, k[t, h], v[t, h])
    assert np.array_equal(host(c.pool), c.host)
    assert int(err) == 0


def hard_blocks(g, n):
    """Blocks where the last bit decides: quants next to halves, ranges next to 15 times an f16, smallest elements next to an
    f16, all equal, subnormal, saturating, one far outlier."""
    x = g.standard_normal((n, 32)).astype(np.float32)
    for i in range(n):
        kind = i % 10
        d = np.float32(np.float16(2.0 ** g.uniform(-23, 8)))
        m = np.float32(np.float16(g.standard_normal() * 2.0 ** g.uniform(-10, 6)))
        if kind == 0:  # exact halves, and a step of f32 beside them
            x[i] = m + d * (g.integers(0, 15, 32) + np.float32(0.5)).astype(np.float32)
            x[i, 0], x[i, 1] = m, m + 15 * d
        elif kind == 1:
            x[i] = m + d * (g.integers(0, 15, 32) + np.float32(0.5)).astype(np.float32)
            x[i, 0], x[i, 1] = m, m + 15 * d
            x[i, 2:17] = np.nextafter(x[i, 2:17], np.float32(np.inf))
            x[i, 17:] = np.nextafter(x[i, 17:], np.float32(-np.inf))
        elif kind == 2:  # a range a step of f32 above or below 15 d
            x[i] = m + d * g.uniform(0, 15, 32).astype(np.float32)
            x[i, 3], x[i, 9] = m, np.nextafter(m + 15 * d, np.float32(np.inf if i & 16 else -np.inf))
        elif kind == 3:  # the smallest a step of f32 above or below an f16
            x[i] = np.abs(x[i]) + m
            x[i, 31] = np.nextafter(m, np.float32(np.inf if i & 16 else -np.inf))
        elif kind == 4:
            x[i] = g.standard_normal() * 10.0 ** g.uniform(-9, 4)
        elif kind == 5:  # around the smallest f16
            x[i] *= np.float32(10.0 ** g.uniform(-9, -5))
        elif kind == 6:  # past the largest
            x[i] *= np.float32(10.0 ** g.uniform(4.5, 38))
            x[i] = np.clip(x[i], -3e38, 3e38)
        elif kind == 7:
            x[i, g.integers(32)] = 10.0 ** g.uniform(0, 6) * g.choice([-1, 1])
        elif kind == 8:
            x[i] = -np.abs(x[i]) * np.float32(10.0 ** g.uniform(-3, 6))
        else:
            x[i] = np.float32(g.choice([0.0, -0.0, 1e-45, 1e-38, 65504, -65504, 65520])) * (np.arange(32) % 2).astype(np.float32)
    return x


def test_append_blocks_where_the_last_bit_decides():
    g = rng(41)
    n, d, ps = 640, 256, 256
    x = hard_blocks(g, 2 * n * d // 32).reshape(2, n, 1, d)
    c = Cache(1, d, ps, 1, -(-n // ps), fill=0x77)
    pos = np.arange(n, dtype=np.int32)
    qg.qkv_append(c.c, cuda(x[0]), cuda(x[1]), cuda(pos))
    got = host(c.pool)
    for t in range(n):
        c.put(0, t, 0, x[0, t, 0], x[1, t, 0])
    bad = np.argwhere(got != c.host)
    assert len(bad) == 0, (len(bad), bad[:5])


def test_append_not_finite():
    """A block with a NaN or an infinity is lost as a whole, and nothing else; a finite one saturates."""
    g = rng(5)
    c = Cache(2, 64, 16, 1, 1)
    k, v = g.standard_normal((2, 5, 2, 64)).astype(np.float32)
    k[0, 0, 3], k[1, 1, 40], v[2, 0, 63], v[3, 1, 0], v[4, 0, 0] = np.nan, np.inf, -np.inf, 1e30, -1e30
    pos = np.arange(5, dtype=np.int32)
    qg.qkv_append(c.c, cuda(k), cuda(v), cuda(pos))
    ko, vo = (torch.empty((5, 2, 64), dtype=torch.float32, device="cuda") for _ in range(2))
    qg.qkv_read(c.c, cuda(pos), ko, vo)
    ko, vo = host(ko), host(vo)
    assert np.isnan(ko[0, 0, :32]).all() and np.isnan(ko[1, 1, 32:]).all() and np.isnan(vo[2, 0, 32:]).all()
    low = np.float32(ref.below(v[3, 1, :32].min()))
    # 1e30 counts as 65504: a range of 65504 to 65508, d the f16 behind 4367 to 4367.2
    assert vo[3, 1, 0] == np.float32(15 * 4368.0 + low) and (vo[3, 1, 1:32] == low).all()
    # m = -65504; the others lie within 4 of 0, so d is the f16 behind 65508 / 15 = 4367.2 (steps of 4): 4368, and they take
    # the quant 15 (65500 / 4368 = 14.9954): 15 * 4368 - 65504 = 16
    assert vo[4, 0, 0] == -65504 and np.abs(v[4, 0, 1:32]).max() < 4 and (vo[4, 0, 1:32] == 16).all()
    assert np.isnan(ko).sum() == 64 and np.isnan(vo).sum() == 32


@pytest.mark.parametrize("d,kv,heads,rot,inter", [(64, 2, 6, 64, False), (128, 8, 40, 128, True), (256, 2, 16, 64, False),
                                                  (128, 1, 3, 20, False), (256, 3, 3, 256, True)])
def test_append_rotated_with_queries(d, kv, heads, rot, inter):
    """One launch: keys rotated into the cache, values as they are, queries rotated to f16; fused rows, seq by default."""
    g = rng(6, d, heads)
    n_seq, each, ps = 3, 4, 32
    n = n_seq * each
    c = Cache(kv, d, ps, n_seq, 2)
    rows = g.standard_normal((n, heads + 2 * kv, d)).astype(np.float32)
    pos = np.tile(np.arange(29, 29 + each, dtype=np.int32), n_seq)
    dev = cuda(rows)
    q_out = torch.full((n, heads, d), float("nan"), dtype=torch.float16, device="cuda")
    qg.qkv_append(c.c, dev[:, heads:heads + kv], dev[:, heads + kv:], cuda(pos), rope=qg.qrope_plan(rot, interleaved=inter),
                  q=dev[:, :heads], q_out=q_out)
    want, size = attn_ref.rotate(rows[:, :heads + kv], pos, attn_ref.thetas(rot, 1e4), inter)
    err = attn_ref.ROT * size
    q = want[:, :heads]
    assert_within(host(q_out), q, err[:, :heads] * (1 + ref.HALF) + ref.HALF * np.abs(q) + ref.SUB, "queries")
    c.host = host(c.pool)
    for t in range(n):
        for h in range(kv):
            (kq, km, _), (vq, vm, _) = c.get(t // each, pos[t], h)
            kw, ke = want[t, heads + h].reshape(-1, 32), err[t, heads + h].reshape(-1, 32)
            # half a step; a step is at most one f16 step above a 15th of the range, which m's rounding down widens by a step of m
            lo, span = kw.min(1), kw.max(1) - kw.min(1) + 2 * ke.max(1)
            d_max = (span + 2 * ref.HALF * np.abs(lo) + 2 * ref.SUB) / 15 * (1 + 2 * ref.HALF) + 2 * ref.SUB
            assert_within(kq + km, kw.reshape(-1), (ke + d_max[:, None] * (0.5 + 15 * 4 * ref.SINGLE)).reshape(-1), "keys")
            vv, vs, vl = ref.quantise(rows[t, heads + kv + h].reshape(-1, 32))
            assert np.array_equal(vq, (vv * vs.astype(np.float64)[:, None]).reshape(-1))
            assert np.array_equal(vm, np.repeat(vl.astype(np.float64), 32))


def test_append_prompt_matches_token_by_token():
    """A prompt written in one call leaves the same bytes as its tokens one by one."""
    n, kv, d, ps = 300, 2, 128, 64
    rows = torch.randn(n, 3 * kv, d, device="cuda")
    plan = qg.qrope_plan(128)
    pos = torch.arange(7, 7 + n, dtype=torch.int32, device="cuda")
    a, b = (Cache(kv, d, ps, 1, 5, seed=3) for _ in range(2))
    args = lambda t: (rows[t, kv:2 * kv], rows[t, 2 * kv:], pos[t])  # noqa: E731
    qa, qb = (torch.empty((n, kv, d), dtype=torch.float16, device="cuda") for _ in range(2))
    qg.qkv_append(a.c, *args(slice(0, n)), rope=plan, q=rows[:, :kv], q_out=qa)
    for t in range(n):
        s = slice(t, t + 1)
        qg.qkv_append(b.c, *args(s), rope=plan, q=rows[s, :kv], q_out=qb[s])
    assert torch.equal(a.pool, b.pool) and torch.equal(qa, qb)


@pytest.mark.parametrize("out", [torch.float16, torch.float32])
@pytest.mark.parametrize("d,kv,ps", [(64, 3, 16), (128, 8, 64), (256, 1, 32), (256, 2, 256)])
def test_read(d, kv, ps, out):
    """Any bytes, f16 NaN and infinities among d and m: q d + m, rounded once."""
    g = rng(7, d, kv)
    c = Cache(kv, d, ps, 2, 2, fill=0)
    c.host[:] = g.integers(0, 256, c.host.size, dtype=np.uint8)
    c.upload()
    n = 29
    seq, pos = g.integers(0, 2, n).astype(np.int32), g.integers(0, 2 * ps, n).astype(np.int32)
    pos[4] = -3
    k, v = (torch.full((n, kv, d), 7.0, dtype=out, device="cuda") for _ in range(2))
    qg.qkv_read(c.c, cuda(pos), k, v, seq=cuda(seq))
    want = np.zeros((2, n, kv, d))
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(n):
            for h in range(kv):
                if pos[t] >= 0:
                    want[:, t, h] = [qd + m for qd, m, _ in c.get(seq[t], pos[t], h)]  # (exact in f64: 4 + 11 bits and 11)
        want = want.astype({torch.float16: np.float16, torch.float32: np.float32}[out])
    for got, w in ((k, want[0]), (v, want[1])):
        np.testing.assert_array_equal(host(got), w)
    only = torch.full((n, kv, d), 7.0, dtype=out, device="cuda")
    qg.qkv_read(c.c, cuda(pos), None, only, seq=cuda(seq))
    assert torch.equal(only.view(torch.int16), v.view(torch.int16))


def test_bad_slots_are_skipped_and_flagged():
    n, kv, d, ps = 6, 2, 64, 16
    c = Cache(kv, d, ps, 2, 3, fill=0x11)
    c.table[1, 2], c.table[0, 1] = -1, 1 << 20
    c.upload()
    seq = np.array([0, 2, -1, 0, 1, 0], np.int32)
    pos = np.array([3, 0, 0, 48, 40, 20], np.int32)
    bits = [0, qg.QG_KV_BAD_SEQ, qg.QG_KV_BAD_SEQ, qg.QG_KV_BAD_POS, qg.QG_KV_BAD_PAGE, qg.QG_KV_BAD_PAGE]
    x = np.ones((n, kv, d), np.float32)
    before = host(c.pool).copy()
    for t in range(n):
        one = slice(t, t + 1)
        for call in ("append", "read"):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            if call == "append":
                qg.qkv_append(c.c, cuda(x[one]), cuda(x[one]), cuda(pos[one]), seq=cuda(seq[one]), err_flag=err)
            else:
                k = torch.full((1, kv, d), 5.0, dtype=torch.float16, device="cuda")
                qg.qkv_read(c.c, cuda(pos[one]), k, torch.empty_like(k), seq=cuda(seq[one]), err_flag=err)
                assert (host(k) == (1 if t == 0 else 0)).all()
            assert int(err) == bits[t], (t, call)
    c.host = before
    for h in range(kv):
        c.put(0, 3, h, x[0, h], x[0, h])
    assert np.array_equal(host(c.pool), c.host)


# ----------------------------------------------------------------- attention
def filled(kv, d, ps, lens, seed, fill=0xFF, extra_pages=0, shift=0.4):
    """A cache whose sequences hold random tokens below lens; every other byte `fill` (NaN d and m)."""
    g = rng(10, seed, d, kv)
    pages = max(1, -(-max(lens) // ps)) + extra_pages
    c = Cache(kv, d, ps, len(lens), pages, seed=seed, fill=fill)
    ks, vs = [], []
    for s, n in enumerate(lens):
        k, v = g.standard_normal((n, kv, d)) * 1.5 + shift, g.standard_normal((n, kv, d)) * 0.7 + 0.1
        parts = np.empty((2, 3, n, kv, d))
        for j in range(n):
            for h in range(kv):
                c.put(s, j, h, k[j, h].astype(np.float32), v[j, h].astype(np.float32))
                parts[:, :, j, h] = c.get(s, j, h)
        ks.append(parts[0])
        vs.append(parts[1])
    c.upload()
    return c, ks, vs


def attend(c, q, lens, window=0, scale=None, ws_fill=0xFF):
    n, ncols, heads, d = q.shape
    y = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    ws = torch.full((qg.qattn_workspace_bytes(c.c, heads, ncols),), ws_fill, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qg.qattn_paged(c.c, cuda(q), cuda(np.array(lens, np.int32)), y, ws, scale=scale, window=window, err_flag=err)
    return host(y), int(err)


def check(kv, heads, d, ps, lens, ncols, window=0, seed=0, size=1.0, extra_pages=0):
    c, ks, vs = filled(kv, d, ps, lens, seed, extra_pages=extra_pages)
    q = (rng(11, seed, heads).standard_normal((len(lens), ncols, heads, d)) * size + 0.1 * size).astype(np.float16)
    y, err = attend(c, q, lens, window)
    want, bound = ref.attention(q, ks, vs, lens, ncols, window, d ** -0.5)
    assert err == 0
    assert_within(y, want, bound, f"{lens} cols {ncols} window {window}")
    return c, q, y


@pytest.mark.parametrize("kv,heads,d", [(1, 1, 64), (2, 16, 256), (8, 40, 128), (3, 9, 64), (2, 14, 128), (1, 6, 256)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 129, 300])
def test_attention_decode_lengths(kv, heads, d, n):
    check(kv, heads, d, 16 if n % 2 else 64, [n], 1, seed=n)


@pytest.mark.parametrize("wide", [0, 2000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_both_ways(d, wide):
    """The same tokens under a narrow table (clusters) and a wide one (runs and a join)."""
    check(2, 10, d, 16, [777, 130], 1, seed=d, extra_pages=wide)


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
def test_attention_ragged_batch(ps):
    """Lengths from nothing to several pages in one call."""
    check(2, 6, 128, ps, [0, 1, 700, 16, 33, 0, 255, 256, 257, 5], 1, seed=ps)


@pytest.mark.parametrize("kv,heads,d", [(2, 10, 64), (1, 7, 128), (2, 4, 256)])
@pytest.mark.parametrize("ncols", [2, 3, 8, 16])
def test_attention_columns(kv, heads, d, ncols):
    """Several new tokens a sequence: causal among themselves; rows before the sequence's start are empty."""
    check(kv, heads, d, 32, [ncols, 1, 0, ncols - 1, 140, 17, 300], ncols, seed=ncols)


@pytest.mark.parametrize("window", [1, 2, 16, 100, 129, 1000])
def test_attention_window(window):
    check(2, 6, 128, 16, [0, 1, 40, 129, 400, 257], 3, window=window, seed=window)


@pytest.mark.parametrize("heads,ncols,d", [(16, 1, 128), (17, 1, 64), (33, 1, 256), (64, 1, 64), (64, 2, 128), (40, 16, 64),
                                           (12, 16, 256)])
def test_attention_many_rows(heads, ncols, d):
    """One key head under many query rows: every row tile, whole and ragged."""
    check(1, heads, d, 64, [200, 90], ncols, seed=heads)


@pytest.mark.parametrize("wide", [0, 2000])
def test_attention_large_scores(wide):
    """Scores of several hundred: one token takes nearly all the weight."""
    check(2, 8, 128, 32, [500, 77], 2, seed=5, size=100.0, extra_pages=wide)


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("step", [0.02, 0.3, -0.3, 3.0])
@pytest.mark.parametrize("d,heads,ncols", [(64, 8, 1), (128, 5, 1), (128, 8, 2), (256, 16, 1), (64, 32, 1)])
def test_attention_rising_scores(d, heads, ncols, step, wide):
    """Scores that rise (or fall) from token to token: the running reference moves again and again, and every sum with it, the
    blocks' m among them."""
    n, lens = 700, [700, 33]
    c, ks, vs = filled(1, d, 16, lens, 17, extra_pages=wide)
    g = rng(18, d)
    for s, n in enumerate(lens):
        for j in range(n):
            k = g.standard_normal(d) * 0.1 + step * j * d ** -0.5
            v = g.standard_normal(d) + 1.5
            c.put(s, j, 0, k.astype(np.float32), v.astype(np.float32))
            ks[s][:, j, 0], vs[s][:, j, 0] = c.get(s, j, 0)
    c.upload()
    q = (1 + 0.1 * g.standard_normal((2, ncols, heads, d))).astype(np.float16)
    y, _ = attend(c, q, lens, scale=1.0)
    want, bound = ref.attention(q, ks, vs, lens, ncols, 0, 1.0)
    assert_within(y, want, bound, f"step {step}")


@pytest.mark.parametrize("size", [1e-4, 1e-2, 1.0, 100.0, 1000.0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_query_sizes(size, d):
    """Queries from f16's subnormals to thousands, one row of each size among others: their blocks' sums as two f16 each."""
    lens, heads, ncols = [150], 6, 2
    c, ks, vs = filled(1, d, 16, lens, 31, shift=2.0)
    q = rng(33, d).standard_normal((1, ncols, heads, d)) + 0.5
    q *= size * 10.0 ** np.arange(-2, heads - 2)[None, None, :, None] if size == 1e-2 else size
    q[0, 1, 2], q[0, 0, 1, :32] = 0, 0
    q = np.clip(q, -60000, 60000).astype(np.float16)
    scale = d ** -0.5 / max(size, 1e-2)
    y, err = attend(c, q, lens, scale=scale)
    want, bound = ref.attention(q, ks, vs, lens, ncols, 0, scale)
    assert err == 0
    assert_within(y, want, bound, f"queries of {size}")


@pytest.mark.parametrize("d", [64, 128])
def test_attention_value_range(d):
    """Values from tiny to near the top of f16 in one sequence, in turn by token and by block of 32."""
    kv, ps, n = 1, 16, 120
    g = rng(21)
    for order in (1, -1):
        c, ks, vs = filled(kv, d, ps, [n], 8)
        for j in range(n):
            size = 10.0 ** (-6 + 10 * j / n) if order > 0 else 10.0 ** (4 - 10 * j / n)
            k, v = g.standard_normal(d) * 0.3, g.standard_normal(d) * np.repeat([size, 1.0], d // 2)
            c.put(0, j, 0, k.astype(np.float32), np.clip(v, -60000, 60000).astype(np.float32))
            ks[0][:, j, 0], vs[0][:, j, 0] = c.get(0, j, 0)
        c.upload()
        q = g.standard_normal((1, 1, 4, d)).astype(np.float16)
        y, _ = attend(c, q, [n])
        want, bound = ref.attention(q, ks, vs, [n], 1, 0, d ** -0.5)
        assert_within(y, want, bound, f"order {order}")


@pytest.mark.parametrize("size", [1e-7, 3e-5, 60000.0])
def test_attention_values_of_one_size(size):
    """All values tiny or near the top of f16: the quants' scales in both f16 factors' range."""
    n, d = 90, 64
    g = rng(22)
    c, ks, vs = filled(1, d, 16, [n], 8)
    for j in range(n):
        k, v = g.standard_normal(d) * 0.3, np.clip(g.standard_normal(d) * 0.3, -1, 1) * size
        c.put(0, j, 0, k.astype(np.float32), v.astype(np.float32))
        ks[0][:, j, 0], vs[0][:, j, 0] = c.get(0, j, 0)
    c.upload()
    q = g.standard_normal((1, 1, 4, d)).astype(np.float16)
    y, _ = attend(c, q, [n])
    want, bound = ref.attention(q, ks, vs, [n], 1, 0, d ** -0.5)
    assert_within(y, want, bound, f"values of {size}")


@pytest.mark.parametrize("where", ["token", "block"])
@pytest.mark.parametrize("large", [60000.0, 300.0])
def test_attention_one_large_value_among_small_ones(where, large):
    """One token, or one block of every token, has values far above the others: the others keep their precision."""
    n, d = 200, 128
    c, ks, vs = filled(1, d, 16, [n], 8)
    g = rng(24)
    for j in range(n):
        k, v = g.standard_normal(d) * 0.3, g.standard_normal(d) * 0.1
        if where == "block":
            v[:32] *= large
        if where == "token" and j == 3:
            v = np.clip(v * 10 * large, -60000, 60000)
            k[:] = -8.0  # and hardly any weight
        c.put(0, j, 0, k.astype(np.float32), v.astype(np.float32))
        ks[0][:, j, 0], vs[0][:, j, 0] = c.get(0, j, 0)
    c.upload()
    q = (np.abs(g.standard_normal((1, 1, 4, d))) * 0.5).astype(np.float16)
    y, _ = attend(c, q, [n])
    want, bound = ref.attention(q, ks, vs, [n], 1, 0, d ** -0.5)
    assert_within(y, want, bound, "one large value")
    rest = slice(32, None) if where == "block" else slice(None)
    assert (bound[..., rest] < 1e-3).all()  # (the values are of 0.1)


@pytest.mark.parametrize("d", [64, 256])
def test_attention_values_past_the_largest_f16(d):
    """Blocks between -65504 and far above 65504, and all above it: what is stored, and the sums of m + 8 d, stay in f16's range."""
    n, kv = 60, 2
    c = Cache(kv, d, 16, 1, 4)
    g = rng(23)
    k, v = g.standard_normal((2, n, kv, d)).astype(np.float32)
    v[0::4, :, :32] *= np.float32(1e6)
    v[1::4, 0], v[2::4, 1] = 1e5, -3e38
    v[3::4, :, 5] = 2e6
    pos = np.arange(n, dtype=np.int32)
    qg.qkv_append(c.c, cuda(k), cuda(v), cuda(pos))
    c.host = host(c.pool)
    ks, vs = np.empty((2, 3, n, kv, d))
    for j in range(n):
        for h in range(kv):
            ks[:, j, h], vs[:, j, h] = c.get(0, j, h)
    assert np.isfinite(vs).all() and np.abs(vs[0] + vs[1]).max() <= 65504 + 131008 * 2.0 ** -10
    q = (g.standard_normal((1, 1, 6, d)) * 0.1).astype(np.float16)
    y, _ = attend(c, q, [n])
    want, bound = ref.attention(q, [ks], [vs], [n], 1, 0, d ** -0.5)
    assert np.isfinite(y).all()
    assert_within(y, want, bound, f"dim {d}")


def test_attention_constant_blocks():
    """Blocks of equal values: d is 0 or nearly so, everything is in m."""
    n, d = 100, 128
    c, ks, vs = filled(1, d, 16, [n], 8)
    g = rng(23)
    for j in range(n):
        k, v = (np.repeat(g.standard_normal(d // 32), 32).astype(np.float32) for _ in range(2))
        if j % 3 == 0:
            k, v = k.astype(np.float16).astype(np.float32), v.astype(np.float16).astype(np.float32)
        c.put(0, j, 0, k, v)
        ks[0][:, j, 0], vs[0][:, j, 0] = c.get(0, j, 0)
    c.upload()
    q = g.standard_normal((1, 2, 4, d)).astype(np.float16)
    y, _ = attend(c, q, [n])
    want, bound = ref.attention(q, ks, vs, [n], 2, 0, d ** -0.5)
    assert_within(y, want, bound, "constant blocks")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_attention_not_finite_where_masked(what, d):
    """A later column's key and value, tokens before the window and past the end: no effect on the rows that do not see
    them; a row that sees one is NaN."""
    kv, heads, ps, ncols, window = 1, 3, 16, 4, 30
    lens = [75, 130]
    c, q, clean = check(kv, heads, d, ps, lens, ncols, window=window, seed=2)
    bad = np.full(d, what, np.float32)
    for s, n in enumerate(lens):
        for j in range(0, n - ncols - window + 1):
            c.put(s, j, 0, bad, bad)
        c.put(s, n - 2, 0, bad, bad)  # column 2's token: columns 0 and 1 do not see it
    c.upload()
    y, _ = attend(c, q, lens, window)
    assert np.array_equal(y[:, :2], clean[:, :2])
    assert np.isnan(y[:, 2:]).all()


@pytest.mark.parametrize("what", ["d", "m"])
@pytest.mark.parametrize("x", [np.nan, np.inf, -np.inf])
def test_attention_value_scale_not_finite_in_one_block(what, x):
    """A value's d or m that is not finite reaches its own block of the rows that see it, no other; an infinite m is one."""
    kv, heads, d, ps = 1, 5, 128, 32
    c, q, clean = check(kv, heads, d, ps, [100], 3, seed=4)
    for j, blk in ((99, 1), (98, 3), (40, 0)):
        off, i = c.where(0, j, 0, True)
        at = off + ref.scale_offset(d, i, blk, True) + (d if what == "m" else 0)
        c.host[at:at + 2] = np.array([x], np.float16).view(np.uint8)
    c.upload()
    y, _ = attend(c, q, [100])
    y, clean = y.reshape(3, heads, 4, 32), clean.reshape(3, heads, 4, 32)
    for col in range(3):
        hit = [0] + [3] * (col >= 1) + [1] * (col >= 2)
        if what == "m" and np.isinf(x):
            assert (y[col][:, hit] == x).all()
        else:
            assert not np.isfinite(y[col][:, hit]).any()
        rest = [b for b in range(4) if b not in hit]
        assert np.array_equal(y[col][:, rest], clean[col][:, rest]), col


def test_attention_bad_pages_and_lengths():
    """Pages outside the pool hold no tokens; a length past the table ends with it; a negative one is empty. Flagged."""
    kv, heads, d, ps, ncols = 2, 6, 64, 16, 2
    lens = [200, 64, 208, 40]
    c, ks, vs = filled(kv, d, ps, lens, 6)
    q = rng(12).standard_normal((4, ncols, heads, d)).astype(np.float16)
    c.table[0, 3], c.table[0, 12], c.table[1, :4] = -1, 1 << 24, -7
    c.upload()
    dead = [set(range(48, 64)) | set(range(192, 208)), set(range(64)), set(), set()]
    y, err = attend(c, q, lens)
    want, bound = ref.attention(q, ks, vs, lens, ncols, 0, d ** -0.5, dead)
    assert err == qg.QG_KV_BAD_PAGE
    assert_within(y, want, bound, "bad pages")
    assert (y[1] == 0).all()
    told = [0, 0, 300, -5]  # the table holds 13 pages of 16
    y, err = attend(c, q, told)
    assert err == qg.QG_KV_BAD_POS
    assert (y[[0, 1, 3]] == 0).all()
    ks[2], vs[2] = ks[2][:, :208], vs[2][:, :208]
    want, bound = ref.attention(q, ks, vs, [0, 0, 300, 0], ncols, 0, d ** -0.5)
    assert_within(y, want, bound, "length past the table")


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0, 1e-30])
@pytest.mark.parametrize("heads,d", [(3, 64), (12, 256)])
def test_attention_any_scale(scale, heads, d):
    """A scale of zero (the mean of the values), a negative, a large and a vanishing one."""
    c, ks, vs = filled(1, d, 16, [70, 3], 9)
    q = rng(14, heads).standard_normal((2, 2, heads, d)).astype(np.float16)
    y, err = attend(c, q, [70, 3], scale=scale)
    want, bound = ref.attention(q, ks, vs, [70, 3], 2, 0, scale)
    assert err == 0
    assert_within(y, want, bound, f"scale {scale}")


def big_reference(c, q, lens, ncols, window=0):
    """(y, bound) by f64 torch on values read back from the cache, for long sequences.

    With a the largest magnitude of a value's block, |m| <= a, 15 d is at most 2 a and a step (q d + m reaches from the smallest to the
    largest), so |q - 8| d <= 8/15 of that and |m + 8 d| (the quant 8, between the smallest and the largest) <= a and a step, 1.2 a. The roundings of different tokens' weights are independent, at
    most h_j = (1.1 + 2 * 1.2) HALF a_j each (attn_ref's and kv4_ref's terms); the sum of n such is within 6 sqrt(sum (w_j h_j)^2) but for one time in 10^7 (Hoeffding). f32 sums as in
    test_parity_attn.big_reference."""
    n, _, heads, d = q.shape
    kv = c.n_kv_heads
    ys, bs = [], []
    for s in range(n):
        L = lens[s]
        if L == 0:
            ys.append(torch.zeros((ncols, heads, d), dtype=torch.float64, device="cuda"))
            bs.append(torch.zeros_like(ys[-1]))
            continue
        pos = torch.arange(L, dtype=torch.int32, device="cuda")
        k, v = (torch.empty((L, kv, d), dtype=torch.float32, device="cuda") for _ in range(2))
        qg.qkv_read(c, pos, k, v, seq=torch.full_like(pos, s))
        k, v = k.double().transpose(0, 1), v.double().transpose(0, 1)
        amp = lambda x: x.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(*x.shape[:-1], d // 32, 32).flatten(-2)  # noqa: E731
        ka, va = amp(k), amp(v)
        qq = q[s].double().view(ncols, kv, heads // kv, d).permute(1, 0, 2, 3).reshape(kv, -1, d)
        sc = qq @ k.transpose(1, 2) / d ** 0.5
        at = torch.arange(ncols, device="cuda").repeat_interleave(heads // kv)[:, None] + L - ncols
        seen = pos[None] <= at
        if window:
            seen &= pos[None] > at - window
        mag = (qq.abs() @ (3.01 * ka).transpose(1, 2) / d ** 0.5).masked_fill(~seen, 0).amax(-1, keepdim=True)
        sc = sc.masked_fill(~seen, -float("inf"))
        top = sc.amax(-1, keepdim=True)
        w = torch.exp(sc - top)
        w = w / w.sum(-1, keepdim=True)
        y = w @ v
        rel = (2 * ((d + 8) * mag + 4 * top.abs()) + 16 + 2 * min(L, 4160)) * ref.SINGLE
        b = rel * (w @ (3.01 * va)) + 6 * ((w * w) @ (3.6 * ref.HALF * va).square()).sqrt() + ref.HALF * y.abs() + ref.SUB + \
            w.amax(-1, keepdim=True) * L * 2.0 ** -28 * va.amax(1, keepdim=True)
        back = lambda t: t.view(kv, ncols, -1, d).permute(1, 0, 2, 3).reshape(ncols, heads, d)  # noqa: E731
        ys.append(back(y))
        bs.append(back(b))
    return torch.stack(ys), torch.stack(bs)


@pytest.mark.parametrize("kv,heads,d,ps,lens,ncols,window", [
    (8, 40, 128, 64, [70001], 1, 0),
    (2, 16, 256, 16, [40000, 123, 9001], 1, 0),
    (4, 32, 64, 128, [5000, 1, 33333, 0, 12345], 8, 0),
    (2, 16, 256, 32, [30011, 17000], 4, 0),
    (1, 12, 64, 256, [50000, 777], 16, 4096),
    (8, 8, 128, 64, [3000] * 40, 1, 0),
    (4, 24, 128, 64, [37 * i % 2100 for i in range(200)], 1, 0),
    (2, 4, 64, 16, [9000, 8999], 2, 777),
])
def test_attention_long(kv, heads, d, ps, lens, ncols, window):
    """Long and many sequences, work split and joined, written through qkv_append; the same bits twice."""
    pages = -(-max(lens) // ps)
    n = len(lens)
    table = torch.randperm(n * pages, device="cuda").to(torch.int32).view(n, pages)
    pool = torch.full((n * pages * qg.qkv_page_bytes(Q4, kv, d, ps),), 0xFF, dtype=torch.uint8, device="cuda")
    c = qg.qkv_cache(Q4, pool, table, kv, d, ps)
    append_random(c, lens)
    g = torch.Generator(device="cuda").manual_seed(kv * d + n)
    q = torch.randn((n, ncols, heads, d), generator=g, device="cuda").half()
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.full((qg.qattn_workspace_bytes(c, heads, ncols),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(q)
    qg.qattn_paged(c, q, lens_d, y, ws, window=window)
    want, bound = big_reference(c, q, lens, ncols, window)
    for s in range(n) if n <= 8 else range(0, n, 7):
        off = (y[s].double() - torch.nan_to_num(want[s])).abs()
        assert (off <= torch.nan_to_num(bound[s], nan=0.0)).all(), (s, lens[s], float(off.max()))
    again = torch.empty_like(q)
    ws.fill_(0x3C)
    qg.qattn_paged(c, q, lens_d, again, ws, window=window)
    assert torch.equal(y, again)


def test_attention_pool_beyond_4_gib():
    """Page offsets past 32 bits: the pages in use lie at the far end of a pool of more than 4 GiB."""
    kv, heads, d, ps = 2, 8, 128, 64
    page = qg.qkv_page_bytes(Q4, kv, d, ps)
    n = (9 << 29) // page
    pool = torch.empty(n * page, dtype=torch.uint8, device="cuda")
    pages = 12
    table = torch.arange(n - pages, n, dtype=torch.int32, device="cuda").flip(0).view(1, pages).contiguous()
    c = qg.qkv_cache(Q4, pool, table, kv, d, ps)
    L = pages * ps - 3
    append_random(c, [L], seed=5)
    q = torch.randn((1, 2, heads, d), device="cuda").half()
    y = torch.empty_like(q)
    ws = torch.empty(qg.qattn_workspace_bytes(c, heads, 2), dtype=torch.uint8, device="cuda")
    qg.qattn_paged(c, q, torch.tensor([L], dtype=torch.int32, device="cuda"), y, ws)
    want, bound = big_reference(c, q, [L], 2)
    assert ((y.double() - want).abs() <= bound).all()


def test_attention_1024_sequences():
    """The most sequences a call takes, of lengths 0 to 40."""
    n, kv, heads, d, ps = 1024, 1, 2, 64, 16
    lens = [(7 * i) % 41 for i in range(n)]
    table = torch.randperm(n * 3, device="cuda").to(torch.int32).view(n, 3)
    pool = torch.full((n * 3 * qg.qkv_page_bytes(Q4, kv, d, ps),), 0xFF, dtype=torch.uint8, device="cuda")
    c = qg.qkv_cache(Q4, pool, table, kv, d, ps)
    seq = torch.tensor([s for s in range(n) for _ in range(lens[s])], dtype=torch.int32, device="cuda")
    pos = torch.tensor([j for s in range(n) for j in range(lens[s])], dtype=torch.int32, device="cuda")
    k, v = torch.randn(2, len(pos), kv, d, device="cuda")
    qg.qkv_append(c, k, v, pos, seq=seq)
    q = torch.randn(n, 1, heads, d, device="cuda").half()
    y = torch.empty_like(q)
    ws = torch.empty(qg.qattn_workspace_bytes(c, heads, 1), dtype=torch.uint8, device="cuda")
    qg.qattn_paged(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), y, ws)
    want, bound = big_reference(c, q, lens, 1)
    assert ((y.double() - want).abs() <= bound).all()


# ------------------------------------------------- streams, graphs, surroundings
def test_decode_steps_in_a_graph_and_on_another_stream():
    """A decode step captured once and replayed with new rows, positions and lengths equals eager steps, bit for bit; so
    does the step on a stream of its own."""
    n_seq, kv, heads, d, ps, pages, start = 3, 2, 8, 128, 16, 12, [0, 40, 111]
    plan = qg.qrope_plan(64)
    table = torch.randperm(n_seq * pages, device="cuda").to(torch.int32).view(n_seq, pages)
    outs = []
    for mode in ("eager", "graph", "stream"):
        pool = torch.full((n_seq * pages * qg.qkv_page_bytes(Q4, kv, d, ps),), 0xFF, dtype=torch.uint8, device="cuda")
        c = qg.qkv_cache(Q4, pool, table, kv, d, ps)
        append_random(c, start, seed=1)
        rows = torch.zeros((n_seq, heads + 2 * kv, d), device="cuda")
        pos, lens = (torch.zeros(n_seq, dtype=torch.int32, device="cuda") for _ in range(2))
        ws = torch.empty(qg.qattn_workspace_bytes(c, heads, 1), dtype=torch.uint8, device="cuda")
        q_out = torch.empty((n_seq, heads, d), dtype=torch.float16, device="cuda")
        y = torch.empty((n_seq, 1, heads, d), dtype=torch.float16, device="cuda")
        graph, side = None, torch.cuda.Stream()
        if mode == "graph":
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(c, plan, rows, pos, heads, kv, lens, ws, q_out, y)
        got = []
        for i in range(5):
            g = torch.Generator(device="cuda").manual_seed(100 + i)
            rows.copy_(torch.randn(rows.shape, generator=g, device="cuda"))
            pos.copy_(torch.tensor([s + i for s in start]))
            lens.copy_(torch.tensor([s + i + 1 for s in start]))
            if mode == "graph":
                graph.replay()
            elif mode == "stream":
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    step(c, plan, rows, pos, heads, kv, lens, ws, q_out, y)
                torch.cuda.current_stream().wait_stream(side)
            else:
                step(c, plan, rows, pos, heads, kv, lens, ws, q_out, y)
            got.append(y.clone())
        outs.append((torch.stack(got), pool))
    for o, p in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(p, outs[0][1])


@pytest.mark.parametrize("d,heads,ncols,lens", [(128, 10, 1, [300, 4]), (64, 6, 3, [1000, 129]), (256, 4, 16, [40, 500])])
def test_guard_bands(d, heads, ncols, lens):
    """Nothing is written outside the outputs and the workspace; inputs keep their bytes."""
    kv, ps, band = 2, 16, 1 << 14
    pages = -(-max(lens) // ps)
    page = qg.qkv_page_bytes(Q4, kv, d, ps)

    def banded(nbytes):
        buf = torch.full((band + nbytes + band,), 0xFF, dtype=torch.uint8, device="cuda")
        return buf, buf[band:band + nbytes]

    def intact(buf):
        return bool((buf[:band] == 0xFF).all() and (buf[-band:] == 0xFF).all())
    pool_buf, pool = banded(2 * pages * page)
    table = torch.randperm(2 * pages, device="cuda").to(torch.int32).view(2, pages)
    c = qg.qkv_cache(Q4, pool, table, kv, d, ps)
    append_random(c, lens)
    assert intact(pool_buf)
    kept = pool.clone()
    q = torch.randn((2, ncols, heads, d), device="cuda").half()
    q_kept = q.clone()
    y_buf, yb = banded(q.numel() * 2)
    ws_buf, ws = banded(qg.qattn_workspace_bytes(c, heads, ncols))
    y = yb.view(torch.float16).view(q.shape)
    qg.qattn_paged(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), y, ws)
    assert intact(y_buf) and intact(ws_buf) and torch.isfinite(y).all()
    assert torch.equal(pool, kept) and torch.equal(q, q_kept)
    pos = torch.arange(min(lens), dtype=torch.int32, device="cuda")
    for out in (torch.float16, torch.float32):
        size = pos.numel() * kv * d * (2 if out == torch.float16 else 4)
        (k_buf, kb), (v_buf, vb) = banded(size), banded(size)
        qg.qkv_read(c, pos, kb.view(out).view(-1, kv, d), vb.view(out).view(-1, kv, d), seq=torch.zeros_like(pos))
        assert intact(k_buf) and intact(v_buf) and torch.isfinite(kb.view(out)).all() and torch.isfinite(vb.view(out)).all()


def test_no_wait_was_given_up():
    torch.cuda.synchronize()
    assert qg.qg_device_error() == 0
