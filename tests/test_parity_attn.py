"""GPU parity of the rotary, cache and attention calls against plain 64-bit forms
(attn_ref.py)."""
import numpy as np
import pytest

import attn_ref as ref
from helpers import assert_within, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gemm_q4_q8_gb300 as qg  # noqa: E402

F16, Q8 = ref.F16, ref.Q8_0
NP = {torch.float32: np.float32, torch.float16: np.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_q4_q8_gb300 import build
    build.build()


def rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


# -------------------------------------------------------------------- rotary
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot,d", [(64, 64), (128, 128), (64, 256), (256, 256), (20, 80), (2, 8), (6, 16), (40, 96), (24, 24)])
def test_rope(rot, d, inter):
    """Layouts, part of the head, odd pair counts, odd head sizes; positions from negative to far."""
    g = rng(1, rot, d)
    pos = np.array([0, 1, 5, 4097, 131071, 2 ** 31 - 1, -1, -2 ** 31], np.int32)
    theta = ref.thetas(rot, 1e6)
    plan = qg.qrope_plan(rot, base=1e6, interleaved=inter)
    for heads in (1, 3, 40):
        x = g.standard_normal((len(pos), heads, d)).astype(np.float32)
        want, size = ref.rotate(x, pos, theta, inter)
        # the plan's frequency is off by 2^-64 of a turn and by the rounding of pow and the division (4 half steps of f64)
        off = 2 * np.pi * np.abs(pos.astype(np.float64)) * (2.0 ** -64 + 4 * 2.0 ** -53 / (2 * np.pi))
        rot_err = (ref.ROT + off[:, None, None]) * size
        for out in (torch.float32, torch.float16):
            y = torch.full((len(pos), heads, d), float("nan"), dtype=out, device="cuda")
            qg.qrope(plan, cuda(x), cuda(pos), y)
            half = ref.HALF * np.abs(want) + ref.SUB if out == torch.float16 else 0
            assert_within(host(y), want, rot_err * (1 + ref.HALF) + half, f"{heads} heads to {out}")


@pytest.mark.parametrize("factor,orig,mscale", [(4.0, 0, 1.0), (8.0, 8192, 1.0), (40.0, 4096, 1.3689)])
def test_rope_scaled(factor, orig, mscale):
    g = rng(2, orig)
    pos = np.array([0, 3, 8191, 100003, 1000003], np.int32)
    x = g.standard_normal((5, 7, 128)).astype(np.float16)
    theta = ref.thetas(128, 5e5, factor, orig, 1.0, 4.0)
    plan = qg.qrope_plan(128, base=5e5, interleaved=True, factor=factor, orig_ctx=orig, low_turns=1.0, high_turns=4.0,
                         mscale=mscale)
    y = torch.empty((5, 7, 128), dtype=torch.float32, device="cuda")
    qg.qrope(plan, cuda(x), cuda(pos), y)
    want, size = ref.rotate(x, pos, theta, True, mscale)
    off = 2 * np.pi * pos * (2.0 ** -64 + 8 * 2.0 ** -53 / (2 * np.pi))
    assert_within(host(y), want, (ref.ROT + off[:, None, None]) * size, "scaled")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("rot,inter", [(128, False), (64, True), (36, False)])
def test_rope_in_place_and_strided(dtype, rot, inter):
    """Inside wider rows: the rest of the rows keeps its bytes; in place equals out of place bit for bit."""
    g = rng(3, rot)
    n, heads, d = 77, 5, 128
    rows = torch.from_numpy(g.standard_normal((n, (heads + 4) * d)).astype(NP[dtype])).cuda()
    keep = rows.clone()
    pos = cuda((g.integers(0, 200000, n)).astype(np.int32))
    plan = qg.qrope_plan(rot, interleaved=inter)
    x = rows[:, 2 * d:(2 + heads) * d].view(n, heads, d)
    y = torch.empty((n, heads, d), dtype=dtype, device="cuda")
    qg.qrope(plan, x, pos, y)
    qg.qrope(plan, x, pos, x)
    assert torch.equal(x, y)
    assert torch.equal(rows[:, :2 * d], keep[:, :2 * d]) and torch.equal(rows[:, (2 + heads) * d:], keep[:, (2 + heads) * d:])
    want, size = ref.rotate(host(keep)[:, 2 * d:(2 + heads) * d].reshape(n, heads, d), host(pos),
                            ref.thetas(rot, 1e4), inter)
    half = ref.HALF * np.abs(want) + ref.SUB if dtype == torch.float16 else 0
    assert_within(host(y), want, (ref.ROT + 1e-9) * size * (1 + ref.HALF) + half, "strided")


def test_rope_many_tokens():
    """More tokens than warps in flight, against f64 torch."""
    n, heads, d = 20011, 3, 64
    x = torch.randn(n, heads, d, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).contiguous()
    y = torch.empty_like(x)
    qg.qrope(qg.qrope_plan(64), x, pos, y)
    a = pos.double()[:, None, None] * torch.from_numpy(ref.thetas(64, 1e4)).cuda()
    u, v = x[..., :32].double(), x[..., 32:].double()
    want = torch.cat([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos()], -1)
    size = (u.abs() + v.abs()).repeat(1, 1, 2)
    assert ((y.double() - want).abs() <= (ref.ROT + 1e-10) * size).all()


# ------------------------------------------------------------ cache, written
class Cache:
    """A cache on the GPU with shuffled pages, every byte of its pool set at the start."""

    def __init__(self, qtype, kv, d, ps, n_seq, max_pages, seed=0, fill=0xFF, spare=2):
        g = rng(9, seed, d, ps)
        self.qtype, self.kv, self.d, self.ps, self.n_seq = qtype, kv, d, ps, n_seq
        n = n_seq * max_pages + spare
        self.table = g.permutation(n)[:n_seq * max_pages].reshape(n_seq, max_pages).astype(np.int32)
        self.host = np.full(n * qg.qkv_page_bytes(qtype, kv, d, ps), fill, np.uint8)
        self.upload()

    def upload(self):
        self.pool = cuda(self.host)
        self.c = qg.qkv_cache(self.qtype, self.pool, cuda(self.table), self.kv, self.d, self.ps)

    def put(self, seq, pos, head, k, v):
        for row, is_v in ((k, False), (v, True)):
            off, i = ref.locate(self.qtype, self.d, self.kv, self.ps, int(self.table[seq, pos // self.ps]), head,
                                pos % self.ps, is_v)
            ref.write_row(self.host, self.qtype, self.d, off, i, row)

    def get(self, seq, pos, head):
        out = []
        for is_v in (False, True):
            off, i = ref.locate(self.qtype, self.d, self.kv, self.ps, int(self.table[seq, pos // self.ps]), head,
                                pos % self.ps, is_v)
            out.append(ref.read_row(self.host, self.qtype, self.d, off, i))
        return out


def odd_rows(g, n, kv, d):
    """Rows with zero blocks, tiny, huge and one-sided blocks among ordinary ones."""
    x = g.standard_normal((n, kv, d)).astype(np.float32)
    flat = x.reshape(-1, 32)
    for i in range(flat.shape[0]):
        flat[i] *= [1, 1, 1, 0, 1e-7, 3e-5, 1e3, 60000, 1e-3][i % 9]
        if i % 11 == 0:
            flat[i, 5] = -abs(flat[i]).max() * 4
    return np.clip(x, -65000, 65000)


@pytest.mark.parametrize("src", [torch.float32, torch.float16])
@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("d,kv,ps", [(64, 1, 16), (64, 5, 32), (128, 8, 64), (256, 2, 128), (256, 3, 16), (128, 3, 256)])
def test_append_bytes(qtype, d, kv, ps, src):
    """Without rotation every byte of the pool is known: the written slots, and all others unchanged."""
    g = rng(4, d, kv, ps)
    c = Cache(qtype, kv, d, ps, 3, 3, seed=ps, fill=0xA5)
    n = 23
    slots = g.permutation(3 * 3 * ps)[:n]
    seq, pos = (slots // (3 * ps)).astype(np.int32), (slots % (3 * ps)).astype(np.int32)
    pos[[3, 17]] = [-1, -2 ** 31]  # padding
    k, v = odd_rows(g, n, kv, d).astype(NP[src]), odd_rows(g, n, kv, d).astype(NP[src])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qg.qkv_append(c.c, cuda(k), cuda(v), cuda(pos), seq=cuda(seq), err_flag=err)
    for t in range(n):
        if pos[t] >= 0:
            for h in range(kv):
                c.put(seq[t], pos[t], h, k[t, h], v[t, h])
    assert np.array_equal(host(c.pool), c.host)
    assert int(err) == 0


@pytest.mark.parametrize("qtype", [F16, Q8])
def test_append_not_finite(qtype):
    g = rng(5, qtype)
    c = Cache(qtype, 2, 64, 16, 1, 1)
    k, v = g.standard_normal((2, 4, 2, 64)).astype(np.float32)
    k[0, 0, 3], k[1, 1, 40], v[2, 0, 63], v[3, 1, 0] = np.nan, np.inf, -np.inf, 1e30
    pos = np.arange(4, dtype=np.int32)
    qg.qkv_append(c.c, cuda(k), cuda(v), cuda(pos))
    ko, vo = (torch.empty((4, 2, 64), dtype=torch.float32, device="cuda") for _ in range(2))
    qg.qkv_read(c.c, cuda(pos), ko, vo)
    ko, vo = host(ko), host(vo)
    if qtype == Q8:  # the whole block of 32 is lost, and nothing else; a finite one saturates
        assert np.isnan(ko[0, 0, :32]).all() and np.isnan(ko[1, 1, 32:]).all() and np.isnan(vo[2, 0, 32:]).all()
        assert vo[3, 1, 0] == 127 * 65504 and (vo[3, 1, 1:32] == 0).all()
        assert np.isnan(ko).sum() == 64 and np.isnan(vo).sum() == 32
    else:
        assert np.isnan(ko[0, 0, 3]) and ko[1, 1, 40] == np.inf and vo[2, 0, 63] == -np.inf and vo[3, 1, 0] == np.inf
        assert np.isnan(ko).sum() == 1 and np.isinf(ko).sum() == 1 and np.isinf(vo).sum() == 2


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("d,kv,heads,rot,inter", [(64, 2, 6, 64, False), (128, 8, 40, 128, True), (256, 2, 16, 64, False),
                                                  (128, 1, 3, 20, False), (256, 3, 3, 256, True)])
def test_append_rotated_with_queries(qtype, d, kv, heads, rot, inter):
    """One launch: keys rotated into the cache, values as they are, queries rotated to f16; fused rows, seq by default."""
    g = rng(6, d, heads)
    n_seq, each, ps = 3, 4, 32
    n = n_seq * each
    c = Cache(qtype, kv, d, ps, n_seq, 2)
    rows = g.standard_normal((n, heads + 2 * kv, d)).astype(np.float32)
    pos = np.tile(np.arange(29, 29 + each, dtype=np.int32), n_seq)
    dev = cuda(rows)
    q_out = torch.full((n, heads, d), float("nan"), dtype=torch.float16, device="cuda")
    qg.qkv_append(c.c, dev[:, heads:heads + kv], dev[:, heads + kv:], cuda(pos), rope=qg.qrope_plan(rot, interleaved=inter),
                  q=dev[:, :heads], q_out=q_out)
    want, size = ref.rotate(rows[:, :heads + kv], pos, ref.thetas(rot, 1e4), inter)
    err = ref.ROT * size
    q = want[:, :heads]
    assert_within(host(q_out), q, err[:, :heads] * (1 + ref.HALF) + ref.HALF * np.abs(q) + ref.SUB, "queries")
    c.host = host(c.pool)
    for t in range(n):
        for h in range(kv):
            k, v = c.get(t // each, pos[t], h)
            kw, ke, vw = want[t, heads + h], err[t, heads + h], rows[t, heads + kv + h].astype(np.float64)
            if qtype == F16:
                assert_within(k, kw, ke * (1 + ref.HALF) + ref.HALF * np.abs(kw) + ref.SUB, "keys")
                assert np.array_equal(v, vw.astype(np.float16).astype(np.float64))
            else:
                # half a quant, of a scale at most one f16 step above amax / 127
                top = (np.abs(kw) + ke).reshape(-1, 32).max(1) / 127
                d_max = np.repeat(top * (1 + 2 * ref.HALF) * (1 + 4 * ref.SINGLE) + 2 * ref.SUB, 32)
                assert_within(k, kw, ke + 0.5 * d_max * (1 + 128 * 4 * ref.SINGLE), "keys")
                qv, sv = ref.quantise(vw.reshape(-1, 32))
                assert np.array_equal(v, (qv * sv.astype(np.float64)[:, None]).reshape(-1))


@pytest.mark.parametrize("qtype", [F16, Q8])
def test_append_prompt_matches_token_by_token(qtype):
    """A prompt written in one call leaves the same bytes as its tokens one by one."""
    n, kv, d, ps = 300, 2, 128, 64
    rows = torch.randn(n, 3 * kv, d, device="cuda")
    plan = qg.qrope_plan(128)
    pos = torch.arange(7, 7 + n, dtype=torch.int32, device="cuda")
    a, b = (Cache(qtype, kv, d, ps, 1, 5, seed=3) for _ in range(2))
    args = lambda t: (rows[t, kv:2 * kv], rows[t, 2 * kv:], pos[t])  # noqa: E731
    qa, qb = (torch.empty((n, kv, d), dtype=torch.float16, device="cuda") for _ in range(2))
    qg.qkv_append(a.c, *args(slice(0, n)), rope=plan, q=rows[:, :kv], q_out=qa)
    for t in range(n):
        s = slice(t, t + 1)
        qg.qkv_append(b.c, *args(s), rope=plan, q=rows[s, :kv], q_out=qb[s])
    assert torch.equal(a.pool, b.pool) and torch.equal(qa, qb)


# --------------------------------------------------------------- cache, read
@pytest.mark.parametrize("out", [torch.float16, torch.float32])
@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("d,kv,ps", [(64, 3, 16), (128, 8, 64), (256, 1, 32), (256, 2, 256)])
def test_read(qtype, d, kv, ps, out):
    g = rng(7, d, kv)
    c = Cache(qtype, kv, d, ps, 2, 2, fill=0)
    c.host[:] = g.integers(0, 256, c.host.size, dtype=np.uint8)  # any bytes: f16 NaN and infinities among them
    c.upload()
    n = 29
    seq, pos = g.integers(0, 2, n).astype(np.int32), g.integers(0, 2 * ps, n).astype(np.int32)
    pos[4] = -3
    k, v = (torch.full((n, kv, d), 7.0, dtype=out, device="cuda") for _ in range(2))
    qg.qkv_read(c.c, cuda(pos), k, v, seq=cuda(seq))
    want = np.zeros((2, n, kv, d))
    for t in range(n):
        for h in range(kv):
            if pos[t] >= 0:
                want[:, t, h] = c.get(seq[t], pos[t], h)
    with np.errstate(over="ignore", invalid="ignore"):
        want = want.astype(NP[out])
    for got, w in ((k, want[0]), (v, want[1])):
        np.testing.assert_array_equal(host(got), w)
    only = torch.full((n, kv, d), 7.0, dtype=out, device="cuda")
    qg.qkv_read(c.c, cuda(pos), None, only, seq=cuda(seq))
    assert torch.equal(only.view(torch.int16), v.view(torch.int16))


def test_bad_slots_are_skipped_and_flagged():
    """Sequences, positions and pages outside the cache: nothing written, zeros read, the reason flagged."""
    n, kv, d, ps = 6, 2, 64, 16
    c = Cache(F16, kv, d, ps, 2, 3, fill=0x11)
    c.table[1, 2], c.table[0, 1] = -1, 1 << 20
    c.upload()
    seq = np.array([0, 2, -1, 0, 1, 0], np.int32)
    pos = np.array([3, 0, 0, 48, 40, 20], np.int32)
    bits = [0, qg.QG_KV_BAD_SEQ, qg.QG_KV_BAD_SEQ, qg.QG_KV_BAD_POS, qg.QG_KV_BAD_PAGE, qg.QG_KV_BAD_PAGE]
    x = np.ones((n, kv, d), np.float32)
    before = host(c.pool).copy()
    for t in range(n):
        for call in ("append", "read"):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            one = slice(t, t + 1)
            if call == "append":
                qg.qkv_append(c.c, cuda(x[one]), cuda(x[one]), cuda(pos[one]), seq=cuda(seq[one]), err_flag=err)
            else:
                k = torch.full((1, kv, d), 5.0, dtype=torch.float16, device="cuda")
                qg.qkv_read(c.c, cuda(pos[one]), k, torch.empty_like(k), seq=cuda(seq[one]), err_flag=err)
                assert (host(k) == (1 if t == 0 else 0)).all()
            assert int(err) == bits[t], (t, call)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qg.qkv_append(c.c, cuda(x), cuda(x), cuda(pos), seq=cuda(seq), err_flag=err)
    assert int(err) == 7
    qg.qkv_append(c.c, cuda(x), cuda(x), cuda(pos), seq=cuda(seq))  # no flag wanted
    c.host = before
    for h in range(kv):
        c.put(0, 3, h, x[0, h], x[0, h])
    assert np.array_equal(host(c.pool), c.host)


# ----------------------------------------------------------------- attention
def filled(qtype, kv, d, ps, lens, seed, fill=0xFF, extra_pages=0):
    """A cache whose sequences hold random tokens below lens; every other byte `fill` (NaN scales and values)."""
    g = rng(10, seed, d, kv)
    pages = max(1, -(-max(lens) // ps)) + extra_pages
    c = Cache(qtype, kv, d, ps, len(lens), pages, seed=seed, fill=fill)
    ks, vs = [], []
    for s, n in enumerate(lens):
        k, v = g.standard_normal((n, kv, d)) * 1.5, g.standard_normal((n, kv, d)) * 0.7 + 0.1
        for j in range(n):
            for h in range(kv):
                c.put(s, j, h, k[j, h].astype(np.float32), v[j, h].astype(np.float32))
                k[j, h], v[j, h] = c.get(s, j, h)
        ks.append(k)
        vs.append(v)
    c.upload()
    return c, ks, vs


def attend(c, q, lens, window=0, scale=None, ws_fill=0xFF):
    n, ncols, heads, d = q.shape
    y = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    ws = torch.full((qg.qattn_workspace_bytes(c.c, heads, ncols),), ws_fill, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qg.qattn_paged(c.c, cuda(q), cuda(np.array(lens, np.int32)), y, ws, scale=scale, window=window, err_flag=err)
    return host(y), int(err)


def check(qtype, kv, heads, d, ps, lens, ncols, window=0, seed=0, size=1.0):
    c, ks, vs = filled(qtype, kv, d, ps, lens, seed)
    q = (rng(11, seed, heads).standard_normal((len(lens), ncols, heads, d)) * size).astype(np.float16)
    y, err = attend(c, q, lens, window)
    want, bound = ref.attention(q, ks, vs, lens, ncols, window, d ** -0.5)
    assert err == 0
    assert_within(y, want, bound, f"{lens} cols {ncols} window {window}")
    return c, q, y


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("kv,heads,d", [(1, 1, 64), (2, 16, 256), (8, 40, 128), (3, 9, 64), (2, 14, 128), (1, 6, 256)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 129, 300])
def test_attention_decode_lengths(qtype, kv, heads, d, n):
    check(qtype, kv, heads, d, 16 if n % 2 else 64, [n], 1, seed=n)


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
def test_attention_ragged_batch(qtype, ps):
    """Lengths from nothing to several pages in one call."""
    check(qtype, 2, 6, 128, ps, [0, 1, 700, 16, 33, 0, 255, 256, 257, 5], 1, seed=ps)


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("kv,heads,d", [(2, 10, 64), (1, 7, 128), (2, 4, 256)])
@pytest.mark.parametrize("ncols", [2, 3, 8, 16])
def test_attention_columns(qtype, kv, heads, d, ncols):
    """Several new tokens a sequence: causal among themselves; rows before the sequence's start are empty."""
    check(qtype, kv, heads, d, 32, [ncols, 1, 0, ncols - 1, 140, 17, 300], ncols, seed=ncols)


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 129, 1000])
def test_attention_window(qtype, window):
    check(qtype, 2, 6, 64, 16, [0, 1, 40, 129, 400, 257], 3, window=window, seed=window)


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("heads,ncols,d", [(16, 1, 128), (17, 1, 64), (33, 1, 256), (64, 1, 64), (64, 2, 128), (40, 16, 64),
                                           (12, 16, 256)])
def test_attention_many_rows(qtype, heads, ncols, d):
    """One key head under many query rows: every row tile, whole and ragged."""
    check(qtype, 1, heads, d, 64, [200, 90], ncols, seed=heads)


@pytest.mark.parametrize("qtype", [F16, Q8])
def test_attention_large_scores(qtype):
    """Scores of several hundred: one token takes nearly all the weight."""
    check(qtype, 2, 8, 128, 32, [500, 77], 2, seed=5, size=100.0)


@pytest.mark.parametrize("qtype", [F16, Q8])
def test_attention_value_range(qtype):
    """Values from tiny to near the top of f16 in one sequence, in turn by token and by block of 32."""
    kv, d, ps, n = 1, 64, 16, 120
    g = rng(21, qtype)
    for order in (1, -1):
        c, ks, vs = filled(qtype, kv, d, ps, [n], 8)
        for j in range(n):
            size = 10.0 ** (-6 + 10 * j / n) if order > 0 else 10.0 ** (4 - 10 * j / n)
            k, v = g.standard_normal(d) * 0.3, g.standard_normal(d) * np.repeat([size, 1.0], 32)
            c.put(0, j, 0, k.astype(np.float32), np.clip(v, -60000, 60000).astype(np.float32))
            ks[0][j, 0], vs[0][j, 0] = c.get(0, j, 0)
        c.upload()
        q = g.standard_normal((1, 1, 4, d)).astype(np.float16)
        y, _ = attend(c, q, [n])
        want, bound = ref.attention(q, ks, vs, [n], 1, 0, d ** -0.5)
        # a weight times its block's scale is rounded to f16: at most 2^-25 of the largest scale seen
        bound += ref.SUB * np.abs(vs[0]).max(0)[0] * n
        assert_within(y, want, bound, f"order {order}")


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_attention_not_finite_where_masked(qtype, what):
    """A later column's key and value, tokens before the window and past the end: no effect on the rows that do not see
    them; a row that sees a NaN is NaN."""
    kv, heads, d, ps, ncols, window = 1, 3, 64, 16, 4, 30
    lens = [75, 130]
    c, q, clean = check(qtype, kv, heads, d, ps, lens, ncols, window=window, seed=2)
    bad = np.full(d, what, np.float32)
    for s, n in enumerate(lens):
        for j in range(0, n - ncols - window + 1):
            c.put(s, j, 0, bad, bad)
        c.put(s, n - 2, 0, bad, bad)  # column 2's token: columns 0 and 1 do not see it
    c.upload()
    y, _ = attend(c, q, lens, window)
    assert np.array_equal(y[:, :2], clean[:, :2])
    if np.isnan(what):
        assert np.isnan(y[:, 2:]).all()


def test_attention_value_not_finite_in_one_dimension():
    """f16: an infinite or NaN value element reaches its own dimension of the rows that see it, no other."""
    kv, heads, d, ps = 1, 5, 128, 32
    c, q, clean = check(F16, kv, heads, d, ps, [100], 3, seed=4)
    for j, e, x in ((99, 5, np.inf), (98, 77, np.nan), (40, 127, -np.inf)):
        off, i = ref.locate(F16, d, kv, ps, int(c.table[0, j // ps]), 0, j % ps, True)
        at = off + ((e // 32) * 512 + i * 32 + e % 32) * 2
        c.host[at:at + 2] = np.array([x], np.float16).view(np.uint8)
    c.upload()
    y, _ = attend(c, q, [100])
    assert (y[0, :, :, 127] == -np.inf).all()
    assert np.isnan(y[0, 1:, :, 77]).all() and (y[0, 2, :, 5] == np.inf).all()
    same = np.ones((3, d), bool)
    same[:, 127], same[1:, 77], same[2, 5] = False, False, False
    for col in range(3):
        assert np.array_equal(y[0, col][:, same[col]], clean[0, col][:, same[col]]), col


@pytest.mark.parametrize("qtype", [F16, Q8])
def test_attention_bad_pages_and_lengths(qtype):
    """Pages outside the pool hold no tokens; a length past the table ends with it; a negative one is empty. Flagged."""
    kv, heads, d, ps, ncols = 2, 6, 64, 16, 2
    lens = [200, 64, 208, 40]
    c, ks, vs = filled(qtype, kv, d, ps, lens, 6)
    q = rng(12).standard_normal((4, ncols, heads, d)).astype(np.float16)
    c.table[0, 3], c.table[0, 12], c.table[1, :4] = -1, 1 << 24, -7
    c.upload()
    dead = [set(range(48, 64)) | set(range(192, 208)), set(range(64)), set(), set()]
    y, err = attend(c, q, lens)
    want, bound = ref.attention(q, ks, vs, lens, ncols, 0, d ** -0.5, dead)
    assert err == qg.QG_KV_BAD_PAGE
    assert_within(y, want, bound, "bad pages")
    assert (y[1] == 0).all()
    # the table holds 13 pages of 16
    told = [0, 0, 300, -5]
    y, err = attend(c, q, told)
    assert err == qg.QG_KV_BAD_POS
    assert (y[[0, 1, 3]] == 0).all()
    ks[2], vs[2] = ks[2][:208], vs[2][:208]
    want, bound = ref.attention(q, ks, vs, [0, 0, 300, 0], ncols, 0, d ** -0.5)
    assert_within(y, want, bound, "length past the table")


def test_attention_spare_table_entries_are_not_read():
    """Entries past the last token's page may hold anything."""
    c, ks, vs = filled(F16, 2, 64, 16, [20, 33], 7, extra_pages=6)
    c.table[0, 2:], c.table[1, 3:] = 1 << 30, -9
    c.upload()
    q = rng(13).standard_normal((2, 1, 4, 64)).astype(np.float16)
    y, err = attend(c, q, [20, 33])
    want, bound = ref.attention(q, ks, vs, [20, 33], 1, 0, 0.125)
    assert err == 0
    assert_within(y, want, bound, "spare entries")


def big_reference(c, q, lens, ncols, window=0):
    """(y, bound) by f64 torch on values read back from the cache, for long sequences."""
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
        qq = q[s].double().view(ncols, kv, heads // kv, d).permute(1, 0, 2, 3).reshape(kv, -1, d)
        sc = qq @ k.transpose(1, 2) / d ** 0.5
        at = torch.arange(ncols, device="cuda").repeat_interleave(heads // kv)[:, None] + L - ncols
        seen = pos[None] <= at
        if window:
            seen &= pos[None] > at - window
        mag = (qq.abs() @ k.abs().transpose(1, 2) / d ** 0.5).masked_fill(~seen, 0).amax(-1, keepdim=True)
        sc = sc.masked_fill(~seen, -float("inf"))
        top = sc.amax(-1, keepdim=True)
        w = torch.exp(sc - top)
        l = w.sum(-1, keepdim=True)
        y = w @ v / l
        # as in attn_ref.attention; f32 sums over at most 64 partial sums of runs of at most 4,096 terms
        rel = 2 * ((d + 4) * mag + 4 * top.abs()) * ref.SINGLE + 16 * ref.SINGLE + ref.HALF + \
            2 * min(L, 4160) * ref.SINGLE
        b = rel * (w @ v.abs() / l) + ref.HALF * y.abs() + ref.SUB + ref.SUB * v.abs().sum(1, keepdim=True) / l
        back = lambda t: t.view(kv, ncols, -1, d).permute(1, 0, 2, 3).reshape(ncols, heads, d)  # noqa: E731
        ys.append(back(y))
        bs.append(back(b))
    return torch.stack(ys), torch.stack(bs)


def append_random(c, lens, scale=1.0, seed=0):
    """Random tokens through qkv_append."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for s, n in enumerate(lens):
        for at in range(0, n, 32768):
            m = min(32768, n - at)
            kv = torch.randn((m, 2 * c.n_kv_heads, c.head_dim), generator=g, device="cuda") * scale
            pos = torch.arange(at, at + m, dtype=torch.int32, device="cuda")
            qg.qkv_append(c, kv[:, :c.n_kv_heads], kv[:, c.n_kv_heads:], pos, seq=torch.full_like(pos, s))


@pytest.mark.parametrize("qtype,kv,heads,d,ps,lens,ncols,window", [
    (Q8, 8, 40, 128, 64, [70001], 1, 0),
    (F16, 2, 16, 256, 16, [40000, 123, 9001], 1, 0),
    (F16, 4, 32, 64, 128, [5000, 1, 33333, 0, 12345], 8, 0),
    (Q8, 2, 16, 256, 32, [30011, 17000], 4, 0),
    (Q8, 1, 12, 64, 256, [50000, 777], 16, 4096),
    (F16, 8, 8, 128, 64, [3000] * 40, 1, 0),
    (Q8, 4, 24, 128, 64, [37 * i % 2100 for i in range(200)], 1, 0),
])
def test_attention_long(qtype, kv, heads, d, ps, lens, ncols, window):
    """Long and many sequences, work split and joined, written through qkv_append; the same bits twice."""
    pages = -(-max(lens) // ps)
    n = len(lens)
    table = torch.randperm(n * pages, device="cuda").to(torch.int32).view(n, pages)
    pool = torch.full((n * pages * qg.qkv_page_bytes(qtype, kv, d, ps),), 0xFF, dtype=torch.uint8, device="cuda")
    c = qg.qkv_cache(qtype, pool, table, kv, d, ps)
    append_random(c, lens)
    q = torch.randn((n, ncols, heads, d), device="cuda").half()
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.full((qg.qattn_workspace_bytes(c, heads, ncols),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(q)
    qg.qattn_paged(c, q, lens_d, y, ws, window=window)
    pick = range(n) if n <= 8 else range(0, n, 7)
    want, bound = big_reference(c, q, lens, ncols, window)
    for s in pick:
        off = (y[s].double() - torch.nan_to_num(want[s])).abs()
        assert (off <= torch.nan_to_num(bound[s], nan=0.0)).all(), (s, lens[s], float(off.max()))
    again = torch.empty_like(q)
    ws.fill_(0x3C)
    qg.qattn_paged(c, q, lens_d, again, ws, window=window)
    assert torch.equal(y, again)


def test_attention_pool_beyond_4_gib():
    """Page offsets past 32 bits: the pages in use lie at the far end of a pool of more than 4 GiB."""
    kv, heads, d, ps = 2, 8, 128, 64
    page = qg.qkv_page_bytes(F16, kv, d, ps)
    n = (9 << 29) // page
    pool = torch.empty(n * page, dtype=torch.uint8, device="cuda")
    pages = 12
    table = torch.arange(n - pages, n, dtype=torch.int32, device="cuda").flip(0).view(1, pages).contiguous()
    c = qg.qkv_cache(F16, pool, table, kv, d, ps)
    L = pages * ps - 3
    append_random(c, [L], seed=5)
    q = torch.randn((1, 2, heads, d), device="cuda").half()
    y = torch.empty_like(q)
    ws = torch.empty(qg.qattn_workspace_bytes(c, heads, 2), dtype=torch.uint8, device="cuda")
    qg.qattn_paged(c, q, torch.tensor([L], dtype=torch.int32, device="cuda"), y, ws)
    want, bound = big_reference(c, q, [L], 2)
    assert ((y.double() - want).abs() <= bound).all()


# ------------------------------------------------- streams, graphs, surroundings
def step(c, plan, rows, pos, heads, kv, lens, ws, q_out, y):
    qg.qkv_append(c, rows[:, heads:heads + kv], rows[:, heads + kv:], pos, rope=plan, q=rows[:, :heads], q_out=q_out)
    qg.qattn_paged(c, q_out.view(c.n_seq, -1, heads, c.head_dim), lens, y, ws)


@pytest.mark.parametrize("qtype", [F16, Q8])
def test_decode_steps_in_a_graph_and_on_another_stream(qtype):
    """A decode step captured once and replayed with new rows, positions and lengths equals eager steps, bit for bit; so
    does the step on a stream of its own."""
    n_seq, kv, heads, d, ps, pages, start = 3, 2, 8, 128, 16, 12, [0, 40, 111]
    plan = qg.qrope_plan(64)
    table = torch.randperm(n_seq * pages, device="cuda").to(torch.int32).view(n_seq, pages)
    size = n_seq * pages * qg.qkv_page_bytes(qtype, kv, d, ps)
    outs = []
    for mode in ("eager", "graph", "stream"):
        pool = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        c = qg.qkv_cache(qtype, pool, table, kv, d, ps)
        append_random(c, start, seed=1)
        rows = torch.zeros((n_seq, heads + 2 * kv, d), device="cuda")
        pos = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
        lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
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


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("d,heads,ncols,lens", [(128, 10, 1, [300, 4]), (64, 6, 3, [1000, 129]), (256, 4, 16, [40, 500])])
def test_guard_bands(qtype, d, heads, ncols, lens):
    """Nothing is written outside the outputs and the workspace; inputs keep their bytes."""
    kv, ps, band = 2, 16, 1 << 14
    pages = -(-max(lens) // ps)
    page = qg.qkv_page_bytes(qtype, kv, d, ps)

    def banded(nbytes):
        buf = torch.full((band + nbytes + band,), 0xFF, dtype=torch.uint8, device="cuda")
        return buf, buf[band:band + nbytes]

    def intact(buf):
        return bool((buf[:band] == 0xFF).all() and (buf[-band:] == 0xFF).all())
    pool_buf, pool = banded(2 * pages * page)
    table = torch.randperm(2 * pages, device="cuda").to(torch.int32).view(2, pages)
    c = qg.qkv_cache(qtype, pool, table, kv, d, ps)
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
    k_buf, kb = banded(pos.numel() * kv * d * 2)
    v_buf, vb = banded(pos.numel() * kv * d * 2)
    qg.qkv_read(c, pos, kb.view(torch.float16).view(-1, kv, d), vb.view(torch.float16).view(-1, kv, d),
                seq=torch.zeros_like(pos))
    assert intact(k_buf) and intact(v_buf) and torch.isfinite(kb.view(torch.float16)).all()
    x = torch.randn((5, 3, d), device="cuda")
    r_buf, rb = banded(x.numel() * 4)
    qg.qrope(qg.qrope_plan(d), x, pos[:5].repeat(5)[:5].contiguous(), rb.view(torch.float32).view(x.shape))
    assert intact(r_buf) and torch.isfinite(rb.view(torch.float32)).all()
    qo_buf, qo = banded(x.numel() * 2)
    qg.qkv_append(c, x[:2, :kv], x[:2, :kv], torch.tensor([0, min(lens) - 1], dtype=torch.int32, device="cuda"),
                  rope=qg.qrope_plan(d), q=x[:2], q_out=qo[:2 * 3 * d * 2].view(torch.float16).view(2, 3, d))
    assert intact(qo_buf) and intact(pool_buf)


# ------------------------------------------------- scale, many sequences, threads
@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0, 1e-30])
@pytest.mark.parametrize("heads,d", [(3, 64), (12, 256)])
def test_attention_any_scale(qtype, scale, heads, d):
    """A scale of zero (the mean of the values), a negative, a large and a vanishing one."""
    c, ks, vs = filled(qtype, 1, d, 16, [70, 3], 9)
    q = rng(14, heads).standard_normal((2, 2, heads, d)).astype(np.float16)
    y, err = attend(c, q, [70, 3], scale=scale)
    want, bound = ref.attention(q, ks, vs, [70, 3], 2, 0, scale)
    assert err == 0
    assert_within(y, want, bound, f"scale {scale}")


def test_attention_1024_sequences():
    """The most sequences a call takes, of lengths 0 to 40."""
    n, kv, heads, d, ps = 1024, 1, 2, 64, 16
    lens = [(7 * i) % 41 for i in range(n)]
    pages = 3
    table = torch.randperm(n * pages, device="cuda").to(torch.int32).view(n, pages)
    pool = torch.full((n * pages * qg.qkv_page_bytes(F16, kv, d, ps),), 0xFF, dtype=torch.uint8, device="cuda")
    c = qg.qkv_cache(F16, pool, table, kv, d, ps)
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


def test_no_wait_was_given_up():
    """After all calls of this file the device error word is 0."""
    torch.cuda.synchronize()
    assert qg.qg_device_error() == 0
