"""The plain forms of the 4-bit cache, held against worked blocks and against their own definition (no GPU)."""
import ctypes as C

import numpy as np
import pytest

import gemm_q4_q8_gb300 as qg
import kv4_ref as ref
from gemm_q4_q8_gb300 import build as qbuild


def test_worked_block():
    """0 to 31 by hand: m = 0, d is the smallest f16 with 15 d >= 31: 31 / 15 = 2.0666..., f16 steps of 2^-9 there, 1059 / 512
    = 2.068359375 (15 times 1058 / 512 is 30.996). Quants round(x / d): 0, 0.48, 0.97, 1.45, 1.93, ..., 14.99."""
    q, d, m = ref.quantise(np.arange(32, dtype=np.float32))
    assert float(m) == 0 and float(d) == 1059 / 512
    assert q.tolist() == [0, 0, 1, 1, 2, 2, 3, 3, 4, 4, 5, 5, 6, 6, 7, 7, 8, 8, 9, 9, 10, 10, 11, 11, 12, 12, 13, 13, 14, 14, 15, 15]


def test_worked_bytes():
    """Elements 0 to 15 twice, d = 1, m = 0: word w holds elements 8w ... 8w + 7."""
    pool = np.zeros(2 * ref.half_bytes(64), np.uint8)
    row = np.tile(np.arange(16, dtype=np.float32), 4)
    ref.write_row(pool, 64, 0, 3, False, row)
    assert pool[48:64].tolist() == [0x40, 0x62, 0x51, 0x73, 0xC8, 0xEA, 0xD9, 0xFB] * 2
    assert pool[512 + 2 * 3 * 2:512 + 2 * 3 * 2 + 4].view(np.float16).tolist() == [1, 1]  # token 3, both blocks
    ref.write_row(pool, 64, 640, 11, True, row + 2)  # token 11 of the values: place 4 * 1 + 1 + 2 = 7
    assert pool[640 + 512:640 + 576].view(np.float16).reshape(2, 16)[:, 7].tolist() == [1, 1]
    assert pool[640 + 576:640 + 640].view(np.float16).reshape(2, 16)[:, 7].tolist() == [2, 2]
    for off, i, is_v, add in ((0, 3, False, 0), (640, 11, True, 2)):
        qd, m, d = ref.read_row(pool, 64, off, i, is_v)
        assert np.array_equal(qd, row) and (m == add).all() and (d == 1).all()


def test_places_are_a_permutation():
    for d in (64, 128, 256):
        for is_v in (False, True):
            at = sorted(ref.scale_offset(d, i, b, is_v) for i in range(16) for b in range(d // 32))
            assert at == list(range(8 * d, 9 * d, 2))
    assert sorted(ref.byte_of(e) for e in range(32)) == sorted((b, s) for b in range(16) for s in (0, 4))


def test_quantised_values_are_near():
    """|x - (q d + m)| <= d / 2 and a rounding of (x - m) / d, for blocks of all sizes that f16 spans."""
    g = np.random.default_rng(1)
    x = (g.standard_normal((4000, 32)) * 10.0 ** g.uniform(-6, 4, (4000, 1)) + 10.0 ** g.uniform(-6, 4, (4000, 1))).astype(np.float32)
    q, d, m = ref.quantise(x)
    d, m = d.astype(np.float64)[:, None], m.astype(np.float64)[:, None]
    assert (m[:, 0] <= x.min(1)).all() and (m[:, 0] + 15 * d[:, 0] >= x.max(1) * (1 - 2.0 ** -23) - 2.0 ** -24 * np.abs(x).max(1)).all()
    assert (np.abs(x - (q * d + m)) <= d * (0.5 + 15 * 2.0 ** -22)).all()


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qg.load()


def test_page_bytes(lib):
    for d in (64, 128, 256):
        for ps in (16, 32, 64, 128, 256):
            for kv in (1, 3, 8, 256):
                assert qg.qkv_page_bytes(qg.Q4_1, kv, d, ps) == kv * (ps // 16) * 2 * ref.half_bytes(d)
    for kv, d, ps in ((0, 64, 16), (257, 64, 16), (1, 96, 16), (1, 64, 8), (1, 64, 48), (1, 64, 512)):
        assert qg.qkv_page_bytes(qg.Q4_1, kv, d, ps) == 0


NULL, SHAPE, ALIGN, TYPE, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 7


def at(i):
    return 0x100000 + i * (1 << 36)


def cache(**kw):
    c = dict(pool=at(1), page_table=at(2), type=3, n_kv_heads=8, head_dim=128, page_size=64, n_pages=10, max_pages=5, n_seq=2)
    c.update(kw)
    return qg.QGKVCache(*[c[f[0]] for f in qg.QGKVCache._fields_])


def calls(lib, c):
    return (lib.qkv_append(c, None, 0, at(3), 1024, at(4), 1024, None, 0, 0, None, at(5), at(6), 4, None, None),
            lib.qkv_read(c, at(5), at(6), 4, 1, at(3), at(4), None, None),
            lib.qattn_paged(c, at(3), 40, 2, at(5), 0, 0.1, at(4), at(6), 1 << 32, None, None))


@pytest.mark.parametrize("kw,status", [(dict(n_kv_heads=0), SHAPE), (dict(head_dim=80), SHAPE), (dict(page_size=24), SHAPE),
                                       (dict(n_pages=0), SHAPE), (dict(n_seq=1025), SHAPE), (dict(max_pages=1 << 25), SHAPE),
                                       (dict(pool=None), NULL), (dict(page_table=None), NULL), (dict(pool=at(1) + 8), ALIGN),
                                       (dict(page_table=at(2) + 2), ALIGN)])
def test_cache_refusals(lib, kw, status):
    assert calls(lib, cache(**kw)) == (status,) * 3


def test_call_refusals(lib):
    """Refusals that depend on the cache's bytes: outputs over a pool of 10 pages, and the attention's workspace."""
    c = cache()
    size = 10 * qg.qkv_page_bytes(3, 8, 128, 64)
    inside = at(1) + size - 16
    assert lib.qkv_append(c, None, 0, inside, 1024, at(4), 1024, None, 0, 0, None, at(5), at(6), 4, None, None) == ALIAS
    assert lib.qkv_read(c, at(5), at(6), 4, 1, inside, at(4), None, None) == ALIAS
    need = lib.qattn_workspace_bytes(2, 40, 8, 128, 2)
    args = lambda y, ws, n: (c, at(3), 40, 2, at(5), 0, 0.1, y, ws, n, None, None)  # noqa: E731
    assert lib.qattn_paged(*args(inside, at(6), need)) == ALIAS
    assert lib.qattn_paged(*args(at(4), at(6), need - 1)) == WORKSPACE and lib.qattn_paged(*args(at(4), None, 0)) == WORKSPACE
    assert lib.qkv_append(c, None, 3, at(3), 1024, at(4), 1024, None, 0, 0, None, at(5), at(6), 4, None, None) == TYPE
    assert lib.qkv_read(c, at(5), at(6), 4, 3, at(3), at(4), None, None) == TYPE


def test_weights_are_not_taken_in_this_type(lib):
    a = (3, at(1), at(2), 64, 64, at(3), 1, None, at(4), None)
    assert lib.qgemm_cols(*a) == TYPE
    assert lib.qrepack(3, at(1), 64, 64, at(2), at(3), None) == TYPE


def test_binding():
    torch = pytest.importorskip("torch")
    table = torch.zeros((2, 5), dtype=torch.int32)
    pool = torch.zeros(10 * qg.qkv_page_bytes(qg.Q4_1, 2, 64, 16), dtype=torch.uint8)
    c = qg.qkv_cache(qg.Q4_1, pool, table, 2, 64, 16)
    assert (c.n_pages, c.max_pages, c.n_seq, c.type) == (10, 5, 2, 3)
    with pytest.raises(ValueError):
        qg.qkv_cache(qg.Q4_1, pool[:-1], table, 2, 64, 16)
    assert C.sizeof(c) == C.sizeof(qg.QGKVCache)
