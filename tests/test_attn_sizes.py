"""Which sizes qattn_paged takes: its kernel numbers units and places in 32 bits. No GPU needed: a call without a workspace is
refused for that, if not for its size."""
import numpy as np
import pytest

import gemm_q4_q8_gb300 as qg
from gemm_q4_q8_gb300 import build as qbuild

SHAPE, WORKSPACE = 2, 5


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qg.load()


def taken(lib, qtype, d, kv, group, ncols, n_seq, max_pages, ps):
    c = qg.QGKVCache(1 << 36, 1 << 40, qtype, kv, d, ps, 10, max_pages, n_seq)
    st = lib.qattn_paged(c, 1 << 44, kv * group, ncols, 1 << 45, 0, 0.1, 1 << 46, None, 0, None, None)
    assert st in (SHAPE, WORKSPACE)
    return st == WORKSPACE


def places(qtype, d, kv, group, ncols, n_seq, max_pages, ps):
    """Units of a sequence's pages (a record of 16 tokens for each of four warps, two where 32 f16 rows of 256 share them) and the
    places behind an item, times the items."""
    rows, most = group * ncols, (8 if d == 64 else 4) // (1 if qtype == qg.QG_F16 else 2)
    nt = 1
    while nt < most and nt * 8 < rows:
        nt *= 2
    unit = 32 if d == 256 and nt == 4 else 64
    return (-(-max_pages * ps // unit) + (2 if nt == 1 else 4)) * n_seq * kv * -(-rows // (8 * nt))


def test_sizes(lib):
    g = np.random.default_rng(3)
    some = {True: 0, False: 0}
    for _ in range(20000):
        qtype, d, ps = int(g.choice([1, 8])), int(g.choice([64, 128, 256])), int(2 ** g.integers(4, 9))
        kv, group, ncols, n_seq = (int(2 ** g.uniform(0, m)) for m in (8, 6, 4, 10))
        # sizes around the border
        border = 2 ** 31 * max(1, ps // 64) / (n_seq * kv * (group * ncols / 8 + 1)) * 64 / ps
        max_pages = int(np.clip(border * 2 ** g.uniform(-2, 2), 1, (2 ** 31 - 1) // ps))
        a = (qtype, d, kv, group, ncols, n_seq, max_pages, ps)
        ok = taken(lib, *a)
        some[ok] += 1
        assert not ok or places(*a) < 2 ** 31, a
        if (max_pages * ps // 32 + 8) * n_seq * kv * (group * ncols // 8 + 1) < 2 ** 31:
            assert ok, a
    assert min(some.values()) > 1000
