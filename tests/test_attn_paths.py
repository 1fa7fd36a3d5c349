"""The two ways attention is done, by what a sequence's pages can hold: a cluster for each (sequence, kv head, row tile) where
that is little, runs over the whole machine and a second kernel where it is much. The same tokens go through both, once with a
table of just their pages and once with a wide one, against the plain 64-bit form; and lengths far below what a narrow table
holds, so that CTAs of a cluster have nothing to do."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref as ref  # noqa: E402
from test_parity_attn import F16, Q8, _lib, assert_within, attend, filled, rng  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("wide", [0, 300])
@pytest.mark.parametrize("kv,heads,d,lens,ncols,window", [
    (2, 16, 256, [300], 1, 0), (1, 5, 64, [1, 700, 0, 64], 1, 0), (4, 4, 128, [129, 33], 2, 0), (2, 8, 128, [500, 65], 4, 0),
    (1, 4, 256, [200, 3], 4, 0), (3, 9, 64, [700, 90], 1, 100), (2, 2, 128, [600], 3, 17), (1, 1, 64, [17] * 40, 1, 0),
    (1, 20, 128, [257], 1, 0)])
def test_both_ways(qtype, wide, kv, heads, d, lens, ncols, window):
    c, ks, vs = filled(qtype, kv, d, 16, lens, seed=wide + d, extra_pages=wide)
    q = rng(21, heads, d).standard_normal((len(lens), ncols, heads, d)).astype(np.float16)
    y, err = attend(c, q, lens, window)
    want, bound = ref.attention(q, ks, vs, lens, ncols, window, d ** -0.5)
    assert err == 0
    assert_within(y, want, bound, f"{lens} cols {ncols} window {window} wide {wide}")


@pytest.mark.parametrize("qtype", [F16, Q8])
@pytest.mark.parametrize("bad", [-1, 10 ** 9])
def test_bad_page_and_length_in_a_cluster(qtype, bad):
    """A page outside the pool takes its tokens away, in any CTA's share; a length past the table is flagged."""
    kv, heads, d, ps, n = 2, 4, 128, 16, 700
    c, ks, vs = filled(qtype, kv, d, ps, [n], seed=5)
    q = rng(22).standard_normal((1, 1, heads, d)).astype(np.float16)
    for page in (0, 20, 43):
        table = c.c.tensors[1]
        keep = int(table[0, page])
        table[0, page] = bad
        y, err = attend(c, q, [n])
        table[0, page] = keep
        assert err == 4
        seen = np.ones(n, bool)
        seen[page * ps:(page + 1) * ps] = False
        k, v = ks[0][seen], vs[0][seen]
        want, bound = ref.attention(q, [k], [v], [len(k)], 1, 0, d ** -0.5)
        assert_within(y, want, bound, f"page {page}")
    y, err = attend(c, q, [10 ** 6])
    assert err == 2
