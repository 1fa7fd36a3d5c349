"""Q8_0 blocks of the cache where their rounding is decided by the last bit: largest magnitudes at and next to 127 times an
f16 (the scale is the smallest f16 not below a 127th of them), elements at and next to the middle of two quants, over the
whole range from f32 subnormals to blocks too large for an f16 scale. Every value read back must be the exact product of
quant and scale: nothing is tolerated."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_q4_q8_gb300 as qg  # noqa: E402

from test_parity_attn import _lib  # noqa: E402, F401

pytestmark = pytest.mark.gpu

ONE = np.float32(1)


def next_to(x, g):
    """x, or one of its two neighbours in f32."""
    x = x.astype(np.float32)
    up = np.where(g.integers(0, 2, x.shape) == 0, np.nextafter(x, np.float32(np.inf)), np.nextafter(x, np.float32(-np.inf)))
    return np.where(g.integers(0, 3, x.shape) == 0, x, up).astype(np.float32)


def blocks(g, n, low, high):
    """n blocks of 32 whose scales are f16 with bit patterns low .. high - 1."""
    d = g.integers(low, high, n).astype(np.uint16).view(np.float16).astype(np.float64)
    q = g.integers(-126, 127, (n, 32))
    with np.errstate(over="ignore"):
        x = next_to((q + g.choice([0.0, 0.5, -0.5], (n, 32))) * d[:, None], g)
        x[np.arange(n), g.integers(0, 32, n)] = next_to(127 * d, g) * g.choice([-ONE, ONE], n)
    return x


def stored(x):
    """quant * scale of every element, in 64 bits."""
    s = np.abs(x).max(1) / np.float32(127)
    with np.errstate(over="ignore", invalid="ignore"):
        h = s.astype(np.float16)
        h = np.where(h.astype(np.float32) < s, np.nextafter(h, np.float16(np.inf)), h).astype(np.float32)
        h = np.minimum(h, np.float32(65504))[:, None]
        q = np.where(h > 0, np.clip(np.rint(x / np.where(h > 0, h, ONE)), -127, 127), 0)
    return q.astype(np.float64) * h.astype(np.float64)


@pytest.mark.parametrize("low,high", [(0x0001, 0x0400), (0x0400, 0x3C00), (0x3C00, 0x7B00), (0x7B00, 0x7C00)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_blocks_at_the_edges(d, low, high):
    n, kv, ps = 512, 2, 32
    g = np.random.default_rng([d, low])
    rows = [blocks(g, n * kv * d // 32, low, high) for _ in range(2)]
    check(rows, n, kv, d, ps)


def test_blocks_out_of_the_scales_range():
    n, kv, d, ps = 64, 1, 64, 64
    g = np.random.default_rng(9)
    size = (n * kv * d // 32, 32)
    tiny = g.integers(0, 300, size).astype(np.uint32).view(np.float32)  # subnormal: scales of 0 and of the least f16
    tiny[::4] = 0
    large = np.clip(g.standard_normal(size) * 10.0 ** g.uniform(6.5, 38, (size[0], 1)), -3e38, 3e38).astype(np.float32)
    check([tiny, large], n, kv, d, ps)


def check(rows, n, kv, d, ps):
    pool = torch.zeros(n // ps * qg.qkv_page_bytes(qg.Q8_0, kv, d, ps), dtype=torch.uint8, device="cuda")
    table = torch.arange(n // ps, dtype=torch.int32, device="cuda").view(1, -1)
    cache = qg.qkv_cache(qg.Q8_0, pool, table, kv, d, ps)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    qg.qkv_append(cache, *(torch.from_numpy(x).cuda().view(n, kv, d) for x in rows), pos)
    got = [torch.empty((n, kv, d), dtype=torch.float32, device="cuda") for _ in range(2)]
    qg.qkv_read(cache, pos, *got)
    for x, y in zip(rows, got):
        np.testing.assert_array_equal(y.cpu().numpy().reshape(-1, 32).astype(np.float64), stored(x))
