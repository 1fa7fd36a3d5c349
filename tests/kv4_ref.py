"""Plain forms of the 4-bit cache (Q4_1 blocks) and of attention over it, for its tests. Shares nothing with the library: numpy,
from the formulas and the documented layout."""
import numpy as np

from attn_ref import HALF, SINGLE, SUB

F16 = np.float16


def below(x):
    """The largest f16 not above f32 x, at least -65504."""
    x = np.asarray(x, np.float32)
    with np.errstate(over="ignore"):
        h = x.astype(F16)
        h = np.where(h.astype(np.float32) > x, np.nextafter(h, F16(-np.inf)), h)
    return np.clip(h, F16(-65504), F16(65504))


def step_of(r):
    """The smallest f16 h >= 0 with 15 h >= r of f32 r, at most 65504."""
    r = np.maximum(np.asarray(r, np.float32).astype(np.float64), 0)
    h = np.minimum(r / 15, 65504).astype(F16)
    with np.errstate(over="ignore"):
        h = np.where(15 * h.astype(np.float64) < r, np.nextafter(h, F16(np.inf)), h)
    lower = np.nextafter(h, F16(0))
    h = np.where((h > 0) & (15 * lower.astype(np.float64) >= r), lower, h)
    return np.minimum(h, F16(65504))


def quantise(x):
    """(q, d, m) of f32 x [..., 32]: whole numbers 0 to 15, f16, f16. The documented rule in f32 operations."""
    x = np.asarray(x, np.float32)
    bad = ~np.isfinite(x).all(-1)
    x = np.clip(np.where(bad[..., None], np.float32(0), x), np.float32(-65504), np.float32(65504))
    m = below(x.min(-1))
    d = step_of(x.max(-1) - m.astype(np.float32))
    m32, d32 = m.astype(np.float32)[..., None], d.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(d32 > 0, np.clip(np.rint((x - m32) / d32), 0, 15), 0).astype(np.int64)
    return np.where(bad[..., None], 0, q), np.where(bad, F16(np.nan), d), np.where(bad, F16(0), m)


def half_bytes(d):
    return 10 * d


def offset(d, kv, ps, page, head, slot, is_v):
    """Byte offset of a token's half record, and its number in the group."""
    rec = 2 * half_bytes(d)
    return ((page * kv + head) * (ps // 16) + slot // 16) * rec + (half_bytes(d) if is_v else 0), slot % 16


def byte_of(e):
    """(byte of a block's 16, shift) of element e."""
    u = e % 8
    return 4 * (e // 8) + (0, 2, 1, 3)[u % 4], 4 * (u // 4)


def scale_offset(d, i, blk, is_v):
    """Byte offset in a half of token i's d of a block; its m lies d bytes behind."""
    place = blk * 16 + 4 * (i % 8 // 2) + i % 2 + 2 * (i // 8) if is_v else i * (d // 32) + blk
    return 8 * d + 2 * place


BYTES, SHIFTS = (np.array(a) for a in zip(*(byte_of(e) for e in range(32))))


def write_row(pool, d, off, i, is_v, row):
    q, dd, m = quantise(np.asarray(row, np.float32).reshape(-1, 32))
    for b in range(d // 32):
        at = off + b * 256 + i * 16
        got = np.zeros(16, np.uint8)
        np.bitwise_or.at(got, BYTES, (q[b] << SHIFTS).astype(np.uint8))
        pool[at:at + 16] = got
        at = off + scale_offset(d, i, b, is_v)
        for k, s in ((0, dd[b]), (d, m[b])):
            pool[at + k:at + k + 2] = np.array([0x7FFF if np.isnan(s) else s.view(np.uint16)], np.uint16).view(np.uint8)


def read_row(pool, d, off, i, is_v):
    """(q d, m, d) of a token's row, f64 [D] each."""
    qd, mm, dd = np.empty(d), np.empty(d), np.empty(d)
    for b in range(d // 32):
        at = off + b * 256 + i * 16
        q = (pool[at:at + 16][BYTES] >> SHIFTS) & 15
        at = off + scale_offset(d, i, b, is_v)
        s, m = (float(pool[at + k:at + k + 2].view(F16)[0]) for k in (0, d))
        at = slice(32 * b, 32 * b + 32)
        qd[at], mm[at], dd[at] = q * s, m, s
    return qd, mm, dd


def attention(q, ks, vs, lens, ncols, window, scale, dead=None):
    """(y, bound) in f64 of q [seq, ncols, heads, D]. ks, vs: per sequence (q d, m, d), each [tokens, kv, D]. dead[s]: positions
    that do not exist.

    bound, with A = sum |Q| (q d + |m|) of a token: its score is an f32 sum of D products, with the blocks' sums of queries as two
    f16 each (2^-22 of them): (D + 8) half steps of f32 of the largest A, scaled; as in attn_ref.attention that is on the weight
    and on the sum, with 16 half steps for the exponential. Values are taken as (q - 8) d + (m + 8 d): a weight times d is rounded
    to f16, so is m + 8 d, and so is the weight that it meets: half a step of |q - 8| d and two of |m + 8 d|. Weights far below their
    run's largest are off by 2^-32 of it, products with d by 2^-30 of the largest weight times the largest d (times |q - 8|). f32 sums of n
    terms add n half steps to numerator and sum; y is rounded once."""
    n, _, heads, d = q.shape
    y = np.zeros(q.shape, np.float64)
    bound = np.zeros(q.shape, np.float64)
    for s in range(n):
        (kq, km, _), (vq, vm, vd) = ks[s], vs[s]
        g = heads // kq.shape[1]
        for c in range(ncols):
            p = lens[s] - ncols + c
            if p < 0:
                continue
            lo = max(0, p - window + 1) if window else 0
            at = [j for j in range(lo, min(p + 1, kq.shape[0])) if not (dead and j in dead[s])]
            if not at:
                continue
            for h in range(heads):
                k1, k2, v1, v2, v3 = (a[at, h // g] for a in (kq, km, vq, vm, vd))
                qq = q[s, c, h].astype(np.float64)
                sc = (k1 + k2) @ qq * scale
                mag = ((k1 + np.abs(k2)) @ np.abs(qq)).max() * abs(scale)
                w = np.exp(sc - sc.max())
                w /= w.sum()
                y[s, c, h] = w @ (v1 + v2)
                e_score = (d + 8) * SINGLE * mag + 4 * SINGLE * np.abs(sc).max()
                rel = 2 * e_score + 16 * SINGLE + 2 * len(at) * SINGLE
                a, c8 = np.abs(v1 - 8 * v3), np.abs(v2 + 8 * v3)
                bound[s, c, h] = rel * (w @ (a + c8)) + 1.01 * HALF * (w @ a) + 2.01 * HALF * (w @ c8) + HALF * np.abs(y[s, c, h]) + \
                    SUB * (1 + w.sum()) + w.max() * (2.0 ** -32 * c8.sum(0) + 8 * len(at) * 2.0 ** -30 * np.nanmax(vd[np.isfinite(vd)]))
    return y, bound
