"""Plain 64-bit forms of the rotary, cache and attention calls, for their tests.
Shares nothing with the library: numpy loops over tokens and blocks."""
import numpy as np

F32, F16, Q8_0 = 0, 1, 8
HALF = 2.0 ** -11    # half a step of f16, relative
SUB = 2.0 ** -25     # half a step of f16 subnormals
SINGLE = 2.0 ** -24  # half a step of f32, relative


def thetas(rot, base, factor=1.0, orig=0, low=1.0, high=32.0):
    out = []
    for i in range(rot // 2):
        t = float(base) ** (-2.0 * i / rot)
        if factor != 1.0:
            keep = 0.0
            if orig:
                keep = min(1.0, max(0.0, (orig * t / (2 * np.pi) - low) / (high - low)))
            t = t * keep + t / factor * (1 - keep)
        out.append(t)
    return np.array(out)


def rotate(x, pos, theta, interleaved, mscale=1.0):
    """(y, size) of x [tok, heads, D] in f64; size = the |u| + |v| of each element's pair (0 past rot)."""
    x = np.asarray(x, np.float64)
    y, size = x.copy(), np.zeros_like(x)
    rot = 2 * len(theta)
    for t, p in enumerate(pos):
        for i, th in enumerate(theta):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            # whole turns taken off in extended precision
            turn = np.longdouble(int(p)) * np.longdouble(th) / (2 * np.pi * np.longdouble(1))
            ang = float((turn - np.floor(turn))) * 2 * np.pi
            c, s = np.cos(ang) * mscale, np.sin(ang) * mscale
            u, v = x[t, :, a].copy(), x[t, :, b].copy()
            y[t, :, a], y[t, :, b] = u * c - v * s, u * s + v * c
            size[t, :, a] = size[t, :, b] = (np.abs(u) + np.abs(v)) * abs(mscale)
    return y, size


# The kernel's f32 rotation against 64 bits, in units of mscale (|u| + |v|): the
# angle is off by pi 2^-25 (its conversion to f32), sine and cosine by 2^-24 (one
# ulp below 1), mscale, product and sum each by half an ulp.
ROT = np.pi * 2.0 ** -25 + 4 * SINGLE


def f16_up(x):
    """The smallest f16 not below f32 x >= 0, at most 65504."""
    x = np.float32(x)
    if x >= 65504:
        return np.float16(65504)
    h = np.float16(x)
    return np.nextafter(h, np.float16(np.inf)) if np.float32(h) < x else h


def quantise(x):
    """Q8_0 of f32 x [..., 32]: (int quants, f16 scales), the documented rule."""
    x = np.asarray(x, np.float32)
    q = np.zeros(x.shape, np.int64)
    d = np.zeros(x.shape[:-1], np.float16)
    for at in np.ndindex(*x.shape[:-1]):
        b = x[at]
        if not np.isfinite(b).all():
            d[at] = np.nan
            continue
        d[at] = f16_up(np.float32(np.abs(b).max()) / np.float32(127))
        if d[at] > 0:
            q[at] = np.clip(np.rint(b / np.float32(d[at])), -127, 127).astype(np.int64)
    return q, d


def record_sizes(qtype, d):
    half = 32 * d if qtype == F16 else 17 * d
    return half, 2 * half


def locate(qtype, d, kv, ps, page, head, slot, is_v):
    """Byte offset of a token's half record in the pool, and its place in the group."""
    half, rec = record_sizes(qtype, d)
    return ((page * kv + head) * (ps // 16) + slot // 16) * rec + (half if is_v else 0), slot % 16


def write_row(pool, qtype, d, off, i, row):
    """row [D] (f32) into the half record at byte offset `off`, token i of its group."""
    for b in range(d // 32):
        x = np.asarray(row[32 * b:32 * b + 32], np.float32)
        if qtype == F16:
            with np.errstate(over="ignore"):
                raw = x.astype(np.float16).view(np.uint8)
            at = off + (b * 512 + i * 32) * 2
            pool[at:at + 64] = raw
        else:
            q, s = quantise(x)
            at = off + b * 512 + i * 32
            pool[at:at + 32] = (q + 128).astype(np.uint8)
            at = off + 16 * d + (b * 16 + 4 * (i % 4) + i // 4) * 2
            pool[at:at + 2] = np.array([s], np.float16).view(np.uint8)


def read_row(pool, qtype, d, off, i):
    out = np.empty(d, np.float64)
    for b in range(d // 32):
        if qtype == F16:
            at = off + (b * 512 + i * 32) * 2
            out[32 * b:32 * b + 32] = pool[at:at + 64].view(np.float16)
        else:
            at = off + b * 512 + i * 32
            sc = off + 16 * d + (b * 16 + 4 * (i % 4) + i // 4) * 2
            out[32 * b:32 * b + 32] = (pool[at:at + 32].astype(np.float64) - 128) * \
                float(pool[sc:sc + 2].view(np.float16)[0])
    return out


def attention(q, ks, vs, lens, ncols, window, scale, dead=None):
    """(y, bound) in f64 of q [seq, ncols, heads, D] over ks, vs: per sequence
    [tokens, kv, D] f64. dead[s]: set of positions that do not exist.

    bound: every weight is off by a factor of at most 1 + e with e from the score
    (an f32 dot product of D terms, scaled: (D + 4) half steps of sum |q||k| scale, on
    both the weight and the sum), from exp (8 half steps and the score's size) and from
    its rounding to f16; f32 sums of n terms add n half steps; weights below the f16
    normals are off by 2^-25 of the largest weight instead, and y is rounded once."""
    n, _, heads, d = q.shape
    y = np.zeros(q.shape, np.float64)
    bound = np.zeros(q.shape, np.float64)
    for s in range(n):
        k, v = ks[s], vs[s]
        g = heads // k.shape[1]
        for c in range(ncols):
            p = lens[s] - ncols + c
            if p < 0:
                continue
            lo = max(0, p - window + 1) if window else 0
            at = [j for j in range(lo, min(p + 1, k.shape[0])) if not (dead and j in dead[s])]
            if not at:
                continue
            for h in range(heads):
                kk, vv = k[at, h // g], v[at, h // g]
                qq = q[s, c, h].astype(np.float64)
                sc = kk @ qq * scale
                mag = (np.abs(kk) @ np.abs(qq)).max() * abs(scale)
                top = sc.max()
                w = np.exp(sc - top)
                y[s, c, h] = (w @ vv) / w.sum()
                e_score = (d + 4) * SINGLE * mag + 4 * SINGLE * np.abs(sc).max()
                rel = 2 * e_score + 16 * SINGLE + HALF + 2 * len(at) * SINGLE
                avg = (w @ np.abs(vv)) / w.sum()
                bound[s, c, h] = rel * avg + HALF * np.abs(y[s, c, h]) + SUB + \
                    SUB * np.abs(vv).sum(0) / w.sum()
    return y, bound
