"""Plain 64-bit forms of the norm, the embedding lookup and the routing, for their tests. Shares nothing with the library."""
import numpy as np

from attn_ref import HALF, SINGLE, SUB, f16_up  # noqa: F401


# ------------------------------------------------------------------- matrices
def stored(b):
    """Bytes [..., 16 m] in the library's order: of each 16 the two halves byte by byte."""
    return np.ascontiguousarray(b.reshape(*b.shape[:-1], -1, 2, 8).swapaxes(-1, -2)).reshape(b.shape)


def unstored(b):
    return np.ascontiguousarray(b.reshape(*b.shape[:-1], -1, 8, 2).swapaxes(-1, -2)).reshape(b.shape)


def weights(qtype, q, scl):
    """f64 [rows, k] of a matrix in the library's layout (Q4_0: 2, Q8_0: 8)."""
    b = unstored(q)
    d = scl.view(np.float16).astype(np.float64)[..., None]
    if qtype == 8:
        w = b.view(np.int8).astype(np.float64).reshape(*d.shape[:-1], 32)
    else:
        b = b.reshape(*d.shape[:-1], 16)
        w = np.concatenate([b & 15, b >> 4], -1).astype(np.float64) - 8
    return (w * d).reshape(q.shape[0], -1)


# ----------------------------------------------------------------------- norm
def add_up(x, add):
    """The sum, f32, rounded to x's type."""
    if add is None:
        return x
    with np.errstate(over="ignore", invalid="ignore"):
        return (x.astype(np.float32) + add.astype(np.float32)).astype(x.dtype)


def norm(s, w, w_add, eps):
    """(y, bound of the f32 arithmetic) of stored sums s [..., n], in f64.

    The mean of the squares is off by its sum's rounding: a product and at most 32 additions a thread, 5 in a warp, 32 of warps: 70
    half steps, and 3 for the division, eps and the root's argument; half of that on the root, and 3 more for the root and its
    reciprocal. Two products and w + w_add: 3. In all 43."""
    s = s.astype(np.float64)
    g = (np.ones(s.shape[-1]) if w is None else w.astype(np.float64)) + w_add
    with np.errstate(divide="ignore", invalid="ignore"):
        y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * g
    return y, 43 * SINGLE * np.abs(y) + 2.0 ** -148


# -------------------------------------------------------------------- routing
def behind(v):
    """Sort key of a number: larger first, NaN last."""
    return (1, 0.0) if np.isnan(v) else (0, -v)


def scores(logits, score):
    """p in f64 of f32 logits [E]."""
    x = logits.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-x))
        ok = ~np.isnan(x)
        top = x[ok].max() if ok.any() else -np.inf
        p = np.where(x == top, 1.0, np.exp(x - top))
        p[~ok] = np.nan
        return p / p[ok].sum() if ok.any() else p


def route(logits, bias, topk, score="softmax", n_group=1, top_group=1, group_top=1, renorm=True, scale=1.0):
    """(ids, weights) of one token; a third value: the smallest distance between c that decides about the ids (of two that differ)."""
    p = scores(logits, score)
    c = p + bias.astype(np.float64) if bias is not None else p
    e = len(p)
    near = np.inf

    def pick(values, n):
        nonlocal near
        order = sorted(range(len(values)), key=lambda i: (behind(values[i]), i))
        for a, b in zip(order[:n], order[1:n + 1]):
            d = abs(values[a] - values[b])
            if d > 0:
                near = min(near, d)
        return order[:n]

    open_ = np.ones(e, bool)
    if top_group < n_group:
        size = e // n_group
        worth = []
        for g in range(n_group):
            best = sorted(c[g * size:(g + 1) * size], key=behind)[:group_top]
            worth.append(sum(best))
        open_[:] = False
        for g in pick(worth, top_group):
            open_[g * size:(g + 1) * size] = True
    values = c if bias is not None else logits.astype(np.float64)
    allowed = np.nonzero(open_)[0]
    ids = np.array([allowed[i] for i in pick(values[allowed], topk)])
    w = p[ids]
    if renorm:
        t = w.sum()
        w = w / t if t != 0 else np.zeros_like(w)
    return ids, w * scale, near
