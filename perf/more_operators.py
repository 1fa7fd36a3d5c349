"""What a decoder layer with routed experts does around its products, measured: the embedding lookup, the root-mean-square
norm with the residual's addition, the key/value cache held in 4 bits and the attention over it, the routing to experts.

A case names one operator ("op") and its sizes. ``prepare`` makes what a serving loop holds in hand: hidden states, tables
and matrices, the pool of cache pages, the page table, the lengths, plans. ``run`` is one pass: the plain form in elementary
torch operations where ``own`` is false, the library's calls where it is true. Both read and write the same bytes.

4-bit blocks (Q4_1, 32 elements of one token's head, value q d + m): m is the largest f16 not above the smallest element,
d the smallest f16 with 15 d >= largest - m, q the integer nearest to (x - m) / d.
Pool layout (bytes): [page][kv head][group of 16 tokens] records; a record is the key half, then the value half. A half:
[D/32][16 tokens][16 bytes] quants, then its 16 D/32 f16 d, then as many m. Byte 4w + b of a block's quants holds element
8w + (0, 2, 1, 3)[b] in its low bits and the element 4 behind that in its high bits. d and m of the keys are stored by
[token][D/32], those of the values by [D/32][16], token i at place 4 (i mod 8 div 2) + i mod 2 + 2 (i div 8).

Matrix layout: quants by row, in every 16-byte group stored byte 2 i + h is byte i + 8 h of the block (Q4_0: byte j holds
elements j and j + 16, value (q - 8) d; Q8_0: int8 q, value q d), f16 scales [row][k/32].
"""
import math

import torch

own = False

F16, F32, Q8, Q4 = "f16", "f32", "q8_0", "q4_0"
_KIND = {F16: torch.float16, F32: torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token looked up in a 5,120-wide table, for the first layer
        dict(name="embed 1 token q4_0", op="embed", type=Q4, rows=248320, k=5120, ntok=1, scale=1.0, dst=F32),
        # a prompt's tokens looked up in the matrix that is the LM head, too
        dict(name="embed 4095 q8_0", op="embed", type=Q8, rows=248320, k=2048, ntok=4095, scale=1.0, dst=F32),
        # one decoded token: the attention's output joins the residual, the norm feeds the next product
        dict(name="norm 1 token", op="norm", ntok=1, heads=1, n=5120, src=F32, add=True, dst=F16, w_add=0.0, eps=1e-6),
        # the same for a prompt
        dict(name="norm prompt", op="norm", ntok=8191, heads=1, n=5120, src=F32, add=True, dst=F16, w_add=0.0, eps=1e-6),
        # an index of embeddings: final hidden states normed to Q8_0 rows, as the Q8_0 products take them, and looked up
        dict(name="norm index q8_0", op="norm", ntok=20011, heads=1, n=2048, src=F16, add=False, dst=Q8, w_add=1.0, eps=1e-5),
        # a prompt of two sequences written to the 4-bit cache (queries rotated on the way) and read back, ragged against
        # pages and groups
        dict(name="append prompt", op="append", seqs=2, ntok=16382, heads=40, kv=8, dim=128, page=64, rot=128,
             inter=False, base=1e6, first=5),
        # one token for one user, a short history: latency
        dict(name="attn 1x1 of 1000", op="attn", seqs=1, cols=1, heads=16, kv=2, dim=256, page=16, short=1000, long=1000,
             window=0),
        # one token for one user over a very long history: what a 4-bit cache is for
        dict(name="attn 1x1 of 262143", op="attn", seqs=1, cols=1, heads=40, kv=8, dim=128, page=64, short=262143,
             long=262143, window=0),
        # a serving batch of ragged lengths, one token each
        dict(name="attn 64x1 ragged", op="attn", seqs=64, cols=1, heads=40, kv=8, dim=128, page=64, short=130, long=16383,
             window=0),
        # speculative verify: 4 new tokens a sequence, small heads, sliding window
        dict(name="attn 8x4 window", op="attn", seqs=8, cols=4, heads=32, kv=8, dim=64, page=32, short=700, long=16001,
             window=4096),
        # one decoded token through the router of 256 experts: sigmoid scores, a bias for balance, 4 of 8 groups, top 8
        dict(name="route 1 token", op="route", ntok=1, hidden=2048, experts=256, k=8, score="sigmoid", bias=True,
             groups=8, keep=4, best=2, renorm=True, scale=2.5),
        # a prompt's logits routed
        dict(name="route prompt", op="route", ntok=16383, hidden=0, experts=256, k=8, score="sigmoid", bias=True,
             groups=8, keep=4, best=2, renorm=True, scale=2.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "norm", "norm", "append", "attn", "attn", "attn", "route", "route"])
    case = dict(op=op)
    shrink = "ntok"
    if op == "embed":
        k = 32 * _log(rng, 2, 160)
        case.update(type=rng.choice([Q4, Q8, F16]), k=k, rows=_log(rng, 1000, min(248320, 500_000_000 // k)),
                    ntok=_log(rng, 1, 16384), scale=rng.choice([1.0, math.sqrt(k)]), dst=rng.choice([F16, F32]))
    elif op == "norm":
        dst = rng.choice([F16, F16, F32, Q8])
        heads = rng.choice([1, 1, 2, 8, 40])
        n = _log(rng, 64, 8192) if heads == 1 else rng.choice([64, 80, 128, 256])
        if dst == Q8:
            n = max(32, n // 32 * 32)
        elif rng.random() < 0.7:
            n = n // 8 * 8
        case.update(ntok=_log(rng, 1, 32768), heads=heads, n=n, src=rng.choice([F16, F32]), add=rng.random() < 0.5, dst=dst,
                    w_add=rng.choice([0.0, 1.0]), eps=rng.choice([1e-6, 1e-5]))
    elif op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 8, 512 // groups)
        keep = rng.randint(1, groups)
        fused = rng.random() < 0.5
        case.update(ntok=rng.randint(1, 16) if fused else _log(rng, 1, 32768), hidden=8 * _log(rng, 16, 640) if fused else 0,
                    experts=experts, k=rng.randint(1, min(8, keep * (experts // groups))),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups, keep=keep,
                    best=rng.choice([1, 2]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
        if fused:
            shrink = "hidden"
    else:
        dim = rng.choice([64, 128, 256])
        kv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        seqs = _log(rng, 1, 64)
        case.update(seqs=seqs, kv=kv, heads=kv * group, dim=dim, page=rng.choice([16, 32, 64, 128]))
        if op == "append":
            case.update(rot=rng.choice([dim, dim // 2, dim // 4]), inter=rng.random() < 0.5,
                        base=rng.choice([1e4, 5e5, 1e6, 1e7]), first=_log(rng, 1, 200000) - 1,
                        ntok=seqs * _log(rng, 1, 16382))
        else:
            long = _log(rng, 1, 262143)
            case.update(cols=rng.choice([1, 1, 1, 2, 3, 4, 8]), long=long, short=_log(rng, 1, long),
                        window=rng.choice([0, 0, 0, 1000]))
            shrink = "long"
    most = [work(c) for c in listed() if c["op"] == op]
    while any(work(case)[w] > max(m[w] for m in most) for w in ("bytes", "flops")):
        if shrink == "long":
            case["long"] = max(1, case["long"] * 3 // 4)
            case["short"] = min(case["short"], case["long"])
        elif shrink == "hidden":
            case["hidden"] = max(8, case["hidden"] * 3 // 32 * 8)
            if case["hidden"] == 8:
                case["ntok"] = max(1, case["ntok"] // 2)
        else:
            each = case["ntok"] // case.get("seqs", 1)
            case["ntok"] = max(1, each * 3 // 4) * case.get("seqs", 1)
    return case


def _lens(case):
    """Tokens of each sequence, the new ones among them: spread from short to long over their logarithm."""
    n, lo, hi = case["seqs"], case["short"], case["long"]
    at = [((b * 0.6180339887498949) % 1.0) for b in range(n)]
    got = [int(round(lo * (hi / lo) ** x)) for x in at]
    got[-1] = hi
    return got


def _visible(case):
    """(keys read, (query, key) pairs) of an attention case, per head."""
    keys = pairs = 0
    for n in _lens(case):
        lows = []
        for t in range(case["cols"]):
            p = n - case["cols"] + t
            if p < 0:
                continue
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            lows.append(lo)
            pairs += p + 1 - lo
        if lows:
            keys += n - min(lows)
    return keys, pairs


_BYTES = {F32: 4.0, F16: 2.0, Q8: 34 / 32, Q4: 18 / 32}


def work(case):
    op = case["op"]
    if op == "embed":
        n = case["ntok"] * case["k"]
        return {"bytes": n * (_BYTES[case["type"]] + _BYTES[case["dst"]]) + 4 * case["ntok"], "flops": 2 * n}
    if op == "norm":  # Q8_0 rows are looked up again, as f16
        n = case["ntok"] * case["heads"] * case["n"]
        moved = _BYTES[case["src"]] * (3 if case["add"] else 1) + _BYTES[case["dst"]]
        if case["dst"] == Q8:
            moved += _BYTES[Q8] + 2
        return {"bytes": n * moved + 4 * case["n"], "flops": n * (5 + (4 if case["dst"] == Q8 else 0))}
    if op == "route":
        n, e = case["ntok"], case["experts"]
        got = 8 * n * case["k"] + (4 * e if case["bias"] else 0)
        if case["hidden"]:
            return {"bytes": got + 4 * e * case["hidden"] + 2 * n * case["hidden"], "flops": 2 * n * e * case["hidden"] + 8 * n * e}
        return {"bytes": got + 4 * n * e, "flops": 8 * n * e}
    d = case["dim"]
    stored = 20 / 32 * 2 * case["kv"] * d  # one token, keys and values
    if op == "append":  # rows of f32 in; the token's cache bytes written, then read back as f16
        n = case["ntok"]
        q = n * case["heads"] * d
        kvs = n * 2 * case["kv"] * d
        return {"bytes": q * (4 + 2) + kvs * (4 + 2) + 2 * n * stored + 8 * n,
                "flops": 3 * n * (case["heads"] + case["kv"]) * case["rot"] + 5 * kvs}
    keys, pairs = _visible(case)
    rows = case["seqs"] * case["cols"] * case["heads"]
    return {"bytes": keys * stored + rows * d * 4 + 4 * case["seqs"], "flops": 4.0 * d * pairs * case["heads"]}


# ------------------------------------------------------------- data in hand
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _bits(h):
    return h.contiguous().view(torch.int16)


def _f16(b):
    return b.to(torch.int16).view(torch.float16)


def _quantise4(x):
    """Q4_1 of f32 [..., 32]: (quants, d, m)."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    m = lo.half()
    b = _bits(m).int()
    down = torch.where(m == 0, torch.full_like(b, -32767), torch.where(b < 0, b + 1, b - 1))  # the f16 below
    m = _f16(torch.where(m.float() > lo, down, b)).float()
    r = hi - m
    d = (r / 15).half()
    b = _bits(d).int()
    b = torch.where(d.float() * 15 < r, b + 1, b)
    b = torch.where((b > 0) & (_f16((b - 1).clamp(min=0)).float() * 15 >= r), b - 1, b)
    d = _f16(b).float()
    q = torch.where(d > 0, torch.round((x - m) / d).clamp(0, 15), torch.zeros_like(x))
    return q, d, m


def _nibbles(q):
    """Bytes [..., 16] of quants [..., 32]."""
    q = q.to(torch.uint8).unflatten(-1, (4, 2, 4))[..., [0, 2, 1, 3]]
    return (q[..., 0, :] | (q[..., 1, :] << 4)).flatten(-2)


def _elements(b):
    """Quants [..., 32] of bytes [..., 16]."""
    b = b.unflatten(-1, (4, 4))[..., [0, 2, 1, 3]]
    return torch.stack([b & 15, b >> 4], -2).flatten(-3)


def _places(device):
    """The place of each of a group's 16 tokens among the values' d and m."""
    i = torch.arange(16, device=device)
    return (i % 8) // 2 * 4 + i % 2 + 2 * (i // 8)


def _pack(case, k, v, stale):
    """Pool bytes of keys and values f32 [pages, kv, page, D]; tokens marked in `stale` hold bytes of all ones."""
    n, h, ps, d = k.shape
    halves = []
    for x, is_v in ((k, False), (v, True)):
        q, dd, m = _quantise4(x.view(n, h, ps // 16, 16, d // 32, 32))  # [n, h, group, token, block, 32]
        old = stale.view(n, 1, ps // 16, 16, 1, 1)
        q = torch.where(old, torch.full_like(q, 15), q)
        quants = _nibbles(q).transpose(3, 4).flatten(3)
        parts = [quants]
        for s in (dd, m):
            s = torch.where(old, torch.full_like(_bits(s.half()), -1), _bits(s.half())).squeeze(-1)
            if is_v:
                t = torch.empty_like(s)
                t[:, :, :, _places(s.device)] = s
                s = t.transpose(3, 4)
            parts.append(s.contiguous().view(torch.uint8).flatten(3))
        halves.append(torch.cat(parts, -1))
    return torch.stack(halves, 3).flatten(1).contiguous()


def _pages(case, g, ends, first=0):
    """(page table, number of pages, first position of each page or -1, its sequence): pages in shuffled order, two spare.
    Positions before `first` belong to pages of another pool (-1 here)."""
    ps = case["page"]
    skip = first // ps
    need = [-(-e // ps) - skip for e in ends]
    wide, total = max(max(need), 1) + skip, sum(need)
    order = torch.randperm(total + 2, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(ends), wide), -1, dtype=torch.int32)
    start = torch.full((total + 2,), -1, dtype=torch.int64)
    owner = torch.zeros(total + 2, dtype=torch.int64)
    at = 0
    for b, n in enumerate(need):
        ids = order[at:at + n]
        table[b, skip:skip + n] = ids
        start[ids.long()] = (skip + torch.arange(n)) * ps
        owner[ids.long()] = b
        at += n
    return table.cuda(), total + 2, start.cuda(), owner.cuda()


def _filled(case, g, lens):
    """A pool whose sequences hold keys and values of tokens below `lens`; stale bytes elsewhere."""
    h, d, ps = case["kv"], case["dim"], case["page"]
    table, n, start, owner = _pages(case, g, lens)
    # channels of unlike size and mean, as keys have them, and values of unlike size by head
    chan, mean = torch.exp(0.6 * _randn(g, 1, h, 1, d)), _randn(g, 1, h, 1, d)
    v_size = torch.exp(0.5 * _randn(g, 1, h, 1, 1))
    lens = torch.tensor(lens, device="cuda")
    pool = []
    for a in range(0, n, 4096):  # a part at a time: the pool is packed far smaller than its values
        z = min(n, a + 4096)
        k = (_randn(g, z - a, h, ps, d) + 0.5 * mean) * chan
        v = _randn(g, z - a, h, ps, d) * v_size
        pos = start[a:z, None] + torch.arange(ps, device="cuda")
        stale = (start[a:z, None] < 0) | (pos >= lens[owner[a:z]][:, None])
        pool.append(_pack(case, k, v, stale))
    return table, torch.cat(pool), chan


def _tokens(case):
    """(sequence, position) of each token of an append: sequence by sequence, positions from `first` on."""
    each = case["ntok"] // case["seqs"]
    seq = torch.arange(case["seqs"]).repeat_interleave(each)
    pos = case["first"] + torch.arange(each).repeat(case["seqs"])
    return seq.to(torch.int32).cuda(), pos.to(torch.int32).cuda(), case["first"] + each


def _prepare_embed(case, g, s, qg):
    rows, k, kind = case["rows"], case["k"], case["type"]
    s["ids"] = torch.randint(0, rows, (case["ntok"],), generator=g, device="cuda").to(torch.int32)
    if kind == F16:
        s["q"], s["scl"] = torch.randn(rows, k, generator=g, device="cuda", dtype=torch.float16) * 0.02, None
    else:
        wide = k // 2 if kind == Q4 else k
        s["q"] = torch.randint(0, 256, (rows, wide), generator=g, device="cuda", dtype=torch.uint8)
        s["scl"] = (_randn(g, rows, k // 32).abs() * 0.02 / (8 if kind == Q4 else 127)).to(torch.float16)
    if qg:
        s["type"] = {Q4: qg.Q4_0, Q8: qg.Q8_0, F16: qg.QG_F16}[kind]
        s["y"] = torch.empty(case["ntok"], k, dtype=_KIND[case["dst"]], device="cuda")


def _prepare_norm(case, g, s, qg):
    n, h, c = case["ntok"], case["heads"], case["n"]
    # hidden states: a few large channels, tokens of unlike size
    x = _randn(g, n, h, c) * torch.exp(0.7 * _randn(g, 1, 1, c)) * torch.exp(0.5 * _randn(g, n, 1, 1))
    s["x"] = x.to(_KIND[case["src"]])
    s["add"] = (0.3 * _randn(g, n, h, c)).to(_KIND[case["src"]]) if case["add"] else None
    s["w"] = 1 - case["w_add"] + 0.2 * _randn(g, c)
    if qg:
        s["sum"] = torch.empty_like(s["x"]) if case["add"] else None
        s["y"] = torch.empty(n, h, c, dtype=_KIND[F16 if case["dst"] == Q8 else case["dst"]], device="cuda")
        if case["dst"] == Q8:
            s["q"] = torch.empty(n, h, c, dtype=torch.int8, device="cuda")
            s["scl"] = torch.empty(n, h, c // 32, dtype=torch.float16, device="cuda")
            s["ids"] = torch.arange(n * h, dtype=torch.int32, device="cuda")


def _prepare_route(case, g, s, qg):
    n, e = case["ntok"], case["experts"]
    if case["hidden"]:
        # activations and router weights of few bits each: the logits come out alike in any order of summing, so that ids can be
        # compared
        s["x"] = (_randn(g, n, case["hidden"]) * 16).round().div(16).to(torch.float16)
        s["w"] = (_randn(g, e, case["hidden"]) * 32).round() / 1024
    else:
        s["logits"] = 1.5 * _randn(g, n, e)
    s["bias"] = 0.1 * _randn(g, e) if case["bias"] else None
    if qg:
        s["plan"] = qg.qroute_plan(case["score"], n_group=case["groups"], top_group=case["keep"], group_top=case["best"],
                                   renorm=case["renorm"], scale=case["scale"])
        s["ids"] = torch.empty(n, case["k"], dtype=torch.int32, device="cuda")
        s["rw"] = torch.empty(n, case["k"], dtype=torch.float32, device="cuda")


def _prepare_cache(case, g, s, qg):
    h, d = case["kv"], case["dim"]
    if case["op"] == "attn":
        lens = _lens(case)
        s["table"], s["pool"], chan = _filled(case, g, lens)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = _randn(g, case["seqs"], case["cols"], h, case["heads"] // h, d) * 2.0 / chan.square().mean(-1).sqrt().view(1, 1, h, 1, 1)
        s["q"] = q.reshape(case["seqs"], case["cols"], case["heads"], d).to(torch.float16)
    else:
        s["seq"], s["pos"], end = _tokens(case)
        s["table"], n, _, _ = _pages(case, g, [end] * case["seqs"], case["first"])
        s["pool"] = torch.full((n, h * (case["page"] // 16) * 20 * d), 0xFF, dtype=torch.uint8, device="cuda")
        # one row of the QKV projection a token: query heads, key heads, value heads (no far outliers: one that a block's
        # quants are stretched over makes a quant next to a half, which the last bit of an angle decides, a large difference)
        s["rows"] = _randn(g, case["ntok"], case["heads"] + 2 * h, d).clamp_(-2, 2)
    if qg:
        s["cache"] = qg.qkv_cache(qg.Q4_1, s["pool"], s["table"], h, d, case["page"])
        if case["op"] == "attn":
            s["ws"] = torch.empty(qg.qattn_workspace_bytes(s["cache"], case["heads"], case["cols"]), dtype=torch.uint8,
                                  device="cuda")
            s["y"] = torch.empty_like(s["q"])
        else:
            s["k"] = torch.empty(case["ntok"], h, d, dtype=torch.float16, device="cuda")
            s["v"] = torch.empty_like(s["k"])
            s["plan"] = qg.qrope_plan(case["rot"], base=case["base"], interleaved=case["inter"])
            s["q_out"] = torch.empty(case["ntok"], case["heads"], d, dtype=torch.float16, device="cuda")


def prepare(case, seed):
    s = {"case": case, "op": case["op"]}
    qg = None
    if own:
        import gemm_q4_q8_gb300 as qg
        s["qg"] = qg
    make = {"embed": _prepare_embed, "norm": _prepare_norm, "route": _prepare_route}.get(case["op"], _prepare_cache)
    make(case, _gen(seed), s, qg)
    return s


# ------------------------------------------------------------ the plain forms
def _stored_bytes(b):
    """Bytes of a matrix's rows in the order of the blocks, of stored ones [..., 16 groups]."""
    return b.unflatten(-1, (-1, 8, 2)).transpose(-1, -2).flatten(-3)


def _looked_up(kind, q, scl, ids):
    """Rows `ids` of a matrix, f32."""
    b = q[ids.long()]
    if kind == F16:
        return b.float()
    d = scl[ids.long()].float()[..., None]
    b = _stored_bytes(b.view(torch.uint8))
    if kind == Q8:
        w = b.view(torch.int8).float().unflatten(-1, (-1, 32))
    else:
        b = b.unflatten(-1, (-1, 16))
        w = torch.cat([b & 15, b >> 4], -1).float() - 8
    return (w * d).flatten(-2)


def _quantise8(x):
    """Q8_0 of f32 [..., 32] as the f32 values that it stands for: the scale amax / 127 rounded up to f16, the quants the
    nearest integers of x / scale."""
    s = x.abs().amax(-1, keepdim=True) / 127
    d = s.half()
    d = torch.where(d.float() < s, _f16(_bits(d) + 1), d).float()
    return torch.where(d > 0, torch.round(x / d) * d, torch.zeros_like(x))


def _plain_norm(s):
    case = s["case"]
    x = s["x"].float()
    out = {}
    if case["add"]:
        out["sum"] = (x + s["add"].float()).to(s["x"].dtype)
        x = out["sum"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + case["eps"]) * (s["w"] + case["w_add"])
    if case["dst"] == Q8:
        y = _quantise8(y.unflatten(-1, (-1, 32))).flatten(-2)
    out["y"] = y.to(_KIND[F16 if case["dst"] == Q8 else case["dst"]])
    return out


def _plain_route(s):
    case = s["case"]
    n, e = case["ntok"], case["experts"]
    logits = (s["x"].float() @ s["w"].t() if case["hidden"] else s["logits"]).double()  # 64 bits: experts next to each other
    p = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.exp(logits - logits.amax(-1, keepdim=True))
    if case["score"] == "softmax":
        p = p / p.sum(-1, keepdim=True)
    c = p + s["bias"].double() if case["bias"] else p
    rank = c if case["bias"] else logits
    if case["keep"] < case["groups"]:
        size = e // case["groups"]
        best = c.view(n, case["groups"], size).sort(dim=-1, descending=True)[0][..., :case["best"]].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True)[1][:, :case["keep"]]
        out = torch.ones(n, case["groups"], dtype=torch.bool, device=c.device).scatter_(1, kept, False)
        rank = rank.masked_fill(out.repeat_interleave(size, 1), -math.inf)
    ids = rank.sort(dim=-1, descending=True, stable=True)[1][:, :case["k"]]
    rw = p.gather(1, ids)
    if case["renorm"]:
        rw = rw / rw.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "rw": (rw * case["scale"]).float()}


def _freqs(rot, base):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


def _rotate(x, pos, rot, inter, freqs):
    """x f32 [tokens, heads, D], the first `rot` of each head rotated. Angles in 64 bits: positions are large."""
    a = pos.double()[:, None] * freqs
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    r = x[..., :rot]
    if inter:
        u, v = r[..., 0::2], r[..., 1::2]
        y = torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2)
    else:
        u, v = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([u * c - v * s, u * s + v * c], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _halves(case, pages):
    """Pool bytes [..., page bytes] as views: (quants [..., kv, page/16, 2, D/32, 16, 16], d and m as f16 [..., kv, page/16, 2,
    2 (d, m), 16 D/32])."""
    h, d, gr = case["kv"], case["dim"], case["page"] // 16
    halves = pages.unflatten(-1, (h, gr, 2, 10 * d))
    scales = halves.view(torch.float16)[..., 4 * d:].unflatten(-1, (2, d // 2))
    return halves[..., :8 * d].unflatten(-1, (d // 32, 16, 16)), scales


def _values(case, pages):
    """Keys and values f32 [..., tokens, kv, D] of pool bytes [..., page bytes]."""
    nb = case["dim"] // 32
    quants, scales = _halves(case, pages)
    got = []
    for is_v in (0, 1):
        q = _elements(quants[..., is_v, :, :, :].transpose(-2, -3)).float()  # [..., kv, group, token, block, 32]
        s = scales[..., is_v, :, :].float()
        s = s.unflatten(-1, (nb, 16))[..., _places(s.device)].transpose(-1, -2) if is_v else s.unflatten(-1, (16, nb))
        x = q * s[..., 0, :, :, None] + s[..., 1, :, :, None]
        x = x.flatten(-2).flatten(-3, -2)  # [..., kv, token, D]
        got.append(x.transpose(-2, -3))
    return got


def _plain_attn(s):
    case = s["case"]
    b, cols, heads, d = s["q"].shape
    h = case["kv"]
    k, v = _values(case, s["pool"][s["table"].clamp(min=0).long()])
    k, v = k.flatten(1, 2), v.flatten(1, 2)  # [seq, tokens, kv, D]
    j = torch.arange(k.shape[1], device="cuda")
    held = (j < s["lens"][:, None])[..., None, None]
    k = torch.where(held, k, torch.zeros_like(k)).transpose(1, 2)
    v = torch.where(held, v, torch.zeros_like(v)).transpose(1, 2)
    q = s["q"].float().view(b, cols, h, heads // h, d).permute(0, 2, 1, 3, 4).reshape(b, h, -1, d)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(b, h, cols, heads // h, -1)
    at = (s["lens"][:, None] - cols + torch.arange(cols, device="cuda")).view(b, 1, cols, 1, 1)
    seen = j <= at
    if case["window"]:
        seen = seen & (j > at - case["window"])
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    y = torch.matmul(p.flatten(2, 3), v).view(b, h, cols, heads // h, d)
    y = torch.where(total > 0, y / total, torch.zeros_like(y))
    return y.permute(0, 2, 1, 3, 4).reshape(b, cols, heads, d).to(torch.float16)


def _plain_append(s):
    case = s["case"]
    rows, a, h, d, n = s["rows"], case["heads"], case["kv"], case["dim"], case["ntok"]
    f = _freqs(case["rot"], case["base"])
    q = _rotate(rows[:, :a], s["pos"], case["rot"], case["inter"], f).to(torch.float16)
    k = _rotate(rows[:, a:a + h], s["pos"], case["rot"], case["inter"], f)
    page = s["table"][s["seq"].long(), (s["pos"] // case["page"]).long()].long()
    slot = (s["pos"] % case["page"]).long()
    grp, i = slot // 16, slot % 16
    quants, scales = _halves(case, s["pool"])
    nb = d // 32
    out = {"q": q}
    for is_v, name, x in ((0, "k", k), (1, "v", rows[:, a + h:])):
        w, dd, m = _quantise4(x.view(n, h, nb, 32))
        quants[page, :, grp, is_v, :, i] = _nibbles(w)
        half = scales[:, :, :, is_v]
        place = _places(x.device)[i]
        for what, v in ((0, dd), (1, m)):
            one = half[:, :, :, what].unflatten(-1, (nb, 16) if is_v else (16, nb))
            if is_v:
                one[page, :, grp, :, place] = v.squeeze(-1).half()
            else:
                one[page, :, grp, i] = v.squeeze(-1).half()
        got = _elements(quants[page, :, grp, is_v, :, i]).float()
        sc = []
        for what in (0, 1):
            one = half[:, :, :, what].unflatten(-1, (nb, 16) if is_v else (16, nb))
            sc.append((one[page, :, grp, :, place] if is_v else one[page, :, grp, i]).float()[..., None])
        out[name] = (got * sc[0] + sc[1]).flatten(-2).to(torch.float16)
    return out


def _plain(s):
    op = s["op"]
    if op == "embed":
        case = s["case"]
        return (_looked_up(case["type"], s["q"], s["scl"], s["ids"]) * case["scale"]).to(_KIND[case["dst"]])
    return {"norm": _plain_norm, "route": _plain_route, "attn": _plain_attn, "append": _plain_append}[op](s)


def run(s):
    if not own:
        return _plain(s)
    qg, op, case = s["qg"], s["op"], s["case"]
    if op == "embed":
        qg.qembed(s["type"], s["q"], s["scl"], s["ids"], s["y"], scale=case["scale"])
        return s["y"]
    if op == "norm":
        if case["dst"] == Q8:
            qg.qrms_norm(s["x"], s["w"], s["q"], y_scl=s["scl"], eps=case["eps"], w_add=case["w_add"], add=s["add"],
                         sum_out=s["sum"])
            n = case["ntok"] * case["heads"]
            qg.qembed(qg.Q8_0, s["q"].view(n, -1), s["scl"].view(n, -1), s["ids"], s["y"].view(n, -1))
        else:
            qg.qrms_norm(s["x"], s["w"], s["y"], eps=case["eps"], w_add=case["w_add"], add=s["add"], sum_out=s["sum"])
        return {"sum": s["sum"], "y": s["y"]} if case["add"] else {"y": s["y"]}
    if op == "route":
        if case["hidden"]:
            qg.qmoe_router_planned(s["plan"], s["w"], s["x"], case["k"], s["ids"], s["rw"], bias=s["bias"])
        else:
            qg.qmoe_route(s["plan"], s["logits"], case["k"], s["ids"], s["rw"], bias=s["bias"])
        return {"ids": s["ids"], "rw": s["rw"]}
    if op == "attn":
        qg.qattn_paged(s["cache"], s["q"], s["lens"], s["y"], s["ws"], window=case["window"])
        return s["y"]
    a, h = case["heads"], case["kv"]
    rows = s["rows"]
    qg.qkv_append(s["cache"], rows[:, a:a + h], rows[:, a + h:], s["pos"], seq=s["seq"], rope=s["plan"], q=rows[:, :a],
                  q_out=s["q_out"])
    qg.qkv_read(s["cache"], s["pos"], s["k"], s["v"], seq=s["seq"])
    return {"k": s["k"], "v": s["v"], "q": s["q_out"]}


# --------------------------------------------------------- 64 bits, set apart
def _turned(x, pos, case):
    """Rotation in 64 bits, as a product of complex numbers."""
    rot = case["rot"]
    step = [math.exp(-2.0 * i / rot * math.log(case["base"])) for i in range(rot // 2)]
    angle = pos.to(torch.float64).view(-1, 1, 1) * torch.tensor(step, dtype=torch.float64, device=x.device)
    unit = torch.polar(torch.ones_like(angle), angle)
    x = x.to(torch.float64).clone()
    part = x[..., :rot]
    pairs = part.unflatten(-1, (-1, 2)) if case["inter"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
    x[..., :rot] = (z if case["inter"] else z.transpose(-1, -2)).flatten(-2)
    return x


def _steps(x):
    """The distance of f16 numbers around f64 |x|."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -14))) - 10)


def _blocks4(x):
    """What 4-bit blocks stand for, of f64 values."""
    b = x.unflatten(-1, (-1, 32))
    lo, hi = b.amin(-1, keepdim=True), b.amax(-1, keepdim=True)
    m = torch.floor(lo / _steps(lo)) * _steps(lo)
    d = (hi - m) / 15
    d = torch.ceil(d / _steps(d)) * _steps(d)
    q = torch.where(d > 0, torch.round((b - m) / torch.where(d > 0, d, torch.ones_like(d))).clamp(0, 15), torch.zeros_like(b))
    return (q * d + m).flatten(-2)


def _blocks8(x):
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True) / 127.0
    d = torch.ceil(top / _steps(top)) * _steps(top)
    return torch.where(d > 0, torch.round(b / torch.where(d > 0, d, torch.ones_like(d))) * d, torch.zeros_like(b)).flatten(-2)


def _token_record(case, pool, page, slot):
    """Keys and values in 64 bits [tokens, kv, D] of the given pages and slots, by byte offsets into the pool."""
    h, d, ps = case["kv"], case["dim"], case["page"]
    flat = pool.reshape(-1)
    halves = flat.view(torch.float16)
    rec = 20 * d
    base = (page.view(-1, 1, 1) * h + torch.arange(h, device=pool.device).view(1, -1, 1)) * (ps // 16) * rec
    base = base + (slot // 16).view(-1, 1, 1) * rec
    i = (slot % 16).view(-1, 1, 1)
    c = torch.arange(d, device=pool.device).view(1, 1, -1)
    u = c % 8
    byte = (c // 32) * 256 + i * 16 + (c % 32) // 8 * 4 + (u % 4 % 2) * 2 + u % 4 // 2
    got = []
    for is_v in (0, 1):
        at = base + is_v * 10 * d
        q = (flat[at + byte].long() >> (4 * (u // 4))) & 15
        if is_v:
            place = (c // 32) * 16 + 4 * (i % 8 // 2) + i % 2 + 2 * (i // 8)
        else:
            place = i * (d // 32) + c // 32
        got.append(q.double() * halves[at // 2 + 4 * d + place].double() + halves[at // 2 + 4 * d + d // 2 + place].double())
    return got


def _exact_embed(s, case):
    rows, k = s["ids"].long(), case["k"]
    if case["type"] == F16:
        return s["q"][rows].double() * case["scale"]
    c = torch.arange(k, device="cuda")
    e = c % 32
    d = s["scl"][rows].double()[:, c // 32]
    j = e % 16  # byte j of 16 is stored at 2 (j mod 8) + j div 8
    if case["type"] == Q4:
        b = s["q"][rows][:, c // 32 * 16 + 2 * (j % 8) + j // 8].long()
        w = ((b >> (4 * (e // 16))) & 15).double() - 8
    else:
        b = s["q"][rows][:, c // 16 * 16 + 2 * (j % 8) + j // 8].long()
        w = torch.where(b > 127, b - 256, b).double()
    return w * d * case["scale"]


def _exact_route(s, case):
    n, e, k = case["ntok"], case["experts"], case["k"]
    ids, rws = [], []
    j = torch.arange(e, device="cuda")
    for a in range(0, n, 1024):
        z = min(n, a + 1024)
        if case["hidden"]:
            logits = torch.einsum("nh,eh->ne", s["x"][a:z].double(), s["w"].double())
        else:
            logits = s["logits"][a:z].double()
        p = 1 / (1 + torch.exp(-logits)) if case["score"] == "sigmoid" else torch.softmax(logits, -1)
        c = p if s["bias"] is None else p + s["bias"].double()
        open_ = torch.ones_like(c, dtype=torch.bool)
        if case["keep"] < case["groups"]:
            best = c.view(z - a, case["groups"], -1).topk(case["best"], -1)[0].sum(-1)
            g = torch.arange(case["groups"], device="cuda")
            ahead = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & (g[None, :] < g[:, None]))
            open_ = (ahead.sum(-1) < case["keep"]).repeat_interleave(e // case["groups"], 1)
        v = torch.where(open_, c if s["bias"] is not None else logits, torch.full_like(c, -math.inf))
        # an expert's place: how many are ahead of it
        ahead = (v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & (j[None, :] < j[:, None]))
        place = ahead.sum(-1)
        chosen = torch.where(place < k, place, torch.full_like(place, k))
        one = torch.zeros(z - a, k + 1, dtype=torch.int64, device="cuda").scatter_(1, chosen, j.expand(z - a, e))[:, :k]
        w = p.gather(1, one)
        if case["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        ids.append(one.to(torch.int32))
        rws.append(w * case["scale"])
    return {"ids": torch.cat(ids), "rw": torch.cat(rws)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        return _exact_embed(s, case)
    if op == "route":
        return _exact_route(s, case)
    if op == "norm":
        x = s["x"].double()
        out = {}
        if case["add"]:
            out["sum"] = x + s["add"].double()
            x = out["sum"]
        y = x / (x.square().mean(-1, keepdim=True) + case["eps"]).sqrt() * (s["w"].double() + case["w_add"])
        out["y"] = _blocks8(y) if case["dst"] == Q8 else y
        return out
    if op == "append":
        a, h = case["heads"], case["kv"]
        rows = s["rows"]
        return {"q": _turned(rows[:, :a], s["pos"], case), "k": _blocks4(_turned(rows[:, a:a + h], s["pos"], case)),
                "v": _blocks4(rows[:, a + h:].double())}
    table, ps = s["table"].long(), case["page"]
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv"]
    for b, n in enumerate(_lens(case)):
        first = None
        for t in range(case["cols"]):
            p = n - case["cols"] + t
            if p < 0:
                continue
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            at = torch.arange(lo, p + 1, device="cuda")
            if first is None or case["window"]:
                first = lo
                every = torch.arange(lo, n, device="cuda")
                k, v = _token_record(case, s["pool"], table[b, every // ps], every % ps)
            m = at.numel()
            kk, vv = k[lo - first:lo - first + m], v[lo - first:lo - first + m]
            q = s["q"][b, t].double().view(case["kv"], group, -1)
            w = torch.softmax(torch.einsum("hgd,jhd->hgj", q, kk) / math.sqrt(case["dim"]), -1)
            y[b, t] = torch.einsum("hgj,jhd->hgd", w, vv).reshape(case["heads"], -1)
    return y
