"""The attention side of a decoder layer, measured: rotary positions, the paged
key/value cache (written in f16 or as Q8_0 blocks, and read back), and the
attention of a few new tokens over it.

A case names one operator ("op") and its sizes. ``prepare`` makes what a serving
loop holds in hand: the outputs of the QKV projection, the pool of cache pages,
the page table, the lengths. ``run`` is one pass: the plain form in elementary
torch operations where ``own`` is false, the library's calls where it is true.
Both read and write the same pool bytes.

Pool layout (bytes): [page][kv head][group of 16 tokens] records; a record is the
key half, then the value half. f16: [D/32][16][32] f16. Q8_0: [D/32][16][32]
quants stored as q + 128, then [D/32][16] f16 scales, token i of the group at
place 4 (i mod 4) + i div 4.
"""
import math

import torch

own = False

F16, Q8 = "f16", "q8_0"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token: the query heads of a 2,048-wide layer, a quarter of each head rotated
        dict(name="rope 1 token", op="rope", ntok=1, heads=16, dim=256, rot=64, inter=False, base=1e7,
             factor=1.0, orig=0, src="f32", dst="f16", first=4097),
        # a prompt of odd length through a 5,120-wide layer, positions scaled for a long context
        dict(name="rope prompt", op="rope", ntok=8191, heads=40, dim=128, rot=128, inter=True, base=5e5,
             factor=8.0, orig=8192, src="f32", dst="f16", first=100000),
        # one decoded token appended (with the queries rotated) to an f16 cache
        dict(name="append 1 token f16", op="append", type=F16, seqs=1, ntok=1, heads=16, kv=2, dim=256,
             page=16, rot=64, inter=False, base=1e7, first=30001),
        # a verify step: 4 new tokens for each of 16 sequences, Q8_0 cache
        dict(name="append 16x4 q8_0", op="append", type=Q8, seqs=16, ntok=64, heads=40, kv=8, dim=128,
             page=64, rot=128, inter=False, base=1e6, first=997),
        # a prompt written at once: two sequences, ragged against pages and groups
        dict(name="append prompt q8_0", op="append", type=Q8, seqs=2, ntok=16382, heads=40, kv=8, dim=128,
             page=64, rot=128, inter=False, base=1e6, first=5),
        # a short prefix read back, then a long one (a session moved out of the cache)
        dict(name="read 300 q8_0", op="read", type=Q8, seqs=1, ntok=300, kv=2, dim=256, page=16, first=0),
        dict(name="read 32767 f16", op="read", type=F16, seqs=1, ntok=32767, kv=8, dim=128, page=64, first=1),
        # one token for one user, a short history: latency
        dict(name="attn 1x1 of 1000 q8_0", op="attn", type=Q8, seqs=1, cols=1, heads=16, kv=2, dim=256,
             page=16, short=1000, long=1000, window=0),
        # one token for one user over a very long history
        dict(name="attn 1x1 of 131071 f16", op="attn", type=F16, seqs=1, cols=1, heads=40, kv=8, dim=128,
             page=64, short=131071, long=131071, window=0),
        # a serving batch of ragged lengths, one token each
        dict(name="attn 64x1 ragged q8_0", op="attn", type=Q8, seqs=64, cols=1, heads=40, kv=8, dim=128,
             page=64, short=130, long=8191, window=0),
        # speculative verify: 8 new tokens a sequence, sliding window, small heads
        dict(name="attn 8x8 window f16", op="attn", type=F16, seqs=8, cols=8, heads=32, kv=8, dim=64,
             page=32, short=700, long=16001, window=4096),
        # speculative verify over wide heads, Q8_0
        dict(name="attn 4x4 q8_0", op="attn", type=Q8, seqs=4, cols=4, heads=16, kv=2, dim=256,
             page=128, short=9000, long=33333, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "read", "attn", "attn", "attn", "attn"])
    dim = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    case = dict(op=op, dim=dim)
    rope = dict(heads=kv * group, rot=rng.choice([dim, dim // 2, dim // 4]), inter=rng.random() < 0.5,
                base=rng.choice([1e4, 5e5, 1e6, 1e7]), first=_log(rng, 1, 200000) - 1)
    if op == "rope":
        case.update(rope, ntok=_log(rng, 1, 65536), factor=rng.choice([1.0, 4.0, 8.0]),
                    orig=rng.choice([0, 4096, 8192]), src=rng.choice(["f32", "f16"]), dst=rng.choice(["f32", "f16"]))
    else:
        seqs = _log(rng, 1, 64)
        case.update(type=rng.choice([F16, Q8]), seqs=seqs, kv=kv, page=rng.choice([16, 32, 64, 128]))
        if op == "append":
            case.update(rope, ntok=seqs * _log(rng, 1, 16382))
        elif op == "read":
            case.update(first=rng.randrange(40), ntok=seqs * _log(rng, 1, 32767))
        else:
            long = _log(rng, 1, 131071)
            case.update(cols=rng.choice([1, 1, 1, 2, 3, 4, 8]), heads=kv * group, long=long,
                        short=_log(rng, 1, long), window=rng.choice([0, 0, 0, 1000]))
    most = [work(c) for c in listed() if c["op"] == op]
    while any(work(case)[w] > max(m[w] for m in most) for w in ("bytes", "flops")):
        if op == "attn":
            case["long"] = max(1, case["long"] * 3 // 4)
            case["short"] = min(case["short"], case["long"])
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


def work(case):
    op, d = case["op"], case["dim"]
    if op == "rope":
        n = case["ntok"] * case["heads"] * d
        size = {"f32": 4, "f16": 2}
        return {"bytes": n * (size[case["src"]] + size[case["dst"]]) + 4 * case["ntok"],
                "flops": 3 * case["ntok"] * case["heads"] * case["rot"]}
    stored = {F16: 2.0, Q8: 1.0 + 2 / 32}[case["type"]] * 2 * case["kv"] * d  # one token, keys and values
    if op == "append":  # rows of f32 in; the token's cache bytes written, then read back as f16
        n = case["ntok"]
        q = n * case["heads"] * d
        kvs = n * 2 * case["kv"] * d
        return {"bytes": q * (4 + 2) + kvs * (4 + 2) + 2 * n * stored + 8 * n,
                "flops": 3 * n * (case["heads"] + case["kv"]) * case["rot"] + (0 if case["type"] == F16 else 4 * kvs)}
    if op == "read":
        n = case["ntok"]
        return {"bytes": n * (stored + 2 * case["kv"] * d * 2) + 8 * n, "flops": n * 2 * case["kv"] * d}
    keys, pairs = _visible(case)
    rows = case["seqs"] * case["cols"] * case["heads"]
    return {"bytes": keys * stored + rows * d * 4 + 4 * case["seqs"], "flops": 4.0 * d * pairs * case["heads"]}


# ------------------------------------------------------------- data in hand
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _quantise(x):
    """Q8_0 of f32 [..., 32]: the scale amax / 127 rounded up to f16, the quants the nearest integers of x / scale."""
    s = x.abs().amax(-1, keepdim=True) / 127
    d = s.half()
    up = (d.view(torch.int16) + 1).view(torch.float16)
    d = torch.where(d.float() < s, up, d)
    d32 = d.float()
    q = torch.where(d32 > 0, torch.round(x / d32), torch.zeros_like(x))
    return q, d


#: the place of each of a group's 16 scales
def _places(device):
    i = torch.arange(16, device=device)
    return (i % 4) * 4 + i // 4


def _pack(case, k, v, stale):
    """Pool bytes of keys and values f32 [pages, kv, page, D]; tokens marked in `stale` hold bytes of all ones."""
    n, h, ps, d = k.shape
    kv = torch.stack([k, v], 2).view(n, h, 2, ps // 16, 16, d // 32, 32).permute(0, 1, 3, 2, 5, 4, 6)
    old = stale.view(n, 1, ps // 16, 1, 1, 16, 1)
    if case["type"] == F16:
        x = kv.to(torch.float16).contiguous().view(torch.int16)
        x = torch.where(old, torch.full_like(x, -1), x)
        return x.view(torch.uint8).view(n, -1)
    q, s = _quantise(kv)
    q = torch.where(old, torch.full_like(q, 127), q)
    q = (q + 128).to(torch.uint8).flatten(4)
    s = s.contiguous().view(torch.int16)
    s = torch.where(old, torch.full_like(s, -1), s).squeeze(-1)
    t = torch.empty_like(s)
    t[..., _places(s.device)] = s
    return torch.cat([q, t.contiguous().view(torch.uint8).flatten(4)], -1).view(n, -1)


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
    # channels of unlike size, as keys have them, and values of unlike size by head
    chan = torch.exp(0.6 * _randn(g, 1, h, 1, d))
    k = _randn(g, n, h, ps, d) * chan
    v = _randn(g, n, h, ps, d) * torch.exp(0.5 * _randn(g, 1, h, 1, 1))
    pos = start[:, None] + torch.arange(ps, device="cuda")
    stale = (start[:, None] < 0) | (pos >= torch.tensor(lens, device="cuda")[owner][:, None])
    return table, _pack(case, k, v, stale), chan


def _tokens(case):
    """(sequence, position) of each token of an append or read: sequence by sequence, positions from `first` on."""
    each = case["ntok"] // case["seqs"]
    seq = torch.arange(case["seqs"]).repeat_interleave(each)
    pos = case["first"] + torch.arange(each).repeat(case["seqs"])
    return seq.to(torch.int32).cuda(), pos.to(torch.int32).cuda(), case["first"] + each


def prepare(case, seed):
    g = _gen(seed)
    op, d = case["op"], case["dim"]
    s = {"case": case, "op": op}
    if own:
        import gemm_q4_q8_gb300 as qg
        s["qg"] = qg
        kind = {"f32": torch.float32, "f16": torch.float16}
    if op == "rope":
        n, h = case["ntok"], case["heads"]
        s["x"] = _randn(g, n, h, d).to({"f32": torch.float32, "f16": torch.float16}[case["src"]])
        s["pos"] = (case["first"] + torch.arange(n, device="cuda")).to(torch.int32)
        if own:
            s["plan"] = qg.qrope_plan(case["rot"], base=case["base"], interleaved=case["inter"],
                                      factor=case["factor"], orig_ctx=case["orig"])
            s["y"] = torch.empty(n, h, d, dtype=kind[case["dst"]], device="cuda")
        return s
    h = case["kv"]
    if op == "attn":
        lens = _lens(case)
        s["table"], s["pool"], chan = _filled(case, g, lens)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = _randn(g, case["seqs"], case["cols"], h, case["heads"] // h, d) * 2.0 / chan.square().mean(-1).sqrt().view(1, 1, h, 1, 1)
        s["q"] = q.reshape(case["seqs"], case["cols"], case["heads"], d).to(torch.float16)
    else:
        seq, pos, end = _tokens(case)
        s["seq"], s["pos"] = seq, pos
        if op == "read":
            s["table"], s["pool"], _ = _filled(case, g, [end] * case["seqs"])
        else:
            s["table"], n, _, _ = _pages(case, g, [end] * case["seqs"], case["first"])
            per = {F16: 64, Q8: 34}[case["type"]] * d  # bytes of a group of 16 tokens
            s["pool"] = torch.full((n, h * (case["page"] // 16) * per), 0xFF, dtype=torch.uint8, device="cuda")
            # one row of the QKV projection a token: query heads, key heads, value heads
            rows = _randn(g, case["ntok"], case["heads"] + 2 * h, d)
            rows[:, case["heads"]:case["heads"] + h] *= torch.exp(0.6 * _randn(g, 1, h, d))
            s["rows"] = rows
    if own:
        qtype = {F16: qg.QG_F16, Q8: qg.Q8_0}[case["type"]]
        s["cache"] = qg.qkv_cache(qtype, s["pool"], s["table"], h, d, case["page"])
        if op == "attn":
            s["ws"] = torch.empty(qg.qattn_workspace_bytes(s["cache"], case["heads"], case["cols"]),
                                  dtype=torch.uint8, device="cuda")
            s["y"] = torch.empty_like(s["q"])
        else:
            s["k"] = torch.empty(case["ntok"], h, d, dtype=torch.float16, device="cuda")
            s["v"] = torch.empty_like(s["k"])
        if op == "append":
            s["plan"] = qg.qrope_plan(case["rot"], base=case["base"], interleaved=case["inter"])
            s["q_out"] = torch.empty(case["ntok"], case["heads"], d, dtype=torch.float16, device="cuda")
    return s


# ------------------------------------------------------------ the plain forms
def _freqs(rot, base, factor=1.0, orig=0):
    """Radians a position of each pair; a factor above 1 slows the pairs that turn less than 32 times (not at all from 32
    on, wholly below 1) over the original context, or all alike where there is none."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if orig:
        keep = ((orig * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
    else:
        keep = torch.zeros_like(f)
    return f * keep + f / factor * (1 - keep)


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
    """(quants or values, scales or None) of pool bytes [..., page bytes], as views
    [..., kv, page/16, 2, D/32, 16(, 32)]: the scales in their stored places."""
    h, d, gr = case["kv"], case["dim"], case["page"] // 16
    nb = d // 32
    if case["type"] == F16:
        return pages.view(torch.float16).unflatten(-1, (h, gr, 2, nb, 16, 32)), None
    halves = pages.unflatten(-1, (h, gr, 2, 17 * d))
    return (halves[..., :16 * d].unflatten(-1, (nb, 16, 32)),
            halves.view(torch.float16)[..., 8 * d:].unflatten(-1, (nb, 16)))


def _values(case, pages):
    """Keys and values f32 [..., tokens, kv, D] of pool bytes [..., page bytes]."""
    x, scales = _halves(case, pages)
    x = x.float()
    if scales is not None:
        x = (x - 128) * scales[..., _places(x.device)].float()[..., None]
    lead = x.dim() - 6
    x = x.permute(*range(lead), lead + 2, lead + 1, lead + 4, lead, lead + 3, lead + 5)
    x = x.flatten(-2).flatten(lead + 1, lead + 2)
    return x.select(lead, 0), x.select(lead, 1)


def _slots(s):
    case = s["case"]
    page = s["table"][s["seq"].long(), (s["pos"] // case["page"]).long()].long()
    slot = (s["pos"] % case["page"]).long()
    return page, slot // 16, slot % 16


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


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "rope":
        f = _freqs(case["rot"], case["base"], case["factor"], case["orig"])
        y = _rotate(s["x"].float(), s["pos"], case["rot"], case["inter"], f)
        return y.to({"f32": torch.float32, "f16": torch.float16}[case["dst"]])
    if op == "attn":
        return _plain_attn(s)
    page, grp, i = _slots(s)
    x, scales = _halves(case, s["pool"])
    h, d, n = case["kv"], case["dim"], case["ntok"]
    q = None
    if op == "append":
        rows, a = s["rows"], case["heads"]
        f = _freqs(case["rot"], case["base"])
        q = _rotate(rows[:, :a], s["pos"], case["rot"], case["inter"], f).to(torch.float16)
        k = _rotate(rows[:, a:a + h], s["pos"], case["rot"], case["inter"], f)
        kv = torch.stack([k, rows[:, a + h:]], 1).view(n, 2, h, d // 32, 32)
        if scales is None:
            w = kv.to(torch.float16)
        else:
            w, sc = _quantise(kv)
            w = (w + 128).to(torch.uint8)
            put = sc.squeeze(-1).transpose(1, 2)
            scales[page, :, grp, :, :, (i % 4) * 4 + i // 4] = put
        x[page, :, grp, :, :, i] = w.transpose(1, 2)
    got = x[page, :, grp, :, :, i].float()  # [tokens, kv, 2, D/32, 32]
    if scales is not None:
        got = (got - 128) * scales[page, :, grp, :, :, (i % 4) * 4 + i // 4].float()[..., None]
    got = got.flatten(-2).to(torch.float16)
    out = {"k": got[:, :, 0], "v": got[:, :, 1]}
    return out if q is None else dict(out, q=q)


def run(s):
    if not own:
        return _plain(s)
    qg, op = s["qg"], s["op"]
    if op == "rope":
        qg.qrope(s["plan"], s["x"], s["pos"], s["y"])
        return s["y"]
    if op == "attn":
        qg.qattn_paged(s["cache"], s["q"], s["lens"], s["y"], s["ws"], window=s["case"]["window"])
        return s["y"]
    if op == "append":
        a, h = s["case"]["heads"], s["case"]["kv"]
        rows = s["rows"]
        qg.qkv_append(s["cache"], rows[:, a:a + h], rows[:, a + h:], s["pos"], seq=s["seq"], rope=s["plan"],
                      q=rows[:, :a], q_out=s["q_out"])
        qg.qkv_read(s["cache"], s["pos"], s["k"], s["v"], seq=s["seq"])
        return {"k": s["k"], "v": s["v"], "q": s["q_out"]}
    qg.qkv_read(s["cache"], s["pos"], s["k"], s["v"], seq=s["seq"])
    return {"k": s["k"], "v": s["v"]}


# --------------------------------------------------------- 64 bits, set apart
def _turned(x, pos, case, factor, orig):
    """Rotation in 64 bits, as a product of complex numbers."""
    rot = case["rot"]
    step = []
    for i in range(rot // 2):
        w = math.exp(-2.0 * i / rot * math.log(case["base"]))
        if factor != 1.0:
            turns = orig * w / (2 * math.pi)
            share = min(1.0, max(0.0, (turns - 1.0) / 31.0)) if orig else 0.0
            w = share * w + (1 - share) * w / factor
        step.append(w)
    angle = pos.to(torch.float64).view(-1, 1, 1) * torch.tensor(step, dtype=torch.float64, device=x.device)
    unit = torch.polar(torch.ones_like(angle), angle)
    x = x.to(torch.float64).clone()
    part = x[..., :rot]
    pairs = part.unflatten(-1, (-1, 2)) if case["inter"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
    x[..., :rot] = (z if case["inter"] else z.transpose(-1, -2)).flatten(-2)
    return x


def _stored(x, kind):
    """What a cache stands for, of f64 values: the values themselves (f16 rounds them once, as it does the outputs), or
    Q8_0 blocks of 32."""
    if kind == F16:
        return x
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True) / 127.0
    # the smallest f16 not below it: multiples of its binade's step
    step = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -14))) - 10)
    d = torch.ceil(top / step) * step
    q = torch.where(d > 0, torch.round(b / torch.where(d > 0, d, torch.ones_like(d))), torch.zeros_like(b))
    return (q * d).flatten(-2)


def _token_record(case, pool, page, slot):
    """Keys and values in 64 bits [tokens, kv, D] of the given pages and slots, by byte offsets into the pool."""
    h, d, ps = case["kv"], case["dim"], case["page"]
    f16 = case["type"] == F16
    half = 32 * d if f16 else 17 * d
    flat = pool.reshape(-1)
    base = page.view(-1, 1, 1) * (h * (ps // 16) * 2 * half) + torch.arange(h, device=pool.device).view(1, -1, 1) * ((ps // 16) * 2 * half)
    base = base + (slot // 16).view(-1, 1, 1) * (2 * half)
    i = (slot % 16).view(-1, 1, 1)
    c = torch.arange(d, device=pool.device).view(1, 1, -1)
    element = (c // 32) * 512 + i * 32 + c % 32
    got = []
    for at in (base, base + half):
        if f16:
            got.append(flat.view(torch.float16)[at // 2 + element].double())
        else:
            scale = flat.view(torch.float16)[(at + 16 * d) // 2 + (c // 32) * 16 + (i % 4) * 4 + i // 4]
            got.append((flat[at + element].double() - 128) * scale.double())
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turned(s["x"], s["pos"], case, case["factor"], case["orig"])
    if op == "append":
        a, h = case["heads"], case["kv"]
        rows = s["rows"]
        return {"q": _turned(rows[:, :a], s["pos"], case, 1.0, 0),
                "k": _stored(_turned(rows[:, a:a + h], s["pos"], case, 1.0, 0), case["type"]),
                "v": _stored(rows[:, a + h:].double(), case["type"])}
    table, ps = s["table"].long(), case["page"]
    if op == "read":
        pos = s["pos"].long()
        k, v = _token_record(case, s["pool"], table[s["seq"].long(), pos // ps], pos % ps)
        return {"k": k, "v": v}
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
