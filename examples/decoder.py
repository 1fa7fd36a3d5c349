"""A small decoder with routed experts, from token ids to logits, served over a cache in 4 bits.

One call of ``Decoder.step`` takes ``ncols`` new tokens for each sequence through

    qembed                the tokens' rows of the matrix that is the LM head, too
    and in each layer
    qrms_norm             the residual's addition and the norm
    qgemm_cols            the fused QKV projection
    qrms_norm             each query and key head
    qkv_append            rotary positions, keys and values into the 4-bit cache
    qattn_paged           attention over everything cached so far
    qgemm_cols            the output projection
    qrms_norm             the residual's addition and the norm
    qmoe_router_planned   scores, bias, groups: each token's experts and their weights
    qmoe_experts          the experts
    and at the end
    qrms_norm, qgemm_cols the logits
    qargmax_f32           the next token

Run it on a GPU: python examples/decoder.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_q4_q8_gb300 as qg  # noqa: E402


class Layer:
    """Weights of a layer, (quants, scales) in the library's layout each: wqkv [(heads + 2 kv) * d, hidden], wo [hidden, heads * d], the
    experts' gate and up [experts * ffn, hidden] and down [experts * hidden, ffn] stacks; f32: the router [experts, hidden], its bias
    [experts], and the norms of the layer's two inputs [hidden] and of query and key heads [d]."""

    def __init__(self, **w):
        self.__dict__.update(w)


class Decoder:
    """n_seq sequences of up to ``tokens`` tokens; pages are handed out in order here, a server would use an allocator of its own."""

    def __init__(self, qtype, table, layers, last_norm, heads, kv_heads, head_dim, n_seq, tokens, route, topk, page_size=16,
                 cache_type=qg.Q4_1, base=1e6, embed_scale=1.0, eps=1e-6):
        self.qtype, self.table, self.layers, self.last_norm = qtype, table, layers, last_norm
        self.heads, self.kv, self.d, self.n_seq, self.topk = heads, kv_heads, head_dim, n_seq, topk
        self.rope, self.route = qg.qrope_plan(head_dim, base=base), route
        self.embed_scale, self.eps = embed_scale, eps
        self.hidden = table[1].shape[1] * 32
        pages = -(-tokens // page_size)
        page = qg.qkv_page_bytes(cache_type, kv_heads, head_dim, page_size)
        place = torch.arange(n_seq * pages, dtype=torch.int32, device="cuda").view(n_seq, pages)
        self.caches = [qg.qkv_cache(cache_type, torch.zeros(n_seq * pages * page, dtype=torch.uint8, device="cuda"), place, kv_heads,
                                    head_dim, page_size) for _ in layers]
        self.lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")  # tokens cached
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        most = max(qg.qattn_workspace_bytes(self.caches[0], heads, c) for c in range(1, 17))
        self.ws = torch.empty(most, dtype=torch.uint8, device="cuda")

    def step(self, ids, keep=None):
        """ids int32 [n_seq * ncols] (at most 16, each sequence's tokens in order) -> (f32 logits [n, vocab], int32 next tokens [n]). keep:
        a list that takes each layer's values in between."""
        n, ncols, h, kv, d, dim = ids.numel(), ids.numel() // self.n_seq, self.heads, self.kv, self.d, self.hidden
        new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
        half = torch.float16
        x = new(n, dim)
        qg.qembed(self.qtype, *self.table, ids, x, scale=self.embed_scale, err_flag=self.err)
        pos = (self.lens[:, None] + torch.arange(ncols, dtype=torch.int32, device="cuda")).reshape(-1).contiguous()
        self.lens += ncols
        delta = None  # what the last block adds to the residual
        for w, cache in zip(self.layers, self.caches):
            residual = new(n, dim)
            a = new(n, dim, dtype=half)
            qg.qrms_norm(x, w.norm1, a, eps=self.eps, add=delta, sum_out=residual)
            rows = new(n, h + 2 * kv, d)
            qg.qgemm_cols(self.qtype, *w.wqkv, a, rows)
            projected = rows.clone() if keep is not None else None
            qg.qrms_norm(rows[:, :h], w.norm_q, rows[:, :h], eps=self.eps)
            qg.qrms_norm(rows[:, h:h + kv], w.norm_k, rows[:, h:h + kv], eps=self.eps)
            q = new(n, h, d, dtype=half)
            qg.qkv_append(cache, rows[:, h:h + kv], rows[:, h + kv:], pos, rope=self.rope, q=rows[:, :h], q_out=q, err_flag=self.err)
            att = new(self.n_seq, ncols, h, d, dtype=half)
            qg.qattn_paged(cache, q.view(self.n_seq, ncols, h, d), self.lens, att, self.ws, err_flag=self.err)
            out = new(n, dim)
            qg.qgemm_cols(self.qtype, *w.wo, att.view(n, h * d), out)
            middle, b = new(n, dim), new(n, dim, dtype=half)
            qg.qrms_norm(residual, w.norm2, b, eps=self.eps, add=out, sum_out=middle)
            experts = w.router.shape[0]
            ffn = w.gate[1].shape[0] // experts
            chosen, rw, logits = new(n, self.topk, dtype=torch.int32), new(n, self.topk), new(n, experts)
            qg.qmoe_router_planned(self.route, w.router, b, self.topk, chosen, rw, bias=w.bias, logits_out=logits)
            moe_ws = new(qg.qmoe_workspace_bytes(experts, ffn, dim, n, self.topk), dtype=torch.uint8)
            delta = new(n, dim)
            qg.qmoe_experts(self.qtype, *w.gate, *w.up, *w.down, experts, ffn, dim, chosen, rw, b, delta, moe_ws)
            if keep is not None:
                keep.append(dict(x=x, residual=residual, a=a, projected=projected, rows=rows, q=q, att=att, out=out, middle=middle, b=b,
                                 logits=logits, chosen=chosen, rw=rw, ws=moe_ws, delta=delta, pos=pos))
            x = middle
        final, c = new(n, dim), new(n, dim, dtype=half)
        qg.qrms_norm(x, self.last_norm, c, eps=self.eps, add=delta, sum_out=final)
        logits = new(n, self.table[1].shape[0])
        qg.qgemm_cols(self.qtype, *self.table, c, logits)
        token = new(n, dtype=torch.int32)
        qg.qargmax_f32(logits, token)
        if keep is not None:
            keep.append(dict(x=x, delta=delta, final=final, c=c, logits=logits))
        return logits, token


def random_decoder(qtype, vocab, hidden, heads, kv_heads, head_dim, experts, ffn, n_layers, seed=0, route=None, **kw):
    """A decoder of random weights, and the GGUF-order (quants, scales) that they were packed from: the table's, then a dict a layer."""
    import numpy as np

    import synth
    g = synth.rng(seed)
    plain = []

    def packed(rows, k):
        q, s = synth.draw_matrix(g, qtype, rows, k)
        blocks = torch.from_numpy(np.ascontiguousarray(synth.to_gguf_blocks(qtype, q, s))).cuda()
        qd, sd = torch.empty(q.shape, dtype=torch.uint8, device="cuda"), torch.empty(s.shape, dtype=torch.int16, device="cuda")
        qg.qrepack(qtype, blocks, rows, k, qd, sd)
        return (qd, sd), (q, s)

    def vector(n, mean=1.0, size=0.1):
        return torch.from_numpy((mean + size * g.standard_normal(n)).astype(np.float32)).cuda()
    table, p = packed(vocab, hidden)
    plain.append(p)
    layers = []
    for _ in range(n_layers):
        dev, host = {}, {}
        for name, rows, k in (("wqkv", (heads + 2 * kv_heads) * head_dim, hidden), ("wo", hidden, heads * head_dim),
                              ("gate", experts * ffn, hidden), ("up", experts * ffn, hidden), ("down", experts * hidden, ffn)):
            dev[name], host[name] = packed(rows, k)
        router = torch.from_numpy((g.standard_normal((experts, hidden)) * hidden ** -0.5).astype(np.float32)).cuda()
        layers.append(Layer(router=router, bias=vector(experts, 0.0), norm1=vector(hidden), norm2=vector(hidden), norm_q=vector(head_dim),
                            norm_k=vector(head_dim), **dev))
        plain.append(host)
    route = route or qg.qroute_plan("sigmoid", n_group=4, top_group=2, group_top=2, scale=2.0)
    return Decoder(qtype, table, layers, vector(hidden), heads, kv_heads, head_dim, route=route, **kw), plain


def main():
    n_seq = 2
    model, _ = random_decoder(qg.Q8_0, vocab=1000, hidden=256, heads=8, kv_heads=2, head_dim=64, experts=32, ffn=64, n_layers=2,
                              n_seq=n_seq, tokens=512, topk=4)
    g = torch.Generator(device="cuda").manual_seed(0)
    prompt = torch.randint(0, 1000, (n_seq, 24), generator=g, device="cuda").to(torch.int32)
    for at in range(0, 24, 8):  # a prompt of 24 tokens in pieces of 8
        _, token = model.step(prompt[:, at:at + 8].reshape(-1).contiguous())
    token = token.view(n_seq, -1)[:, -1].contiguous()
    said = [token.tolist()]
    for _ in range(8):
        _, token = model.step(token)
        said.append(token.tolist())
    print(f"{model.lens.tolist()} tokens cached, decoded {said}, errors {int(model.err)}, device errors {qg.qg_device_error()}")


if __name__ == "__main__":
    main()
