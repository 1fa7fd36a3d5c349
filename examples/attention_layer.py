"""An attention layer of a decoder, served from the paged cache.

One call of ``AttentionLayer.step`` takes the hidden states of ``ncols`` new
tokens for each sequence (a prompt in pieces, one decoded token, or the tokens
of a speculative verify) through

    qgemm_cols   the fused QKV projection (Q4_0 / Q8_0 weights)
    qkv_append   rotary positions on q and k, k and v into the cache
    qattn_paged  attention over everything cached so far
    qgemm_cols   the output projection, added to the residual

``shift`` drops the first tokens of a sequence and moves the rest to the front
(a context shift): qkv_read, qrope by a negative position, qkv_append.

Run it on a GPU: python examples/attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_q4_q8_gb300 as qg  # noqa: E402


class AttentionLayer:
    """wqkv, wo: (quants, scales) of the fused projection [(heads + 2 kv_heads) * head_dim, hidden] and of the output
    projection [hidden, heads * head_dim], in the library's layout. The cache holds n_seq sequences of up to
    ``tokens`` tokens; pages are handed out in order here, a server would use an allocator of its own."""

    def __init__(self, qtype, wqkv, wo, heads, kv_heads, head_dim, n_seq, tokens, cache_type=qg.Q8_0, page_size=64,
                 rot_dim=None, base=1e6):
        self.qtype, self.wqkv, self.wo = qtype, wqkv, wo
        self.heads, self.kv, self.d, self.n_seq = heads, kv_heads, head_dim, n_seq
        pages = -(-tokens // page_size)
        nbytes = n_seq * pages * qg.qkv_page_bytes(cache_type, kv_heads, head_dim, page_size)
        self.pool = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        self.table = torch.arange(n_seq * pages, dtype=torch.int32, device="cuda").view(n_seq, pages)
        self.cache = qg.qkv_cache(cache_type, self.pool, self.table, kv_heads, head_dim, page_size)
        self.rope = qg.qrope_plan(rot_dim or head_dim, base=base)
        self.lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")  # tokens cached
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        most = max(qg.qattn_workspace_bytes(self.cache, heads, c) for c in range(1, 17))
        self.ws = torch.empty(most, dtype=torch.uint8, device="cuda")

    def step(self, x, residual):
        """x f16 [n_seq * ncols, hidden] (at most 16 rows, each sequence's tokens in order), residual f32 alike ->
        (residual + attention, and the values in between: QKV rows, rotated queries, attention output)."""
        ncols = x.shape[0] // self.n_seq
        n, h, kv, d = x.shape[0], self.heads, self.kv, self.d
        rows = torch.empty((n, h + 2 * kv, d), dtype=torch.float32, device="cuda")
        qg.qgemm_cols(self.qtype, *self.wqkv, x, rows)
        pos = (self.lens[:, None] + torch.arange(ncols, dtype=torch.int32, device="cuda")).reshape(-1).contiguous()
        self.lens += ncols
        q = torch.empty((n, h, d), dtype=torch.float16, device="cuda")
        qg.qkv_append(self.cache, rows[:, h:h + kv], rows[:, h + kv:], pos, rope=self.rope, q=rows[:, :h], q_out=q,
                      err_flag=self.err)
        att = torch.empty((self.n_seq, ncols, h, d), dtype=torch.float16, device="cuda")
        qg.qattn_paged(self.cache, q.view(self.n_seq, ncols, h, d), self.lens, att, self.ws, err_flag=self.err)
        y = torch.empty_like(residual)
        qg.qgemm_cols(self.qtype, *self.wo, att.view(n, h * d), y, residual)
        return y, (rows, q, att)

    def shift(self, seq, drop):
        """Forget the first ``drop`` tokens of a sequence: what is left moves to position 0 onward, its keys turned back
        by ``drop`` positions (rotations add up, so the scores among them stay what they were)."""
        n = int(self.lens[seq]) - drop
        if n > 0:
            at = torch.arange(drop, drop + n, dtype=torch.int32, device="cuda")
            which = torch.full_like(at, seq)
            k, v = (torch.empty((n, self.kv, self.d), dtype=torch.float32, device="cuda") for _ in range(2))
            qg.qkv_read(self.cache, at, k, v, seq=which, err_flag=self.err)
            qg.qrope(self.rope, k, torch.full_like(at, -drop), k)
            qg.qkv_append(self.cache, k, v, at - drop, seq=which, err_flag=self.err)
        self.lens[seq] = max(n, 0)


def random_layer(qtype, hidden, heads, kv_heads, head_dim, seed=0, **kw):
    """A layer of random weights (and the GGUF blocks they were packed from)."""
    import numpy as np

    import synth
    g = synth.rng(seed)
    packed, plain = [], []
    for rows, k in (((heads + 2 * kv_heads) * head_dim, hidden), (hidden, heads * head_dim)):
        q, s = synth.draw_matrix(g, qtype, rows, k)
        blocks = torch.from_numpy(np.ascontiguousarray(synth.to_gguf_blocks(qtype, q, s))).cuda()
        qd = torch.empty(q.shape, dtype=torch.uint8, device="cuda")
        sd = torch.empty(s.shape, dtype=torch.int16, device="cuda")
        qg.qrepack(qtype, blocks, rows, k, qd, sd)
        packed.append((qd, sd))
        plain.append((q, s))
    return AttentionLayer(qtype, *packed, heads, kv_heads, head_dim, **kw), plain


def main():
    torch.manual_seed(0)
    hidden, n_seq = 2048, 2
    layer, _ = random_layer(qg.Q8_0, hidden, heads=16, kv_heads=2, head_dim=256, n_seq=n_seq, tokens=4096, rot_dim=64)
    for piece in (8, 8, 8, 1, 1, 4):  # a prompt of 24 tokens, two decoded ones, a verify of four
        x = torch.randn(n_seq * piece, hidden, device="cuda")
        y, _ = layer.step(x.half(), x)
        print(f"{piece} tokens a sequence -> {layer.lens.tolist()} cached, mean |y| {y.abs().mean().item():.3f}")
    layer.shift(0, 10)
    x = torch.randn(n_seq, hidden, device="cuda")
    y, _ = layer.step(x.half(), x)
    print(f"after a shift by 10: {layer.lens.tolist()} cached, errors {int(layer.err)}, "
          f"device errors {qg.qg_device_error()}, mean |y| {y.abs().mean().item():.3f}")


if __name__ == "__main__":
    main()
