"""Decoding with drafted tokens through one MoE transformer block.

Each step feeds every sequence its last decided token and a few drafts, and
runs, without a host synchronisation between the calls:

    qkv projection -> moe_rope_append -> moe_paged_attention -> output projection
    -> moe_layer_forward -> logits -> moe_verify_drafts

moe_verify_drafts leaves the decided tokens and the cache length that the next
step starts from. The drafts come from a bigram model (the block's embedding
and output matrix alone). Weights are random; run it as

    python examples/decode_step.py
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_mixture_experts_router_gb300 as moe  # noqa: E402


class Block:
    """Random weights and the buffers of up to `seqs` sequences of `longest` tokens."""

    def __init__(self, seqs, drafts, longest, d_model=256, heads=8, kv_heads=2, dim=64, experts=8, top_k=2,
                 d_ff=512, vocab=512, page=16, cache=moe.MOE_BF16, temperature=1.0, seed=0):
        self.B, self.n, self.V, self.temperature = seqs, drafts + 1, vocab, temperature
        self.T = T = seqs * self.n
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

        self.embed = torch.randn((vocab, d_model), generator=g, device="cuda").bfloat16()
        self.w_qkv = weight((heads + 2 * kv_heads) * dim, d_model)
        self.w_o = weight(d_model, heads * dim)
        self.w_router = weight(experts, d_model)
        self.w_gate, self.w_up = weight(experts, d_ff, d_model), weight(experts, d_ff, d_model)
        self.w_down = weight(experts, d_model, d_ff)
        self.w_out = 4 * weight(vocab, d_model)
        self.random = torch.Generator(device="cuda").manual_seed(seed + 1)

        # the cache: a pool of pages and each sequence's table into it
        per_seq = -(-longest // page)
        pages = seqs * per_seq
        shape = (pages, page, kv_heads, dim)
        kind = torch.uint8 if cache == moe.MOE_E4M3 else torch.bfloat16
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=kind, device="cuda") for _ in range(2))
        scale = (pages, kv_heads, page)
        self.k_scale, self.v_scale = ((torch.zeros(scale, device="cuda") for _ in range(2))
                                      if cache == moe.MOE_E4M3 else (None, None))
        self.table = torch.randperm(pages, generator=g, device="cuda").int().view(seqs, per_seq)
        self.cu = (self.n * torch.arange(seqs + 1, device="cuda")).int()

        wide = (heads + 2 * kv_heads) * dim
        self.attn = moe.attn_config(
            n_seqs=seqs, n_tokens=T, max_new=self.n, n_heads=heads, n_kv_heads=kv_heads, head_dim=dim,
            page_size=page, n_pages=pages, max_pages=per_seq, cache_dtype=cache, rot_dim=dim,
            q_stride=wide, k_stride=wide, v_stride=wide)
        self.attn_packed = moe.attn_config(
            n_seqs=seqs, n_tokens=T, max_new=self.n, n_heads=heads, n_kv_heads=kv_heads, head_dim=dim,
            page_size=page, n_pages=pages, max_pages=per_seq, cache_dtype=cache)
        self.layer = moe.config(T=T, d_model=d_model, n_experts=experts, top_k=top_k, d_ff=d_ff)
        self.verify = moe.verify_config(n_seqs=seqs, n_tokens=T, max_new=self.n, vocab=vocab)
        self.ws = {"append": moe.workspace(self.attn, "append"),
                   "attention": moe.workspace(self.attn_packed, "attention"),
                   "layer": moe.workspace(self.layer), "verify": moe.workspace(self.verify, "verify")}
        self.q = torch.empty((T, heads, dim), dtype=torch.bfloat16, device="cuda")
        self.context = torch.empty_like(self.q)
        self.y = torch.empty((T, d_model), dtype=torch.bfloat16, device="cuda")
        self.decided = torch.empty(T, dtype=torch.int32, device="cuda")
        self.accepted = torch.empty(seqs, dtype=torch.int32, device="cuda")
        self.next = torch.empty(seqs, dtype=torch.int32, device="cuda")

    def distribution(self, logits):
        """Probabilities at the block's temperature; 0: all on the best token."""
        if self.temperature == 0:
            return torch.nn.functional.one_hot(logits.argmax(-1), self.V).float()
        return torch.softmax(logits.float() / self.temperature, -1)

    def draft(self, last):
        """The step's tokens [B][n] (the last decided and the drafts) and the draft
        model's distributions [T][V]."""
        tokens, q = [last], []
        for _ in range(self.n):
            q.append(self.distribution(self.embed[tokens[-1].long()] @ self.w_out.t()))
            tokens.append(torch.multinomial(q[-1], 1, generator=self.random)[:, 0].int())
        return torch.stack(tokens[:-1], 1), torch.stack(q, 1).reshape(self.T, self.V)

    def target(self, tokens, kv_len):
        """The block's distributions [T][V] after each token; kv_len holds the new
        tokens too."""
        x = self.embed[tokens.reshape(-1).long()]
        qkv = (x @ self.w_qkv.t()).unflatten(1, (-1, self.dim))
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        moe.moe_rope_append(self.attn, q, k, v, None, self.cu, kv_len, self.table, self.q, self.k_cache,
                            self.v_cache, self.k_scale, self.v_scale, self.ws["append"])
        moe.moe_paged_attention(self.attn_packed, self.q, self.cu, kv_len, self.table, self.k_cache,
                                self.v_cache, self.k_scale, self.v_scale, self.context, None,
                                self.ws["attention"])
        x = x + self.context.flatten(1) @ self.w_o.t()
        moe.moe_layer_forward(self.layer, x, self.w_router, None, None, self.w_gate, self.w_up,
                              self.w_down, self.y, None, None, None, None, self.ws["layer"])
        return self.distribution((x + self.y) @ self.w_out.t())

    def step(self, last, cached):
        """One decoding step: the decided tokens [B][n] (-1 behind the last), the next
        `last` and `cached`."""
        tokens, q = self.draft(last)
        kv_len = cached + self.n
        p = self.target(tokens, kv_len)
        u = torch.rand(self.T, generator=self.random, device="cuda")
        u_sample = torch.rand(self.B, generator=self.random, device="cuda")
        moe.moe_verify_drafts(self.verify, p, q, tokens, u, u_sample, self.cu, kv_len, self.decided,
                              self.accepted, self.next, self.ws["verify"])
        decided = self.decided.view(self.B, self.n).clone()
        last = decided.gather(1, self.accepted.long()[:, None])[:, 0]
        return decided, last, self.next.clone()

    def status(self):
        return {name: moe.moe_stream_status(ws) for name, ws in self.ws.items()}


def decode(block, first, steps):
    """Runs the steps from one token a sequence; a list of each sequence's tokens."""
    last, cached = first, torch.zeros(block.B, dtype=torch.int32, device="cuda")
    rows = []
    for _ in range(steps):
        decided, last, cached = block.step(last, cached)
        rows.append(decided)
    out = torch.cat(rows, 1).tolist()
    return [[t for t in row if t >= 0] for row in out]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--e4m3", action="store_true", help="an E4M3 cache")
    a = ap.parse_args()
    block = Block(a.seqs, a.drafts, a.steps * (a.drafts + 1), cache=moe.MOE_E4M3 if a.e4m3 else moe.MOE_BF16)
    out = decode(block, torch.arange(a.seqs, device="cuda").int(), a.steps)
    assert not any(block.status().values()), block.status()
    total = sum(len(row) for row in out)
    print(f"{total} tokens for {a.seqs} sequences in {a.steps} steps: "
          f"{total / a.seqs / a.steps:.2f} a step with {a.drafts} drafts")
    print("first sequence:", out[0][:16], "...")


if __name__ == "__main__":
    main()
