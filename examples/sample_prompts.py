"""Several samples of each of a few prompts through one MoE transformer block, over one
pool of pages: a prompt is computed and kept once, its samples share its pages.

    moe_pages_update     room for the prompts
    prompts              qkv -> moe_rope_append -> moe_paged_attention -> layer
    moe_pages_update     each prompt forked into its samples (the page it ends in is copied)
    each step            moe_logits_probs -> moe_verify_drafts (which draws, as nothing is
                         drafted) -> moe_pages_update -> qkv -> ... -> logits

without a host synchronisation between the calls. The cache holds E4M3 codes under one scale
a page and head; tokens that a sample has had are penalised. A sample that the pool has no
room for appends nothing, and stops or waits for the next step. Weights are random; run it as

    python examples/sample_prompts.py
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_mixture_experts_router_gb300 as moe  # noqa: E402


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Samples:
    """`samples` sequences for each of `prompts` (lists of tokens), with room for `steps` tokens, or in
    a pool of so many `pages`."""

    def __init__(self, prompts, samples, steps, d_model=256, heads=8, kv_heads=2, dim=64, experts=8, top_k=2, d_ff=512, vocab=512,
                 page=32, temperature=1.0, frequency=0.5, repetition=1.1, seed=0, pages=None):
        self.prompts, self.S, self.V = prompts, samples, vocab
        self.B = B = len(prompts) * samples
        self.heads, self.kv_heads, self.dim, self.d_model = heads, kv_heads, dim, d_model
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

        self.embed = torch.randn((vocab, d_model), generator=g, device="cuda").bfloat16()
        self.w_qkv, self.w_o = weight((heads + 2 * kv_heads) * dim, d_model), weight(d_model, heads * dim)
        self.w_router = weight(experts, d_model)
        self.w_gate, self.w_up = weight(experts, d_ff, d_model), weight(experts, d_ff, d_model)
        self.w_down, self.w_out = weight(experts, d_model, d_ff), 4 * weight(vocab, d_model)
        self.random = torch.Generator(device="cuda").manual_seed(seed + 1)

        # the pool: the prompts' pages, and each sample's own
        longest = max(len(p) for p in prompts) + steps + 1
        columns = -(-longest // page)
        self.pages = pages or sum(-(-len(p) // page) for p in prompts) + B * (-(-(steps + 1) // page) + 2)
        self.k_cache, self.v_cache = (torch.zeros((self.pages, page, kv_heads, dim), dtype=torch.uint8, device="cuda") for _ in range(2))
        self.k_scale, self.v_scale = (torch.zeros((self.pages, kv_heads), device="cuda") for _ in range(2))
        self.tables = [torch.zeros((B, columns), dtype=torch.int32, device="cuda") for _ in range(2)]
        self.refs = torch.zeros(self.pages, dtype=torch.int32, device="cuda")
        self.length = torch.zeros(B, dtype=torch.int32, device="cuda")  # tokens there is room for
        self.live = torch.ones(B, dtype=torch.bool, device="cuda")  # samples that go on
        self.ws, self.columns, self.page = {}, columns, page
        self.layers = dict(d_model=d_model, n_experts=experts, top_k=top_k, d_ff=d_ff)

        # what each sample has had: the prompt, and room for what is generated
        width = longest
        history = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        for i, p in enumerate(prompts):
            history[i * samples:(i + 1) * samples, :len(p)] = ints(p)
        self.history, self.cu_history = history, ints([b * width for b in range(B + 1)])
        self.n_prompt = ints([len(p) for p in prompts for _ in range(samples)])
        full = lambda x: torch.full((B,), x, device="cuda")  # noqa: E731
        self.temperature, self.frequency, self.repetition = full(float(temperature)), full(float(frequency)), full(float(repetition))
        self.logits_cfg = moe.logits_config(n_seqs=B, n_tokens=B, vocab=vocab, n_history=B * width)
        self.verify_cfg = moe.verify_config(n_seqs=B, n_tokens=B, vocab=vocab)
        self.one_each = ints(list(range(B + 1)))
        self.p = torch.empty((B, vocab), device="cuda")
        self.ones = torch.ones(B, device="cuda")
        self.accepted = torch.empty(B, dtype=torch.int32, device="cuda")

    def cfg(self, tokens, most, **kw):
        return moe.attn_config(n_seqs=self.B, n_tokens=tokens, max_new=most, n_heads=self.heads, n_kv_heads=self.kv_heads,
                               head_dim=self.dim, page_size=self.page, n_pages=self.pages, max_pages=self.columns,
                               cache_dtype=moe.MOE_E4M3_PAGE, **kw)

    def workspace(self, name, cfg, kind):
        if name not in self.ws:
            self.ws[name] = moe.workspace(cfg, kind)
        return self.ws[name]

    def update(self, parent, kept, need):
        """Sequences made anew; `need` becomes what was granted."""
        cfg, (old, new) = self.cfg(0, 1), self.tables
        moe.moe_pages_update(cfg, parent, self.length, kept, need, old, self.refs, new, self.refs, need, self.k_cache, self.v_cache,
                             self.k_scale, self.v_scale, self.workspace("pages", cfg, "pages"))
        self.tables, self.length = [new, old], need

    def grow(self, parent, kept):
        """Room for one more token behind `kept` of each sample that goes on. A refused one keeps what it
        has (its granted length is `kept`): a token written all the same would go over the last one it
        has, in a page that others may hold. The first refused one does not fit, and stops; those behind
        it are refused with it, and ask again with the next step."""
        self.update(parent, kept, kept + self.live.int())
        self.room = self.live & (self.length > kept)
        refused = self.live & ~self.room
        self.live = self.live & ~(refused & (refused.cumsum(0) == 1))

    def block(self, name, tokens, cu, length, most):
        """The block's output rows of new tokens, whose keys and values go into the pages."""
        T, wide = tokens.numel(), (self.heads + 2 * self.kv_heads) * self.dim
        x = self.embed[tokens.long()]
        q, k, v = (x @ self.w_qkv.t()).unflatten(1, (-1, self.dim)).split([self.heads, self.kv_heads, self.kv_heads], 1)
        caches, table = (self.k_cache, self.v_cache, self.k_scale, self.v_scale), self.tables[0]
        rows = torch.empty((T, self.heads, self.dim), dtype=torch.bfloat16, device="cuda")
        cfg = self.cfg(T, most, rot_dim=self.dim, q_stride=wide, k_stride=wide, v_stride=wide)
        moe.moe_rope_append(cfg, q, k, v, None, cu, length, table, rows, *caches, self.workspace(name + " append", cfg, "append"))
        cfg, context = self.cfg(T, most), torch.empty_like(rows)
        moe.moe_paged_attention(cfg, rows, cu, length, table, *caches, context, None, self.workspace(name + " attention", cfg, "attention"))
        x = x + context.flatten(1) @ self.w_o.t()
        layer, y = moe.config(T=T, **self.layers), torch.empty_like(x)
        moe.moe_layer_forward(layer, x, self.w_router, None, None, self.w_gate, self.w_up, self.w_down, y, None, None, None, None,
                              self.workspace(name + " layer", layer, "layer"))
        return x + y

    def start(self):
        """Computes the prompts, by the first sample of each, and forks them: the logits that
        every sample starts from."""
        first = [len(p) if s == 0 else 0 for p in self.prompts for s in range(self.S)]
        none = torch.zeros_like(self.length)
        self.update(None, none, ints(first))
        cu = [0]
        for n in first:
            cu.append(cu[-1] + n)
        x = self.block("prompts", ints([t for p in self.prompts for t in p]), ints(cu), self.length, max(first))
        ends = ints([cu[i * self.S + 1] - 1 for i in range(len(self.prompts))]).long().repeat_interleave(self.S)
        parent = ints([b // self.S * self.S for b in range(self.B)])
        kept = self.length[parent.long()]
        self.live = kept > 0  # a prompt that found no room has none
        self.grow(parent, kept)
        return (x[ends] @ self.w_out.t()).float()

    def draw(self, logits):
        """The samples' next tokens."""
        cfg = self.logits_cfg
        moe.moe_logits_probs(cfg, logits, self.one_each, None, self.history, self.cu_history, self.n_prompt, self.repetition, None,
                             self.frequency, None, None, None, None, None, self.temperature, self.p, self.workspace("logits", cfg, "logits"))
        tokens = torch.empty(self.B, dtype=torch.int32, device="cuda")
        u = torch.rand(self.B, generator=self.random, device="cuda")
        moe.moe_verify_drafts(self.verify_cfg, self.p, None, tokens, self.ones, u, self.one_each, None, tokens, self.accepted, None,
                              self.workspace("verify", self.verify_cfg, "verify"))
        return tokens

    def generate(self, steps):
        """[B][steps] tokens, -1 where a sample had no room."""
        logits, out = self.start(), []
        for _ in range(steps):
            tokens = torch.where(self.room, self.draw(logits), -1)
            out.append(tokens)
            # self.length counts the token just drawn: it goes behind what is cached
            at = (self.length.long()[:, None] - 1).clamp(min=0)
            self.history.scatter_(1, at, torch.where(self.room[:, None], tokens[:, None], self.history.gather(1, at)))
            # length 0: a token without a slot is not written (and recorded by the append)
            x = self.block("step", tokens, self.one_each, torch.where(self.room, self.length, 0), 1)
            logits = torch.where(self.room[:, None], (x @ self.w_out.t()).float(), logits)
            self.grow(None, self.length)
        return torch.stack(out, 1)

    def status(self):
        return {name: moe.moe_stream_status(ws) for name, ws in self.ws.items()}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--prompts", type=int, default=4)
    ap.add_argument("--samples", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    prompts = [[(7 * i + 3 * t) % 512 for t in range(40 + 25 * i)] for i in range(a.prompts)]
    s = Samples(prompts, a.samples, a.steps)
    out = s.generate(a.steps)
    stopped = int((~s.live).sum())
    assert stopped or not any(s.status().values()), s.status()
    held = int((s.refs > 0).sum())
    alone = sum(-(-int(n) // s.page) for n in s.length.tolist())
    print(f"{out.numel()} tokens of {s.B} samples; {held} pages held, {alone} if none were shared; {stopped} stopped for want of room")
    print("first samples:", *out[:2, :12].tolist(), sep="\n  ")


if __name__ == "__main__":
    main()
