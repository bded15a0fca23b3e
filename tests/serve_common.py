"""Helpers of the decode-step tests: a batch with its block table and cache,
and 64-bit implementations of the three operators written from their
definitions (numpy, one row at a time)."""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch

import sparse_mixture_experts_router_gb300 as moe

# Largest relative error of one rounding to nearest, half a step.
STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
DTYPE = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "e4m3": moe.MOE_E4M3}


@dataclasses.dataclass
class Batch:
    """Lists of a batch and a cache of the kind asked for. Slots that no
    position uses hold NaN (E4M3: NaN codes and scales)."""
    new: list
    length: list
    heads: int
    kv_heads: int
    dim: int
    page: int
    cache: str = "bf16"
    window: int = 0
    order: str = "token"      # "token": [page][token][head][dim], "head": [page][head][token][dim]
    q_pad: int = 0            # elements between one token's heads and the next token's
    spare: int = 3
    seed: int = 0
    max_new: int = 0
    values: float = 1.0       # standard deviation of q
    columns: int = 1          # of the block table, at least

    def __post_init__(self):
        rs = self.rs = np.random.RandomState(self.seed)
        self.B, self.T = len(self.new), int(sum(self.new))
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        pages = [-(-max(n, 0) // self.page) for n in self.length]
        self.n_pages = sum(pages) + self.spare
        ids = rs.permutation(self.n_pages)
        self.table = np.full((self.B, max(self.columns, max(pages, default=1))), -7, np.int32)  # unused: no page
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.dtype = "f32" if self.cache == "f32" else "bf16"
        g = torch.Generator().manual_seed(self.seed)
        used = torch.zeros((self.n_pages, self.page), dtype=torch.bool)
        for b, n in enumerate(self.length):
            for i in range(max(n, 0)):
                used[int(self.table[b, i // self.page]), i % self.page] = True
        self.used = used
        shape = (self.n_pages, self.page, self.kv_heads, self.dim)

        def make():
            x = torch.randn(shape, generator=g)
            if self.cache != "e4m3":
                x = x.to(TORCH[self.cache])
                x[~used] = float("nan")
                return x, None
            amax = x.abs().amax(-1)
            codes = (x * (448 / amax)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[~used] = 0x7F  # NaN
            scale = amax / 448
            scale[~used] = float("nan")
            return codes, scale.transpose(1, 2).contiguous()

        self.k, self.k_scale = make()
        self.v, self.v_scale = make()
        row = self.heads * self.dim + self.q_pad
        self.q_rows = (self.values * torch.randn((max(self.T, 1), row), generator=g)).to(TORCH[self.dtype])
        self.q = self.q_rows[:self.T, :self.heads * self.dim].unflatten(1, (self.heads, self.dim))

    # -- device side
    def cfg(self, **kw):
        strides = {}
        if self.order == "head":
            strides = dict(page_stride=self.page * self.kv_heads * self.dim, token_stride=self.dim,
                           head_stride=self.page * self.dim)
        return moe.attn_config(**{**dict(
            n_seqs=self.B, n_tokens=self.T, max_new=self.max_new or max(1, max(self.new, default=1)),
            n_heads=self.heads, n_kv_heads=self.kv_heads, head_dim=self.dim, page_size=self.page,
            n_pages=self.n_pages, max_pages=self.table.shape[1], dtype=DTYPE[self.dtype],
            cache_dtype=DTYPE[self.cache], window=self.window,
            q_stride=self.heads * self.dim + self.q_pad), **strides, **kw})

    def lists(self):
        return tuple(torch.from_numpy(np.asarray(x, np.int32)).cuda()
                     for x in (self.cu, self.length, self.table))

    def device_cache(self):
        """(k, v, k_scale, v_scale) on the GPU, in this batch's order."""
        def put(x):
            x = x.transpose(1, 2).contiguous() if self.order == "head" else x
            return x.cuda()
        s = [None if x is None else x.cuda() for x in (self.k_scale, self.v_scale)]
        return put(self.k), put(self.v), s[0], s[1]

    def back(self, x):
        """A device cache in [page][token][head][dim] order on the host."""
        x = x.cpu()
        return x.transpose(1, 2) if self.order == "head" else x

    # -- 64-bit values
    def line(self, which, b, i, h):
        x, s = (self.k, self.k_scale) if which == "k" else (self.v, self.v_scale)
        page, at = int(self.table[b, i // self.page]), i % self.page
        if s is None:
            return x[page, at, h].double().numpy()
        return (x[page, at, h].view(torch.float8_e4m3fn).double() * s[page, h, at].double()).numpy()


def attention64(bt: Batch, scale=None):
    """out, lse, and for each output the bound of what fp32 scores, sums and
    one rounding of the weights and of the result may move it by."""
    scale = scale or 1 / math.sqrt(bt.dim)
    out = np.zeros((bt.T, bt.heads, bt.dim))
    lse = np.full((bt.T, bt.heads), -np.inf)
    tol_out, tol_lse = np.zeros_like(out), np.zeros_like(lse)
    G = bt.heads // bt.kv_heads
    weight_step = STEP["f16"] if bt.cache == "e4m3" else STEP[bt.cache]
    u = STEP["f32"]
    for b in range(bt.B):
        n = bt.length[b]
        for kh in range(bt.kv_heads):
            if n <= 0:
                continue
            K = np.stack([bt.line("k", b, i, kh) for i in range(n)])
            V = np.stack([bt.line("v", b, i, kh) for i in range(n)])
            for j in range(bt.new[b]):
                pos = n - bt.new[b] + j
                if pos < 0:
                    continue
                first = max(0, pos - bt.window + 1) if bt.window else 0
                k, v = K[first:pos + 1], V[first:pos + 1]
                for h in range(kh * G, kh * G + G):
                    t = bt.cu[b] + j
                    q = bt.q[t, h].double().numpy()
                    s = k @ q * scale
                    m = s.max()
                    w = np.exp(s - m)
                    l = w.sum()
                    out[t, h] = w @ v / l
                    lse[t, h] = m + math.log(l)
                    # a score: D products and sums in fp32, the scale, and exp
                    ds = (bt.dim + 4) * u * (np.abs(k) @ np.abs(q)).max() * abs(scale) + 8 * u * (np.abs(s).max() + 1)
                    sums = (len(k) + 8) * u
                    reach = w @ np.abs(v) / l
                    tol_out[t, h] = STEP[bt.dtype] * np.abs(out[t, h]) + (weight_step + 2 * ds + 2 * sums) * reach * 1.01 + 1e-30
                    tol_lse[t, h] = ds + sums + 4 * u * abs(lse[t, h])
    return out, lse, tol_out, tol_lse


def verify64(p, q, tokens, u, us, cu, length):
    """Tokens, accepted counts and next lengths, exactly: Python integers over
    2^-1100 for the sums (p, q fp32 values as numpy float64)."""
    from fractions import Fraction
    out, acc, nxt = [], [], []
    V = p.shape[1]
    for b in range(len(cu) - 1):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if hi == lo:
            acc.append(0)
            nxt.append(int(length[b]))
            continue
        got = []
        while len(got) < hi - lo - 1:
            j = lo + len(got)
            x = int(tokens[j + 1])
            if not 0 <= x < V:
                break
            qx = Fraction(1) if q is None else Fraction(float(q[j, x]))
            if not Fraction(float(u[j])) * qx < Fraction(float(p[j, x])):
                break
            got.append(x)
        a = len(got)
        target = [Fraction(float(v)) for v in p[lo + a]]
        rest = target
        if a < hi - lo - 1:
            if q is None:
                x = int(tokens[lo + a + 1])
                rest = [max(v - (1 if i == x else 0), Fraction(0)) for i, v in enumerate(target)]
            else:
                rest = [max(v - Fraction(float(w)), Fraction(0)) for v, w in zip(target, q[lo + a])]
        total = sum(rest)
        if total == 0:
            rest, total = target, sum(target)
        drawn, run = -1, Fraction(0)
        for i, v in enumerate(rest):
            run += v
            if run > Fraction(float(us[b])) * total:
                drawn = i
                break
        out += got + [drawn] + [-1] * (hi - lo - a - 1)
        acc.append(a)
        nxt.append(int(length[b]) - (hi - lo - 1 - a))
    return np.array(out), np.array(acc), np.array(nxt)
