"""Batches whose outputs show the rounding of the attention's weights, and its bound."""
import math

import numpy as np
import torch

from serve_common import STEP, Batch

# Weights of a bf16 cache are two bf16 terms: hi rounded down leaves less than
# 2^-7 of the weight, rounding that is off by 2^-8 of it, in the worst case
# (weight at a power of two) 2^-16 of the weight, and hi 2^-23 is added.
WEIGHT_STEP = {"bf16": 2.0 ** -16 + 2.0 ** -23, "e4m3": STEP["f16"], "f32": STEP["f32"]}


def cancelling(new, length, heads, kv_heads, dim, cache="bf16", **kw):
    """Keys in pairs of nearly the same weight (2^-9 apart) and opposite values: a row's
    sum is far below the sum of its terms' magnitudes, and so is its rounding."""
    bt = Batch(new=new, length=length, heads=heads, kv_heads=kv_heads, dim=dim, page=16, cache=cache, values=0.5, **kw)
    bt.q[..., dim - 1] = 1
    for b, n in enumerate(length):
        for i in range(1, n, 2):
            a = int(bt.table[b, (i - 1) // 16]), (i - 1) % 16
            c = int(bt.table[b, i // 16]), i % 16
            bt.k[a][..., dim - 1] = 0
            bt.k[c] = bt.k[a]
            bt.k[c][..., dim - 1] = 2.0 ** -9 * math.sqrt(dim)
            bt.v[c] = -bt.v[a]
    return bt


def rows64(bt, round_weights=lambda w: w):
    """out in 64 bits with the weights (relative to a row's largest) rounded by the
    function given, and the bound of the difference from unrounded ones."""
    scale = 1 / math.sqrt(bt.dim)
    out, tol = np.zeros((bt.T, bt.heads, bt.dim)), np.zeros((bt.T, bt.heads, bt.dim))
    G, u = bt.heads // bt.kv_heads, STEP["f32"]
    for b in range(bt.B):
        n = bt.length[b]
        for kh in range(bt.kv_heads if n > 0 else 0):
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
                    w = np.exp(s - s.max())
                    out[t, h] = round_weights(w) @ v / w.sum()
                    # a score: dim products and sums in fp32, the scale, and exp
                    ds = (bt.dim + 4) * u * (np.abs(k) @ np.abs(q)).max() * scale + 8 * u * (np.abs(s).max() + 1)
                    sums = (len(k) + 8) * u
                    tol[t, h] = STEP[bt.dtype] * np.abs(out[t, h]) + (WEIGHT_STEP[bt.cache] + 2 * ds + 2 * sums) * (w @ np.abs(v) / w.sum()) * 1.01 + 1e-30
    return out, tol


def bf16(x):
    return torch.from_numpy(x).float().bfloat16().double().numpy()


def one_term(w):
    return bf16(w)


def two_terms(w):
    w = w.astype(np.float32)
    hi = (w.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
    return hi + bf16(w.astype(np.float64) - hi * (1 - 2.0 ** -23))


def rounding_of_sums(dim, sums):
    """The most that `dim` additions of numbers next to 1 can be off in that many sums (of
    equal length, added pairwise), each addition by half a step of its result."""
    def half_step(x):
        return 2.0 ** math.floor(math.log2(x)) * STEP["f32"]
    length, total = dim // sums, 0.0
    total += sums * sum(half_step(i + 1e-3) for i in range(1, length + 1))
    while sums > 1:
        length, sums = 2 * length, sums // 2
        total += sums * half_step(length + 1e-3)
    return total
