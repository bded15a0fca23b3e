"""Helpers of the tests of E4M3 caches with one scale per page and head: a batch over such
a cache, and the append in 64 bits, written from its definition."""
from __future__ import annotations

import math

import numpy as np
import torch

import sparse_mixture_experts_router_gb300 as moe
from serve_common import Batch

MIN_EXP, MAX_EXP = -110, 119


def scale64(amax):
    """The least power of two 2^e (in the range of scales) with amax <= 448 2^e."""
    if not amax > 0:
        return 2.0 ** MIN_EXP
    m, e = math.frexp(amax / 512)
    return 2.0 ** min(max(e + (m > 448 / 512), MIN_EXP), MAX_EXP)


class PageBatch(Batch):
    """A Batch whose pages hold E4M3 codes under one scale a head. Unused slots hold NaN
    codes, unused pages NaN scales. spread: powers of two that a page's elements range over."""

    def __init__(self, *a, spread=2.0, **kw):
        self.spread = spread
        super().__init__(*a, **{**kw, "cache": "e4m3"})
        g = torch.Generator().manual_seed(self.seed + 1)

        def make():
            x = torch.randn((self.n_pages, self.page, self.kv_heads, self.dim), generator=g)
            x *= torch.exp2(torch.empty(self.n_pages, 1, self.kv_heads, 1).uniform_(-self.spread, self.spread, generator=g))
            x[~self.used] = 0
            scale = torch.tensor([[scale64(float(x[p, :, h].abs().max())) for h in range(self.kv_heads)]
                                  for p in range(self.n_pages)], dtype=torch.float32).view(self.n_pages, self.kv_heads)
            codes = (x / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[~self.used] = 0x7F
            scale[~self.used.any(1)] = float("nan")
            return codes, scale

        self.k, self.k_scale = make()
        self.v, self.v_scale = make()

    def cfg(self, **kw):
        return super().cfg(**{"cache_dtype": moe.MOE_E4M3_PAGE, **kw})

    def line(self, which, b, i, h):
        x, s = (self.k, self.k_scale) if which == "k" else (self.v, self.v_scale)
        page, at = int(self.table[b, i // self.page]), i % self.page
        return (x[page, at, h].view(torch.float8_e4m3fn).double() * s[page, h].double()).numpy()


def rotated64(x, pos, rot, interleaved, sections, base=10000.0):
    """[T][heads][D] turned by positions [3][T], in 64 bits."""
    x = x.double().numpy().copy()
    pairs = rot // 2
    axis = np.repeat(np.arange(3), sections if sum(sections) else (pairs, 0, 0))
    for i in range(pairs):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        angle = (pos[axis[i]] * base ** (-2.0 * i / rot))[:, None]
        a, b = x[..., lo].copy(), x[..., hi].copy()
        x[..., lo] = a * np.cos(angle) - b * np.sin(angle)
        x[..., hi] = b * np.cos(angle) + a * np.sin(angle)
    return x


def append64(bt, codes, scale, x):
    """A cache (codes [page][place][head][dim], scales [page][head]) after x [T][heads][D]
    has been written: values in units of the new scales, the scales, and a mask of the rows
    that the call may change."""
    value = codes.view(torch.float8_e4m3fn).double().numpy().copy()
    scale = scale.double().numpy().copy()
    touched = np.zeros(value.shape[:2], bool)
    for b in range(bt.B):
        places = {}
        for j in range(bt.new[b]):
            at = bt.length[b] - bt.new[b] + j
            places.setdefault(int(bt.table[b, at // bt.page]), []).append((at % bt.page, int(bt.cu[b]) + j))
        for page, rows in places.items():
            first = rows[0][0]
            for h in range(value.shape[2]):
                new = np.stack([x[t, h] for _, t in rows])
                amax = np.abs(new[np.isfinite(new)]).max(initial=0.0)
                s = scale64(amax)
                if first > 0:
                    s = max(s, scale[page, h])
                    value[page, :first, h] *= scale[page, h] / s
                for place, t in rows:
                    value[page, place, h] = np.where(np.isfinite(x[t, h]), x[t, h] / s, np.nan)
                scale[page, h] = s
            touched[page, :rows[-1][0] + 1] = True
    return value, scale, touched
