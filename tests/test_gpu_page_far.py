"""Caches whose pages lie behind 2^32 bytes: append over page scales, attention by both kernels, copy on
write, compaction and copies give there what they give near the start."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from page_common import PageBatch

pytestmark = pytest.mark.gpu
PAGE, HEADS, DIM = 64, 2, 128
FAR = (5 << 30) // (PAGE * HEADS * DIM)  # a page behind 5 GB of each cache


@pytest.fixture(scope="module")
def caches():
    n = FAR + 64
    k, v = (torch.zeros((n, PAGE, HEADS, DIM), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((n, HEADS), device="cuda") for _ in range(2))
    return k, v, ks, vs


@pytest.mark.parametrize("new,heads", [(2, 4), (50, 8)])
def test_append_and_attention(caches, new, heads):
    bt = PageBatch(new=[new, 1], length=[200, 70], heads=heads, kv_heads=HEADS, dim=DIM, page=PAGE)
    near = bt.device_cache()
    for big, small in zip(caches, near):
        big[FAR:FAR + bt.n_pages] = small
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((bt.T, HEADS, DIM), generator=g).bfloat16().cuda() for _ in range(2))
    q = bt.q_rows.cuda()
    cu, length, table = bt.lists()
    outs = []
    for base, (kc, vc, ks, vs) in ((0, near), (FAR, caches)):
        cfg = bt.cfg(n_pages=kc.shape[0], rot_dim=64)
        out, lse = torch.empty((bt.T, heads, DIM), dtype=torch.bfloat16, device="cuda"), torch.empty((bt.T, heads), device="cuda")
        at, ws = table + base, moe.workspace(cfg, "append")
        turned = torch.empty_like(out)
        moe.moe_rope_append(cfg, q, k, v, None, cu, length, at, turned, kc, vc, ks, vs, ws)
        assert moe.moe_stream_status(ws) == 0
        ws = moe.workspace(cfg, "attention")
        moe.moe_paged_attention(cfg, turned, cu, length, at, kc, vc, ks, vs, out, lse, ws)
        assert moe.moe_stream_status(ws) == 0
        outs.append((out, lse, *(x[base:base + bt.n_pages] for x in (kc, vc, ks, vs))))
    for a, b in zip(*outs):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert torch.isfinite(outs[1][0].float()).all()


def test_pages(caches):
    k, v, ks, vs = caches
    n, g = k.shape[0], torch.Generator(device="cuda").manual_seed(2)
    for x in (k, v):
        x[FAR:] = torch.randint(0, 100, x[FAR:].shape, dtype=torch.uint8, device="cuda", generator=g)
    for x in (ks, vs):
        x[FAR:] = torch.rand(x[FAR:].shape, device="cuda", generator=g)
    cfg = moe.attn_config(n_seqs=2, n_tokens=0, n_heads=HEADS, n_kv_heads=HEADS, head_dim=DIM, page_size=PAGE, n_pages=n, max_pages=4,
                          cache_dtype=moe.MOE_E4M3_PAGE)
    ws = moe.workspace(cfg, "pages")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # one sequence of two pages, forked; all pages but a few far ones are held by others
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    refs[FAR + 40:FAR + 44] = 0
    table, out = i32([[FAR + 3, FAR + 5, -1, -1], [-1] * 4]), torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    granted = i32([100, 101])
    moe.moe_pages_update(cfg, i32([0, 0]), i32([100, 0]), i32([100, 100]), granted, table, refs, out, refs, granted, k, v, ks, vs, ws)
    assert moe.moe_stream_status(ws) == 0 and granted.tolist() == [100, 101]
    assert out.tolist() == [[FAR + 3, FAR + 5, -1, -1], [FAR + 3, FAR + 40, -1, -1]]
    for x in (k, v):
        assert torch.equal(x[FAR + 40, :36], x[FAR + 5, :36]) and not torch.equal(x[FAR + 40, 36:], x[FAR + 5, 36:])
    for x in (ks, vs):
        assert torch.equal(x[FAR + 40], x[FAR + 5])
    # out of the far end and back in
    src, dst = i32([FAR + 3, FAR + 40, 7]), i32([11, FAR + 20, FAR + 21])
    want = [x[src.long()].clone() for x in caches]
    moe.moe_pages_copy(cfg, src, dst, n, k, v, ks, vs, k, v, ks, vs, ws)
    assert moe.moe_stream_status(ws) == 0
    assert all(torch.equal(x[dst.long()], w) for x, w in zip(caches, want))
    # compaction: the highest page of those in use goes to the one free page, far from it
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    refs[2], page_map, live = 0, torch.empty_like(refs), i32([0])
    table, want = i32([[n - 1, FAR + 3, 0, 0], [0] * 4]), [x[n - 1].clone() for x in caches]
    moe.moe_pages_compact(cfg, i32([100, 0]), table, refs, out, refs, page_map, live, k, v, ks, vs, ws)
    assert moe.moe_stream_status(ws) == 0 and live.item() == n - 1 and out[0, :2].tolist() == [2, FAR + 3]
    assert all(torch.equal(x[2], w) for x, w in zip(caches, want))
