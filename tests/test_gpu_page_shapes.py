"""Attention of many rows over E4M3 caches with page scales: head sizes and groups of every kind, orders
and strides, sequences that begin before their cache, bounds far above the batch, negative scales."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from page_common import PageBatch
from serve_common import attention64

pytestmark = pytest.mark.gpu


def check(bt, scale=0.0):
    cfg, (k, v, ks, vs) = bt.cfg(scale=scale), bt.device_cache()
    out = torch.full((bt.T, bt.heads, bt.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((bt.T, bt.heads), 7.0, device="cuda")
    ws = moe.workspace(cfg, "attention")
    ws.fill_(0xA5)
    moe.moe_paged_attention(cfg, bt.q_rows.cuda(), *bt.lists(), k, v, ks, vs, out, lse, ws)
    assert moe.moe_stream_status(ws) == 0
    want, want_lse, tol, tol_lse = attention64(bt, scale)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(out - want) <= tol).all(), (np.abs(out - want) / tol).max()
    seen = np.isfinite(want_lse)
    assert (np.isneginf(lse) == ~seen).all()
    assert (np.abs(lse - want_lse)[seen] <= tol_lse[seen]).all()


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("new", [[36, 2], [90]])
def test_head_sizes(new, dim, page):
    check(PageBatch(new=new, length=[150, 40][:len(new)], heads=4, kv_heads=2, dim=dim, page=page, seed=dim))


@pytest.mark.parametrize("heads,kv_heads,new", [(71, 1, 2), (5, 1, 27), (65, 1, 1), (129, 1, 1), (3, 3, 100), (17, 1, 8), (66, 2, 4), (1, 1, 300)])
def test_groups(heads, kv_heads, new):
    """Rows of 65, 128, 129, 256 and 257 and more, odd groups among them."""
    check(PageBatch(new=[new, 1], length=[330, 9], heads=heads, kv_heads=kv_heads, dim=64, page=64, seed=heads))


@pytest.mark.parametrize("rows", [64, 65, 127, 128, 129, 255, 256, 257, 385])
def test_numbers_of_rows(rows):
    check(PageBatch(new=[rows], length=[rows + 70], heads=1, kv_heads=1, dim=64, page=32, seed=rows))


@pytest.mark.parametrize("page", [7, 16, 64])
@pytest.mark.parametrize("new", [40, 90])
def test_orders_and_strides(new, page):
    check(PageBatch(new=[new, 5], length=[200, 90], heads=4, kv_heads=2, dim=96, page=page, order="head", q_pad=64))


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("window", [0, 1, 7, 200])
def test_rows_before_the_first_key(page, window):
    """More new tokens than the cache has: the first rows see nothing; sequences of nothing and of one."""
    check(PageBatch(new=[100, 40, 1, 0, 70], length=[30, 0, 1, 5, 70], heads=4, kv_heads=2, dim=64, page=page, window=window))


@pytest.mark.parametrize("new", [[1, 3, 1], [70, 1, 2]])
def test_bounds_far_above_the_batch(new):
    check(PageBatch(new=new, length=[300, 1000, 64], heads=8, kv_heads=2, dim=128, page=64, max_new=2000, columns=40))


@pytest.mark.parametrize("new,heads", [(1, 8), (12, 4), (40, 4), (90, 4)])
@pytest.mark.parametrize("scale", [-0.2, 0.7, 1e-30])
def test_scales_of_scores(new, heads, scale):
    bt = PageBatch(new=[new], length=[170], heads=heads, kv_heads=2, dim=64, page=32, spread=1.0)
    check(bt, scale)
    bt.v[int(bt.table[0, 160 // 32]), 160 % 32] = 0x7F  # a NaN value, which the rows from its position on see
    cfg, (k, v, ks, vs) = bt.cfg(scale=scale), bt.device_cache()
    out = torch.empty((bt.T, heads, 64), dtype=torch.bfloat16, device="cuda")
    ws = moe.workspace(cfg, "attention")
    moe.moe_paged_attention(cfg, bt.q_rows.cuda(), *bt.lists(), k, v, ks, vs, out, None, ws)
    want, _, tol, _ = attention64(bt, scale)
    got, bad = out.double().cpu().numpy(), np.isnan(want)
    assert np.array_equal(np.isnan(got), bad) and (np.abs(got - want)[~bad] <= tol[~bad]).all()


def test_two_streams_at_once():
    """Two batches on two streams with workspaces of their own, and each graph replayed beside the other's."""
    batches = [PageBatch(new=[40, 3], length=[900, 200], heads=8, kv_heads=2, dim=128, page=16, seed=1),
               PageBatch(new=[90], length=[3000], heads=4, kv_heads=1, dim=64, page=64, seed=2)]
    calls, streams = [], [torch.cuda.Stream() for _ in batches]
    for bt in batches:
        cfg = bt.cfg()
        out = [torch.zeros((bt.T, bt.heads, bt.dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        calls.append((cfg, bt.q_rows.cuda(), bt.lists(), bt.device_cache(), out, moe.workspace(cfg, "attention")))

    def run(c, which, stream=None):
        cfg, q, lists, caches, out, ws = c
        moe.moe_paged_attention(cfg, q, *lists, *caches, out[which], None, ws, stream)

    for c in calls:
        run(c, 0)
    torch.cuda.synchronize()
    graphs = []
    for c, s in zip(calls, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(c, 1, s)
        graphs.append(g)
    for _ in range(10):
        for c in calls:
            c[4][1].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for c, s in zip(calls, streams):
            run(c, 1, s)
        torch.cuda.synchronize()
        assert all(torch.equal(c[4][0], c[4][1]) for c in calls)
        assert all(moe.moe_stream_status(c[5]) == 0 for c in calls)
