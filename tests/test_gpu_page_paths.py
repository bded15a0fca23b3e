"""Attention over E4M3 caches with page scales on the paths that ordinary batches do not take: values
that are not finite and that some rows see, long tables (checked as they are used), bad lists, and
caches that appends have built, scales raised within a page."""
import math

import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from page_common import PageBatch, append64
from serve_common import attention64
from test_gpu_page_cache import attend

pytestmark = pytest.mark.gpu

# up to 64 rows: the warp-level kernel; to 128: two streams of keys; above: two streams of rows
WILD = {
    "24 rows": dict(new=[6], length=[100], heads=4, kv_heads=1, dim=64, page=16),
    "120 rows, several blocks": dict(new=[60], length=[3000], heads=2, kv_heads=1, dim=64, page=32),
    "180 rows": dict(new=[90, 3], length=[300, 70], heads=2, kv_heads=1, dim=128, page=64),
    "180 rows, pages of 7": dict(new=[90, 3], length=[300, 70], heads=2, kv_heads=1, dim=64, page=7),
    "180 rows, several blocks": dict(new=[90], length=[2500], heads=2, kv_heads=1, dim=64, page=64),
    "180 rows, all of them new": dict(new=[90], length=[90], heads=2, kv_heads=1, dim=64, page=32),
    "100 rows in splits": dict(new=[25], length=[9100], heads=4, kv_heads=1, dim=64, page=64),
}


def matches(bt, more=0.0):
    """more: of the bound, for scales beyond 2^-40 .. 2^40, whose logarithms are in the weights' exponents
    (2^-15 of a weight, which fp16 rounds by 2^-11)."""
    out, lse = attend(bt)
    want, want_lse, tol, tol_lse = attention64(bt)
    tol *= 1 + more
    bad = np.isnan(want)
    assert np.array_equal(np.isnan(out), bad)
    assert (np.abs(out - want)[~bad] <= tol[~bad]).all()
    seen = np.isfinite(want_lse)
    assert (np.isneginf(lse) == ~seen).all()
    assert (np.abs(lse - want_lse)[seen] <= tol_lse[seen]).all()
    return bad


@pytest.mark.parametrize("window", [0, 40, 150])
@pytest.mark.parametrize("shape", WILD)
def test_nan_values_that_some_rows_see(shape, window):
    """At either end of what the rows see: rows that do not see them are as without them."""
    for spread in (1.0, 30.0):
        bt = PageBatch(**WILD[shape], window=window, spread=1.0)
        rs = np.random.RandomState(1)
        if spread > 1:  # scales of all sizes beside them
            used = bt.used.any(1)
            bt.v_scale[used] = torch.from_numpy(2.0 ** rs.randint(-90, 90, (int(used.sum()), bt.kv_heads))).float()
            bt.v[(bt.v & 0x7F) < 0x38] = 0x38
        n, new = bt.length[0], bt.new[0]
        for key, elements in ((n - 1, slice(None)), (n - new // 2, slice(3, 20)), (max(0, n - new - window + new // 3), slice(40, 41))):
            if window or key >= n - new:
                bt.v[int(bt.table[0, key // bt.page]), key % bt.page, :, elements] = 0x7F
        bad = matches(bt, 0.0 if spread == 1 else 2.0 ** -4)
        assert bad.any() and not bad.all()


@pytest.mark.parametrize("shape", [s for s in WILD if "splits" not in s])
def test_a_value_scale_that_is_not_finite_and_that_some_rows_see(shape):
    bt = PageBatch(**WILD[shape], spread=1.0)
    bt.v_scale[int(bt.table[0, (bt.length[0] - 1) // bt.page])] = math.nan
    matches(bt)


LONG = [dict(new=[2, 1], length=[150, 40], heads=4, kv_heads=2, dim=64, page=16), dict(new=[3], length=[100], heads=8, kv_heads=1, dim=256, page=16),
        dict(new=[40, 2], length=[150, 40], heads=4, kv_heads=2, dim=64, page=16), dict(new=[40], length=[700], heads=4, kv_heads=1, dim=128, page=64)]


@pytest.mark.parametrize("case", LONG, ids=lambda c: f"{c['new']}x{c['heads']}p{c['page']}")
def test_long_tables(case):
    """More than 4096 entries: the lists are checked where they are used, most blocks have no key, and
    entries behind a sequence's last page are not looked at (the batch has -7 there)."""
    bt = PageBatch(**case, columns=5000)
    matches(bt)
    cfg, (k, v, ks, vs), lists = bt.cfg(), bt.device_cache(), bt.lists()
    q, ws = bt.q_rows.cuda(), moe.workspace(cfg, "attention")
    out = torch.zeros((bt.T, bt.heads, bt.dim), dtype=torch.bfloat16, device="cuda")
    for page in (-1, bt.n_pages, 1 << 30):
        table = lists[2].clone()
        table[0, 1] = page
        moe.moe_paged_attention(cfg, q, lists[0], lists[1], table, k, v, ks, vs, out, None, ws)
        assert moe.moe_stream_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    moe.moe_paged_attention(cfg, q, *lists, k, v, ks, vs, out, None, ws)
    assert moe.moe_stream_status(ws) == 0


@pytest.mark.parametrize("columns", [1, 5000])
@pytest.mark.parametrize("new", [2, 40])
@pytest.mark.parametrize("name,at,value", [("table", (1, 1), 1 << 20), ("table", (1, 0), -1), ("length", 1, -1), ("length", 1, 1 << 29), ("cu", 2, 1000),
                                           ("cu", 1, -5), ("cu", 0, 1)])
def test_bad_lists_in_attention(name, at, value, new, columns):
    """Recorded; a sequence whose own lists are good is as ever (the first, where the table or a length
    of the second is wrong)."""
    bt = PageBatch(new=[new, 3], length=[100, 40], heads=4, kv_heads=1, dim=64, page=32, columns=columns)
    cfg, caches = bt.cfg(), bt.device_cache()
    q, ws = bt.q_rows.cuda(), moe.workspace(cfg, "attention")
    out = [torch.zeros((bt.T, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    moe.moe_paged_attention(cfg, q, *bt.lists(), *caches, out[0], None, ws)
    assert moe.moe_stream_status(ws) == 0
    lists = dict(cu=bt.cu.copy(), length=np.array(bt.length, np.int32), table=bt.table.copy())
    lists[name][at] = value
    dev = [torch.from_numpy(lists[n]).cuda() for n in ("cu", "length", "table")]
    moe.moe_paged_attention(cfg, q, *dev, *caches, out[1], None, ws)
    assert moe.moe_stream_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    if name != "cu":
        assert torch.equal(out[0][:new], out[1][:new])


@pytest.mark.parametrize("heads,page,dim", [(2, 8, 64), (32, 8, 64), (32, 32, 128), (4, 32, 256)])
def test_appended_caches_are_attended(heads, page, dim):
    """Tokens appended one to three at a time, some of them 2^6 times as large, so that pages' scales
    are raised and older codes multiplied; after each append the cache is what the definition says, and
    attention over it matches 64 bits over the codes and scales that it holds."""
    g = torch.Generator().manual_seed(heads + page)
    steps = [1, 3, 2, 1, 1, 3, 3, 2, 3, 1, 2]
    total = sum(steps)
    bt = PageBatch(new=[total], length=[total], heads=heads, kv_heads=1, dim=dim, page=page, spread=0.0, max_new=3)
    bt.k[:], bt.v[:], bt.k_scale[:], bt.v_scale[:] = 0, 0, 0.0, 0.0
    loud = torch.tensor([64.0 if i % 7 == 4 else 1.0 for i in range(total)])[:, None, None]
    keys, values = ((torch.randn((total, 1, dim), generator=g) * loud).bfloat16() for _ in range(2))
    kc, vc, ks, vs = bt.device_cache()
    at, raised = 0, 0
    for n in steps:
        k, v = keys[at:at + n], values[at:at + n]
        at += n
        bt.new, bt.length, bt.T, bt.cu = [n], [at], n, np.array([0, n], np.int32)
        bt.q_rows = (0.1 * torch.randn((n, heads * dim), generator=g)).bfloat16()
        bt.q = bt.q_rows.unflatten(1, (heads, dim))
        want = [append64(bt, c, s, x.double().numpy()) for c, s, x in ((bt.k, bt.k_scale, k), (bt.v, bt.v_scale, v))]
        cfg = bt.cfg(q_stride=0)
        ws = moe.workspace(cfg, "append")
        moe.moe_rope_append(cfg, None, k.cuda(), v.cuda(), None, *bt.lists(), None, kc, vc, ks, vs, ws)
        assert moe.moe_stream_status(ws) == 0
        was = bt.k_scale.clone()
        bt.k, bt.v, bt.k_scale, bt.v_scale = kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu()
        raised += int(((bt.k_scale > was) & (was > 0)).sum())
        for codes, scale, (value, scale64, touched) in ((bt.k, bt.k_scale, want[0]), (bt.v, bt.v_scale, want[1])):
            assert np.array_equal(scale.double().numpy(), scale64)
            have = codes.view(torch.float8_e4m3fn).double().numpy()
            # a code is rounded to half a step, 2^-4 of it or 2^-10 among the subnormals
            assert (np.abs(have - value)[touched] <= 2.0 ** -4 * np.abs(value[touched]) + 2.0 ** -10).all()
        cfg = bt.cfg(q_stride=0)
        out = torch.empty((n, heads, dim), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((n, heads), device="cuda")
        ws = moe.workspace(cfg, "attention")
        moe.moe_paged_attention(cfg, bt.q_rows.cuda(), *bt.lists(), kc, vc, ks, vs, out, lse, ws)
        assert moe.moe_stream_status(ws) == 0
        want_out, want_lse, tol, tol_lse = attention64(bt)
        assert (np.abs(out.double().cpu().numpy() - want_out) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - want_lse) <= tol_lse).all()
    assert raised > 0
