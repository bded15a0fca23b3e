"""Attention over E4M3 caches whose values' scales lie anywhere between 2^-110 and 2^119: the sum of
weights has no scales in it, the weighted values have, and neither may push the other out of range."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from page_common import PageBatch
from serve_common import Batch, attention64
from test_gpu_page_cache import attend as attend_pages
from test_gpu_paged_attention import Call

pytestmark = pytest.mark.gpu

# The warp-level kernel (up to 64 rows a head group, heads above 128) with its tile counts, the
# tcgen05 kernel by keys (to 128 rows) and by rows, over pages of whole groups of 32 keys and others;
# several blocks an item; splits.
SHAPES = {
    "1 row": dict(new=[1, 1], length=[200, 33], heads=2, kv_heads=2, dim=128, page=16),
    "12 rows": dict(new=[3, 1], length=[100, 300], heads=8, kv_heads=2, dim=64, page=32),
    "wide heads": dict(new=[5], length=[150], heads=4, kv_heads=2, dim=256, page=16),
    "long": dict(new=[1], length=[5000], heads=8, kv_heads=1, dim=64, page=64),
    "80 rows, pages of 16": dict(new=[40, 2], length=[170, 60], heads=2, kv_heads=1, dim=64, page=16),
    "80 rows, pages of 64": dict(new=[40, 2], length=[170, 60], heads=2, kv_heads=1, dim=128, page=64),
    "200 rows": dict(new=[50], length=[400], heads=4, kv_heads=1, dim=128, page=32),
    "200 rows, pages of 7": dict(new=[50], length=[400], heads=4, kv_heads=1, dim=64, page=7),
    "100 rows in splits": dict(new=[25], length=[9100], heads=4, kv_heads=1, dim=64, page=64),
    "100 rows in splits, pages of 48": dict(new=[25], length=[9100], heads=4, kv_heads=1, dim=64, page=48),
}


def close(out, lse, want, want_lse, tol, tol_lse, k=0):
    """want and tol are those of scales 2^k times smaller, without an absolute term that would hide
    small outputs. Beside attention64's terms the exponent of a weight has the scale's logarithm in it:
    numbers of up to 2^7.2 added (2^-17 of rounding each, two of them; two more where the references
    meet) and a logarithm good to 2^-22 make 2^-15 of a weight, which fp16 rounds by 2^-11: 1/16 on the
    bound's term of the weights. bf16's least step is 2^-133."""
    out, bound = out / 2.0 ** k, (tol - 1e-30) * (1 + 2.0 ** -4) + 2.0 ** (-134 - k)
    assert np.isfinite(out).all()
    assert (np.abs(out - want) <= bound).all(), (np.abs(out - want) / bound).max()
    assert (np.abs(lse - want_lse) <= tol_lse).all()


@pytest.mark.parametrize("shape", SHAPES)
def test_scaling_all_values_scales_the_output(shape):
    bt = PageBatch(**SHAPES[shape], spread=2.0)
    bt.v_scale[bt.used.any(1)] = 1.0
    want = attention64(bt)
    for k in (-110, -100, -85, -76, -60, -50, 0, 50, 80, 100, 112, 119):
        bt.v_scale[bt.used.any(1)] = 2.0 ** k
        close(*attend_pages(bt), *want, k)


@pytest.mark.parametrize("shape", SHAPES)
def test_pages_of_all_scales_side_by_side(shape):
    """Each page its own scale, the largest anywhere: every row's sum is right, and its output to the
    magnitude of what it weighs. Rows whose window holds small pages alone keep their own magnitude.
    (Codes of 1 and more: a weight is off by up to 2^-32 of the largest times its scale, which shows
    where the page of that has codes near 0.)"""
    for window, seed in ((0, 1), (5, 2)):
        bt = PageBatch(**SHAPES[shape], spread=2.0, window=window, seed=seed)
        rs = np.random.RandomState(seed)
        used = bt.used.any(1)
        e = rs.choice([-110, -90, -60, -30, 0, 30, 60, 90, 110, 118], (int(used.sum()), bt.kv_heads))
        bt.v_scale[used] = torch.from_numpy(2.0 ** e).float()
        bt.v[(bt.v & 0x7F) < 0x38] = 0x38
        out, lse = attend_pages(bt)
        want, want_lse, tol, tol_lse = attention64(bt)
        close(out, lse, want, want_lse, tol, tol_lse)


def dominated(bt, page, score):
    """Keys of zeros but for the first `page` of each sequence, whose score is `score` for every row."""
    bt.k[bt.used] = 0
    bt.k_scale[bt.used.any(1)] = 1.0
    bt.q_rows[:] = 0
    bt.q[..., 0] = score / 8 * bt.dim ** 0.5 / 8  # times 64, over sqrt(dim)
    one = torch.tensor([64.0]).to(torch.float8_e4m3fn).view(torch.uint8)[0]
    for b in range(bt.B):
        for i in range(page):
            bt.k[int(bt.table[b, i // bt.page]), i % bt.page, :, 0] = one


@pytest.mark.parametrize("k", [119, 100, 60, -60, -110])
@pytest.mark.parametrize("shape", ["long", "100 rows in splits", "100 rows in splits, pages of 48", "200 rows"])
def test_many_small_weights_beside_a_large_one(shape, k):
    """One key's weight is 2^15 times that of each other one: 9100 others are a fifth of the sum, under
    every scale."""
    bt = PageBatch(**SHAPES[shape], spread=2.0)
    dominated(bt, 1, 10.4)
    bt.v_scale[bt.used.any(1)] = 1.0
    want = attention64(bt)
    bt.v_scale[bt.used.any(1)] = 2.0 ** k
    close(*attend_pages(bt), *want, k)


@pytest.mark.parametrize("shape", [s for s in SHAPES if "splits" not in s and s != "long"])
def test_a_page_of_zero_values_takes_nearly_all_weight(shape):
    """The first page's keys weigh 2^87 times the others' and their values are 0 under the least scale:
    the output is 2^-87 of the others' values, to its own precision."""
    bt = PageBatch(**SHAPES[shape], spread=1.0)
    first = min(bt.page, 16, *bt.length)
    dominated(bt, first, 60.0)
    for b in range(bt.B):
        for i in range(-(-first // bt.page) * bt.page):
            bt.v[int(bt.table[b, i // bt.page]), i % bt.page] = 0
        bt.v_scale[int(bt.table[b, 0])] = 2.0 ** -110
    out, lse = attend_pages(bt)
    want, want_lse, tol, tol_lse = attention64(bt)
    assert 0 < np.abs(want).max() < 1e-20
    close(out, lse, want, want_lse, tol, tol_lse)


@pytest.mark.parametrize("shape", ["1 row", "12 rows", "wide heads", "long"])
def test_scales_of_tokens(shape):
    """The same of caches with a scale a token: scaled as a whole, and a key that takes nearly all
    weight with a scale of 0."""
    bt = Batch(**SHAPES[shape], cache="e4m3")
    used = bt.used[:, None].expand_as(bt.v_scale)
    base = bt.v_scale.clone()
    want = attention64(bt)
    for k in (-100, -60, 0, 60, 100):
        bt.v_scale = torch.where(used, base * 2.0 ** k, base)
        r = Call(bt)()
        assert r.status == 0
        close(r.out.double().cpu().numpy(), r.lse.double().cpu().numpy(), *want, k)
    bt.v_scale = base
    dominated_tokens(bt, 60.0)
    for least in (0.0, 2.0 ** -110):
        for b in range(bt.B):
            bt.v_scale[int(bt.table[b, 0]), :, 0] = least
            bt.v[int(bt.table[b, 0]), 0] = 0
        r = Call(bt)()
        assert r.status == 0
        close(r.out.double().cpu().numpy(), r.lse.double().cpu().numpy(), *attention64(bt))


def dominated_tokens(bt, score):
    bt.k[bt.used] = 0
    bt.q_rows[:] = 0
    bt.q[..., 0] = score / 8 * bt.dim ** 0.5 / 8
    one = torch.tensor([64.0]).to(torch.float8_e4m3fn).view(torch.uint8)[0]
    bt.k_scale[bt.used[:, None].expand_as(bt.k_scale)] = 1.0
    for b in range(bt.B):
        bt.k[int(bt.table[b, 0]), 0, :, 0] = one
