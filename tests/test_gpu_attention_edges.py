"""moe_paged_attention where its parts could come apart: bounds of its own, derived beside them."""
import numpy as np
import pytest
import torch

import attention_bounds as ab
from serve_common import Batch, attention64
from test_gpu_paged_attention import Call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,heads", [(7, 16), (16, 16)])  # 56 and 128 rows a head group
def test_maxima_that_rise_with_every_tile(new, heads):
    """Scores that grow by more than 8 (log2 units) from one tile of 128 keys to the
    next, from the half of the tile that the other thread of a row holds: a row's
    two threads scale their halves of the output alike only if both saw both maxima."""
    bt = Batch(new=[new], length=[1500], heads=heads, kv_heads=2, dim=64, page=16, seed=30)
    direction = torch.randn(64, generator=torch.Generator().manual_seed(31))
    direction /= direction.norm()
    bt.q_rows[:] = (8 * direction).repeat(heads).bfloat16()
    for i in range(1500):
        # tile by tile upwards, the larger scores in alternate halves of 64 keys
        rise = i // 128 + (0.5 if (i // 64 + i // 128) % 2 else 0.0)
        bt.k[int(bt.table[0, i // 16]), i % 16] = (8.0 * rise * direction + 0.01 * bt.k[int(bt.table[0, i // 16]), i % 16].float()).bfloat16()
    a = check(bt)
    for _ in range(5):
        b = Call(bt)()
        assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


@pytest.mark.parametrize("cache,group", [("bf16", 1), ("bf16", 4), ("e4m3", 1), ("e4m3", 4), ("f32", 1), ("f32", 4)])
@pytest.mark.parametrize("dim", [64, 128])
def test_keys_that_only_some_rows_see_at_both_ends(cache, group, dim):
    """A window and 20 new tokens: 19 keys at either end are seen by some of the rows only.
    NaN in the first and in the last of them reaches the first and the last token alone."""
    new, window, length = 20, 100, 400
    bt = Batch(new=[new, 3], length=[length, 90], heads=2 * group, kv_heads=2, dim=dim, page=16, cache=cache, window=window, seed=32)
    for i in (length - new - window + 1, length - 1):
        page, at = int(bt.table[0, i // 16]), i % 16
        bt.v[page, at] = 0x7F if cache == "e4m3" else float("nan")
    out, lse, tol, tol_lse = attention64(bt)
    r = Call(bt)()
    got, got_lse = r.out.double().cpu().numpy(), r.lse.double().cpu().numpy()
    wild = [0, new - 1]
    tame = [t for t in range(bt.T) if t not in wild]
    assert np.isnan(got[wild]).all() and (np.abs(got[tame] - out[tame]) <= tol[tame]).all()
    assert (np.abs(got_lse - lse) <= tol_lse).all()


def same_kinds(got, want):
    """Infinities of the same sign, and NaN, in the same places."""
    return all(np.array_equal(f(got), f(want)) for f in (np.isposinf, np.isneginf, np.isnan))


def check_not_finite(bt):
    with np.errstate(invalid="ignore"):
        out, lse, tol, tol_lse = attention64(bt)
    r = Call(bt)()
    got, got_lse = r.out.double().cpu().numpy(), r.lse.double().cpu().numpy()
    assert same_kinds(got, out)
    fine = np.isfinite(out)
    assert (np.abs(got[fine] - out[fine]) <= tol[fine]).all()
    assert (np.abs(got_lse - lse) <= tol_lse).all()  # takes no part in it


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("new,heads,dim", [(1, 2, 64), (1, 16, 128), (2, 16, 128), (3, 24, 64), (7, 16, 64), (16, 16, 128), (1, 4, 256), (2, 16, 192)])
@pytest.mark.parametrize("columns", [1, 16384])
def test_infinite_values(cache, new, heads, dim, columns):
    """A positive weight times an infinite value is that infinity, wherever the key
    stands; both infinities together are NaN. lse does not see values."""
    length = 700
    bt = Batch(new=[new], length=[length], heads=heads, kv_heads=2, dim=dim, page=16, cache=cache, columns=columns, seed=33, values=0.5)
    inf = float("inf")
    for i, e, v in ((0, 1, inf), (37, 2, -inf), (300, 3, inf), (301, 3, inf), (302, 4, inf), (600, 4, -inf), (length - 1, 5, inf),
                    (length - new, 6, -inf), (length - new, 7, inf), (length - 1, 7, -inf), (128, 0, inf)):
        page, at = int(bt.table[0, i // 16]), i % 16
        bt.v[page, at, :, e] = v
    check_not_finite(bt)


@pytest.mark.parametrize("new,heads,dim", [(1, 2, 64), (2, 16, 128), (7, 16, 64), (2, 16, 256)])
@pytest.mark.parametrize("columns", [1, 16384])
def test_value_scales_that_are_not_finite(new, heads, dim, columns):
    """An infinite scale makes its token's values infinite (those of code 0 NaN) for who
    sees it, and leaves lse alone; so does a NaN."""
    length = 500
    for v in (float("inf"), float("nan")):
        for places in ((3,), (200, 201), (length - 1,), (0, length - new)):
            bt = Batch(new=[new], length=[length], heads=heads, kv_heads=2, dim=dim, page=16, cache="e4m3", columns=columns,
                       seed=34, values=0.5)
            for i in places:
                page, at = int(bt.table[0, i // 16]), i % 16
                bt.v_scale[page, :, at] = v
                bt.v[page, at, :, 3] = 0
            check_not_finite(bt)


@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 64), (16, 1, 64), (4, 1, 256)])
def test_many_small_weights_beside_a_large_one(heads, kv_heads, dim):
    """E4M3: of every 32 keys one has nearly all the weight, and the others, 2^-25.5 of
    it each, are the only ones with a value in element 0."""
    n = 8000
    bt = Batch(new=[1], length=[n], heads=heads, kv_heads=kv_heads, dim=dim, page=16, cache="e4m3", seed=35)

    def e4m3(v):
        return int(torch.tensor(v).to(torch.float8_e4m3fn).view(torch.uint8))
    large = torch.zeros((bt.n_pages, bt.page), dtype=torch.bool)
    for i in range(0, n, 32):
        large[int(bt.table[0, i // 16]), i % 16] = True
    small = bt.used & ~large
    bt.q_rows[:] = 0
    bt.q[..., 0] = 1
    for x, s in ((bt.k, bt.k_scale), (bt.v, bt.v_scale)):
        x[bt.used] = 0
        s[~s.isnan()] = 1.0
    bt.v_scale /= 64
    bt.k[..., 0] = torch.where(large[..., None], e4m3(24.0), bt.k[..., 0]).to(torch.uint8)
    bt.v[..., 1] = torch.where(large[..., None], e4m3(448.0), bt.v[..., 1]).to(torch.uint8)
    bt.v[..., 0] = torch.where(small[..., None], e4m3(448.0), bt.v[..., 0]).to(torch.uint8)
    scale = 25.5 * np.log(2) / 24
    out, lse, tol, tol_lse = attention64(bt, scale)
    r = Call(bt, scale)()
    got = r.out.double().cpu().numpy()
    # a weight is off by 2^-32 of the largest at most: n of them, against n / 32 of the largest's weight
    tol = tol + 2.0 ** -32 * 32 * 7.0 * 1.01
    assert 1e-6 < out[0, 0, 0] < 1e-4
    assert (np.abs(got - out) <= tol).all()
    assert abs(got[0, 0, 0] - out[0, 0, 0]) <= 0.02 * out[0, 0, 0]
    assert (np.abs(r.lse.double().cpu().numpy() - lse) <= tol_lse).all()


@pytest.mark.parametrize("outlier", [2.0 ** 10, 2.0 ** 18, 2.0 ** 22])
@pytest.mark.parametrize("new,heads", [(1, 2), (2, 16)])
def test_queries_with_one_large_element(outlier, new, heads):
    """E4M3: an element of q far above the others, where the keys are 0, takes nothing
    from the products of the others (exact above 2^-31 of it: but for a few within 0.002 of 0)."""
    bt = Batch(new=[new, 1], length=[300, 40], heads=heads, kv_heads=2, dim=64, page=16, cache="e4m3", seed=36)
    bt.q[..., 5] = outlier
    bt.k[..., 5] = torch.where(bt.used[..., None], 0, bt.k[..., 5]).to(torch.uint8)
    check(bt)


def test_query_rows_over_the_whole_range():
    """E4M3: rows whose largest element is near the ends of bf16's range, and zero."""
    for values, scale in ((2.0 ** 124, 2.0 ** -126), (2.0 ** -100, 2.0 ** 97), (0.0, 0.5)):
        check(Batch(new=[1, 2], length=[45, 70], heads=4, kv_heads=2, dim=64, page=16, cache="e4m3", values=values, seed=37), scale)


@pytest.mark.parametrize("new,length,heads,dim", [
    ([1], [48], 4, 64), ([1, 1], [48, 20], 4, 128), ([2, 1], [64, 31], 8, 128), ([1], [40], 4, 256), ([4], [44], 8, 256), ([4], [64], 8, 64),
    ([7], [64], 16, 64), ([16, 5], [130, 64], 16, 128)])
@pytest.mark.parametrize("columns", [1, 16384])
def test_weights_of_two_terms(new, length, heads, dim, columns):
    """bf16 caches: values that cancel leave the weights' rounding, 2^-16, as the largest
    part of the error; one bf16 term would pass the bound 4 times and more."""
    bt = ab.cancelling(new, length, heads, 2, dim, seed=50, columns=columns)
    out, tol = ab.rows64(bt)
    got = Call(bt)().out.double().cpu().numpy()
    assert (np.abs(got - out) <= tol).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("heads,dim,window", [(8, 64, 0), (2, 128, 0), (4, 80, 333)])
def test_a_prompt_beside_decoding_sequences(cache, heads, dim, window):
    """A chunk of a prompt of more than a thousand tokens, in one batch with single tokens,
    drafts, an idle sequence and the start of another prompt."""
    check(Batch(new=[1, 1100, 1, 3, 0, 1, 260], length=[900, 1500, 2500, 70, 10, 1, 260], heads=heads, kv_heads=2, dim=dim, page=16, cache=cache,
                window=window, seed=51))


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "f32"])
def test_the_most_new_tokens(cache):
    """4096 of a sequence, some of them before the cache's first position."""
    check(Batch(new=[4096, 2], length=[4000, 50], heads=1, kv_heads=1, dim=32, page=64, cache=cache, seed=52))


@pytest.mark.parametrize("heads", [2, 8, 16, 24])  # 1, 4, 8 and 12 rows a head group
@pytest.mark.parametrize("dim,sums", [(128, 2), (256, 4)])
def test_fp32_scores_are_not_one_sum(heads, dim, sums):
    """fp32: products of 1 and not quite half a step of the last binade more, which a
    single running sum drops dim / 2 times. One key: lse is its score."""
    step = dim // 128 * 31 * 2.0 ** -23  # 0.484 of a step between dim / 2 and dim
    bt = Batch(new=[1], length=[1], heads=heads, kv_heads=2, dim=dim, page=16, cache="f32", seed=53)
    bt.q_rows[:] = 1
    bt.k[bt.used] = 1 + step
    want = dim * (1 + step)
    # and the roundings of the factor log2 e, its product, the factor ln 2 and its product
    bound = ab.rounding_of_sums(dim, sums) + 4 * 2.0 ** -24 * want
    r = Call(bt, 1.0)()
    got = r.lse.double().cpu().numpy()
    assert (np.abs(got - want) <= bound).all(), np.abs(got - want).max() / bound
    assert torch.equal(r.out.cpu(), bt.v[bt.used][0].repeat_interleave(heads // 2, 0)[None])
    # what one sum would give
    one = np.float32(0)
    for _ in range(dim):
        one = np.float32(one + np.float32(1 + step))
    assert abs(float(one) - want) > bound
