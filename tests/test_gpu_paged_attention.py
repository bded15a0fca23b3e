"""moe_paged_attention against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from serve_common import TORCH, Batch, attention64

pytestmark = pytest.mark.gpu


class Call:
    def __init__(self, bt, scale=0.0, stream=None):
        self.bt, self.stream = bt, stream
        self.cfg = bt.cfg(scale=scale)
        self.lists, self.cache = bt.lists(), bt.device_cache()
        self.q = bt.q_rows.cuda()
        self.out = torch.full((bt.T, bt.heads, bt.dim), float("nan"), dtype=TORCH[bt.dtype], device="cuda")
        self.lse = torch.full((bt.T, bt.heads), float("nan"), device="cuda")
        self.ws = moe.workspace(self.cfg, "attention")
        self.ws.fill_(0xA5)  # its contents need not be initialised
        torch.cuda.synchronize()

    def launch(self):
        k, v, ks, vs = self.cache
        moe.moe_paged_attention(self.cfg, self.q, *self.lists, k, v, ks, vs, self.out, self.lse, self.ws, self.stream)

    def __call__(self):
        self.launch()
        self.status = moe.moe_stream_status(self.ws, self.stream)
        return self


def check(bt, scale=0.0, stream=None):
    r = Call(bt, scale, stream)()
    assert r.status == moe.MOE_OK
    out, lse, tol_out, tol_lse = attention64(bt, scale)
    got, got_lse = r.out.double().cpu().numpy(), r.lse.double().cpu().numpy()
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert (got[empty] == 0).all()
    worst = np.max(np.abs(got - out) / np.maximum(tol_out, 1e-30), initial=0)
    assert worst <= 1, f"out: {worst:.3f} of the bound"
    d = np.abs(got_lse - lse, out=np.zeros_like(lse), where=~empty)
    assert (d <= tol_lse).all(), f"lse off by {d.max():.3g}"
    return r


CACHES = ["bf16", "e4m3", "f32"]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257])
def test_lengths_of_one_sequence(cache, length):
    check(Batch(new=[1], length=[length], heads=4, kv_heads=2, dim=64, page=16, cache=cache, seed=length))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128, 160, 192, 256])
def test_head_sizes(cache, dim):
    check(Batch(new=[1, 2], length=[70, 33], heads=6, kv_heads=2, dim=dim, page=16, cache=cache, seed=dim))


@pytest.mark.parametrize("dim", [8, 24, 72, 200, 248])
def test_head_sizes_not_of_16(dim):
    for cache in ("bf16", "f32"):
        check(Batch(new=[1, 2], length=[70, 33], heads=6, kv_heads=2, dim=dim, page=16, cache=cache, seed=dim))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (8, 1), (9, 1), (14, 2), (16, 1), (17, 1), (24, 1), (33, 1), (64, 1), (71, 1)])
def test_shared_heads(cache, heads, kv_heads):
    check(Batch(new=[1, 1], length=[50, 3], heads=heads, kv_heads=kv_heads, dim=64, page=8, cache=cache, seed=heads))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("page", [1, 3, 7, 8, 16, 32, 48, 100, 128])
@pytest.mark.parametrize("order", ["token", "head"])
def test_pages_and_orders(cache, page, order):
    check(Batch(new=[1, 1, 1], length=[130, 16, 77], heads=4, kv_heads=2, dim=128, page=page, cache=cache, order=order,
                seed=page))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_drafts(cache, dim, group):
    """Several new tokens: each sees up to its own position; some of them stand
    before the cache's first position and see nothing."""
    check(Batch(new=[5, 1, 8, 0, 3, 4], length=[40, 1, 8, 9, 1, 100], heads=2 * group, kv_heads=2, dim=dim, page=16,
                cache=cache, seed=group))


def test_many_new_tokens():
    check(Batch(new=[70, 1], length=[90, 20], heads=4, kv_heads=1, dim=64, page=16, seed=3))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("window", [1, 2, 16, 17, 63, 1000])
def test_window(cache, window):
    check(Batch(new=[1, 4, 2], length=[200, 90, 1], heads=4, kv_heads=2, dim=64, page=16, cache=cache, window=window,
                seed=window))


@pytest.mark.parametrize("cache", CACHES)
def test_batch_of_uneven_lengths(cache):
    rs = np.random.RandomState(5)
    n = rs.randint(0, 400, 40).tolist()
    check(Batch(new=[1] * 40, length=n, heads=8, kv_heads=2, dim=64, page=16, cache=cache, seed=6))


@pytest.mark.parametrize("cache", CACHES)
def test_long_sequences(cache):
    check(Batch(new=[1, 2], length=[5003, 2049], heads=8, kv_heads=1, dim=128, page=32, cache=cache, seed=7))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 64), (20, 2, 128), (3, 3, 256)])
def test_splits_of_few_sequences(cache, heads, kv_heads, dim):
    """A wide block table with a sequence or two: the keys are cut into more
    parts than a cluster has, most of them empty for a short sequence."""
    for new, length in (([1], [1999]), ([3, 1], [700, 1]), ([1, 2], [0, 40])):
        bt = Batch(new=new, length=length, heads=heads, kv_heads=kv_heads, dim=dim, page=16, cache=cache,
                   columns=16384, seed=19)
        assert len(new) > 1 or moe.workspace_size(bt.cfg(), "attention") > 256  # room for splits
        check(bt)


@pytest.mark.parametrize("cache", CACHES)
def test_values_not_finite_behind_a_row(cache):
    """The last new token's value holds infinities: only its own row shows it."""
    bt = Batch(new=[3], length=[45], heads=4, kv_heads=2, dim=64, page=16, cache=cache, seed=20)
    page, at = int(bt.table[0, 44 // 16]), 44 % 16
    if cache == "e4m3":
        bt.v[page, at] = 0x7F
    else:
        bt.v[page, at] = float("inf")
    out, lse, tol, _ = attention64(bt)
    r = Call(bt)()
    got = r.out.double().cpu().numpy()
    assert (np.abs(got[:2] - out[:2]) <= tol[:2]).all()
    assert not np.isfinite(got[2]).any()


@pytest.mark.parametrize("cache", CACHES)
def test_scale_and_strides(cache):
    for scale in (1.0, 1e-6, -0.2):
        check(Batch(new=[1, 2], length=[45, 70], heads=4, kv_heads=2, dim=64, page=16, cache=cache, q_pad=64, seed=8), scale)


@pytest.mark.parametrize("cache", CACHES)
def test_peaked_scores(cache):
    """Scores of hundreds: the weights underflow except at the largest, which
    moves from key to key."""
    check(Batch(new=[1, 3], length=[300, 65], heads=4, kv_heads=2, dim=64, page=16, cache=cache, values=60.0, seed=9))


@pytest.mark.parametrize("cache", CACHES)
def test_large_and_small_values(cache):
    """Values over the types' range; a token's E4M3 scales may lie far from
    its neighbours'."""
    bt = Batch(new=[1, 1], length=[90, 40], heads=4, kv_heads=2, dim=64, page=16, cache=cache, seed=10)
    g = torch.Generator().manual_seed(1)
    f = torch.exp2(torch.randint(-30, 30, (bt.n_pages, bt.page, bt.kv_heads), generator=g).float())
    if cache == "e4m3":
        bt.v_scale *= f.transpose(1, 2)
        bt.k_scale[:, :, ::5] = 0  # rows of zeros
        bt.v_scale[:, :, ::7] = 0
        bt.k_scale[~bt.used[:, None].expand(bt.k_scale.shape)] = float("nan")
    else:
        bt.v = (bt.v.float() * f[..., None]).to(bt.v.dtype)
        bt.k[:, ::5] = torch.where(bt.k[:, ::5].isnan(), bt.k[:, ::5], torch.zeros_like(bt.k[:, ::5]))
    check(bt)


@pytest.mark.parametrize("cache", CACHES)
def test_query_scale(cache):
    """Queries far from 1 (E4M3 caches multiply in fp16)."""
    for values, scale in ((2.0 ** 40, 2.0 ** -43), (2.0 ** -40, 2.0 ** 37)):
        check(Batch(new=[1, 2], length=[45, 70], heads=4, kv_heads=2, dim=64, page=16, cache=cache, values=values, seed=11), scale)


def test_infinite_score_of_a_masked_key_reaches_nothing():
    """Positions behind the window or past the token hold infinities and NaN."""
    bt = Batch(new=[2], length=[60], heads=2, kv_heads=1, dim=64, page=16, window=10, seed=12)
    for i in list(range(0, 48)):  # token 58 sees 49.., token 59 sees 50..
        page, at = int(bt.table[0, i // 16]), i % 16
        bt.k[page, at], bt.v[page, at] = float("inf"), float("nan")
    check(bt)


def test_no_tokens():
    check(Batch(new=[0, 0], length=[3, 0], heads=4, kv_heads=1, dim=64, page=16, seed=13))
    check(Batch(new=[], length=[], heads=4, kv_heads=1, dim=64, page=16, seed=13))


@pytest.mark.parametrize("cache", CACHES)
def test_equal_calls_give_equal_bits(cache):
    bt = Batch(new=[1, 5], length=[3000, 700], heads=8, kv_heads=1, dim=64, page=16, cache=cache, seed=14)
    a, b = Call(bt)(), Call(bt)()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_own_stream():
    check(Batch(new=[1, 3], length=[300, 65], heads=4, kv_heads=2, dim=64, page=16, seed=15), stream=torch.cuda.Stream())


def test_in_a_graph_while_the_cache_grows():
    """Captured once and replayed: lengths and tables are read on the device."""
    bt = Batch(new=[1, 1], length=[300, 65], heads=8, kv_heads=2, dim=64, page=16, seed=16)
    r = Call(bt)
    r()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.launch()
    for length in ([300, 65], [123, 1], [17, 64]):
        bt.length = length
        r.lists[1].copy_(torch.tensor(length, dtype=torch.int32))
        r.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        out, lse, tol, _ = attention64(bt)
        assert (np.abs(r.out.double().cpu().numpy() - out) <= tol).all()


@pytest.mark.parametrize("columns", [1, 8000])  # a long table is checked as it is used
@pytest.mark.parametrize("cache,heads", [("bf16", 2), ("e4m3", 2), ("f32", 2), ("bf16", 40)])
def test_bad_lists_are_reported(columns, cache, heads):
    def status(edit):
        bt = Batch(new=[2, 1], length=[50, 35], heads=heads, kv_heads=1, dim=64, page=16, cache=cache, columns=columns,
                   seed=17)
        edit(bt)
        return Call(bt)().status

    def put(name, i, v):
        def edit(bt):
            getattr(bt, name)[i] = v
        return edit
    assert status(lambda bt: None) == moe.MOE_OK
    for edit in (put("length", 1, -4), put("length", 0, 16 * columns + 64), put("table", (0, 1), 99), put("table", (0, 0), -1),
                 put("table", (1, 2), 1 << 30), put("cu", 1, 1000), put("cu", 0, -1), put("cu", 2, 2)):
        assert status(edit) == moe.MOE_ERR_DEVICE_CHECK
    assert status(put("table", (0, 3), 1 << 20)) == moe.MOE_ERR_DEVICE_CHECK  # positions 48 and 49
    if columns > 4:
        assert status(put("table", (0, 4), 1 << 20)) == moe.MOE_OK  # behind the last


def test_lse_is_optional():
    bt = Batch(new=[1], length=[33], heads=2, kv_heads=1, dim=64, page=16, seed=18)
    r = Call(bt)
    want = Call(bt)()
    r.lse = None
    r()
    assert torch.equal(r.out, want.out)


@pytest.mark.parametrize("dim", [8, 64, 80, 128])
@pytest.mark.parametrize("group,new", [(33, 1), (12, 4), (8, 8), (16, 8), (40, 4), (5, 30)])
def test_many_query_rows(dim, group, new):
    """Head groups of 33 rows and more, in blocks of 16 and (from 49 rows, bf16)
    of 128: the keys that all rows see, and those that only some do."""
    check(Batch(new=[new, 1, new, max(1, new - 1)], length=[300, 1, new, 129 + new], heads=2 * group, kv_heads=2, dim=dim,
                page=16, seed=group))


@pytest.mark.parametrize("length", [1, 7, 127, 128, 129, 135, 136, 255, 256, 257, 640, 1500])
@pytest.mark.parametrize("new", [8, 9])  # 48 and 54 rows
def test_many_query_rows_lengths(length, new):
    check(Batch(new=[new, 3], length=[length, length], heads=12, kv_heads=2, dim=64, page=7, seed=length))


@pytest.mark.parametrize("window", [1, 3, 8, 64, 129, 300])
def test_many_query_rows_window(window):
    check(Batch(new=[8, 5, 2], length=[700, 90, 1], heads=16, kv_heads=2, dim=64, page=16, window=window, seed=window))


def test_many_query_rows_split_and_peaked():
    for columns, lengths in ((1, [3000, 2049]), (16384, [2500, 3])):
        check(Batch(new=[6, 3], length=lengths, heads=24, kv_heads=2, dim=128, page=32, columns=columns, seed=21))
        check(Batch(new=[6, 3], length=lengths, heads=24, kv_heads=2, dim=128, page=32, columns=columns, values=60.0,
                    order="head", q_pad=64, seed=22))


@pytest.mark.parametrize("new", [5, 7])  # 40 and 56 rows
def test_many_query_rows_values_not_finite(new):
    bt = Batch(new=[new], length=[300], heads=16, kv_heads=2, dim=64, page=16, seed=23)
    page, at = int(bt.table[0, 299 // 16]), 299 % 16
    bt.v[page, at] = float("nan")
    out, lse, tol, _ = attention64(bt)
    got = Call(bt)().out.double().cpu().numpy()
    assert (np.abs(got[:-1] - out[:-1]) <= tol[:-1]).all() and np.isnan(got[-1]).all()


@pytest.mark.parametrize("new", [5, 7])
def test_many_query_rows_equal_bits_and_bad_pages(new):
    bt = Batch(new=[new, 2], length=[900, 300], heads=16, kv_heads=2, dim=64, page=16, seed=24)
    a, b = Call(bt)(), Call(bt)()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse) and a.status == moe.MOE_OK
    bt.table[0, 3] = 1 << 20
    bt.table[1, 18] = -5
    assert Call(bt)().status == moe.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("max_new", [2, 7, 50])
def test_bound_of_new_tokens_above_what_comes(cache, max_new):
    """max_new is a bound: it chooses the kernel's rows, not the result."""
    check(Batch(new=[1, 0, 2], length=[90, 3, 200], heads=16, kv_heads=2, dim=64, page=16, cache=cache, max_new=max_new,
                seed=25))


@pytest.mark.parametrize("new", [5, 7])
def test_many_query_rows_negative_scale(new):
    check(Batch(new=[new, 4], length=[300, 70], heads=16, kv_heads=2, dim=64, page=16, seed=26), -0.1)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("group", [2, 40])
def test_cache_beyond_32_bits(cache, group):
    """Pages whose elements lie past 2^32 bytes and 2^31 elements."""
    bt = Batch(new=[1, 2], length=[70, 33], heads=2 * group, kv_heads=2, dim=64, page=16, cache=cache, seed=27)
    r = Call(bt)
    small = [r.cache[i] for i in (0, 1)]
    pages = (1 << 31) // (16 * 2 * 64) + 5000
    big = [torch.empty((pages,) + x.shape[1:], dtype=x.dtype, device="cuda") for x in small]
    first = pages - bt.n_pages
    for b, x in zip(big, small):
        b[first:] = x
    scales = [None, None]
    if cache == "e4m3":
        scales = [torch.empty((pages,) + x.shape[1:], device="cuda") for x in r.cache[2:]]
        for b, x in zip(scales, r.cache[2:]):
            b[first:] = x
    want = Call(bt)()
    r.cache = (*big, *scales)
    r.cfg = moe.attn_config(**{n: getattr(r.cfg, n) for n in (
        "n_seqs", "n_tokens", "max_new", "n_heads", "n_kv_heads", "head_dim", "page_size", "max_pages", "dtype",
        "cache_dtype", "q_stride")}, n_pages=pages)
    r.lists = (r.lists[0], r.lists[1], torch.where(r.lists[2] >= 0, r.lists[2] + first, r.lists[2]))
    r()
    assert r.status == moe.MOE_OK
    assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)
