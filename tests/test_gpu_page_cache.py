"""E4M3 caches with one scale per page and head: the append that writes them and the attention
that reads them, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from page_common import PageBatch, append64, rotated64
from serve_common import STEP, attention64

pytestmark = pytest.mark.gpu
U = STEP["f32"]


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(11)


def attend(bt, **kw):
    cfg, (k, v, ks, vs) = bt.cfg(**kw), bt.device_cache()
    out = torch.full((max(bt.T, 1), bt.heads, bt.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((max(bt.T, 1), bt.heads), 7.0, device="cuda")
    ws = moe.workspace(cfg, "attention")
    moe.moe_paged_attention(cfg, bt.q_rows.cuda(), *bt.lists(), k, v, ks, vs, out, lse, ws)
    assert moe.moe_stream_status(ws) == 0
    return out[:bt.T].double().cpu().numpy(), lse[:bt.T].double().cpu().numpy()


CASES = [
    dict(new=[1], length=[1], heads=1, kv_heads=1, dim=16, page=1),
    dict(new=[1, 0, 1], length=[40, 9, 33], heads=8, kv_heads=2, dim=64, page=16),
    dict(new=[1] * 5, length=[1, 31, 32, 33, 200], heads=16, kv_heads=2, dim=128, page=32),
    dict(new=[2, 5, 1], length=[2, 300, 70], heads=15, kv_heads=5, dim=80, page=7),  # rows before the first key
    dict(new=[4, 4], length=[129, 61], heads=12, kv_heads=2, dim=128, page=64),      # 24 rows a head group
    dict(new=[7, 3], length=[500, 90], heads=16, kv_heads=2, dim=64, page=16, order="head"),   # 56 rows
    dict(new=[40, 3], length=[260, 3], heads=4, kv_heads=2, dim=128, page=48),       # 80 rows
    dict(new=[33], length=[400], heads=4, kv_heads=1, dim=112, page=64, window=70),  # 132 rows
    dict(new=[20, 1], length=[150, 40], heads=8, kv_heads=1, dim=96, page=1),        # 160 rows
    dict(new=[3, 9], length=[200, 77], heads=4, kv_heads=2, dim=256, page=32),
    dict(new=[18], length=[100], heads=2, kv_heads=1, dim=192, page=16, q_pad=64),
    dict(new=[130], length=[700], heads=2, kv_heads=1, dim=128, page=128),
    dict(new=[1], length=[9000], heads=8, kv_heads=1, dim=128, page=64),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['new']}of{c['length']}x{c['heads']}d{c['dim']}p{c['page']}"[:60])
@pytest.mark.parametrize("spread", [1.0, 20.0])
def test_attention_matches_64_bits(case, spread):
    # queries so small that scores stay of order 1 whatever the pages' scales
    bt = PageBatch(**case, spread=spread, values=2.0 ** -spread * 2)
    out, lse = attend(bt)
    want, want_lse, tol, tol_lse = attention64(bt)
    assert (np.abs(out - want) <= tol).all(), (np.abs(out - want) / tol).max()
    seen = np.isfinite(want_lse)
    assert (np.isneginf(lse) == ~seen).all()
    assert (np.abs(lse - want_lse)[seen] <= tol_lse[seen]).all()


def test_scales_at_the_ends_of_their_range():
    """Pages of zeros (the least scale) and pages of the largest scale: products of a code and its
    scale that are bf16's smallest and largest."""
    for new in (1, 60):
        bt = PageBatch(new=[new], length=[200], heads=2, kv_heads=1, dim=64, page=16)
        for x in (bt.k_scale, bt.v_scale):
            x[int(bt.table[0, 0])] = 2.0 ** -110
            x[int(bt.table[0, 3])] = 2.0 ** 100
        bt.k_scale[int(bt.table[0, 3])] = 2.0 ** -3  # large values, ordinary scores
        bt.q_rows *= 0.1
        out, _ = attend(bt)
        want, _, tol, _ = attention64(bt)
        assert (np.abs(out - want) <= tol).all()


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new", [1, 12, 60])
def test_queries_and_keys_of_zeros(new, page):
    """Some rows' queries are 0, and keys too, whose pages have the least scale: every score is 0, and a
    masked place is masked all the same."""
    bt = PageBatch(new=[new, new], length=[200, new], heads=4, kv_heads=2, dim=64, page=page)
    bt.k[bt.used] = 0
    bt.k_scale[bt.used.any(1)] = 2.0 ** -110
    bt.q_rows[::2] = 0
    out, lse = attend(bt)
    want, want_lse, tol, tol_lse = attention64(bt)
    assert (np.abs(out - want) <= tol).all()
    # n terms summed in fp32 are off by up to n 2^-24 of the sum, 2^-16.3 for 200, and so is its
    # logarithm: attention64 counts those
    assert (np.abs(lse - want_lse) <= tol_lse).all()


def test_unseen_codes_reach_nothing():
    """NaN codes and NaN scales wherever no row looks (the batch's own), and in the last page's
    places behind the length."""
    for new, heads in ((1, 8), (30, 4)):
        bt = PageBatch(new=[new, new], length=[new + 3, 77], heads=heads, kv_heads=2, dim=64, page=32)
        out, lse = attend(bt)
        assert np.isfinite(out).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("new", [3, 40])
def test_nan_codes_that_some_rows_see(new):
    bt = PageBatch(new=[new], length=[100], heads=4, kv_heads=2, dim=64, page=16)
    last = int(bt.table[0, 99 // 16])
    bt.v[last, 99 % 16] = 0x7F
    out, _ = attend(bt)
    assert np.isnan(out[-1]).all() and np.isfinite(out[:-1]).all()
    clean = PageBatch(new=[new], length=[100], heads=4, kv_heads=2, dim=64, page=16)
    want, _, tol, _ = attention64(clean)
    assert (np.abs(out[:-1] - want[:-1]) <= tol[:-1]).all()


def test_attention_captured_and_repeated_gives_equal_bits():
    bt = PageBatch(new=[40, 2], length=[300, 1000], heads=8, kv_heads=2, dim=128, page=16)
    cfg, (k, v, ks, vs) = bt.cfg(), bt.device_cache()
    q, lists = bt.q_rows.cuda(), bt.lists()
    out = [torch.zeros((bt.T, bt.heads, bt.dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = moe.workspace(cfg, "attention")
    run = lambda o: moe.moe_paged_attention(cfg, q, *lists, k, v, ks, vs, o, None, ws)  # noqa: E731
    run(out[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(out[1])
    for _ in range(3):
        out[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1])


# ---- append -------------------------------------------------------------------------------------

APPENDS = [
    dict(new=[1], length=[1], heads=1, kv_heads=1, dim=16, page=1, rot=0),
    dict(new=[1, 1, 0, 1], length=[1, 17, 40, 32], heads=8, kv_heads=2, dim=64, page=16, rot=64),
    dict(new=[5, 3, 1], length=[5, 40, 96], heads=4, kv_heads=2, dim=128, page=32, rot=96, interleaved=True),
    dict(new=[40, 1, 17], length=[90, 200, 17], heads=4, kv_heads=2, dim=128, page=16, rot=128),
    dict(new=[100, 64], length=[131, 64], heads=3, kv_heads=3, dim=80, page=64, rot=42),
    dict(new=[70], length=[100], heads=2, kv_heads=1, dim=256, page=48, rot=200, sections=(50, 30, 20)),
    dict(new=[9, 2], length=[30, 2], heads=6, kv_heads=2, dim=96, page=7, rot=10, interleaved=True, sections=(3, 0, 2)),
    dict(new=[300], length=[333], heads=2, kv_heads=2, dim=48, page=256, rot=48),
    dict(new=[33] * 20, length=[50 + i for i in range(20)], heads=2, kv_heads=1, dim=64, page=16, rot=32),
]


def append(bt, k, v, q, case, pos=None, **kw):
    rot = case["rot"]
    sections = case.get("sections", (0, 0, 0))
    cfg = bt.cfg(rot_dim=rot, rot_interleaved=case.get("interleaved", False), rot_sections=sections, q_stride=0, **kw)
    kc, vc, ks, vs = bt.device_cache()
    q_out = torch.empty_like(q, device="cuda")
    ws = moe.workspace(cfg, "append")
    moe.moe_rope_append(cfg, q.cuda(), k.cuda(), v.cuda(), None if pos is None else pos.cuda(), *bt.lists(), q_out, kc, vc,
                        ks, vs, ws)
    assert moe.moe_stream_status(ws) == 0
    return q_out.cpu(), bt.back(kc), bt.back(vc), ks.cpu(), vs.cpu()


def check_cache(bt, before, before_scale, x, got, got_scale, reach):
    """Codes within half a step of the value in units of the page's scale (a subnormal's step is
    2^-9), after fp32's error of the rotation: `reach` is the norm of each element's pair."""
    value, scale, touched = append64(bt, before, before_scale, x)
    written = touched.any(1)
    assert np.array_equal(got_scale.double().numpy()[written], scale[written])
    same = ~torch.from_numpy(touched)
    assert torch.equal(got[same], before[same])
    assert torch.equal(got_scale.view(torch.int32)[~torch.from_numpy(written)], before_scale.view(torch.int32)[~torch.from_numpy(written)])
    have = got.view(torch.float8_e4m3fn).double().numpy()
    for page in np.flatnonzero(written):
        a, b = have[page][touched[page]], value[page][touched[page]]
        assert (np.isnan(a) == np.isnan(b)).all()
        # 8 U of a pair's norm (angle 1.6 U, sine and cosine 2 U each, two products and a sum)
        tol = STEP["e4m3"] * np.abs(b) + 2.0 ** -10 + 8 * U * reach / scale[page][None, :, None]
        ok = np.isfinite(b)
        assert (np.abs(a - b)[ok] <= (tol * 1.01)[ok]).all()


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"{c['new'][:3]}of{c['length'][:3]}d{c['dim']}p{c['page']}")
def test_append_matches_64_bits(case, order):
    bt = PageBatch(**{k: case[k] for k in ("new", "length", "heads", "kv_heads", "dim", "page")}, order=order, spread=3.0)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((bt.T, bt.kv_heads, bt.dim), generator=g) * torch.exp2(
        torch.empty(bt.T, bt.kv_heads, 1).uniform_(-4, 4, generator=g)) for _ in range(2))
    k, v, q = k.bfloat16(), v.bfloat16(), torch.randn((bt.T, bt.heads, bt.dim), generator=g).bfloat16()
    at = np.concatenate([np.arange(n - m, n) for m, n in zip(bt.new, bt.length)])
    sections = case.get("sections", (0, 0, 0))
    pos = torch.randint(-1000, 1 << 20, (3, bt.T), generator=g).int() if sum(sections) else None
    places = np.stack([at] * 3) if pos is None else pos.numpy()
    turn = lambda x: rotated64(x, places, case["rot"], case.get("interleaved", False), sections)  # noqa: E731
    q_out, kc, vc, ks, vs = append(bt, k, v, q, case, pos)
    top = float(max(k.abs().max(), v.abs().max(), q.abs().max())) * 1.5
    want = turn(q)
    assert (np.abs(q_out.double().numpy() - want) <= STEP["bf16"] * np.abs(want) + 8 * U * top).all()
    check_cache(bt, bt.k, bt.k_scale, turn(k), kc, ks, top)
    check_cache(bt, bt.v, bt.v_scale, v.double().numpy(), vc, vs, top)


def test_append_raises_a_scale_and_rescales_older_codes():
    """Page 0 holds small elements; the token behind them is 2^12 times as large, then again as
    small: the scale stays, codes lose what falls below the subnormals and no more."""
    case = dict(new=[1], length=[11], heads=2, kv_heads=2, dim=64, page=16, rot=0)
    bt = PageBatch(**{k: case[k] for k in ("new", "length", "heads", "kv_heads", "dim", "page")}, spread=0.0)
    k = torch.randn((1, 2, 64)).bfloat16()
    k[:, 0] *= 2.0 ** 12
    q = torch.zeros((1, 2, 64)).bfloat16()
    _, kc, vc, ks, vs = append(bt, k, k, q, case)
    check_cache(bt, bt.k, bt.k_scale, k.double().numpy(), kc, ks, 0.0)
    page = int(bt.table[0, 0])
    assert ks[page, 0] > bt.k_scale[page, 0]
    # once more over the same place with a small token: the scale stays
    bt.k, bt.k_scale, bt.v, bt.v_scale = kc, ks, vc, vs
    _, kc2, _, ks2, _ = append(bt, k * 2.0 ** -12, k, q, case)
    assert torch.equal(ks2[page], ks[page]) and torch.equal(kc2[page, :10], kc[page, :10])


def test_append_from_the_first_place_starts_anew():
    case = dict(new=[2], length=[18], heads=1, kv_heads=1, dim=32, page=16, rot=0)
    bt = PageBatch(**{k: case[k] for k in ("new", "length", "heads", "kv_heads", "dim", "page")})
    page = int(bt.table[0, 1])
    bt.k_scale[page] = bt.v_scale[page] = 2.0 ** 60  # of a sequence that had the page before
    k = torch.randn((2, 1, 32)).bfloat16()
    _, kc, _, ks, _ = append(bt, k, k, torch.zeros((2, 1, 32)).bfloat16(), case)
    assert ks[page] < 1
    check_cache(bt, bt.k, bt.k_scale, k.double().numpy(), kc, ks, 0.0)


def test_append_keeps_infinities_and_nan_out_of_the_scale():
    case = dict(new=[3], length=[20], heads=1, kv_heads=2, dim=32, page=16, rot=0)
    bt = PageBatch(**{k: case[k] for k in ("new", "length", "heads", "kv_heads", "dim", "page")} | {"heads": 2})
    k = torch.randn((3, 2, 32)).bfloat16()
    k[1, 0, 5], k[2, 0, 6], k[0, 1, 7] = math.inf, math.nan, -math.inf
    _, kc, _, ks, _ = append(bt, k, k, torch.zeros((3, 2, 32)).bfloat16(), case)
    check_cache(bt, bt.k, bt.k_scale, k.double().numpy(), kc, ks, 0.0)
    assert int((kc[int(bt.table[0, 1])] & 0x7F == 0x7F).sum()) >= 3


def test_append_zeros_and_the_largest_numbers():
    case = dict(new=[2, 2], length=[2, 2], heads=1, kv_heads=1, dim=16, page=4, rot=0)
    bt = PageBatch(**{k: case[k] for k in ("new", "length", "heads", "kv_heads", "dim", "page")})
    k = torch.zeros((4, 1, 16)).bfloat16()
    k[2:] = torch.finfo(torch.bfloat16).max
    _, kc, _, ks, _ = append(bt, k, k, torch.zeros((4, 1, 16)).bfloat16(), case)
    a, b = int(bt.table[0, 0]), int(bt.table[1, 0])
    assert float(ks[a, 0]) == 2.0 ** -110 and (kc[a, :2] == 0).all()
    assert float(ks[b, 0]) == 2.0 ** 119 and (kc[b, :2] == 0x7E).all()


def test_append_in_place_of_q_and_on_another_stream():
    case = dict(rot=48)
    bt = PageBatch(new=[20, 3], length=[30, 50], heads=4, kv_heads=2, dim=64, page=16)
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn((bt.T, 2, 64), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((bt.T, 4, 64), generator=g).bfloat16()
    want, kc0, vc0, ks0, vs0 = append(bt, k, v, q, case)
    cfg = bt.cfg(rot_dim=48, q_stride=0)
    kc, vc, ks, vs = bt.device_cache()
    dq, dk, dv, lists, ws = q.cuda(), k.cuda(), v.cuda(), bt.lists(), moe.workspace(cfg, "append")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    moe.moe_rope_append(cfg, dq, dk, dv, None, *lists, dq, kc, vc, ks, vs, ws, stream=s)
    assert moe.moe_stream_status(ws, s) == 0
    assert torch.equal(dq.cpu(), want) and torch.equal(kc.cpu(), kc0) and torch.equal(vc.cpu(), vc0)
    assert torch.equal(ks.cpu().view(torch.int32), ks0.view(torch.int32))
    # only the cache
    kc, vc, ks, vs = bt.device_cache()
    moe.moe_rope_append(cfg, None, dk, dv, None, *lists, None, kc, vc, ks, vs, ws)
    assert moe.moe_stream_status(ws) == 0 and torch.equal(kc.cpu(), kc0) and torch.equal(vc.cpu(), vc0)


def test_append_then_attend_over_growing_pages():
    """Tokens appended one to three at a time, each step attended: the attention of the end is that
    of the cache's own values, and those are within E4M3's step (twice it, where a page was
    rescaled into subnormals never here) of the tokens."""
    g = torch.Generator().manual_seed(9)
    page, D, steps = 8, 64, [1, 3, 2, 1, 1, 3, 3, 2]
    total = sum(steps)
    toks = torch.randn((total, 1, D), generator=g).bfloat16()
    kc, vc = (torch.zeros((4, page, 1, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((4, 1), device="cuda") for _ in range(2))
    table = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device="cuda")
    at = 0
    for n in steps:
        cfg = moe.attn_config(n_seqs=1, n_tokens=n, max_new=n, n_heads=1, n_kv_heads=1, head_dim=D, page_size=page, n_pages=4,
                              max_pages=4, cache_dtype=moe.MOE_E4M3_PAGE)
        ws = moe.workspace(cfg, "append")
        x = toks[at:at + n].cuda()
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        at += n
        length = torch.tensor([at], dtype=torch.int32, device="cuda")
        moe.moe_rope_append(cfg, None, x, x, None, cu, length, table, None, kc, vc, ks, vs, ws)
        assert moe.moe_stream_status(ws) == 0
    have = (vc.view(torch.float8_e4m3fn).double() * vs.double()[:, None, :, None]).cpu()[[2, 0, 3, 1]].reshape(-1, D)[:total]
    want = toks.double()[:, 0]
    step = vs.double().cpu()[[2, 0, 3, 1]].repeat_interleave(page)[:total, None] * 2.0 ** -9
    # a code rounded once for itself and once more where a raise made it subnormal
    assert ((have - want).abs() <= STEP["e4m3"] * want.abs() + step).all()


@pytest.mark.parametrize("name,at,value", [("table", (0, 1), 5), ("table", (0, 1), -1), ("length", 1, 0), ("length", 0, 1),
                                           ("length", 0, 1 << 20), ("cu", 1, 9), ("cu", 0, 1)])
def test_bad_lists_are_recorded(name, at, value):
    bt = PageBatch(new=[2, 1], length=[20, 5], heads=2, kv_heads=1, dim=32, page=16, spare=2)
    assert bt.n_pages == 5
    k = torch.randn((3, 1, 32)).bfloat16().cuda()
    lists = dict(cu=bt.cu.copy(), length=np.array(bt.length, np.int32), table=bt.table.copy())
    lists[name][at] = value
    dev = [torch.from_numpy(lists[n]).cuda() for n in ("cu", "length", "table")]
    cfg = bt.cfg(q_stride=0)
    kc, vc, ks, vs = bt.device_cache()
    ws = moe.workspace(cfg, "append")
    moe.moe_rope_append(cfg, None, k, k, None, *dev, None, kc, vc, ks, vs, ws)
    status = moe.moe_stream_status(ws)
    assert status == moe.MOE_ERR_DEVICE_CHECK


def test_append_to_an_empty_sequence_is_recorded_for_every_cache():
    """kv_len 0 with a new token: the token has no slot, whatever the cache."""
    for kind in (moe.MOE_BF16, moe.MOE_E4M3, moe.MOE_E4M3_PAGE):
        cfg = moe.attn_config(n_seqs=1, n_tokens=1, n_heads=1, n_kv_heads=1, head_dim=16, page_size=4, n_pages=1, max_pages=1,
                              cache_dtype=kind)
        x = torch.zeros((1, 1, 16), dtype=torch.bfloat16, device="cuda")
        cache = torch.zeros(4 * 16, dtype=torch.bfloat16, device="cuda")
        scale = None if kind == moe.MOE_BF16 else torch.zeros(4, device="cuda")
        cu, length, table = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1], [0], [[0]]))
        ws = moe.workspace(cfg, "append")
        moe.moe_rope_append(cfg, None, x, x, None, cu, length, table, None, cache, cache, scale, scale, ws)
        status = moe.moe_stream_status(ws)
        assert status == moe.MOE_ERR_DEVICE_CHECK
