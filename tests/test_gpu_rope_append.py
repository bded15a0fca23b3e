"""moe_rope_append against the definition in 64 bits: rotated queries, the
cache's new rows (and every other slot untouched), E4M3 codes and scales."""
import math

import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from serve_common import STEP, TORCH, Batch

pytestmark = pytest.mark.gpu


def rotate64(x, pos, rot, interleaved, sections, base):
    """x [heads][dim] fp64, pos one position an axis."""
    y = x.copy()
    pairs = rot // 2
    sections = sections if sum(sections) else (pairs, 0, 0)
    axis = np.repeat([0, 1, 2], sections)
    for i in range(pairs):
        th = float(pos[axis[i]]) * base ** (-2.0 * i / rot)
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        y[:, lo] = x[:, lo] * math.cos(th) - x[:, hi] * math.sin(th)
        y[:, hi] = x[:, hi] * math.cos(th) + x[:, lo] * math.sin(th)
    return y


def reach(x, rot, interleaved):
    """|x_lo| + |x_hi| of each element's pair: what an error of the sine or
    cosine is multiplied by."""
    y = np.abs(x)
    pairs = rot // 2
    for i in range(pairs):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        y[:, lo] = y[:, hi] = np.abs(x[:, lo]) + np.abs(x[:, hi])
    return y


def run(bt, rot, interleaved=False, sections=(0, 0, 0), base=0.0, positions=None, inplace=False,
        stream=None, fused=False):
    g = torch.Generator().manual_seed(bt.seed + 1)
    kind = TORCH[bt.dtype]
    kv = (bt.T, bt.kv_heads, bt.dim)
    k, v = torch.randn(kv, generator=g).to(kind), torch.randn(kv, generator=g).to(kind)
    if bt.T:
        k[0, 0] = 0  # a row of zeros (E4M3: scale 0)
    strides = {}
    q_d, k_d, v_d = bt.q_rows.cuda(), k.cuda(), v.cuda()
    if fused:  # slices of one projection's rows
        wide = torch.cat([bt.q.flatten(1), k.flatten(1), v.flatten(1)], 1).cuda()
        nq, nk = bt.heads * bt.dim, bt.kv_heads * bt.dim
        q_d, k_d, v_d = wide[:, :nq], wide[:, nq:nq + nk], wide[:, nq + nk:]
        strides = dict(q_stride=wide.shape[1], k_stride=wide.shape[1], v_stride=wide.shape[1])
    cfg = bt.cfg(rot_dim=rot, rot_interleaved=interleaved, rot_sections=sections, rope_base=base, **strides)
    kc, vc, ks, vs = bt.device_cache()
    before = [bt.back(x).clone() if x is not None else None for x in (kc, vc)] + [None if x is None else x.cpu() for x in (ks, vs)]
    out = q_d if inplace else torch.full((bt.T, bt.heads, bt.dim), float("nan"), dtype=kind, device="cuda")
    pos = None if positions is None else torch.from_numpy(positions.astype(np.int32)).cuda()
    ws = moe.workspace(cfg, "append")
    lists = bt.lists()
    torch.cuda.synchronize()
    moe.moe_rope_append(cfg, q_d, k_d, v_d, pos, *lists, out, kc, vc, ks, vs, ws, stream)
    status = moe.moe_stream_status(ws, stream)
    after = [bt.back(kc), bt.back(vc), None if ks is None else ks.cpu(), None if vs is None else vs.cpu()]
    return status, out[:bt.T].reshape(bt.T, bt.heads, bt.dim).cpu(), k, v, before, after


def check(bt, rot, interleaved=False, sections=(0, 0, 0), base=0.0, positions=None, **kw):
    status, q_out, k, v, before, after = run(bt, rot, interleaved, sections, base, positions, **kw)
    assert status == moe.MOE_OK
    step, u = STEP[bt.dtype], STEP["f32"]
    base = base or 10000.0
    written = torch.zeros((bt.n_pages, bt.page), dtype=torch.bool)
    for b in range(bt.B):
        for j in range(bt.new[b]):
            t, at = int(bt.cu[b]) + j, bt.length[b] - bt.new[b] + j
            pos = [at] * 3 if positions is None else positions[:, t]
            page, place = int(bt.table[b, at // bt.page]), at % bt.page
            written[page, place] = True

            def bound(x):
                # sine and cosine to 2 ulp of 1 and the angle's 2^-30, two products and a sum
                return 8 * u * reach(x, rot, interleaved)
            x = bt.q[t].double().numpy()
            want = rotate64(x, pos, rot, interleaved, sections, base)
            assert (np.abs(q_out[t].double().numpy() - want) <= step * np.abs(want) + bound(x)).all(), (t, "q")
            for which, src, cache, scale in (("k", k, after[0], after[2]), ("v", v, after[1], after[3])):
                x = src[t].double().numpy()
                want = rotate64(x, pos, rot, interleaved, sections, base) if which == "k" else x
                err = bound(x) if which == "k" else np.zeros_like(x)
                if bt.cache != "e4m3":
                    got = cache[page, place].double().numpy()
                    assert (np.abs(got - want) <= step * np.abs(want) + err).all(), (t, which)
                    continue
                s = scale[page, :, place].double().numpy()
                amax = np.abs(want).max(1)
                assert (np.abs(s - amax / 448) <= (err.max(1) + 2 * u * amax) / 448).all(), (t, which)
                got = cache[page, place].view(torch.float8_e4m3fn).double().numpy() * s[:, None]
                # half a step of the code, at least that of the smallest (2^-10 of the scale's unit)
                half = np.maximum(STEP["e4m3"] * np.abs(want), 2.0 ** -10 * s[:, None])
                assert (np.abs(got - want) <= half * (1 + 8 * u) + 2 * err + 8 * u * np.abs(want)).all(), (t, which)
    for x, y in zip(before, after):  # nothing else was touched, bit for bit
        if x is None:
            continue
        keep = ~written if x.dim() == 4 else None
        if keep is not None:
            raw = (torch.uint8, torch.int16, None, torch.int32)[x.element_size() - 1]
            assert torch.equal(x[keep].contiguous().view(raw), y[keep].contiguous().view(raw))
        else:
            m = ~written[:, None, :].expand(x.shape)
            assert torch.equal(x[m].view(torch.int32), y[m].view(torch.int32))


@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("order", ["token", "head"])
def test_types_and_orders(cache, order):
    check(Batch(new=[1, 3, 0, 2], length=[1, 20, 5, 33], heads=8, kv_heads=2, dim=64, page=16, cache=cache,
                order=order, seed=1), 64)


@pytest.mark.parametrize("dim,rot", [(16, 16), (64, 42), (80, 80), (96, 2), (128, 128), (128, 0), (256, 256), (112, 70)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
def test_head_sizes(dim, rot, interleaved, cache):
    check(Batch(new=[2, 1], length=[17, 9], heads=6, kv_heads=3, dim=dim, page=5, cache=cache, seed=2), rot, interleaved)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (7, 7), (64, 8), (48, 1), (71, 1)])
def test_head_counts(heads, kv_heads):
    check(Batch(new=[1, 2], length=[3, 4], heads=heads, kv_heads=kv_heads, dim=128, page=1, seed=3), 128)


@pytest.mark.parametrize("sections", [(16, 24, 24), (64, 0, 0), (0, 64, 0), (1, 62, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes_and_far_positions(sections, interleaved):
    """Positions of three axes over the whole int32 range: the angle of each is
    exact to a 64-bit fraction of a turn (the check's own angle, in 64 bits,
    limits the position to 2^20)."""
    bt = Batch(new=[5, 7], length=[40, 7], heads=4, kv_heads=2, dim=128, page=8, cache="f32", seed=4)
    pos = bt.rs.randint(-(1 << 20), 1 << 20, (3, bt.T))
    pos[:, 0] = [0, 1, -1]
    check(bt, 128, interleaved, sections, 1e6, positions=pos)


def test_whole_int32_range_of_positions():
    """At rot_dim = 2 the one pair turns by the position itself, in radians:
    checked with the angle reduced in Python's integers."""
    bt = Batch(new=[4], length=[4], heads=1, kv_heads=1, dim=8, page=4, cache="f32", seed=5)
    pos = np.array([[2147483647, -2147483648, 1234567890, 710]] * 3)
    status, q, *_ = run(bt, 2, positions=pos)
    assert status == moe.MOE_OK
    two_pi = (314159265358979323846264338327950288419716939937510 * 2, 10 ** 50)
    for t in range(4):
        turns = int(pos[0, t]) * two_pi[1] % two_pi[0]
        th = turns / two_pi[1]
        x = bt.q[t, 0].double().numpy()
        want = x[0] * math.cos(th) - x[1] * math.sin(th)
        # f_i is rounded to 53 bits: 2^31 * 2^-54 of a radian, far below fp32
        assert abs(q[t, 0, 0].item() - want) <= 8 * STEP["f32"] * (abs(x[0]) + abs(x[1]))


def test_strided_in_place_and_without_queries():
    check(Batch(new=[2, 3], length=[9, 3], heads=4, kv_heads=2, dim=64, page=4, q_pad=64, seed=6), 64)
    check(Batch(new=[2, 3], length=[9, 3], heads=4, kv_heads=2, dim=64, page=4, seed=7), 64, fused=True)
    for rot, inter in ((64, False), (42, False), (64, True)):
        check(Batch(new=[2, 3], length=[9, 3], heads=40, kv_heads=2, dim=64, page=4, seed=8), rot, inter, inplace=True)
    bt = Batch(new=[2], length=[2], heads=4, kv_heads=2, dim=64, page=4, seed=9)
    cfg, (cu, length, table), (kc, vc, _, _) = bt.cfg(rot_dim=64), bt.lists(), bt.device_cache()
    k = torch.randn(2, 2, 64).bfloat16().cuda()
    ws = moe.workspace(cfg, "append")
    moe.moe_rope_append(cfg, None, k, k, None, cu, length, table, None, kc, vc, None, None, ws)
    assert moe.moe_stream_status(ws) == moe.MOE_OK
    page = int(bt.table[0, 0])
    assert torch.equal(vc[page, :2], k) and torch.equal(kc[page, 0], k[0])


@pytest.mark.parametrize("rot,interleaved", [(32, False), (32, True), (20, False), (0, False)])
@pytest.mark.parametrize("tokens", [2, 1500])
def test_elements_that_do_not_turn_pass_as_they_are(rot, interleaved, tokens):
    """Infinities past rot_dim reach their own element only."""
    bt = Batch(new=[tokens], length=[tokens], heads=2, kv_heads=1, dim=64, page=16, seed=14)
    bt.q_rows[:, 40] = float("inf")
    bt.q_rows[:, 64 + 63] = float("-inf")
    status, q, *_ = run(bt, rot, interleaved)
    assert status == moe.MOE_OK
    assert torch.equal(q[..., rot:], bt.q[..., rot:]) and torch.isfinite(q[..., :rot]).all()


@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("rot,interleaved", [(64, False), (42, False), (64, True)])
def test_runs_of_tokens(cache, rot, interleaved):
    """Enough tokens that a warp takes a run of them, over the ends of sequences,
    idle ones and pages; in place as well."""
    rs = np.random.RandomState(6)
    new = [700, 0, 0, 1, 3, 0, 511, 1, 80, 0, 1, 44]
    bt = dict(new=new, length=[n + int(rs.randint(0, 30)) for n in new], heads=6, kv_heads=2, dim=64, page=7, cache=cache)
    check(Batch(**bt, seed=15), rot, interleaved)
    check(Batch(**bt, seed=16), rot, interleaved, inplace=True)
    one = Batch(new=[1] * 1300, length=[1 + i % 9 for i in range(1300)], heads=2, kv_heads=1, dim=80, page=4, cache=cache, seed=17)
    check(one, rot, interleaved, (rot // 2 - 10, 5, 5), positions=one.rs.randint(0, 5000, (3, one.T)))


def test_runs_of_tokens_bad_lists():
    new = [700, 600]
    for name, i, v in (("length", 0, 699), ("table", (0, 5), 9999), ("cu", 1, 701), ("cu", 2, 1299)):
        bt = Batch(new=new, length=[710, 600], heads=2, kv_heads=1, dim=64, page=16, seed=18)
        getattr(bt, name)[i] = v
        assert run(bt, 64)[0] == moe.MOE_ERR_DEVICE_CHECK, name


def test_many_tokens():
    rs = np.random.RandomState(3)
    new = rs.randint(0, 40, 50).tolist()
    check(Batch(new=new, length=[n + int(rs.randint(0, 30)) for n in new], heads=4, kv_heads=1, dim=64, page=16,
                cache="e4m3", seed=10), 32)


def test_no_tokens():
    check(Batch(new=[0, 0], length=[3, 0], heads=4, kv_heads=1, dim=64, page=16, seed=11), 32)
    check(Batch(new=[], length=[], heads=4, kv_heads=1, dim=64, page=16, seed=11), 32)


def test_own_stream():
    s = torch.cuda.Stream()
    check(Batch(new=[2, 3], length=[9, 3], heads=4, kv_heads=2, dim=64, page=4, seed=12), 64, stream=s)


def test_bad_lists_are_reported():
    """A token without a slot, a page outside the cache and counts that do not
    add up set the status; the good tokens are still written."""
    def status(edit):
        bt = Batch(new=[2, 1], length=[5, 3], heads=2, kv_heads=1, dim=64, page=4, seed=13)
        edit(bt)
        cfg, lists, (kc, vc, _, _) = bt.cfg(rot_dim=64), bt.lists(), bt.device_cache()
        x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        ws = moe.workspace(cfg, "append")
        moe.moe_rope_append(cfg, x, x, x, None, *lists, torch.empty_like(x), kc, vc, None, None, ws)
        return moe.moe_stream_status(ws)

    def put(name, i, v):
        def edit(bt):
            getattr(bt, name)[i] = v
        return edit
    assert status(lambda bt: None) == moe.MOE_OK
    for edit in (put("length", 0, 1), put("length", 1, -4), put("length", 0, 9), put("table", (0, 1), 99),
                 put("table", (0, 1), -1), put("cu", 1, 1000), put("cu", 0, -1), put("cu", 2, 2)):
        assert status(edit) == moe.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_cache_beyond_32_bits(cache):
    bt = Batch(new=[3, 2], length=[20, 17], heads=2, kv_heads=2, dim=64, page=16, cache=cache, seed=19)
    kind = torch.uint8 if cache == "e4m3" else torch.bfloat16
    pages = (1 << 31) // (16 * 2 * 64) + 5000
    first = pages - bt.n_pages
    caches = [torch.zeros((pages, 16, 2, 64), dtype=kind, device="cuda") for _ in range(2)]
    scales = [torch.zeros((pages, 2, 16), device="cuda") for _ in range(2)] if cache == "e4m3" else [None, None]
    cfg = bt.cfg(rot_dim=0, n_pages=pages)
    cu, length, table = bt.lists()
    x = torch.randn(5, 2, 64).bfloat16().cuda()
    ws = moe.workspace(cfg, "append")
    moe.moe_rope_append(cfg, x, x, x, None, cu, length, table + first, torch.empty_like(x), *caches, *scales, ws)
    assert moe.moe_stream_status(ws) == moe.MOE_OK
    for b in range(2):
        for j in range(bt.new[b]):
            at, t = bt.length[b] - bt.new[b] + j, int(bt.cu[b]) + j
            page = first + int(bt.table[b, at // 16])
            for c, s in zip(caches, scales):
                got = c[page, at % 16]
                if cache == "e4m3":
                    got = got.view(torch.float8_e4m3fn).float() * s[page, :, at % 16, None]
                assert torch.allclose(got.float(), x[t].float(), rtol=2.0 ** -4, atol=2.0 ** -6)
    assert sum(int((c != 0).any(-1).sum()) for c in caches) == 2 * 5 * 2
