"""Logits to probabilities (penalties, biases, masks, temperature, softmax) against 64 bits."""
import math

import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from serve_common import STEP, TORCH

pytestmark = pytest.mark.gpu
U = STEP["f32"]
KIND = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16}


def dev(x, t=np.int32):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, t)).cuda()


class Rows:
    """A batch: logits, lists and parameters on the host (numpy; logits as torch)."""

    def __init__(self, new, V, dtype="f32", out="f32", history=20, biases=0, masks=0, pad=0, p_pad=0, seed=0, neutral=False):
        rs = self.rs = np.random.RandomState(seed)
        self.new, self.V, self.dtype, self.out, self.pad, self.p_pad = new, V, dtype, out, pad, p_pad
        self.B, self.T = len(new), sum(new)
        self.cu = np.concatenate([[0], np.cumsum(new)])
        self.logits = torch.from_numpy(rs.randn(max(self.T, 1), V + pad) * 3).to(TORCH[dtype])
        self.tokens = rs.randint(0, V, max(self.T, 1))
        lengths = rs.randint(0, history + 1, self.B)
        self.cu_history = np.concatenate([[0], np.cumsum(lengths)])
        self.history = rs.randint(0, min(V, 50), lengths.sum())  # with repeats
        self.n_prompt = np.array([rs.randint(0, n + 1) for n in lengths])
        few = [int(rs.randint(0, min(biases, V) + 1)) for _ in range(self.B)]
        self.cu_bias = np.concatenate([[0], np.cumsum(few)])
        self.bias_token = np.concatenate([np.sort(rs.choice(V, n, replace=False)) for n in few] + [np.zeros(0)]).astype(int)
        self.bias = rs.randn(sum(few)).astype(np.float32) * 2
        self.allowed = rs.rand(masks, V) < 0.5 if masks else None
        self.mask_row = rs.randint(-1, masks, max(self.T, 1)) if masks else None
        f = lambda lo, hi: rs.uniform(lo, hi, self.B).astype(np.float32)  # noqa: E731
        self.rep, self.pres, self.freq, self.temp = f(0.8, 1.5), f(-1, 1), f(-0.5, 0.5), f(0.4, 1.6)
        if neutral:
            self.rep = self.pres = self.freq = self.temp = None

    def words(self):
        if self.allowed is None:
            return None
        n = -(-self.V // 32)
        bits = np.zeros((len(self.allowed), n * 32), np.uint8)
        bits[:, :self.V] = self.allowed
        bits[:, self.V:] = self.rs.randint(0, 2, (len(self.allowed), n * 32 - self.V))  # behind the vocabulary: anything
        return np.packbits(bits, axis=1, bitorder="little").view(np.int32)

    def cfg(self, **kw):
        return moe.logits_config(**{**dict(
            n_seqs=self.B, n_tokens=self.T, vocab=self.V, max_new=max([1, *self.new]), dtype=KIND[self.dtype], out_dtype=KIND[self.out],
            n_history=len(self.history), n_bias=len(self.bias), n_masks=0 if self.allowed is None else len(self.allowed),
            logits_stride=self.V + self.pad, p_stride=self.V + self.p_pad), **kw})

    def lists(self):
        f = lambda x: dev(x, np.float32)  # noqa: E731
        h, n = len(self.history) > 0, len(self.bias) > 0
        return dict(cu=dev(self.cu), tokens=dev(self.tokens), history=dev(self.history) if h else None, cu_history=dev(self.cu_history) if h else None,
                    n_prompt=dev(self.n_prompt) if h else None, rep=f(self.rep), pres=f(self.pres), freq=f(self.freq),
                    bias_token=dev(self.bias_token) if n else None, bias=f(self.bias) if n else None, cu_bias=dev(self.cu_bias) if n else None,
                    mask=dev(self.words()), mask_row=dev(self.mask_row), temp=f(self.temp))

    def run(self, lists=None, stream=None, **kw):
        cfg = self.cfg(**kw)
        ws = moe.workspace(cfg, "logits")
        p = torch.full((max(self.T, 1), self.V + self.p_pad), 7.0, dtype=TORCH[self.out], device="cuda")
        moe.moe_logits_probs(cfg, self.logits.cuda(), *(lists or self.lists()).values(), p, ws)
        self.status = moe.moe_stream_status(ws)
        got = p.double().cpu().numpy()
        assert (got[:, self.V:] == 7).all() and (self.T or (got == 7).all())  # nothing behind a row
        return got[:self.T, :self.V]

    def processed(self, t, b):
        """x of row t in 64 bits, its fp32 error and the row's counts."""
        x = self.logits[t, :self.V].double().numpy().copy()
        x[np.isnan(x)] = -np.inf
        lo, hi = self.cu_history[b], self.cu_history[b + 1]
        fed = self.tokens[self.cu[b]:t + 1]
        words = self.history[lo:hi]
        count = np.bincount(np.concatenate([words[self.n_prompt[b]:], fed]).astype(int), minlength=self.V)
        seen = np.bincount(np.concatenate([words, fed]).astype(int), minlength=self.V) > 0
        one = lambda v, d: d if v is None else float(v[b])  # noqa: E731
        rep, pres, freq = one(self.rep, 1.0), one(self.pres, 0.0), one(self.freq, 0.0)
        size = np.abs(x)
        x[seen] = np.where(x[seen] > 0, x[seen] / rep, x[seen] * rep)
        x = np.where(count > 0, x - freq * count - pres, x)
        size = size * max(1, rep, 1 / rep) + np.abs(freq) * count + np.abs(pres)
        lo, hi = self.cu_bias[b], self.cu_bias[b + 1]
        x[self.bias_token[lo:hi]] += self.bias[lo:hi]
        size[self.bias_token[lo:hi]] += np.abs(self.bias[lo:hi])
        x[np.isnan(x)] = -np.inf
        if self.allowed is not None and self.mask_row[t] >= 0:
            x[~self.allowed[self.mask_row[t]]] = -np.inf
        return x, 6 * U * size  # six roundings: 1 / repetition, its product, frequency's, two differences, a sum

    def want(self):
        p = np.zeros((self.T, self.V))
        tol = np.zeros_like(p)
        for b in range(self.B):
            for t in range(self.cu[b], self.cu[b + 1]):
                x, err = self.processed(t, b)
                temp = 1.0 if self.temp is None else float(self.temp[b])
                top = x.max(initial=-np.inf)
                if top == -np.inf:
                    continue
                if temp == 0:
                    p[t, np.argmax(x)] = 1
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    d = np.where(x == top, 0.0, (x - top) / temp)
                    w = np.where(np.isneginf(d), 0.0, np.exp(d))
                    p[t] = w / w.sum()
                    # an exponent's error: of x and of the maximum, the difference, 1 / temperature and the
                    # product (4 roundings of d), taken twice (a block's maximum, then the row's), exp 2 ulp
                    # each, the factors and the sum of V terms in 32 by 32 steps
                    e = (np.where(np.isfinite(err), err, 0) + np.where(np.isfinite(err), err, 0)[np.argmax(x)]) / temp
                    mean = (p[t] * e).sum()
                    rel = e + mean + 2 * 4 * U * np.where(np.isfinite(d), np.abs(d), 0) + 2 * 4 * U * (p[t] * np.where(p[t] > 0, np.abs(d), 0)).sum() + 110 * U
                    tol[t] = p[t] * (rel * 1.01 + STEP[self.out]) + 1e-37  # fp32's subnormals are flushed
        return p, tol

    def check(self, **kw):
        got = self.run(**kw)
        assert self.status == 0
        p, tol = self.want()
        bad = np.abs(got - p) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], p[bad][:5])
        return got


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("case", [
    dict(new=[1], V=1, history=3, masks=2), dict(new=[1], V=7, history=0), dict(new=[3, 0, 1], V=33, biases=5, masks=3),
    dict(new=[2, 4], V=1000, history=200, biases=40, masks=4, pad=3), dict(new=[1, 1, 1], V=4099, history=500, biases=3, p_pad=5),
    dict(new=[1], V=32000, history=700, biases=20), dict(new=[5] * 9, V=16385, history=60, masks=5), dict(new=[1] * 40, V=50021, biases=100),
    dict(new=[2], V=129280, history=3000, biases=300, masks=1, pad=1, p_pad=2), dict(new=[1, 1], V=1003, neutral=True, masks=2),
], ids=lambda c: f"{len(c['new'])}x{c['V']}")
def test_matches_64_bits(dtype, out, case):
    Rows(**case, dtype=dtype, out=out).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_vocabulary_of_many_tiles(dtype):
    """More tokens than the registers of 16 blocks hold: the row is read twice."""
    r = Rows([1, 2], 16 * 16384 * 3 + 77, dtype=dtype, history=400, biases=50, masks=2, pad=1)
    r.temp[1] = 0
    r.check()
    r = Rows([1], 16 * 16384 + 9, dtype=dtype, history=400, neutral=True)
    r.check()


def test_greedy_takes_the_lowest_of_equal_logits():
    for V, at in ((40, (3, 17)), (32000, (1999, 2000, 31999)), (300000, (299999, 12))):
        r = Rows([1], V, history=0)
        r.rep = r.pres = r.freq = None
        r.logits.clamp_(max=5)
        r.logits[0, list(at)] = 9.0
        r.temp[:] = 0
        got = r.check()
        assert got[0].argmax() == min(at) and got.sum() == 1


def test_masks_that_leave_one_or_nothing():
    r = Rows([4], 5000, masks=3, history=0)
    r.allowed[:] = False
    r.allowed[1, 4321] = True
    r.mask_row[:4] = [0, 1, 2, -1]
    got = r.check()
    assert got[0].sum() == 0 and got[1, 4321] == 1 and got[2].sum() == 0 and abs(got[3].sum() - 1) < 1e-5
    r.temp[:] = 0
    got = r.check()
    assert got[0].sum() == 0 and got[1, 4321] == 1


def test_infinities_and_nan():
    """NaN counts as -inf, masked or not; +inf takes the row, shared among equals; a row of -inf is 0."""
    r = Rows([6], 3000, masks=1, history=0, neutral=True)
    r.mask_row[:] = -1
    inf, nan = math.inf, math.nan
    r.logits[0, ::2] = nan
    r.logits[1, 5] = inf
    r.logits[2, [7, 2999]] = inf
    r.logits[3] = -inf
    r.logits[4] = nan
    r.logits[5, 100:200] = nan
    r.logits[5, 300] = inf
    r.allowed[0] = True
    r.allowed[0, 100:301] = False
    r.mask_row[5] = 0
    got = r.check()
    assert got[1, 5] == 1 and got[2, 7] == 0.5 and got[2, 2999] == 0.5 and got[3].sum() == 0 and got[4].sum() == 0
    assert np.isfinite(got).all()


def test_the_lowest_number_as_a_mask():
    """Logits masked by the caller with the type's lowest number, whole rows among them."""
    for dtype in ("f32", "bf16"):
        r = Rows([3], 999, dtype=dtype, history=0)
        r.logits[0, 10:] = torch.finfo(TORCH[dtype]).min
        r.logits[1] = torch.finfo(TORCH[dtype]).min
        r.rep = r.pres = r.freq = None
        got = r.check()
        assert abs(got[1].sum() - 1) < 1e-4


def test_history_counts():
    """A token 1000 times in the history, prompt and generated apart; the new tokens before a row's own."""
    r = Rows([3, 1], 64, history=0)
    r.cu_history, r.history, r.n_prompt = np.array([0, 1003, 1004]), np.array([5] * 1000 + [6, 7, 7] + [9]), np.array([1001, 1])
    r.tokens = np.array([11, 12, 11, 13])
    r.rep[:], r.pres[:], r.freq[:] = 1.5, 0.25, 0.125
    r.check()
    r.freq[:] = -0.01
    r.n_prompt[:] = 0
    r.check()
    x = Rows([3, 1], 64, history=0)
    lists = x.lists()
    lists["tokens"] = None  # new tokens not counted
    got = x.run(lists)
    x.rep = x.pres = x.freq = None
    p, tol = x.want()
    assert (np.abs(got - p) <= tol).all()


def test_empty_places_of_the_history():
    """Lists with room to grow: entries -1 change nothing."""
    r = Rows([2, 1], 500, history=30, biases=5, seed=2)
    want = r.run()
    grown, cu, at = [], [0], r.cu_history
    for b in range(2):
        grown += list(r.history[at[b]:at[b + 1]]) + [-1] * 7
        cu.append(len(grown))
    r.history, r.cu_history = np.array(grown), np.array(cu)
    assert np.array_equal(r.run(), want) and r.status == 0


@pytest.mark.parametrize("V,pad", [(40, 3), (20011, 1)])
def test_long_histories(V, pad):
    """Histories of 2040 to 9000 tokens that start and end anywhere, some places of them empty."""
    lengths = [2040, 2047, 2048, 2049, 2050, 2051, 2052, 2053, 2055, 9000, 1, 4099]
    r = Rows([1, 2] * 6, V, history=0, pad=pad, seed=9)
    r.cu_history = np.concatenate([[0], np.cumsum(lengths)])
    r.history = r.rs.randint(0, V, sum(lengths))
    r.n_prompt = np.array([r.rs.randint(0, n + 1) for n in lengths])
    want = r.check()
    empty = r.rs.rand(len(r.history)) < 0.3
    full, r.history = r.history, np.where(empty, -1, r.history)
    got = r.run()
    assert r.status == 0 and not np.array_equal(got, want)
    # the same without the empty places
    at = np.concatenate([[0], np.cumsum(~empty)])
    r.n_prompt = at[r.cu_history[:-1] + r.n_prompt] - at[r.cu_history[:-1]]
    r.cu_history, r.history = at[r.cu_history], full[~empty]
    assert np.array_equal(r.check(), got)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_logits_out(out):
    r = Rows([2, 1], 5003, history=100, biases=30, masks=2, out=out, p_pad=1)
    r.temp[1] = 0
    r.logits[0, 3] = math.nan
    got = r.run(out_logits=1)
    assert r.status == 0
    for b in range(2):
        for t in range(r.cu[b], r.cu[b + 1]):
            x, err = r.processed(t, b)
            temp = float(r.temp[b]) or 1.0
            assert (np.isneginf(got[t]) == np.isneginf(x)).all()
            ok = np.isfinite(x)
            tol = err / temp + (2 * U + STEP[out]) * np.abs(x / temp)
            assert (np.abs(got[t] - x / temp)[ok] <= 1.01 * tol[ok]).all()


def test_temperatures_at_the_ends():
    r = Rows([1] * 4, 2000, history=0)
    r.rep = r.pres = r.freq = None
    r.temp[:] = [1e-30, 1e30, 1e-3, 100.0]
    got = r.check()
    assert got[0].max() == 1 and abs(got[1].max() - 1 / 2000) < 1e-6


def test_in_place_on_another_stream_and_captured():
    r = Rows([2, 3], 30011, history=100, biases=10, masks=2)
    want = r.run()
    cfg, lists, ws = r.cfg(), r.lists(), moe.workspace(r.cfg(), "logits")
    source, p = r.logits.cuda(), torch.empty((r.T, r.V), device="cuda")
    p.copy_(source)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_logits_probs(cfg, p, *lists.values(), p, ws, stream=s)
    assert moe.moe_stream_status(ws, s) == 0 and np.array_equal(p.double().cpu().numpy(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.copy_(source)
        moe.moe_logits_probs(cfg, p, *lists.values(), p, ws)
    for _ in range(3):
        p.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(p.double().cpu().numpy(), want)


@pytest.mark.parametrize("name,at,value", [
    ("cu", 1, 9), ("cu_history", 1, -1), ("cu_history", 2, 0), ("cu_history", 0, 1), ("n_prompt", 0, -1), ("n_prompt", 0, 1000), ("history", 2, 100),
    ("history", 0, -2), ("tokens", 1, 100), ("bias_token", 1, 0), ("bias_token", 0, -1), ("bias_token", 3, 100), ("cu_bias", 1, 77), ("mask_row", 0, 2),
    ("mask_row", 2, -2), ("rep", 0, 0.0), ("rep", 1, math.nan), ("temp", 0, -1.0), ("temp", 0, math.inf), ("pres", 1, math.nan), ("freq", 1, math.inf),
])
def test_bad_lists_are_recorded(name, at, value):
    r = Rows([2, 1], 100, history=30, biases=0, masks=2, seed=4)
    assert r.cu_history[1] > 3
    r.cu_bias, r.bias_token, r.bias = np.array([0, 4, 6]), np.array([0, 5, 7, 99, 3, 4]), np.ones(6, np.float32)
    lists = r.lists()
    assert r.run(lists) is not None and r.status == 0
    lists[name][at] = value
    r.run(lists)
    assert r.status == moe.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("B", [2, 600])
def test_rows_behind_the_last_sequence(B):
    """Recorded, and left as they were; rows of sequences are not touched by that."""
    r = Rows([1] * B, 1000, history=30, biases=5, masks=2, seed=6)
    want = r.run()
    lists = r.lists()
    lists["cu"][B:] = B - 1  # the last sequence has no row
    got = r.run(lists)
    assert r.status == moe.MOE_ERR_DEVICE_CHECK
    assert np.array_equal(got[:B - 1], want[:B - 1]) and (got[B - 1:] == 7).all()


def test_no_rows():
    r = Rows([0, 0], 50, history=5)
    r.run()
    assert r.status == 0


def test_probabilities_verify_their_drafts():
    """Greedy sequences draft what the logits say: verification accepts it all and draws the next."""
    r = Rows([4, 1], 999, history=0)
    r.temp[:] = 0
    r.rep = r.pres = r.freq = None
    best = r.logits[:, :999].float().argmax(1).numpy()
    r.tokens[1:4] = best[:3]
    lists = r.lists()
    cfg, p = r.cfg(), torch.empty((r.T, r.V), device="cuda")
    moe.moe_logits_probs(cfg, r.logits.cuda(), *lists.values(), p, moe.workspace(cfg, "logits"))
    v = moe.verify_config(n_seqs=2, n_tokens=5, max_new=4, vocab=999)
    ws = moe.workspace(v, "verify")
    out, acc = dev([-9] * 5), dev([0, 0])
    u = torch.full((5,), 0.5, device="cuda")
    moe.moe_verify_drafts(v, p, None, lists["tokens"], u, u[:2], lists["cu"], None, out, acc, None, ws)
    assert moe.moe_stream_status(ws) == 0
    assert acc.tolist() == [3, 0] and out.tolist() == best.tolist()
