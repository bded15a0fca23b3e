"""moe_verify_drafts against the definition in exact fractions: every token,
count and length equal."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from serve_common import TORCH, verify64

pytestmark = pytest.mark.gpu


def inputs(new, V, kind="f32", seed=0, noise=0.6, pad=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(new)
    logits = 3 * torch.randn((T, V), generator=g)
    p = torch.softmax(logits, 1).to(TORCH[kind])
    q = torch.softmax(logits + noise * torch.randn((T, V), generator=g), 1).to(TORCH[kind])
    drawn = torch.multinomial(q.float(), 1, generator=g)[:, 0] if T else torch.zeros(0, dtype=torch.long)
    tokens = drawn.roll(1).int()
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(p=p, q=q, tokens=tokens, u=torch.rand(T, generator=g), us=torch.rand(len(new), generator=g), cu=cu,
                length=(np.array(new, np.int64) + 7).astype(np.int32), pad=pad, max_new=max(1, max(new, default=1)))


def rows(x, pad):
    """x on the GPU, its rows `pad` elements apart (NaN between)."""
    if x is None:
        return None
    wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype)
    wide[:, :x.shape[1]] = x
    return wide.cuda()


def call(d, stream=None, q_pad=None):
    T, V = d["p"].shape
    B = len(d["cu"]) - 1
    q_pad = d["pad"] if q_pad is None else q_pad
    cfg = moe.verify_config(n_seqs=B, n_tokens=T, max_new=d["max_new"], vocab=V,
                            dtype=moe.MOE_F32 if d["p"].dtype == torch.float32 else moe.MOE_BF16,
                            p_stride=V + d["pad"], q_stride=V + q_pad)
    args = [rows(d["p"], d["pad"]), rows(d["q"], q_pad), d["tokens"].cuda(), d["u"].cuda(), d["us"].cuda(),
            torch.from_numpy(d["cu"]).cuda(), torch.from_numpy(d["length"]).cuda()]
    out = torch.full((T,), -9, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    nxt = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    ws = moe.workspace(cfg, "verify")
    ws.fill_(0xA5)
    torch.cuda.synchronize()
    moe.moe_verify_drafts(cfg, *args, out, acc, nxt, ws, stream)
    return moe.moe_stream_status(ws, stream), out.cpu().numpy(), acc.cpu().numpy(), nxt.cpu().numpy()


def check(d, status=moe.MOE_OK, **kw):
    st, out, acc, nxt = call(d, **kw)
    assert st == status
    p = np.nan_to_num(d["p"].double().numpy(), nan=0.0).clip(0, 1)
    q = None if d["q"] is None else np.nan_to_num(d["q"].double().numpy(), nan=0.0).clip(0, 1)
    want = verify64(p, q, d["tokens"].numpy(), d["u"].numpy(), d["us"].numpy(), d["cu"], d["length"])
    for got, w in zip((acc, out, nxt), (want[1], want[0], want[2])):
        assert np.array_equal(got, w)
    return acc


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 5, 31, 100, 1003, 4096, 5001])
def test_vocabularies(kind, V):
    check(inputs([5, 1, 3, 2, 4], V, kind, seed=V))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [1, 2, 3, 5, 8])
def test_row_strides(kind, pad):
    d = inputs([4, 2, 5], 997, kind, seed=pad, pad=pad)
    check(d)
    check(d, q_pad=pad + 1)  # the two rows aligned differently


@pytest.mark.parametrize("B", [1, 2, 9, 40, 200, 700])
def test_batches(B):
    rs = np.random.RandomState(B)
    acc = check(inputs(rs.randint(0, 6, B).tolist(), 211, seed=B))
    assert B < 40 or len(set(acc.tolist())) > 3


def test_many_drafts():
    acc = check(inputs([70, 33, 34, 1], 50, seed=3, noise=0.01))
    assert acc.max() > 31


def test_large_vocabulary():
    check(inputs([3, 2], 70001, seed=4))


def test_all_accepted_and_all_rejected():
    d = inputs([5, 5], 300, seed=5)
    d["u"].zero_()
    assert check(d).tolist() == [4, 4]
    d = inputs([5, 5], 300, seed=6)
    for b in range(2):  # the target gives the first draft nothing
        d["p"][5 * b, d["tokens"][5 * b + 1].long()] = 0
    assert check(d).tolist() == [0, 0]


def test_without_a_draft_distribution():
    d = inputs([5, 4, 1], 40, seed=7)
    d["q"] = None
    check(d)


def test_next_to_borders():
    """u q = p exactly is a rejection; u R on a running sum takes the next
    token. Probabilities of a few powers of two make both happen."""
    V = 64
    rs = np.random.RandomState(8)
    new = [3] * 60
    d = inputs(new, V, seed=8)
    d["p"] = torch.full((180, V), 1.0 / V)
    d["q"] = torch.full((180, V), 1.0 / V)
    d["q"][:, ::2] *= 1.5
    d["q"][:, 1::2] *= 0.5
    d["u"] = torch.from_numpy(rs.choice([0.0, 0.5, 0.75, 2 / 3, 1 - 2.0 ** -24], 180).astype(np.float32))
    d["us"] = torch.from_numpy(rs.choice(np.arange(64) / 64.0, 60).astype(np.float32))
    d["us"][0], d["us"][1] = 0.0, 1 - 2.0 ** -24
    check(d)


def test_residual_without_a_positive_entry():
    """p below q everywhere (rows that do not sum to one): drawn from p; and
    from nothing where p is all zero."""
    d = inputs([2, 2], 33, seed=9)
    d["p"] = d["q"] * 0.25
    d["u"].fill_(0.9)
    check(d)
    d["p"][:] = 0
    st, out, acc, _ = call(d)
    assert st == moe.MOE_OK and out.tolist() == [-1] * 4 and acc.tolist() == [0, 0]


def test_values_that_are_no_probabilities():
    d = inputs([3, 3, 3], 500, seed=10)
    d["p"][::2, 7] = float("nan")
    d["p"][1::2, 9] = -0.5
    d["q"][::3, 11] = float("nan")
    d["p"][2, 13] = 3.0
    check(d)


def test_tiny_and_lonely_probabilities():
    d = inputs([2] * 6, 2000, seed=11)
    d["p"].zero_()
    for t in range(12):
        d["p"][t, 100 * t + 3] = [1.0, 2.0 ** -30, 2.0 ** -59][t % 3]
        d["q"][t, 100 * t + 3] = 0
    check(d)


def test_no_sequences_and_idle_ones():
    check(inputs([0, 0, 3, 0], 50, seed=12))
    check(inputs([], 50, seed=12))


def test_own_stream():
    check(inputs([4, 2, 5], 997, seed=13), stream=torch.cuda.Stream())


def test_bad_lists_are_reported():
    for name, i, v in (("tokens", 1, 50), ("tokens", 2, -1), ("cu", 1, 100), ("cu", 0, -3), ("cu", 2, 5)):
        d = inputs([3, 3], 50, seed=14)
        d["u"].zero_()
        d[name][i] = v
        assert call(d)[0] == moe.MOE_ERR_DEVICE_CHECK, (name, i)
    d = inputs([3, 3], 50, seed=14)  # a draft outside the vocabulary is rejected
    d["u"].zero_()
    d["tokens"][1] = 50
    assert call(d)[2].tolist() == [0, 2]


def test_frequencies_follow_the_target():
    """Over many draws with q far from p the decided first tokens follow p:
    chi-square over 8 outcomes, 4000 draws (7 degrees: above 35 once in 10^5)."""
    n, V = 4000, 8
    g = torch.Generator().manual_seed(15)
    p = torch.tensor([0.3, 0.2, 0.15, 0.1, 0.1, 0.08, 0.05, 0.02])
    q = torch.tensor([0.05, 0.3, 0.05, 0.2, 0.02, 0.08, 0.2, 0.1])
    tokens = torch.zeros(2 * n, dtype=torch.int32)
    tokens[1::2] = torch.multinomial(q.expand(n, V), 1, generator=g)[:, 0].int()
    d = dict(p=p.expand(2 * n, V).contiguous(), q=q.expand(2 * n, V).contiguous(), tokens=tokens,
             u=torch.rand(2 * n, generator=g), us=torch.rand(n, generator=g), cu=np.arange(0, 2 * n + 1, 2, dtype=np.int32),
             length=np.full(n, 2, np.int32), pad=0, max_new=2)
    _, out, _, _ = call(d)
    seen = np.bincount(out[::2], minlength=V)
    want = n * p.double().numpy()
    assert ((seen - want) ** 2 / want).sum() < 35
