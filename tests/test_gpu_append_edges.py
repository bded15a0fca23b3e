"""moe_rope_append at the ends of what it takes, with bounds derived beside them."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from serve_common import STEP, Batch
from test_gpu_rope_append import run

pytestmark = pytest.mark.gpu


def angle(position, base, pair, pairs):
    """position * base^(-pair / pairs) modulo a turn, reduced with 60 digits."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    turns = Decimal(int(position)) * Decimal(base) ** (Decimal(-pair) / pairs) / two_pi
    return float((turns - int(turns)) * two_pi)


@pytest.mark.parametrize("rot,base", [(256, 10000.0), (256, 500000.0), (128, 10000.0), (128, 1e6), (80, 1.0 + 2.0 ** -20), (2, 10000.0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_every_pair_at_the_farthest_positions(rot, base, interleaved):
    """sine and cosine: the angle's rounding to fp32 half turns, 1.6 units of 2^-24,
    2 of sincospi, and one each for the products and their sum."""
    pairs = rot // 2
    bt = Batch(new=[24], length=[24], heads=2, kv_heads=1, dim=max(8, rot), page=8, cache="f32", seed=40)
    pos = bt.rs.randint(2 ** 31 - 10 ** 6, 2 ** 31 - 1, (1, 24)) * bt.rs.choice([-1, 1], (1, 24))
    pos[0, :2] = 2 ** 31 - 1, -2 ** 31
    status, q, *_ = run(bt, rot, interleaved, base=base, positions=np.repeat(pos, 3, 0))
    assert status == moe.MOE_OK
    th = np.array([[angle(p, base, i, pairs) for i in range(pairs)] for p in pos[0]])[:, None]
    cos, sin = np.cos(th), np.sin(th)
    x, got = bt.q.double().numpy(), q.double().numpy()
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, pairs), slice(pairs, rot))
    bound = 6 * STEP["f32"] * (np.abs(x[..., lo]) + np.abs(x[..., hi]))
    assert (np.abs(got[..., lo] - (x[..., lo] * cos - x[..., hi] * sin)) <= bound).all()
    assert (np.abs(got[..., hi] - (x[..., hi] * cos + x[..., lo] * sin)) <= bound).all()


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("rot,interleaved", [(32, False), (32, True), (20, False), (0, False)])
@pytest.mark.parametrize("tokens", [2, 1500])
def test_zeros_that_do_not_turn_keep_their_sign(cache, rot, interleaved, tokens):
    bt = Batch(new=[tokens], length=[tokens], heads=2, kv_heads=1, dim=64, page=16, cache=cache, seed=41)
    bt.q_rows[:, rot:64] = -0.0
    bt.q_rows[:, 64 + rot:] = 0.0
    status, q, *_ = run(bt, rot, interleaved)
    assert status == moe.MOE_OK
    raw = torch.int32 if cache == "f32" else torch.int16
    assert torch.equal(q[..., rot:].contiguous().view(raw), bt.q[..., rot:].contiguous().view(raw))
