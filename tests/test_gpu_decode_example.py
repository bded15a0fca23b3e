"""The decode-step calls together, as examples/decode_step.py runs them."""
import os
import sys

import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_step  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", [moe.MOE_BF16, moe.MOE_E4M3])
def test_steps_decide_tokens(cache):
    B, steps, drafts = 5, 12, 3
    block = decode_step.Block(B, drafts, steps * (drafts + 1), cache=cache)
    out = decode_step.decode(block, torch.arange(B, device="cuda").int(), steps)
    assert not any(block.status().values())
    assert all(steps <= len(row) <= steps * (drafts + 1) and all(0 <= t < block.V for t in row) for row in out)


def test_drafts_do_not_change_what_is_decided():
    """Without temperature the decided tokens are the block's best ones, however
    many drafts a step has: a step of one token is the plain decoder. (The two
    run products of other sizes, whose roundings differ; the seed's best tokens
    are ahead by more than those.)"""
    first = torch.arange(4, device="cuda").int()
    plain = decode_step.decode(decode_step.Block(4, 0, 24, temperature=0), first, 24)
    for drafts in (1, 3):
        block = decode_step.Block(4, drafts, 24 * (drafts + 1), temperature=0)
        got = decode_step.decode(block, first, 24)
        for a, b in zip(plain, got):
            assert a == b[:24]
