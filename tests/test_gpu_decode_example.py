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


def test_calls_of_a_step_in_one_graph():
    """The step's calls captured once and replayed give what they give launched."""
    B, n = 4, 3
    block = decode_step.Block(B, n - 1, 64, seed=3)
    tokens = torch.randint(0, block.V, (B, n), device="cuda").int()
    kv_len = torch.tensor([3, 10, 40, 64], device="cuda").int()
    u, us = torch.rand(B * n, device="cuda"), torch.rand(B, device="cuda")
    _, q = block.draft(tokens[:, 0].contiguous())

    def calls():
        p = block.target(tokens, kv_len)
        moe.moe_verify_drafts(block.verify, p, q, tokens, u, us, block.cu, kv_len, block.decided, block.accepted,
                              block.next, block.ws["verify"])

    calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in (block.context, block.y, block.decided, block.accepted, block.next)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for t in (block.context, block.y, block.decided, block.accepted, block.next):
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert not any(block.status().values())
    for a, b in zip(want, (block.context, block.y, block.decided, block.accepted, block.next)):
        assert torch.equal(a, b)
