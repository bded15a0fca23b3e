"""The example that samples prompts over shared pages, and its calls in one graph."""
import os
import sys

import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
PROMPTS = [[(11 * i + 5 * t) % 512 for t in range(n)] for i, n in enumerate((33, 1, 64, 90))]


def run(**kw):
    import sample_prompts
    s = sample_prompts.Samples(PROMPTS, 3, 20, **kw)
    out = s.generate(20)
    assert not any(s.status().values()), s.status()
    return s, out.cpu()


def test_samples_of_a_prompt_without_chance_are_equal():
    s, out = run(temperature=0.0)
    rows = out.view(4, 3, 20)
    assert (rows == rows[:, :1]).all() and (out >= 0).all() and (out < 512).all()
    # three samples hold a prompt's whole pages, one each the pages they write
    want = torch.zeros(s.pages, dtype=torch.int32)
    for row, n in zip(s.tables[0].cpu(), s.length.tolist()):
        for page in row[:-(-n // s.page)].tolist():
            want[page] += 1
    assert torch.equal(s.refs.cpu(), want) and s.length.tolist() == [len(p) + 21 for p in PROMPTS for _ in range(3)]
    assert want.max() == 3


def test_a_large_penalty_lets_no_token_come_again():
    _, out = run(frequency=1e4, temperature=0.7)
    assert all(len(set(row)) == 20 for row in out.tolist())


def test_chance_makes_samples_differ():
    _, out = run(temperature=1.5)
    rows = out.view(4, 3, 20)
    assert (rows[:, 0] != rows[:, 1]).any()


def test_a_step_captured_and_replayed():
    """A step's calls in one graph, on state that the host puts back: equal tokens each time."""
    import sample_prompts
    s = sample_prompts.Samples(PROMPTS, 2, 4, temperature=0.0)
    logits = s.start()
    tokens = s.draw(logits)
    length, need, tables, refs = s.length.clone(), s.length + 1, s.tables, s.refs.clone()
    keep = [t.clone() for t in (s.k_cache, s.v_cache, s.k_scale, s.v_scale)]

    def step():
        s.length, s.tables = length, tables
        x = s.block("step", tokens, s.one_each, s.length, 1)
        out = s.draw((x @ s.w_out.t()).float())
        s.update(None, length, need)
        return out

    def put_back():
        for t, k in zip((s.k_cache, s.v_cache, s.k_scale, s.v_scale), keep):
            t.copy_(k)
        s.refs.copy_(refs)
        need.copy_(length + 1)

    want = step().clone()
    put_back()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.random = torch.Generator(device="cuda").manual_seed(3)
        s.draw = lambda logits: sample(s, logits)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = step()
    for _ in range(3):
        put_back()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert not any(s.status().values())


def sample(s, logits):
    """draw() with random numbers of its own making, for a capture."""
    moe.moe_logits_probs(s.logits_cfg, logits, s.one_each, None, s.history, s.cu_history, s.n_prompt, s.repetition, None, s.frequency,
                         None, None, None, None, None, s.temperature, s.p, s.ws["logits"])
    tokens = torch.empty(s.B, dtype=torch.int32, device="cuda")
    moe.moe_verify_drafts(s.verify_cfg, s.p, None, tokens, s.ones, s.ones * 0.5, s.one_each, None, tokens, s.accepted, None, s.ws["verify"])
    return tokens
