"""The example that samples prompts, over pools that run out."""
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from test_gpu_sample_example import PROMPTS, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def whole():
    return run(temperature=0.0)


@pytest.mark.parametrize("fewer", [1, 3, 5, 9])
def test_refused_samples_write_over_nobody(whole, fewer):
    """Every sample's tokens are the first of those that it draws in a pool with room: nobody's cached
    tokens are written over. What was refused is recorded, and the counts are those of the tables."""
    import sample_prompts
    full, want = whole
    s = sample_prompts.Samples(PROMPTS, 3, 20, temperature=0.0, pages=int((full.refs > 0).sum()) - fewer)
    got = s.generate(20).cpu()
    assert (got == -1).any() and (got >= 0).any()
    for row, all_of_it in zip(got, want):
        row = row[row >= 0]
        assert torch.equal(row, all_of_it[:len(row)])
    status = s.status()
    assert status.pop("step append") == moe.MOE_ERR_DEVICE_CHECK and not any(status.values()), status
    check_counts(s)


def check_counts(s):
    count = torch.zeros(s.pages, dtype=torch.int32)
    for row, n in zip(s.tables[0].cpu(), s.length.tolist()):
        for page in row[:-(-n // s.page)].tolist():
            count[page] += 1
    assert torch.equal(s.refs.cpu(), count)


def test_prompts_that_find_no_room():
    """The third prompt and those behind it have none: their samples draw nothing, and those of the
    first two have no page for their first token."""
    import sample_prompts
    s = sample_prompts.Samples(PROMPTS, 3, 5, temperature=0.0, pages=3)
    got = s.generate(5).cpu()
    assert (got[6:] == -1).all() and not s.live[6:].any() and s.length[6:].sum() == 0
    assert s.status()["prompts append"] == moe.MOE_ERR_DEVICE_CHECK and not s.status()["pages"]
    check_counts(s)
