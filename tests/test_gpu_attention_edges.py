"""moe_paged_attention where its parts could come apart: bounds of its own, derived beside them."""
import pytest
import torch

from serve_common import Batch
from test_gpu_paged_attention import Call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,heads", [(7, 16), (16, 16)])  # 56 and 128 rows a head group
def test_maxima_that_rise_with_every_tile(new, heads):
    """Scores that grow by more than 8 (log2 units) from one tile of 128 keys to the
    next, from the half of the tile that the other thread of a row holds: a row's
    two threads scale their halves of the output alike only if both saw both maxima."""
    bt = Batch(new=[new], length=[1500], heads=heads, kv_heads=2, dim=64, page=16, seed=30)
    direction = torch.randn(64, generator=torch.Generator().manual_seed(31))
    direction /= direction.norm()
    bt.q_rows[:] = (8 * direction).repeat(heads).bfloat16()
    for i in range(1500):
        # tile by tile upwards, the larger scores in alternate halves of 64 keys
        rise = i // 128 + (0.5 if (i // 64 + i // 128) % 2 else 0.0)
        bt.k[int(bt.table[0, i // 16]), i % 16] = (8.0 * rise * direction + 0.01 * bt.k[int(bt.table[0, i // 16]), i % 16].float()).bfloat16()
    a = check(bt)
    for _ in range(5):
        b = Call(bt)()
        assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
