"""moe_rope_append over page scales where no sequence has more than one new token: batches smaller and
larger than a block, some sequences without one, pages of one token."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from page_common import PageBatch
from test_gpu_page_cache import append, check_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [1, 3, 16])
@pytest.mark.parametrize("B", [1, 2, 255, 256, 257, 700])
def test_one_token_or_none_of_each_sequence(B, page):
    rs = np.random.RandomState(B + page)
    new = (rs.rand(B) < 0.7).astype(int).tolist()
    new[-1] = 1
    length = rs.randint(1, 3 * page + 2, B).tolist()
    bt = PageBatch(new=new, length=length, heads=2, kv_heads=1, dim=32, page=page, spread=1.0)
    g = torch.Generator().manual_seed(B)
    k, v = ((torch.randn((bt.T, 1, 32), generator=g) * 4).bfloat16() for _ in range(2))
    q = torch.randn((bt.T, 2, 32), generator=g).bfloat16()
    q_out, kc, vc, ks, vs = append(bt, k, v, q, dict(rot=0))
    assert torch.equal(q_out, q)
    check_cache(bt, bt.k, bt.k_scale, k.double().numpy(), kc, ks, 0.0)
    check_cache(bt, bt.v, bt.v_scale, v.double().numpy(), vc, vs, 0.0)


def test_lists_of_two_tokens_where_one_is_the_most():
    """Recorded, and nothing outside the caches' pages of good sequences is written."""
    bt = PageBatch(new=[1, 1, 1], length=[5, 9, 17], heads=1, kv_heads=1, dim=16, page=8)
    k = torch.ones((3, 1, 16)).bfloat16().cuda()
    kc, vc, ks, vs = bt.device_cache()
    cfg, ws = bt.cfg(q_stride=0), moe.workspace(bt.cfg(), "append")
    cu, length, table = bt.lists()
    for bad in ([0, 2, 2, 3], [0, 1, 0, 3], [1, 1, 2, 3], [0, 1, 2, 2]):
        moe.moe_rope_append(cfg, None, k, k, None, torch.tensor(bad, dtype=torch.int32, device="cuda"), length, table, None, kc, vc, ks, vs, ws)
        assert moe.moe_stream_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    untouched = torch.ones(bt.n_pages, dtype=torch.bool)
    for b, n in enumerate(bt.length):
        untouched[int(bt.table[b, (n - 1) // 8])] = False
    assert torch.equal(kc.cpu()[untouched], bt.k[untouched]) and torch.equal(vc.cpu()[untouched], bt.v[untouched])
