"""moe_logits_probs at the edges of its ranges: rows that start anywhere on the 16-byte grid, and
temperatures at the end of fp32."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from serve_common import TORCH
from test_gpu_logits import Rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 9, 31, 4097, 33003])
def test_rows_start_and_end_anywhere_in_a_vector(dtype, out, V):
    """Eleven rows V + 1, 3 or 5 elements apart begin at every offset of a 16-byte vector."""
    for pad, p_pad in ((1, 0), (3, 1), (5, 3)):
        r = Rows([1] * 11, V, dtype=dtype, out=out, history=5, biases=2, masks=2, pad=pad, p_pad=p_pad, seed=V + pad)
        r.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_in_place_leave_what_is_between_them(dtype):
    r = Rows([1] * 11, 45, dtype=dtype, out=dtype, history=5, pad=7, seed=3)
    want = Rows([1] * 11, 45, dtype=dtype, out=dtype, history=5, pad=7, seed=3).run()
    p = r.logits.cuda()
    cfg = r.cfg(p_stride=52)
    ws = moe.workspace(cfg, "logits")
    moe.moe_logits_probs(cfg, p, *r.lists().values(), p, ws)
    assert moe.moe_stream_status(ws) == 0
    assert np.array_equal(p[:, :45].double().cpu().numpy(), want)
    assert torch.equal(p[:, 45:].cpu(), r.logits[:, 45:].to(TORCH[dtype]))


def test_logits_out_over_the_least_temperatures():
    """1 / temperature is infinite in fp32 from 2^-128 down: 0 stays 0, others become large or infinite
    with their sign, by fp32's largest number."""
    x = torch.tensor([0.0, -0.0, 1e-10, -1e-10, 1.0, -1.0, 3.0, -3.0, float("-inf"), float("inf")])
    top = float(torch.finfo(torch.float32).max)
    for temp in (2.0 ** -149, 1e-40, 2.0 ** -129):
        cfg = moe.logits_config(n_seqs=1, n_tokens=1, vocab=x.numel(), out_logits=True)
        ws = moe.workspace(cfg, "logits")
        p = torch.empty((1, x.numel()), device="cuda")
        cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        t = torch.tensor([temp], device="cuda")
        moe.moe_logits_probs(cfg, x[None].cuda(), cu, *[None] * 12, t, p, ws)
        assert moe.moe_stream_status(ws) == 0
        want = (x.double() * min(1 / temp, top)).float()
        assert torch.allclose(p[0].cpu(), want, rtol=2.0 ** -23, atol=0.0), (temp, p)
