"""E4M3 caches with page scales on the host (CPU only): configurations and refusals."""
import pytest

import sparse_mixture_experts_router_gb300 as moe
from page_common import scale64
from test_serve_host import A, APPEND, ATTEND, INV, OK, UNS, attn, call, lib  # noqa: F401


@pytest.mark.parametrize("kw,rc", [
    ({}, OK), ({"head_dim": 72}, UNS), ({"head_dim": 80}, OK), ({"dtype": moe.MOE_F32}, INV), ({"page_size": 1}, OK),
    ({"page_stride": 4096, "token_stride": 256, "head_stride": 136}, UNS),
    ({"page_stride": 4096, "token_stride": 256, "head_stride": 128}, OK), ({"cache_dtype": 4}, INV),
])
def test_check_attn_config(lib, kw, rc):  # noqa: F811
    c = attn(**{"cache_dtype": moe.MOE_E4M3_PAGE, **kw})
    assert moe.check_config(c) == rc
    for kind in ("append", "attention"):
        assert (moe.workspace_size(c, kind) > 0) == (rc == OK)


def test_scales_come_with_the_cache(lib):  # noqa: F811
    c = attn(cache_dtype=moe.MOE_E4M3_PAGE)
    before = moe.launch_count()
    assert call(lib, "moe_paged_attention", c, ATTEND.values(), kind="attention") == INV
    assert call(lib, "moe_rope_append", c, {**APPEND, "ks": A}.values(), kind="append") == INV
    assert call(lib, "moe_rope_append", c, {**APPEND, "ks": A, "vs": A + 4}.values(), kind="append") == moe.MOE_ERR_MISALIGNED
    assert moe.launch_count() == before


def test_scale_of_the_tests():
    assert scale64(448) == 1 and scale64(448.0001) == 2 and scale64(224) == 0.5 and scale64(0) == 2.0 ** -110
    assert scale64(3.3e38) == 2.0 ** 119 and scale64(1e-45) == 2.0 ** -110
