"""moe_pages_copy's lists in the binding (CPU only): the number of copies is src's, so a dst of another
length would be read behind its end."""
import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe
from test_serve_host import attn, lib  # noqa: F401


class Stand:
    """In the library's place: notes what it is called with."""

    def __init__(self, real):
        self.real, self.got = real, []

    def __getattr__(self, name):
        return getattr(self.real, name)

    def moe_pages_copy(self, cfg, n, src, dst, n_src, *rest):
        self.got.append((n, src, dst, n_src))
        return moe.MOE_OK


@pytest.fixture
def stand(lib, monkeypatch):  # noqa: F811
    s = Stand(lib)
    monkeypatch.setattr(moe, "lib", lambda: s)
    return s


def copy(src, dst):
    moe.moe_pages_copy(attn(), src, dst, 4, None, None, None, None, None, None, None, None, None, stream=0)


@pytest.mark.parametrize("n_src,n_dst", [(3, 2), (2, 3), (1, 0), (0, 1)])
def test_lists_of_different_lengths_are_refused(stand, n_src, n_dst):
    src, dst = torch.zeros(n_src, dtype=torch.int32), torch.zeros(n_dst, dtype=torch.int32)
    with pytest.raises(moe.MoeError) as e:
        copy(src, dst)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG and not stand.got


def test_equal_lists_reach_the_library(stand):
    src, dst = (torch.zeros(5, dtype=torch.int32) for _ in range(2))
    copy(src, dst)
    assert stand.got == [(5, src.data_ptr(), dst.data_ptr(), 4)]
