"""The page calls and the logits call on the host (CPU only): configurations and refusals, none of
which reaches the GPU."""
import ctypes

import pytest

import sparse_mixture_experts_router_gb300 as moe
from test_serve_host import A, INV, OK, UNS, attn, call, lib  # noqa: F401

BASE = dict(n_seqs=4, n_tokens=8, max_new=3, vocab=1000, n_history=5, n_bias=3, n_masks=2)


@pytest.mark.parametrize("kw,rc", [
    ({}, OK), ({"n_seqs": 0, "n_tokens": 0}, OK), ({"n_seqs": -1}, INV), ({"n_tokens": 13}, INV), ({"n_tokens": -1}, INV), ({"max_new": 0}, INV),
    ({"max_new": 4097}, UNS), ({"vocab": 0}, INV), ({"vocab": 1}, OK), ({"vocab": (1 << 24) + 1}, UNS), ({"n_history": 1 << 30}, OK),
    ({"n_history": (1 << 30) + 1}, UNS), ({"n_bias": (1 << 30) + 1}, UNS), ({"dtype": 2}, INV), ({"out_dtype": 3}, INV),
    ({"dtype": moe.MOE_BF16, "out_dtype": moe.MOE_BF16}, OK), ({"n_history": -1}, INV), ({"n_bias": -1}, INV), ({"n_masks": -1}, INV),
    ({"logits_stride": 999}, INV), ({"p_stride": 999}, INV), ({"p_stride": 1001}, OK), ({"n_seqs": 65535}, UNS), ({"p_stride": (1 << 40) + 1}, UNS),
    ({"n_seqs": 65534, "max_new": 4096, "n_tokens": (1 << 26) + 1}, UNS),
])
def test_check_logits_config(lib, kw, rc):  # noqa: F811
    c = moe.logits_config(**{**BASE, **kw})
    assert moe.check_config(c) == rc
    assert (moe.workspace_size(c, "logits") > 0) == (rc == OK)
    assert lib.moe_check_logits_config(None) == INV
    c.out_logits = 2
    assert moe.check_config(c) == INV


LOGITS = dict(x=A, cu=A, tokens=A, history=A, cu_history=A, n_prompt=A, rep=A, pres=A, freq=A, bias_token=A, bias=A, cu_bias=A, mask=A, mask_row=A,
              temp=A, p=A + 256)


def test_logits_refusals(lib):  # noqa: F811
    c = moe.logits_config(**BASE)
    before = moe.launch_count()
    for name in LOGITS:
        if name not in ("tokens", "rep", "pres", "freq", "temp"):
            assert call(lib, "moe_logits_probs", c, {**LOGITS, name: None}.values(), kind="logits") == INV, name
        assert call(lib, "moe_logits_probs", c, {**LOGITS, name: A + 8}.values(), kind="logits") == moe.MOE_ERR_MISALIGNED, name
    need = moe.workspace_size(c, "logits")
    assert call(lib, "moe_logits_probs", c, LOGITS.values(), ws=None, nbytes=need) == INV
    assert call(lib, "moe_logits_probs", c, LOGITS.values(), ws=A + 16, nbytes=need) == moe.MOE_ERR_MISALIGNED
    assert call(lib, "moe_logits_probs", c, LOGITS.values(), nbytes=need - 1) == moe.MOE_ERR_WORKSPACE
    # entries without their number
    for kw, name in (({"n_history": 0}, "history"), ({"n_bias": 0}, "bias"), ({"n_masks": 0}, "mask")):
        assert call(lib, "moe_logits_probs", moe.logits_config(**{**BASE, **kw}), LOGITS.values(), kind="logits") == INV, name
    # in place for equal types and strides alone
    for kw in ({"out_dtype": moe.MOE_BF16}, {"p_stride": 1008}):
        assert call(lib, "moe_logits_probs", moe.logits_config(**{**BASE, **kw}), {**LOGITS, "p": A}.values(), kind="logits") == INV
    assert lib.moe_logits_probs(None, *[None] * 16, None, 0, None) == INV
    assert moe.launch_count() == before


UPDATE = dict(parent=A, len=A, kept=A, need=A, table=A, refs=A, table_out=A + 64, refs_out=A, granted=A + 64, kc=A, vc=A, ks=None, vs=None)
COMPACT = dict(len=A, table=A, refs=A, table_out=A, refs_out=A, map=A, live=A, kc=A, vc=A, ks=None, vs=None)


@pytest.mark.parametrize("fn,base,optional", [("moe_pages_update", UPDATE, {"parent", "ks", "vs"}), ("moe_pages_compact", COMPACT, {"ks", "vs"})])
def test_page_refusals(lib, fn, base, optional):  # noqa: F811
    before, c = moe.launch_count(), attn()
    for name in base:
        if name not in optional:
            assert call(lib, fn, c, {**base, name: None}.values(), kind="pages") == INV, name
        if base[name] is not None:
            assert call(lib, fn, c, {**base, name: A + 8}.values(), kind="pages") == moe.MOE_ERR_MISALIGNED, name
    need = moe.workspace_size(c, "pages")
    assert call(lib, fn, c, base.values(), ws=None, kind="pages") == INV
    assert call(lib, fn, c, base.values(), ws=A + 16, kind="pages") == moe.MOE_ERR_MISALIGNED
    assert call(lib, fn, c, base.values(), nbytes=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(lib, fn, c, {**base, "ks": A}.values(), kind="pages") == INV  # no scales for bf16
    for kind in (moe.MOE_E4M3, moe.MOE_E4M3_PAGE):
        assert call(lib, fn, attn(cache_dtype=kind), {**base, "ks": A}.values(), kind="pages") == INV
    assert getattr(lib, fn)(None, *[None] * len(base), None, 0, None) == INV
    assert moe.launch_count() == before


def test_update_in_place_needs_sequences_to_be_their_own_parents(lib):  # noqa: F811
    c = attn()
    assert call(lib, "moe_pages_update", c, {**UPDATE, "table_out": A}.values(), kind="pages") == INV
    assert call(lib, "moe_pages_update", c, {**UPDATE, "granted": A}.values(), kind="pages") == INV


def test_copy_refusals(lib):  # noqa: F811
    c = attn()
    need = moe.workspace_size(c, "pages")

    def copy(cfg=c, n=2, src=A, dst=A, n_src=4, kf=A, vf=A, ksf=None, vsf=None, kc=A, vc=A, ks=None, vs=None, ws=A, nbytes=need):
        p = [None if x is None else ctypes.c_void_p(x) for x in (kf, vf, ksf, vsf, kc, vc, ks, vs, ws)]
        return lib.moe_pages_copy(ctypes.byref(cfg) if cfg else None, n, src, dst, n_src, *p, nbytes, None)

    before = moe.launch_count()
    assert copy(cfg=None) == INV and copy(n=-1) == INV and copy(n_src=-1) == INV
    for name in ("src", "dst", "kf", "vf", "kc", "vc", "ws"):
        assert copy(**{name: None}) == INV, name
        assert copy(**{name: A + 8}) == moe.MOE_ERR_MISALIGNED, name
    assert copy(ksf=A, vsf=A) == INV and copy(ks=A, vs=A) == INV
    assert copy(cfg=attn(cache_dtype=moe.MOE_E4M3_PAGE), ks=A, vs=A) == INV
    assert copy(nbytes=need - 1) == moe.MOE_ERR_WORKSPACE
    assert moe.launch_count() == before


def test_page_limits(lib):  # noqa: F811
    assert moe.workspace_size(attn(n_pages=(1 << 30) + 1, page_size=1), "pages") == 0
    assert moe.workspace_size(attn(n_pages=1, page_size=1 << 26, max_pages=1), "pages") == 0
    assert moe.workspace_size(attn(n_pages=1 << 20), "pages") > 0
    assert moe.workspace_size(attn(n_pages=0, n_seqs=0, n_tokens=0), "pages") > 0
