"""The decode-step calls on the host (CPU only): what their configurations
allow, that every bad argument is refused before any CUDA call, and that the
lists' clamps, run as host code, form no index outside the arrays."""
import ctypes
import math
import os
import subprocess

import pytest

import sparse_mixture_experts_router_gb300 as moe
from sparse_mixture_experts_router_gb300 import _build

A = 0x10000  # an aligned address that no test dereferences


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.lib()


def attn(**kw):
    base = dict(n_seqs=4, n_tokens=8, max_new=3, n_heads=8, n_kv_heads=2, head_dim=128, page_size=16,
                n_pages=64, max_pages=16, rot_dim=64)
    base.update(kw)
    return moe.attn_config(**base)


OK, INV, UNS = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,rc", [
    ({}, OK), ({"n_seqs": 0, "n_tokens": 0}, OK), ({"n_seqs": -1}, INV), ({"n_tokens": -1}, INV),
    ({"n_tokens": 13}, INV), ({"max_new": 0}, INV), ({"max_new": 4097}, UNS), ({"n_heads": 7}, INV),
    ({"n_heads": 0}, INV), ({"n_kv_heads": 0}, INV), ({"head_dim": 0, "rot_dim": 0}, INV),
    ({"head_dim": 264}, UNS), ({"head_dim": 68}, UNS), ({"head_dim": 72}, OK),
    ({"head_dim": 72, "cache_dtype": moe.MOE_E4M3}, UNS), ({"head_dim": 256}, OK),
    ({"page_size": 0}, INV), ({"page_size": 1}, OK), ({"page_size": 1 << 27}, UNS),
    ({"n_pages": 0}, OK), ({"max_pages": 0}, OK), ({"dtype": 2}, INV), ({"dtype": moe.MOE_F32}, OK),
    ({"cache_dtype": moe.MOE_F32}, INV), ({"cache_dtype": moe.MOE_E4M3}, OK),
    ({"dtype": moe.MOE_F32, "cache_dtype": moe.MOE_E4M3}, INV), ({"window": -1}, INV),
    ({"rot_dim": 63}, INV), ({"rot_dim": 130}, INV), ({"rot_dim": 0}, OK), ({"rot_dim": 42}, OK),
    ({"rot_sections": (16, 8, 8)}, OK), ({"rot_sections": (16, 8, 9)}, INV),
    ({"rot_sections": (40, -8, 0)}, INV), ({"rope_base": 0.5}, INV), ({"rope_base": math.nan}, INV),
    ({"rope_base": math.inf}, INV), ({"rope_base": 1.0}, OK), ({"scale": math.nan}, INV),
    ({"scale": math.inf}, INV), ({"scale": -0.1}, OK), ({"q_stride": 1023}, INV),
    ({"q_stride": 1028}, UNS), ({"q_stride": 1536}, OK), ({"k_stride": 255}, INV),
    ({"page_stride": 4096}, INV), ({"page_stride": 4096, "token_stride": 256, "head_stride": 128}, OK),
    ({"page_stride": 4096, "token_stride": 256, "head_stride": 132}, UNS),
    ({"n_seqs": 65535}, UNS),
])
def test_check_attn_config(lib, kw, rc):
    c = attn(**kw)
    assert moe.check_config(c) == rc
    for kind in ("append", "attention"):
        assert (moe.workspace_size(c, kind) > 0) == (rc == OK)
    assert lib.moe_check_attn_config(None) == INV


@pytest.mark.parametrize("kw,rc", [
    ({}, OK), ({"n_seqs": 0, "n_tokens": 0}, OK), ({"vocab": 0}, INV), ({"vocab": 1}, OK),
    ({"vocab": 1 << 25}, UNS), ({"n_tokens": 21}, INV), ({"max_new": 0}, INV), ({"dtype": 2}, INV),
    ({"dtype": moe.MOE_BF16}, OK), ({"p_stride": 999}, INV), ({"q_stride": 999}, INV),
    ({"p_stride": 1001}, OK), ({"n_seqs": -1}, INV),
])
def test_check_verify_config(lib, kw, rc):
    c = moe.verify_config(**{**dict(n_seqs=4, n_tokens=20, max_new=5, vocab=1000), **kw})
    assert moe.check_config(c) == rc
    assert (moe.workspace_size(c, "verify") > 0) == (rc == OK)
    assert lib.moe_check_verify_config(None) == INV


def call(lib, fn, cfg, ptrs, ws=A, nbytes=None, kind=None):
    nbytes = moe.workspace_size(cfg, kind) if nbytes is None else nbytes
    return getattr(lib, fn)(ctypes.byref(cfg), *[None if p is None else ctypes.c_void_p(p) for p in ptrs],
                            None if ws is None else ctypes.c_void_p(ws), nbytes, None)


APPEND = dict(q=A, k=A, v=A, pos=A, cu=A, len=A, table=A, q_out=A, kc=A, vc=A, ks=None, vs=None)
ATTEND = dict(q=A, cu=A, len=A, table=A, kc=A, vc=A, ks=None, vs=None, out=A, lse=A)
VERIFY = dict(p=A, q=A, tokens=A, ua=A, us=A, cu=A, len=A, out=A, acc=A, next=A)


@pytest.mark.parametrize("fn,kind,base,optional,conf", [
    ("moe_rope_append", "append", APPEND, {"pos", "ks", "vs"}, attn()),
    ("moe_paged_attention", "attention", ATTEND, {"ks", "vs", "lse"}, attn()),
    ("moe_verify_drafts", "verify", VERIFY, {"q", "len", "next"},
     moe.verify_config(n_seqs=4, n_tokens=20, max_new=5, vocab=1000)),
])
def test_refusals_launch_nothing(lib, fn, kind, base, optional, conf):
    before = moe.launch_count()
    for name in base:
        if name not in optional:
            assert call(lib, fn, conf, {**base, name: None}.values(), kind=kind) == INV, name
        if base[name] is not None:
            assert call(lib, fn, conf, {**base, name: A + 8}.values(), kind=kind) == \
                moe.MOE_ERR_MISALIGNED, name
    need = moe.workspace_size(conf, kind)
    assert call(lib, fn, conf, base.values(), ws=None, kind=kind) == INV
    assert call(lib, fn, conf, base.values(), ws=A + 16, kind=kind) == moe.MOE_ERR_MISALIGNED
    assert call(lib, fn, conf, base.values(), nbytes=need - 1, kind=kind) == moe.MOE_ERR_WORKSPACE
    assert getattr(lib, fn)(None, *[None] * len(base), None, 0, None) == INV
    assert moe.launch_count() == before


def test_refusals_of_combinations(lib):
    e4 = attn(cache_dtype=moe.MOE_E4M3)
    # scales with an E4M3 cache, and only with one
    assert call(lib, "moe_paged_attention", e4, ATTEND.values(), kind="attention") == INV
    assert call(lib, "moe_paged_attention", attn(), {**ATTEND, "ks": A}.values(), kind="attention") == INV
    assert call(lib, "moe_rope_append", e4, {**APPEND, "ks": A}.values(), kind="append") == INV
    # q and q_out come together; in place only for packed rows
    assert call(lib, "moe_rope_append", attn(), {**APPEND, "q_out": None}.values(), kind="append") == INV
    assert call(lib, "moe_rope_append", attn(q_stride=2048), APPEND.values(), kind="append") == INV
    # kv_next is formed from kv_len
    v = moe.verify_config(n_seqs=4, n_tokens=20, max_new=5, vocab=1000)
    assert call(lib, "moe_verify_drafts", v, {**VERIFY, "len": None}.values(), kind="verify") == INV


HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "serve_util.cuh"
// Lists of arbitrary values (and valid ones) through the clamps the kernels
// use: rows inside [0, T), lengths and pages inside the cache.
int main() {
  unsigned long long x = 88172645463325252ull;
  auto rnd = [&] { x ^= x << 13; x ^= x >> 7; x ^= x << 17; return (int)(x >> 20); };
  int bad_seen = 0, good_seen = 0;
  for (int trial = 0; trial < 200000; ++trial) {
    moe::AttnArgs a = {};
    const int B = 1 + (unsigned)rnd() % 4;
    a.c.n_seqs = B;
    a.c.max_new = 1 + (unsigned)rnd() % 5;
    a.c.page_size = 1 + (unsigned)rnd() % 7;
    a.c.max_pages = (unsigned)rnd() % 5;
    a.c.n_pages = (unsigned)rnd() % 6;
    std::vector<int> cu(B + 1), len(B), table(B * a.c.max_pages + 1);
    const bool wild = trial % 2;
    int t = 0;
    for (int b = 0; b <= B; ++b) {
      cu[b] = wild && rnd() % 2 ? rnd() >> ((unsigned)rnd() % 31) : t;
      if (b < B) t += (unsigned)rnd() % (a.c.max_new + 1);
    }
    a.c.n_tokens = wild ? (unsigned)rnd() % (B * a.c.max_new + 1) : cu[B];
    for (int& v : len) v = wild ? rnd() >> ((unsigned)rnd() % 31) : (unsigned)rnd() % (a.c.max_pages * a.c.page_size + 1);
    for (int& v : table) v = rnd() >> ((unsigned)rnd() % 31);
    a.cu_new = cu.data(); a.kv_len = len.data(); a.table = table.data();
    for (int b = 0; b < B; ++b) {
      const moe::SeqRange r = moe::seq_range(a, b);
      if (r.row0 < 0 || r.n < 0 || r.n > a.c.max_new || r.row0 + r.n > a.c.n_tokens) return 1;
      if (r.len < 0 || r.len > a.c.max_pages * a.c.page_size) return 2;
      if (!wild && !r.ok) return 3;
      if (r.ok && (r.row0 != cu[b] || r.n != cu[b + 1] - cu[b] || r.len != len[b])) return 4;
      (r.ok ? good_seen : bad_seen)++;
      for (int i = 0; i < r.len; ++i) {
        const int page = moe::page_of(a, b, i);
        if (page < -1 || page >= a.c.n_pages) return 5;
      }
    }
  }
  return bad_seen > 1000 && good_seen > 1000 ? 0 : 6;
}
"""


def test_list_clamps_form_no_index_outside(tmp_path):
    src = tmp_path / "clamps.cu"
    src.write_text(HARNESS)
    exe = str(tmp_path / "clamps")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O1", "-std=c++17", "-I", _build.CSRC, str(src), "-o", exe],
                   check=True, capture_output=True)
    assert subprocess.run([exe], timeout=120).returncode == 0
