"""What the attention kernels' host-side functions promise (CPU only)."""
import subprocess

import numpy as np
import pytest

import attention_bounds as ab
import sparse_mixture_experts_router_gb300 as moe
from sparse_mixture_experts_router_gb300 import _build

# Two threads of a row, one barrier a tile: each leaves tile i's value, passes
# the barrier and reads the other's. Between barriers they run in any order.
ORDER = r"""
#include <cstdio>
#include "paged_attention.cuh"
constexpr int kRows = 4, kTiles = 9;
struct Thread { int tile = 0, at = 0; };  // at 0: to write, 1: at the barrier, 2: to read
template <typename Slot>
bool reads_own_tiles(Slot slot) {
  unsigned long long x = 88172645463325252ull;
  for (int trial = 0; trial < 20000; ++trial) {
    int mem[8 * kRows];
    for (int& m : mem) m = -1;
    Thread t[2];
    const int row = trial % kRows;
    while (t[0].tile < kTiles || t[1].tile < kTiles) {
      x ^= x << 13; x ^= x >> 7; x ^= x << 17;
      // runs of one thread's steps, so that it gets as far ahead as it can
      const int h = (x >> 40) % 8 ? (int)(x >> 20) & 1 : trial & 1;
      Thread& a = t[h];
      Thread& b = t[h ^ 1];
      if (a.tile == kTiles) continue;
      if (a.at == 0) {
        mem[slot(a.tile, h, row)] = a.tile;
        a.at = 1;
      } else if (a.at == 1) {
        // passes once the other has arrived at the same barrier, or passed it
        if (b.tile > a.tile || (b.tile == a.tile && b.at >= 1)) a.at = 2;
      } else {
        if (mem[slot(a.tile, h ^ 1, row)] != a.tile) return false;
        a.at = 0;
        ++a.tile;
      }
    }
  }
  return true;
}
int main() {
  bool used[4 * kRows] = {};
  for (int i = 0; i < 2; ++i)
    for (int h = 0; h < 2; ++h)
      for (int r = 0; r < kRows; ++r) {
        const int s = moe::attn::max_slot(i, h, r, kRows);
        if (s < 0 || s >= 4 * kRows || used[s]) return 1;
        used[s] = true;
      }
  if (!reads_own_tiles([](int i, int h, int r) { return moe::attn::max_slot(i, h, r, kRows); })) return 2;
  // one place for all tiles is overwritten in some order
  if (reads_own_tiles([](int, int h, int r) { return h * kRows + r; })) return 3;
  return 0;
}
"""


def run(tmp_path, name, source):
    src, exe = tmp_path / f"{name}.cu", str(tmp_path / name)
    src.write_text(source)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.CSRC, str(src),
                    "-o", exe], check=True, capture_output=True)
    return subprocess.run([exe], timeout=120, capture_output=True, text=True)


def test_a_rows_two_maxima_are_read_before_they_are_overwritten(tmp_path):
    assert run(tmp_path, "order", ORDER).returncode == 0


@pytest.mark.parametrize("pages,page,max_pages,kv_heads,rc", [
    (1 << 30, 1 << 30, 0, 16, moe.MOE_ERR_UNSUPPORTED), (2 ** 31 - 1, 1 << 29, 1, 16, moe.MOE_ERR_UNSUPPORTED),
    (2 ** 31 - 1, 2 ** 31 - 1, 0, 1024, moe.MOE_ERR_UNSUPPORTED), (1 << 20, 1 << 16, 1, 16, moe.MOE_ERR_UNSUPPORTED),
    ((1 << 20) - 1, 1 << 16, 1, 16, moe.MOE_OK), (1 << 24, 16, 1 << 16, 8, moe.MOE_OK)])
def test_caches_of_2_to_the_40_rows_are_refused(pages, page, max_pages, kv_heads, rc):
    """The product passes 64 bits for the first three."""
    _build.build()
    c = moe.attn_config(n_seqs=1, n_tokens=1, n_heads=kv_heads, n_kv_heads=kv_heads, head_dim=64, page_size=page, n_pages=pages,
                        max_pages=max_pages)
    assert moe.check_config(c) == rc
    assert (moe.workspace_size(c, "attention") > 0) == (rc == moe.MOE_OK)


@pytest.mark.parametrize("new,length,heads,dim", [([1], [48], 4, 64), ([2, 1], [64, 31], 8, 128), ([7], [64], 16, 64), ([1], [40], 4, 256)])
def test_the_bound_of_weights_tells_one_term_from_two(new, length, heads, dim):
    """What test_gpu_attention_edges.py holds the kernels to: weights of one bf16 term pass
    it by far, two terms stay inside."""
    bt = ab.cancelling(new, length, heads, 2, dim, seed=50)
    out, tol = ab.rows64(bt)
    assert (np.abs(ab.rows64(bt, ab.two_terms)[0] - out) <= tol / 2).all()
    off = np.abs(ab.rows64(bt, ab.one_term)[0] - out) / tol
    assert off.max() > 4 and (off > 1).any(-1).mean() > 0.9
