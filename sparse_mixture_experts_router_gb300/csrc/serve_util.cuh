// What the decode-step kernels (rope_append.cu, paged_attention.cu,
// verify_drafts.cu) share: reading the batch's lists so that no value in
// them can form an address outside the arrays. Host functions too, so that
// the clamps can be run over arbitrary lists without a GPU.
#pragma once
#include "device_util.cuh"
#include "moe_internal.h"

namespace moe {

__host__ __device__ __forceinline__ int clamp_int(int v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// A sequence as its lists give it, clamped to the arrays: its new tokens are
// rows row0 .. row0+n-1 and its cached tokens positions 0 .. len-1, new
// token j at position len - n + j. ok: nothing had to be clamped.
struct SeqRange {
  int row0, n, len;
  bool ok;
};
__host__ __device__ __forceinline__ SeqRange seq_rows(const int32_t* cu_new, int b, int n_seqs,
                                                      int n_tokens, int max_new) {
  const int lo = cu_new[b], hi = cu_new[b + 1];
  SeqRange r;
  r.ok = lo >= 0 && hi >= lo && hi <= n_tokens && hi - lo <= max_new && (b > 0 || lo == 0) &&
         (b < n_seqs - 1 || hi == n_tokens);
  r.row0 = clamp_int(lo, 0, n_tokens);
  r.n = clamp_int(clamp_int(hi, r.row0, n_tokens) - r.row0, 0, max_new);
  r.len = 0;
  return r;
}
__host__ __device__ __forceinline__ SeqRange seq_range(const AttnArgs& a, int b) {
  SeqRange r = seq_rows(a.cu_new, b, a.c.n_seqs, a.c.n_tokens, a.c.max_new);
  const int len = a.kv_len[b], most = a.c.max_pages * a.c.page_size;
  r.ok = r.ok && len >= 0 && len <= most;
  r.len = clamp_int(len, 0, most);
  return r;
}

// The page that holds position `at` (0 <= at < max_pages * page_size) of
// sequence b, or -1 where the table names none of the cache's.
__host__ __device__ __forceinline__ int page_of(const AttnArgs& a, int b, int at) {
  const int page = a.table[(int64_t)b * a.c.max_pages + at / a.c.page_size];
  return page >= 0 && page < a.c.n_pages ? page : -1;
}

// The lists' check, by one block of kThreads: a few threads a sequence look
// at its rows, its length and the pages from position first(range) on, and
// the status word is written. The other blocks of the launch only leave out
// what the clamps above leave out, so no launch to clear the word comes first.
template <int kThreads, typename First>
__device__ void check_lists(const AttnArgs& a, First first) {
  const moe_attn_config& c = a.c;
  const int per = max(1, kThreads / c.n_seqs), sub = threadIdx.x % per;
  bool bad = false;
  for (int b = threadIdx.x / per; b < c.n_seqs; b += kThreads / per) {
    const SeqRange r = seq_range(a, b);
    bad = bad || !r.ok;
    if (r.n == 0 || r.len == 0) continue;
    const int at = first(r);
    bad = bad || at < 0;
    const int last = (r.len - 1) / c.page_size;
    const int32_t* table = a.table + (int64_t)b * c.max_pages;
#pragma unroll 4
    for (int i = max(at, 0) / c.page_size + sub; i <= last; i += per) {
      const int page = __ldg(table + i);
      bad |= page < 0 || page >= c.n_pages;
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *a.status = bad ? status_check() : MOE_OK;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace moe
