// What the paged attention kernels share: the cut of the work into items and
// parts, the lookup of keys in the pages, and the join of the parts.
//
// An item is one (sequence, key-value head, block of query rows): row r of a
// head group is query head r % G of new token r / G, G heads a key-value
// head. An item's keys are cut into splits x parts ranges, a thread block
// each. The parts of a split are a cluster and join through its distributed
// shared memory; the splits, where there are several (an item or two of very
// many keys), leave unnormalised rows in the workspace that a second kernel
// joins.
#pragma once
#include "serve_util.cuh"
#include "serve_ptx.cuh"

namespace moe {
namespace attn {

constexpr int kMaxParts = 16;   // the largest cluster
constexpr int kMaxSplits = 32;
constexpr int kPlanSms = 152;   // the plan does not ask the device, so that the workspace's size is a constant of cfg

// Blocks an SM holds, by registers and by shared memory: of the bf16 and E4M3
// kernel, and of the fp32 one with nt groups of four rows.
constexpr int blocks_per_sm(int dim) { return dim > 128 ? 1 : 3; }
constexpr int f32_blocks_per_sm(int dim, int nt) {
  return dim > 128 ? (nt == 1 ? 3 : 2) : nt > 2 ? 3 : dim <= 64 && nt == 1 ? 8 : 5;
}

// Keys of a tile of the bf16 and E4M3 kernel.
constexpr int keys_of(int dim, bool f8) { return f8 || dim <= 64 ? 32 : 16; }

// n / d for 0 <= n < 2^30 and 1 <= d < 2^30 as a multiplication.
struct FastDiv {
  uint64_t mul;
  int shift;
};
inline FastDiv fast_div(uint32_t d) {
  int bits = 0;
  while ((1u << bits) < d) ++bits;
  const int shift = 30 + bits;
  return {((1ull << shift) + d - 1) / d, shift};
}
__device__ __forceinline__ int div(const FastDiv& f, int n) {
  return (int)(((uint64_t)n * f.mul) >> f.shift);
}

struct Params {
  AttnArgs a;
  int parts, splits;
  int row_blocks;  // of one (sequence, key-value head)
  int group;       // heads a key-value head
  // The lists are checked as they are used, after a launch that clears the
  // status word, and not by a block of their own: for long tables.
  int check_in_use;
  // divisions by page_size, heads a key-value head, parts, splits,
  // row_blocks, n_kv_heads and head_dim / 4
  FastDiv by_page, by_group, by_parts, by_splits, by_rows, by_heads, by_vecs;
  int item_rows;   // query rows of an item
  // splits > 1: O [item][split][item_rows][head_dim] relative to its maximum,
  // and (maximum in log2 units, sum) [item][split][item_rows]
  float* split_o;
  float2* split_ml;
};

// The first position that a sequence's new tokens see.
struct FirstKey {
  int window;
  __device__ int operator()(const SeqRange& r) const {
    return window ? max(0, r.len - r.n - window + 1) : 0;
  }
};

struct Item {
  SeqRange sq;
  int index, split, part;  // of this thread block
  int b, kh, G;
  int row0, rows;          // its query rows: row0 .. row0 + rows - 1 of the head group
  int window;
  __device__ __forceinline__ int clip(int r) const { return row0 + min(r, rows - 1); }
  // Position of row r's token and the first it sees. Rows past the last one
  // repeat it and are not written.
  __device__ __forceinline__ int pos(const Params& p, int r) const {
    return sq.len - sq.n + div(p.by_group, clip(r));
  }
  __device__ __forceinline__ int first(int at) const {
    return window ? max(0, at - window + 1) : 0;
  }
  // Elements from q's start to row r.
  __device__ __forceinline__ int64_t q_at(const Params& p, int r) const {
    const int g = clip(r), j = div(p.by_group, g);
    return (int64_t)(sq.row0 + j) * p.a.c.q_stride + (kh * G + g - j * G) * p.a.c.head_dim;
  }
};
// This block's item, false where it has none (the first cluster checks the
// lists; the whole cluster returns alike).
template <int kThreads>
__device__ __forceinline__ bool item_of(const Params& p, int block_rows, Item& it) {
  const moe_attn_config& c = p.a.c;
  int i = div(p.by_parts, (int)blockIdx.x);
  it.part = (int)blockIdx.x - i * p.parts;
  if (--i < 0) {
    if (it.part == 0 && !p.check_in_use) check_lists<kThreads>(p.a, FirstKey{c.window});
    return false;
  }
  auto next = [&](const FastDiv& f, int d) {  // i / d, and the remainder
    const int q = div(f, i), r = i - q * d;
    i = q;
    return r;
  };
  it.split = next(p.by_splits, p.splits);
  it.index = i;
  const int rb = next(p.by_rows, p.row_blocks);
  it.kh = next(p.by_heads, c.n_kv_heads);
  it.b = i;
  it.sq = seq_range(p.a, it.b);
  if (p.check_in_use && !it.sq.ok && threadIdx.x == 0) set_status(p.a.status, status_check());
  it.G = p.group;
  it.row0 = rb * block_rows;
  it.rows = min(block_rows, it.G * it.sq.n - it.row0);
  it.window = c.window;
  return it.rows > 0;
}

// The keys an item's rows see, in tiles of kKeys from `base` on; this block's
// are t0 .. t1-1.
struct Range {
  int hi_min, hi_max;  // last position of the first and of the last row
  int lo_min, lo_max;  // first position of the same
  int base, t0, t1;
};
__device__ __forceinline__ Range range_of(const Params& p, const Item& it, int block_rows,
                                          int keys) {
  Range r;
  r.hi_min = it.pos(p, 0);
  r.hi_max = it.pos(p, block_rows - 1);
  r.lo_min = it.first(r.hi_min);
  r.lo_max = it.first(r.hi_max);
  r.base = r.lo_min / keys * keys;
  const int tiles = r.hi_max < 0 ? 0 : (r.hi_max - r.base) / keys + 1;
  const int at = it.split * p.parts + it.part, of = p.splits * p.parts;
  const int each = tiles / of, more = tiles - each * of;  // the first `more` blocks take one more
  r.t0 = at * each + min(at, more);
  r.t1 = r.t0 + each + (at < more);
  return r;
}

// A key's place in the cache: its page as the table has it and its place in the
// page (both -1 for a key no row sees). Nothing here uses the page, so a lookup
// for a later tile does not wait for the table.
struct Slot {
  int page, place;
  __device__ __forceinline__ void check(const Params& p) const {
    if (p.check_in_use && place >= 0 && !in(p.a.c)) set_status(p.a.status, status_check());
  }
  __device__ __forceinline__ bool in(const moe_attn_config& c) const {
    return page >= 0 && page < c.n_pages;
  }
  __device__ __forceinline__ int64_t at(const moe_attn_config& c, int kh) const {
    return (int64_t)page * c.page_stride + (int64_t)place * c.token_stride +
           (int64_t)kh * c.head_stride;
  }
  __device__ __forceinline__ int64_t scale_at(const moe_attn_config& c, int kh) const {
    return ((int64_t)page * c.n_kv_heads + kh) * c.page_size + place;
  }
};
__device__ __forceinline__ Slot slot_of(const Params& p, const Item& it, const Range& r, int key) {
  Slot s = {-1, -1};
  if (key >= r.lo_min && key <= r.hi_max) {
    const int n = div(p.by_page, key);
    s.place = key - n * p.a.c.page_size;
    s.page = __ldg(p.a.table + (int64_t)it.b * p.a.c.max_pages + n);
  }
  return s;
}

// Where the thread with half `half` (0, 1) of a row's keys leaves its maximum of
// tile i for the other. Between the write and the read stands the tile's only
// barrier, and nothing holds a thread back from writing tile i + 1's before the
// other has read tile i's: the tiles alternate between two places, and that of
// tile i + 2 is written behind the barrier of tile i + 1.
__host__ __device__ constexpr int max_slot(int tile, int half, int row, int rows) {
  return ((tile & 1) * 2 + half) * rows + row;
}

// Two weights (a pair of fp32) as two bf16 terms each, together within 2^-16 of
// the weight: hi, and the rounded rest. Were hi rounded to nearest (2^-17), the
// rest could be 0 or negative, and against an infinite value hi inf + lo inf
// would be NaN. So hi is rounded down, and the rest is taken from hi (1 - 2^-23),
// which leaves it positive for a weight above 2^-110. A weight of 0 has both
// terms 0, a NaN has NaN.
__device__ __forceinline__ void split_bf16(uint64_t p, uint32_t& hi, uint32_t& lo) {
  hi = ptx::bf16x2_down(ptx::f32x2_lo(p), ptx::f32x2_hi(p));
  const uint64_t h = (uint64_t)(hi & 0xffff0000u) << 32 | (hi << 16);
  const uint64_t rest = ptx::fma_f32x2(h, ptx::f32x2(0x1p-23f - 1.f, 0x1p-23f - 1.f), p);
  lo = f32x2_to_bf16x2(ptx::f32x2_lo(rest), ptx::f32x2_hi(rest));
}

// ---- the join ----------------------------------------------------------------
__device__ __forceinline__ void store4(float* out, int64_t at, float4 x) {
  reinterpret_cast<float4*>(out)[at] = x;
}
__device__ __forceinline__ void store4(__nv_bfloat16* out, int64_t at, float4 x) {
  reinterpret_cast<uint2*>(out)[at] =
      make_uint2(f32x2_to_bf16x2(x.x, x.y), f32x2_to_bf16x2(x.z, x.w));
}
// Four elements (v) of row r from their sum relative to 2^top and the sum of
// weights: the output, or the split's part of it.
template <typename Elem>
__device__ __forceinline__ void write_row(const Params& p, const Item& it, int r, int v, float4 x,
                                          float top, float sum) {
  const moe_attn_config& c = p.a.c;
  const int vecs = c.head_dim / 4;
  if (p.splits > 1) {
    const int64_t row = ((int64_t)it.index * p.splits + it.split) * p.item_rows + r;
    reinterpret_cast<float4*>(p.split_o)[row * vecs + v] = x;
    if (v == 0) p.split_ml[row] = make_float2(top, sum);
    return;
  }
  const float f = 1.f / sum;  // a NaN stays one
  x = sum == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                 : make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
  const int g = it.row0 + r, j = div(p.by_group, g);
  const int at = (it.sq.row0 + j) * c.n_heads + it.kh * it.G + g - j * it.G;  // T * Hq < 2^30
  store4(static_cast<Elem*>(p.a.out), (int64_t)at * vecs + v, x);
  if (v == 0 && p.a.lse)
    p.a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// Where the blocks of a cluster leave what one of them joins: (maximum, sum)
// of every block's rows, and of O the slice of rows x vectors that this block
// writes, from every block.
template <int kRows, int kDim>
struct Inbox {
  float2 ml[kMaxParts][kRows];
  // slices of ceil(n / parts) of the n <= kRows * kDim / 4 vectors
  float4 o[kRows * kDim / 4 + kMaxParts];
};

// Joins a block's kWarps partial O (row r at o + w * stride + r * ld floats,
// all relative to the block's maximum joined[r]; joined[kRows + r] its sum of
// weights) and then the cluster's blocks, and writes the rows. Each block
// sends every other its slice and then reads its own shared memory only, so no
// barrier has to keep blocks from leaving. With kOwnInbox the inbox is memory
// of its own and a block sends as soon as all have started (start_cluster);
// otherwise it lies over the stages of the warps after the first, and blocks
// send when all have read theirs: one barrier more, 8 to 16 KB less.
template <int kRows, int kDim, int kWarps, int kThreads, bool kOwnInbox, typename Elem>
__device__ __forceinline__ void finish(const Params& p, const Item& it, float* o, int stride, int ld,
                                       const float* joined, Inbox<kRows, kDim>* inbox) {
  const int vecs = p.a.c.head_dim / 4, n = it.rows * vecs;
  auto at = [&](int w, int r, int v) {
    return reinterpret_cast<float4*>(o + w * stride + r * ld + 4 * v);
  };
  auto block_sum = [&](int r, int v) {
    float4 x = *at(0, r, v);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 y = *at(w, r, v);
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    return x;
  };
  if (p.parts == 1) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int r = div(p.by_vecs, i), v = i - r * vecs;
      write_row<Elem>(p, it, r, v, block_sum(r, v), joined[r], joined[kRows + r]);
    }
    return;
  }
  const int slice = div(p.by_parts, n + p.parts - 1);
  __syncwarp();
  ptx::cluster_wait();  // pairs with start_cluster
  if (!kOwnInbox) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int r = div(p.by_vecs, i), v = i - r * vecs;
      *at(0, r, v) = block_sum(r, v);
    }
    __syncwarp();
    ptx::cluster_sync();
  }
  for (int i = threadIdx.x; i < kRows * p.parts; i += kThreads) {
    const int r = div(p.by_parts, i);
    ptx::st_cluster_v2(
        ptx::mapa_shared(ptx::smem_addr(&inbox->ml[it.part][r]), i - r * p.parts), joined[r],
        joined[kRows + r]);
  }
  int to = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int r = div(p.by_vecs, i), v = i - r * vecs;
    while ((to + 1) * slice <= i) ++to;
    ptx::st_cluster_v4(
        ptx::mapa_shared(ptx::smem_addr(&inbox->o[it.part * slice + i - to * slice]), to),
        kOwnInbox ? block_sum(r, v) : *at(0, r, v));
  }
  __syncwarp();
  ptx::cluster_sync();
  const int i0 = it.part * slice;
  for (int i = i0 + threadIdx.x; i < min(i0 + slice, n); i += kThreads) {
    const int r = div(p.by_vecs, i), v = i - r * vecs;
    float top = -INFINITY, sum = 0.f;
#pragma unroll 4
    for (int b = 0; b < p.parts; ++b) top = fmaxf(top, inbox->ml[b][r].x);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int b = 0; b < p.parts; ++b) {
      const float2 ml = inbox->ml[b][r];
      const float4 y = inbox->o[b * slice + i - i0];
      const float f = ptx::ex2(ml.x - top);
      sum += ml.y * f;
      x.x += y.x * f, x.y += y.y * f, x.z += y.z * f, x.w += y.w * f;
    }
    write_row<Elem>(p, it, r, v, x, top, sum);
  }
}
__device__ __forceinline__ void start_cluster(const Params& p) {
  if (p.parts > 1) ptx::cluster_arrive();
}

// Sets a kernel's shared memory and cluster attributes (once a thread and
// device) and launches it.
template <typename Kernel>
cudaError_t launch(Kernel kernel, int* configured, const Params& p, unsigned blocks, int threads,
                   int smem, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (*configured != dev) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    *configured = dev;
  }
  return launch_pdl(kernel, dim3(blocks), dim3((unsigned)threads), (size_t)smem, s, p.parts, p);
}

}  // namespace attn
}  // namespace moe
