// Rotary append into an E4M3 cache with one scale per page and head.
//
// The scale of a page's head is 2^e, the least power of two with |x| <= 448 2^e
// for the elements the page holds. A power of two costs E4M3 no precision (it
// moves the exponent) and makes two things exact: raising the scale for a later,
// larger token (older codes are multiplied by 2^(old - new), a change of
// exponent that rounds only codes that become subnormal), and widening a code
// times its scale to bf16, which attention of many rows does.
//
// So the new tokens of one page have to meet before any of them is written: an
// item is a (sequence, page) that the call touches. Sequence b's items start at
// floor(cu_new[b] / page_size) + 2 b, which leaves each sequence at least as many
// as n tokens can touch (1 + ceil((n - 1) / page_size)); with one new token a
// sequence, at b. A warp takes a head of the item's keys, values or queries: its
// rows (8 for each group of lanes that holds a row) stay in registers between
// the maximum and the write. The item's sines and cosines are computed once a
// block, in chunks of that many rows; a page with more new rows than a chunk is
// read twice. One block more checks the lists and writes the status.
//
// Bound by memory for prompts and by the latency of one chain (sequence, page,
// old scale, rows) for a few tokens.
#include <cfloat>

#include <cuda_fp16.h>

#include "rope_append.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsLane = 8;  // rows a group of lanes holds
// Chunk rows x pairs: 8 (32 / lanes) rows of at most 4 lanes pairs.
constexpr int kTurns = kRowsLane * 32 * 4;
constexpr int kMinExp = -110, kMaxExp = 119;

// 2^e for elements up to amax (finite, >= 0): 448 = 1.75 x 2^8.
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)(clamp_int(e, kMinExp, kMaxExp) + 127) << 23);
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= FLT_MAX; }

__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio) {
  uint32_t r = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)(codes >> 16 * h)));
    const __half2 x = *reinterpret_cast<const __half2*>(&f);
    r |= e4m3x2(__low2float(x) * ratio, __high2float(x) * ratio) << 16 * h;
  }
  return r;
}

// What an item is: rows row0 .. row0 + rows - 1 of the call's tokens, at
// positions at0 .. of their sequence, in places place0 .. of page.
struct PageItem {
  int row0, rows, at0, place0, page;
};
// The item of index i (false: none), found by a whole warp.
__device__ __forceinline__ bool page_item(const AttnArgs& a, int per_seq, int index, int lane,
                                          PageItem& it) {
  const moe_attn_config& c = a.c;
  auto start = [&](int b) {
    return clamp_int(__ldg(a.cu_new + b), 0, c.n_tokens) / c.page_size + per_seq * b;
  };
  int lo = 0, hi = c.n_seqs;  // the first sequence whose items end after index
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step - 1;
    const unsigned after = __ballot_sync(0xffffffffu, i >= hi || start(i + 1) > index);
    if (!after) return false;  // only where the list does not ascend
    const int f = __ffs(after) - 1;
    hi = min(hi, lo + (f + 1) * step - 1);
    lo += f * step;
  }
  if (lo >= c.n_seqs) return false;
  const SeqRange r = seq_range(a, lo);
  const int first = max(r.len - r.n, 0);  // below 0: no slot, recorded by the check
  const int page = first / c.page_size + index - start(lo);
  if (!r.ok || index < start(lo) || page > (r.len - 1) / c.page_size || r.len - r.n < 0 || r.n == 0)
    return false;
  it.at0 = max(first, page * c.page_size);
  it.rows = min(r.len, (page + 1) * c.page_size) - it.at0;
  it.row0 = r.row0 + it.at0 - first;
  it.place0 = it.at0 - page * c.page_size;
  it.page = page_of(a, lo, it.at0);
  return true;
}

// kBits: a row is held by 1 << kBits lanes.
template <int kBits>
__global__ void __launch_bounds__(kThreads, 2)
    rope_append_page_kernel(const AttnArgs a, const __grid_constant__ RopeTable rope, int per_seq) {
  constexpr int kLanes = 1 << kBits, kGroups = 32 / kLanes, kChunk = kRowsLane * kGroups;
  __shared__ float2 turns[kTurns + kTurns / 8];  // (cos, sin) of a chunk's pairs, padded
  __shared__ float scales[2 * kAttnMaxHeads];    // of keys and values: maximum, then scale
  const moe_attn_config& c = a.c;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int group = lane / kLanes, gl = lane % kLanes, e0 = gl * 8;
  const int pairs = c.rot_dim / 2, nk = c.n_kv_heads;
  const bool held = e0 < c.head_dim, turns_here = e0 < c.rot_dim;

  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) {
    // a token before the first position has no slot
    if (blockIdx.y == 0) check_lists<kThreads>(a, [](const SeqRange& r) { return r.len - r.n; });
    return;
  }
  PageItem it;
  if (!page_item(a, per_seq, (int)blockIdx.x - 1, lane, it)) return;
  const int units = 2 * nk + (a.q ? c.n_heads : 0), u0 = (int)blockIdx.y * kWarps + warp;
  const int u_step = (int)gridDim.y * kWarps;
  const bool whole = it.rows <= kChunk;

  // Row `row` of unit u: keys, values, queries.
  using T = __nv_bfloat16;
  auto source = [&](int u, int row) {
    const int64_t t = it.row0 + row;
    const T* p = u < nk       ? static_cast<const T*>(a.k) + t * c.k_stride + u * c.head_dim
                 : u < 2 * nk ? static_cast<const T*>(a.v) + t * c.v_stride + (u - nk) * c.head_dim
                              : static_cast<const T*>(a.q) + t * c.q_stride + (u - 2 * nk) * c.head_dim;
    return p + e0;
  };
  const bool vec_partner = !c.rot_interleaved && pairs % 8 == 0;
  const int from = lane + (e0 < pairs ? pairs : -pairs) / 8;
  // The chunk's rows of unit u as they are, and turned (0 where there is none).
  auto read = [&](int u, int r0, int rows, float (&o)[kRowsLane][8]) {
    Eight<T> x[kRowsLane];
#pragma unroll
    for (int i = 0; i < kRowsLane; ++i) {
      x[i] = {};
      const int r = i * kGroups + group;
      if (r < rows && held) x[i] = load8(source(u, r0 + r));
    }
    const bool turned = u < nk || u >= 2 * nk;
#pragma unroll
    for (int i = 0; i < kRowsLane; ++i) {
      widen(x[i], o[i]);
      if (!turned || pairs == 0 || i * kGroups >= rows) continue;
      const int r = i * kGroups + group;
      float y[8];
      if (vec_partner) {
        Eight<T> z;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          reinterpret_cast<uint32_t*>(&z)[w] =
              __shfl_sync(0xffffffffu, reinterpret_cast<const uint32_t*>(&x[i])[w], from);
        widen(z, y);
      } else if (c.rot_interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = o[i][e ^ 1];
      } else {
        const T* p = source(u, r0 + min(r, rows - 1));
#pragma unroll
        for (int e = 0; e < 8; ++e)
          y[e] = e0 + e < c.rot_dim ? to_f32(p[e0 + e < pairs ? e + pairs : e - pairs]) : 0.f;
      }
      if (r < rows && turns_here) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = e0 + e;
          if (at >= c.rot_dim) break;
          const bool first = c.rot_interleaved ? e % 2 == 0 : at < pairs;
          const int n = r * pairs + (c.rot_interleaved ? at / 2 : first ? at : at - pairs);
          const float2 cs = turns[n + n / 8];
          const float own = cs.x, other = first ? -cs.y : cs.y;
          o[i][e] = o[i][e] * own + y[e] * other;
        }
      }
    }
  };
  auto largest = [&](const float (&o)[kRowsLane][8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kRowsLane; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, finite(o[i][e]) ? fabsf(o[i][e]) : 0.f);
#pragma unroll
    for (int x = 16; x > 0; x /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    return m;
  };

  for (int pass = whole ? 1 : 0; pass < 2; ++pass) {
    for (int r0 = 0; r0 < it.rows; r0 += kChunk) {
      const int rows = min(kChunk, it.rows - r0);
      __syncthreads();  // the chunk before has been used
      for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
        const int r = i / pairs, n = i - r * pairs;
        const int axis = (n >= c.rot_sections[0]) + (n >= c.rot_sections[0] + c.rot_sections[1]);
        const int64_t pos = a.positions
                                ? a.positions[(int64_t)axis * c.n_tokens + it.row0 + r0 + r]
                                : it.at0 + r0 + r;
        const int64_t angle = (int64_t)((uint64_t)pos * rope.turns[n]);
        float2 cs;
        sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &cs.y, &cs.x);
        turns[i + i / 8] = cs;
      }
      __syncthreads();
      for (int u = u0; u < units; u += u_step) {
        const bool cached = u < 2 * nk;
        if (pass == 0 && !cached) continue;
        float o[kRowsLane][8];
        read(u, r0, rows, o);
        __syncwarp();  // in place: the partners are read before they are overwritten
        if (!cached) {
#pragma unroll
          for (int i = 0; i < kRowsLane; ++i) {
            const int r = i * kGroups + group;
            if (r < rows && held)
              store8(static_cast<T*>(a.out) + ((int64_t)(it.row0 + r0 + r) * c.n_heads + u - 2 * nk) *
                                                  c.head_dim + e0,
                     o[i]);
          }
          continue;
        }
        if (pass == 0) {
          const float m = largest(o);
          if (lane == 0) scales[u] = r0 == 0 ? m : fmaxf(scales[u], m);
          __syncwarp();
          continue;
        }
        if (it.page < 0) continue;
        const int h = u < nk ? u : u - nk;
        uint8_t* cache = static_cast<uint8_t*>(u < nk ? a.k_cache : a.v_cache) +
                         (int64_t)it.page * c.page_stride + (int64_t)h * c.head_stride;
        float scale;
        if (r0 == 0) {
          scale = page_scale(whole ? largest(o) : scales[u]);
          float* stored = (u < nk ? a.k_scale : a.v_scale) + (int64_t)it.page * nk + h;
          if (it.place0 > 0) {
            const float was = *stored;
            if (was >= scale) {
              scale = was;
            } else if (was < scale) {  // neither for a NaN
              const float ratio = __fdiv_rn(was, scale);
              const int vecs = c.head_dim / 16;
              for (int i = lane; i < it.place0 * vecs; i += 32) {
                uint4* p = reinterpret_cast<uint4*>(cache + (int64_t)(i / vecs) * c.token_stride) +
                           i % vecs;
                uint4 w = *p;
                w.x = rescale4(w.x, ratio), w.y = rescale4(w.y, ratio);
                w.z = rescale4(w.z, ratio), w.w = rescale4(w.w, ratio);
                *p = w;
              }
            }
          }
          __syncwarp();
          if (lane == 0) {
            *stored = scale;
            scales[u] = scale;
          }
          __syncwarp();
        } else {
          scale = scales[u];
        }
        const float inv = __fdiv_rn(1.f, scale);
#pragma unroll
        for (int i = 0; i < kRowsLane; ++i) {
          const int r = i * kGroups + group;
          if (r >= rows || !held) continue;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 8; ++e)  // E4M3 has no infinity
            o[i][e] = finite(o[i][e]) ? __fmul_rn(o[i][e], inv) : __uint_as_float(0x7fc00000u);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = e4m3x2(o[i][2 * e], o[i][2 * e + 1]);
          *reinterpret_cast<uint2*>(cache + (int64_t)(it.place0 + r0 + r) * c.token_stride + e0) =
              make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_append_page(const AttnArgs& a, const RopeTable& rope, int lane_bits,
                                    cudaStream_t s) {
  const moe_attn_config& c = a.c;
  const int per_seq = c.max_new == 1 ? 1 : 2;
  const long long items = c.n_tokens / c.page_size + (long long)per_seq * c.n_seqs;
  const int units = 2 * c.n_kv_heads + (a.q ? c.n_heads : 0);
  // A block for every 8 heads where that leaves the GPU's slots unfilled.
  int groups = 1;
  while (groups < ceil_div(units, kWarps) && items * (groups + 1) <= 2LL * num_sms()) ++groups;
  const dim3 grid((unsigned)items + 1, (unsigned)groups), block(kThreads);
  switch (lane_bits) {
    case 0:
    case 1: return launch_pdl(rope_append_page_kernel<1>, grid, block, 0, s, 1, a, rope, per_seq);
    case 2: return launch_pdl(rope_append_page_kernel<2>, grid, block, 0, s, 1, a, rope, per_seq);
    case 3: return launch_pdl(rope_append_page_kernel<3>, grid, block, 0, s, 1, a, rope, per_seq);
    case 4: return launch_pdl(rope_append_page_kernel<4>, grid, block, 0, s, 1, a, rope, per_seq);
    default: return launch_pdl(rope_append_page_kernel<5>, grid, block, 0, s, 1, a, rope, per_seq);
  }
}

}  // namespace moe
