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
// sequence, at b. A block takes an item, or some heads of it: a warp a row (several
// a row where there are few), so that a row's sines are computed once for all its
// heads, a group of lanes a head. It goes over the rows twice, for the maxima (and the
// queries, which are done then) and to write keys and values; a warp with one row
// and few heads keeps them in registers in between. One block more checks the lists
// and writes the status.
//
// Bound by memory for prompts and by the latency of one chain (sequence, page,
// old scale, rows) for a few tokens.
#include <cfloat>

#include <cuda_fp16.h>

#include "rope_append.cuh"

namespace moe {
namespace {

constexpr int kUnits = 4;  // heads a group of lanes has in flight
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

// kWarps warps a block.
template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 24 / kWarps)
    rope_append_page_kernel(const AttnArgs a, const __grid_constant__ RopeTable rope, int lane_bits,
                            int per_seq) {
  using T = __nv_bfloat16;
  constexpr int kThreads = 32 * kWarps;
  __shared__ float2 turns[kWarps][kMaxPairs + kMaxPairs / 8];  // (cos, sin) of a row's pairs, padded
  // Of this block's keys' and values' heads: the maximum, then 1 / scale; old scale / new.
  __shared__ uint32_t largest[2 * kAttnMaxHeads];
  __shared__ float ratios[2 * kAttnMaxHeads];
  const moe_attn_config& c = a.c;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int lanes = 1 << lane_bits, groups = 32 >> lane_bits;
  const int group = lane >> lane_bits, gl = lane & (lanes - 1), e0 = gl * 8;
  const unsigned group_mask = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1) << (group * lanes);
  const int pairs = c.rot_dim / 2, nk = c.n_kv_heads;
  const bool held = e0 < c.head_dim, turns_here = e0 < c.rot_dim;
  float2* turn = turns[warp];

  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) {
    // a token before the first position has no slot
    if (blockIdx.y == 0) check_lists<kThreads>(a, [](const SeqRange& r) { return r.len - r.n; });
    return;
  }
  PageItem it;
  if (!page_item(a, per_seq, (int)blockIdx.x - 1, lane, it)) return;

  // This block's heads j: unit j * G + y of the keys', values' and queries'.
  const int y = blockIdx.y, G = gridDim.y;
  const int heads = (2 * nk + (a.q ? c.n_heads : 0) - y + G - 1) / G, cached = (2 * nk - y + G - 1) / G;
  // Its rows: per_row warps a row.
  int per_row = kWarps;
  while (per_row > 1 && it.rows >= 2 * kWarps / per_row) per_row /= 2;
  const int row_step = kWarps / per_row, first_row = warp / per_row;
  const int j0 = warp % per_row * groups + group, j_step = per_row * groups, batch = kUnits * j_step;
  const bool keep = it.rows <= row_step && cached <= batch;

  for (int j = threadIdx.x; j < cached; j += kThreads) largest[j] = 0;
  // A row's keys, values and queries, at this lane's elements.
  struct Row {
    const T *k, *v, *q;
  };
  auto row_of = [&](int row) {
    const int64_t t = it.row0 + row;
    return Row{static_cast<const T*>(a.k) + t * c.k_stride + e0,
               static_cast<const T*>(a.v) + t * c.v_stride - nk * c.head_dim + e0,
               static_cast<const T*>(a.q) + t * c.q_stride - 2 * nk * c.head_dim + e0};
  };
  auto source = [&](const Row& r, int u) {
    return (u < nk ? r.k : u < 2 * nk ? r.v : r.q) + u * c.head_dim;
  };
  Eight<T> x[kUnits];
  auto load = [&](const Row& r, int j, int n) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      x[k] = {};
      if (j + k * j_step < n && held) x[k] = load8(source(r, (j + k * j_step) * G + y));
    }
  };
  float own[8], other[8];  // factors of this lane's elements and of their partners
  auto turn_of = [&](int row) {
    for (int i = lane; i < pairs; i += 32) {
      const int axis = (i >= c.rot_sections[0]) + (i >= c.rot_sections[0] + c.rot_sections[1]);
      const int64_t pos = a.positions ? a.positions[(int64_t)axis * c.n_tokens + it.row0 + row] : it.at0 + row;
      const int64_t angle = (int64_t)((uint64_t)pos * rope.turns[i]);
      float2 cs;
      sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &cs.y, &cs.x);
      turn[i + i / 8] = cs;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + i;
      own[i] = 1.f, other[i] = -0.f;  // x 1 + 0 (-0) is x for a zero of either sign
      if (e < c.rot_dim) {
        const bool first = c.rot_interleaved ? i % 2 == 0 : e < pairs;
        const int n = c.rot_interleaved ? e / 2 : first ? e : e - pairs;
        const float2 cs = turn[n + n / 8];
        own[i] = cs.x;
        other[i] = first ? -cs.y : cs.y;
      }
    }
    __syncwarp();
  };
  const bool vec_partner = !c.rot_interleaved && pairs % 8 == 0;
  const int from = lane + (e0 < pairs ? pairs : -pairs) / 8;
  // Unit u of a row (x as it was read), turned if it turns; all lanes of a warp alike where
  // `some` is false: nothing does.
  auto turned = [&](const Row& r, int u, bool some, const Eight<T>& x, float (&o)[8]) {
    widen(x, o);
    if (!some) return;
    float z[8];
    if (vec_partner) {
      Eight<T> w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t p = __shfl_sync(0xffffffffu, reinterpret_cast<const uint32_t*>(&x)[i], from);
        reinterpret_cast<uint32_t*>(&w)[i] = turns_here ? p : 0u;
      }
      widen(w, z);
    } else {
      const T* p = source(r, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        z[i] = e >= c.rot_dim      ? 0.f
               : c.rot_interleaved ? to_f32(x.v[i ^ 1])
                                   : to_f32(p[e < pairs ? i + pairs : i - pairs]);
      }
    }
    if (u < nk || u >= 2 * nk) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = o[i] * own[i] + z[i] * other[i];
    }
  };

  __syncthreads();
  for (int row = first_row; row < it.rows; row += row_step) {
    const Row r = row_of(row);
    T* out = static_cast<T*>(a.out) + (int64_t)(it.row0 + row) * c.n_heads * c.head_dim - 2 * nk * c.head_dim + e0;
    // backwards: the keys and values, which may be kept, last
    const int last = j0 + max(heads - 1 - (j0 - group), 0) / batch * batch;
    load(r, last, heads);  // in flight while the row's sines are computed
    turn_of(row);
    for (int jb = last; jb >= j0; jb -= batch) {
      if (jb != last) load(r, jb, heads);
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int j = jb + k * j_step, u = j * G + y;
        if (j - group >= heads) break;  // the same for the whole warp
        float o[8];
        turned(r, min(u, (heads - 1) * G + y), pairs > 0 && __any_sync(0xffffffffu, u < nk || u >= 2 * nk), x[k], o);
        __syncwarp();  // in place: the partners are read before they are overwritten
        if (j < cached) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(o[i]) & 0x7fffffffu);
          if (m >= 0x7f800000u) {  // some are not finite
            m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              m = max(m, finite(o[i]) ? __float_as_uint(o[i]) & 0x7fffffffu : 0u);
          }
          m = __reduce_max_sync(group_mask, m);
          if (gl == 0) atomicMax(largest + j, m);
        } else if (j < heads && held) {
          store8(out + u * c.head_dim, o);
        }
      }
    }
  }
  __syncthreads();
  if (it.page < 0) return;
  for (int j = threadIdx.x; j < cached; j += kThreads) {
    const int u = j * G + y, h = u < nk ? u : u - nk;
    float* stored = (u < nk ? a.k_scale : a.v_scale) + (int64_t)it.page * nk + h;
    float scale = page_scale(__uint_as_float(largest[j])), ratio = 1.f;
    if (it.place0 > 0) {
      const float was = *stored;
      if (was >= scale)
        scale = was;
      else if (was < scale)  // neither for a NaN
        ratio = __fdiv_rn(was, scale);
    }
    *stored = scale;
    largest[j] = __float_as_uint(__fdiv_rn(1.f, scale));
    ratios[j] = ratio;
  }
  __syncthreads();
  for (int j = warp; j < cached; j += kWarps) {
    const float ratio = ratios[j];
    if (ratio == 1.f) continue;
    // the page's older codes under the raised scale
    const int u = j * G + y, vecs = c.head_dim / 16;
    uint8_t* cache = static_cast<uint8_t*>(u < nk ? a.k_cache : a.v_cache) +
                     (int64_t)it.page * c.page_stride + (int64_t)(u < nk ? u : u - nk) * c.head_stride;
    for (int i = lane; i < it.place0 * vecs; i += 32) {
      uint4* p = reinterpret_cast<uint4*>(cache + (int64_t)(i / vecs) * c.token_stride) + i % vecs;
      uint4 w = *p;
      w.x = rescale4(w.x, ratio), w.y = rescale4(w.y, ratio);
      w.z = rescale4(w.z, ratio), w.w = rescale4(w.w, ratio);
      *p = w;
    }
  }
  for (int row = first_row; row < it.rows; row += row_step) {
    const Row r = row_of(row);
    const int64_t at = (int64_t)it.page * c.page_stride + (int64_t)(it.place0 + row) * c.token_stride + e0;
    uint8_t* k_out = static_cast<uint8_t*>(a.k_cache) + at;
    uint8_t* v_out = static_cast<uint8_t*>(a.v_cache) + at - nk * c.head_stride;
    if (!keep) {
      load(r, j0, cached);
      turn_of(row);
    }
    for (int jb = j0; jb - group < cached; jb += batch) {
      if (jb != j0) load(r, jb, cached);
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int j = jb + k * j_step, u = j * G + y;
        if (j - group >= cached) break;
        float o[8];
        turned(r, min(u, (cached - 1) * G + y), pairs > 0 && __any_sync(0xffffffffu, u < nk), x[k], o);
        if (j >= cached || !held) continue;
        const float inv = __uint_as_float(largest[j]);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 8; ++i)  // E4M3 has no infinity: inf 0 makes it a NaN
          o[i] = fmaf(o[i], 0.f, __fmul_rn(o[i], inv));
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = e4m3x2(o[2 * i], o[2 * i + 1]);
        *reinterpret_cast<uint2*>((u < nk ? k_out : v_out) + u * c.head_stride) =
            make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
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
  // A block takes all heads of an item where a warp has a row, or where the GPU's
  // slots (24 warps an SM) are filled; else some of them. 16 warps a block where items
  // are few and have the rows.
  const int heads = 2 * c.n_kv_heads + (a.q ? c.n_heads : 0);
  const int rows = c.max_new < c.page_size ? c.max_new : c.page_size;
  const bool wide = rows >= 16 && items < 3LL * num_sms();
  const int warps = wide ? 16 : 8;
  int split = 1;
  while (split < c.n_kv_heads && rows < warps && 2 * split * warps <= heads * rows &&
         items * split * warps < 24LL * num_sms())
    split *= 2;
  const dim3 grid((unsigned)items + 1, (unsigned)split), block((unsigned)(32 * warps));
  return wide ? launch_pdl(rope_append_page_kernel<16>, grid, block, 0, s, 1, a, rope, lane_bits, per_seq)
              : launch_pdl(rope_append_page_kernel<8>, grid, block, 0, s, 1, a, rope, lane_bits, per_seq);
}

}  // namespace moe
