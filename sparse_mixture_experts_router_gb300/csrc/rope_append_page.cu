// Rotary append into an E4M3 cache with one scale per page and head.
//
// The scale of a page's head is 2^e, the least power of two with |x| <= 448 2^e
// for the elements the page holds. A power of two costs E4M3 no precision (it
// moves the exponent) and makes raising the scale for a later, larger token exact:
// older codes are multiplied by 2^(old - new), a change of exponent that rounds
// only codes that become subnormal. Attention widens the codes alone, and takes
// a page's scale into its softmax.
//
// So the new tokens of one page have to meet before any of them is written: an
// item is a (sequence, page) that the call touches. Sequence b's items start at
// floor(cu_new[b] / page_size) + 2 b, which leaves each sequence at least as many
// as n tokens can touch (1 + ceil((n - 1) / page_size)); where no sequence has more
// than one new token, item b is sequence b's. A block takes an item, or some heads of it: a warp a row (several
// a row where there are few), so that a row's sines are computed once for all its
// heads, a group of lanes a head. It goes over the rows twice, for the maxima (and the
// queries, which are done then) and to write keys and values; a warp with one row
// and few heads keeps them in registers in between. One block more checks the lists
// and writes the status.
//
// Prompts (8197 tokens, 32/8 heads of 128): 59 us, 3.15 TB/s, 0.46 of a copy's rate: bound
// by issue, 1.8 instructions a cycle from 16 warps an SM (128 registers a thread: four heads
// in flight), 2.5 million a thousand tokens for the angles, the turn, the maxima and
// the conversions. A few tokens: by the latency of one chain (sequence, page, old scale,
// rows, maxima, codes), 11.1 us for 225 tokens of 64 sequences, 7.1 for one of each of 256
// and 6.1 to 6.9 for one.
#include <cfloat>

#include <cuda_fp16.h>

#include "rope_append.cuh"
#include "serve_ptx.cuh"

namespace moe {
namespace {

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
// The item of index i (false: none), found by a whole block.
template <int kThreads>
__device__ __forceinline__ bool page_item(const AttnArgs& a, const FastDiv& by_page, int index, int lane,
                                          PageItem& it) {
  const moe_attn_config& c = a.c;
  auto start_of = [&](int cu, int b) {
    return c.max_new == 1 ? b : div(by_page, clamp_int(cu, 0, c.n_tokens)) + 2 * b;
  };
  auto start = [&](int b) { return start_of(__ldg(a.cu_new + b), b); };
  // the first sequence whose items end after index: counted in one round trip where the
  // threads hold the list, else found in steps of 32 comparisons
  int lo = 0;
  if (c.max_new == 1) {
    lo = index;
  } else if (c.n_seqs <= kThreads) {
    const int t = threadIdx.x;
    lo = __syncthreads_count(t < c.n_seqs && start(t + 1) <= index);
  } else {
    int hi = c.n_seqs;
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step - 1;
      const unsigned after = __ballot_sync(0xffffffffu, i >= hi || start(i + 1) > index);
      if (!after) return false;  // only where the list does not ascend
      const int f = __ffs(after) - 1;
      hi = min(hi, lo + (f + 1) * step - 1);
      lo += f * step;
    }
  }
  if (lo >= c.n_seqs) return false;
  const SeqRange r = seq_range(a, lo);
  const int first = r.len - r.n;  // below 0: no slot, recorded by the check
  if (!r.ok || first < 0 || r.n == 0) return false;
  const int nth = index - start_of(r.row0, lo), page = div(by_page, first) + nth;
  if (nth < 0 || page > div(by_page, r.len - 1)) return false;
  it.at0 = max(first, page * c.page_size);
  it.rows = min(r.len, (page + 1) * c.page_size) - it.at0;
  it.row0 = r.row0 + it.at0 - first;
  it.place0 = it.at0 - page * c.page_size;
  const int id = __ldg(a.table + (int64_t)lo * c.max_pages + page);
  it.page = id >= 0 && id < c.n_pages ? id : -1;
  return true;
}

// kWarps warps a block; kUnits heads of a kind that a group of lanes has in flight.
template <int kWarps, int kUnits>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps)
    rope_append_page_kernel(const AttnArgs a, const __grid_constant__ RopeTable rope,
                            const FastDiv by_page, int lane_bits) {
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
  if (!page_item<kThreads>(a, by_page, (int)blockIdx.x - 1, lane, it)) return;

  // This block's heads: j * G + y of the keys, of the values and of the queries.
  const int y = blockIdx.y, G = gridDim.y;
  const int n_kv = (nk - y + G - 1) / G, n_q = a.q ? (c.n_heads - y + G - 1) / G : 0;
  // Its rows: per_row warps a row.
  int per_row = kWarps;
  while (per_row > 1 && it.rows >= 2 * kWarps / per_row) per_row /= 2;
  const int row_step = kWarps / per_row, first_row = warp / per_row;
  // A group's heads: every j_step-th, kUnits at a time.
  const int j_first = warp % per_row * groups, j0 = j_first + group, j_step = per_row * groups;
  const int batch = kUnits * j_step, head0 = (j0 * G + y) * c.head_dim, head_step = j_step * G * c.head_dim;
  const bool keep = it.rows <= row_step && n_kv <= batch;

  auto stored_scale = [&](int j) {  // keys', then values'
    return (j < n_kv ? a.k_scale + j * G : a.v_scale + (j - n_kv) * G) + (int64_t)it.page * nk + y;
  };
  for (int j = threadIdx.x; j < 2 * n_kv; j += kThreads) largest[j] = 0;
  float was0 = 0.f;  // of scale threadIdx.x, in flight with the rows
  if (it.page >= 0 && it.place0 > 0 && (int)threadIdx.x < 2 * n_kv) was0 = *stored_scale(threadIdx.x);
  // Heads jb .. of a row (`row`: its first head at this lane's elements), of n in all.
  auto load = [&](const T* row, int jb, int n, Eight<T> (&x)[kUnits]) {
    const T* p = row + (int64_t)(jb - j_first) * G * c.head_dim + head0;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      x[k] = {};
      if (jb + group + k * j_step < n && held) x[k] = load8(p + k * head_step);
    }
  };
  auto row_at = [&](const void* base, int64_t stride, int row) {
    return static_cast<const T*>(base) + (it.row0 + row) * stride + e0;
  };
  Eight<T> xk[kUnits], xv[kUnits], xq[kUnits];
  uint64_t own[4], other[4];  // factors of this lane's elements, in pairs, and of their partners
  auto turn_of = [&](int row) {
    for (int i = lane; i < pairs; i += 32) {
      const int axis = (i >= c.rot_sections[0]) + (i >= c.rot_sections[0] + c.rot_sections[1]);
      const int64_t pos = a.positions ? __ldg(a.positions + (int64_t)axis * c.n_tokens + it.row0 + row) : it.at0 + row;
      const int64_t angle = (int64_t)((uint64_t)pos * rope.turns[i]);
      float2 cs;
      sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &cs.y, &cs.x);
      turn[i + i / 8] = cs;
    }
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float f[2] = {1.f, 1.f}, g[2] = {-0.f, -0.f};  // x 1 + 0 (-0) is x for a zero of either sign
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = e0 + 2 * p + h;
        if (e >= c.rot_dim) continue;
        const bool first = c.rot_interleaved ? h == 0 : e < pairs;
        const int n = c.rot_interleaved ? e / 2 : first ? e : e - pairs;
        const float2 cs = turn[n + n / 8];
        f[h] = cs.x;
        g[h] = first ? -cs.y : cs.y;
      }
      own[p] = ptx::f32x2(f[0], f[1]);
      other[p] = ptx::f32x2(g[0], g[1]);
    }
    __syncwarp();
  };
  const bool vec_partner = !c.rot_interleaved && pairs % 8 == 0;
  const int from = lane + (e0 < pairs ? pairs : -pairs) / 8;
  auto pair = [](uint32_t w) { return ptx::f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); };
  const uint64_t zero = ptx::f32x2(0.f, 0.f), minus_zero = ptx::f32x2(-0.f, -0.f);
  auto widen2 = [&](const Eight<T>& x, uint64_t (&o)[4]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = pair(reinterpret_cast<const uint32_t*>(&x)[p]);
  };
  // Head j of a row, x as it was read, turned. All lanes of the warp.
  auto turned = [&](const T* row, int j, int n, const Eight<T>& x, uint64_t (&o)[4]) {
    widen2(x, o);
    if (pairs == 0) return;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
    uint64_t z[4];
    if (vec_partner) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t q = __shfl_sync(0xffffffffu, w[p], from);
        z[p] = pair(turns_here ? q : 0u);
      }
    } else if (c.rot_interleaved) {
#pragma unroll
      for (int p = 0; p < 4; ++p) z[p] = pair(e0 + 2 * p < c.rot_dim ? w[p] << 16 | w[p] >> 16 : 0u);
    } else {
      const T* at = row + (min(j, n - 1) * G + y) * c.head_dim;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        v[i] = e >= c.rot_dim ? 0.f : to_f32(at[e < pairs ? i + pairs : i - pairs]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = ptx::f32x2(v[2 * i], v[2 * i + 1]);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = ptx::fma_f32x2(z[p], other[p], ptx::fma_f32x2(o[p], own[p], minus_zero));
  };
  // The largest finite element of a head into its place.
  auto raise = [&](int j, int n, uint32_t* place, const uint64_t (&o)[4]) {
    if (j >= n) return;
    float m = 0.f;  // a NaN is passed over
#pragma unroll
    for (int p = 0; p < 4; ++p) m = fmaxf(m, fmaxf(fabsf(ptx::f32x2_lo(o[p])), fabsf(ptx::f32x2_hi(o[p]))));
    if (m == INFINITY) {
      m = 0.f;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float lo = fabsf(ptx::f32x2_lo(o[p])), hi = fabsf(ptx::f32x2_hi(o[p]));
        m = fmaxf(m, fmaxf(finite(lo) ? lo : 0.f, finite(hi) ? hi : 0.f));
      }
    }
    const uint32_t bits = __reduce_max_sync(group_mask, __float_as_uint(m));
    if (gl == 0) atomicMax(place + j, bits);
  };

  __syncthreads();
  for (int row = first_row; row < it.rows; row += row_step) {
    const T *k_row = row_at(a.k, c.k_stride, row), *v_row = row_at(a.v, c.v_stride, row);
    const T* q_row = row_at(a.q, c.q_stride, row);
    // backwards, for the first heads to be kept; in flight while the sines are computed
    const int last = j_first + max(n_kv - 1 - j_first, 0) / batch * batch;
    load(k_row, last, n_kv, xk);
    load(v_row, last, n_kv, xv);
    load(q_row, j_first, n_q, xq);
    turn_of(row);
    for (int jb = last; jb >= j_first; jb -= batch) {
      if (jb != last) {
        load(k_row, jb, n_kv, xk);
        load(v_row, jb, n_kv, xv);
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        if (jb + k * j_step >= n_kv) break;  // the same for the whole warp
        const int j = jb + k * j_step + group;
        uint64_t o[4];
        turned(k_row, j, n_kv, xk[k], o);
        raise(j, n_kv, largest, o);
        widen2(xv[k], o);
        raise(j, n_kv, largest + n_kv, o);
      }
    }
    T* out = static_cast<T*>(a.out) + (int64_t)(it.row0 + row) * c.n_heads * c.head_dim + e0 + head0;
    for (int jb = j_first; jb < n_q; jb += batch, out += kUnits * head_step) {
      if (jb != j_first) load(q_row, jb, n_q, xq);
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        if (jb + k * j_step >= n_q) break;
        const int j = jb + k * j_step + group;
        uint64_t o[4];
        turned(q_row, j, n_q, xq[k], o);
        __syncwarp();  // in place: the partners are read before they are overwritten
        if (j >= n_q || !held) continue;
        uint32_t w[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) w[p] = f32x2_to_bf16x2(ptx::f32x2_lo(o[p]), ptx::f32x2_hi(o[p]));
        *reinterpret_cast<uint4*>(out + k * head_step) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  __syncthreads();
  if (it.page < 0) return;
  for (int j = threadIdx.x; j < 2 * n_kv; j += kThreads) {
    float scale = page_scale(__uint_as_float(largest[j])), ratio = 1.f;
    if (it.place0 > 0) {
      const float was = j < kThreads ? was0 : *stored_scale(j);
      if (was >= scale)
        scale = was;
      else if (was < scale)  // neither for a NaN
        ratio = __fdiv_rn(was, scale);
    }
    *stored_scale(j) = scale;
    largest[j] = __float_as_uint(__fdiv_rn(1.f, scale));
    ratios[j] = ratio;
  }
  __syncthreads();
  uint8_t* k_page = static_cast<uint8_t*>(a.k_cache) + (int64_t)it.page * c.page_stride + y * c.head_stride;
  uint8_t* v_page = static_cast<uint8_t*>(a.v_cache) + (int64_t)it.page * c.page_stride + y * c.head_stride;
  for (int j = warp; j < 2 * n_kv; j += kWarps) {
    const float ratio = ratios[j];
    if (ratio == 1.f) continue;
    // the page's older codes under the raised scale
    const int vecs = c.head_dim / 16;
    uint8_t* cache = j < n_kv ? k_page + j * G * c.head_stride : v_page + (j - n_kv) * G * c.head_stride;
    for (int i = lane; i < it.place0 * vecs; i += 32) {
      uint4* p = reinterpret_cast<uint4*>(cache + (int64_t)(i / vecs) * c.token_stride) + i % vecs;
      uint4 w = *p;
      w.x = rescale4(w.x, ratio), w.y = rescale4(w.y, ratio);
      w.z = rescale4(w.z, ratio), w.w = rescale4(w.w, ratio);
      *p = w;
    }
  }
  // Elements o of a head over its scale, as codes.
  auto put = [&](uint8_t* to, uint32_t inv, const uint64_t (&o)[4]) {
    const uint64_t by = (uint64_t)inv << 32 | inv;
    uint32_t w[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {  // E4M3 has no infinity: inf 0 makes it a NaN
      const uint64_t q = ptx::fma_f32x2(o[p], zero, ptx::fma_f32x2(o[p], by, minus_zero));
      w[p] = e4m3x2(ptx::f32x2_lo(q), ptx::f32x2_hi(q));
    }
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  };
  for (int row = first_row; row < it.rows; row += row_step) {
    const T *k_row = row_at(a.k, c.k_stride, row), *v_row = row_at(a.v, c.v_stride, row);
    if (!keep) {
      load(k_row, j_first, n_kv, xk);
      load(v_row, j_first, n_kv, xv);
      turn_of(row);
    }
    const int64_t at = (int64_t)(it.place0 + row) * c.token_stride + e0;
    for (int jb = j_first; jb < n_kv; jb += batch) {
      if (jb != j_first) {
        load(k_row, jb, n_kv, xk);
        load(v_row, jb, n_kv, xv);
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        if (jb + k * j_step >= n_kv) break;
        const int j = jb + k * j_step + group;
        uint64_t o[4], v[4];
        turned(k_row, j, n_kv, xk[k], o);
        if (j >= n_kv || !held) continue;
        widen2(xv[k], v);
        const int64_t head = at + (int64_t)j * G * c.head_stride;
        put(k_page + head, largest[j], o);
        put(v_page + head, largest[n_kv + j], v);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_append_page(const AttnArgs& a, const RopeTable& rope, int lane_bits,
                                    cudaStream_t s) {
  const moe_attn_config& c = a.c;
  const long long items = c.max_new == 1 ? c.n_seqs : c.n_tokens / c.page_size + 2LL * c.n_seqs;
  // Prompts, whose items have a row for each of 16 warps: a block an item, with four heads
  // in flight (two: 67 us for 59, 8197 tokens). Else blocks of 8 warps with two (four: 12.6
  // us for 11.2, 225 tokens of 64 sequences), and an item's heads over several
  // blocks while there are less than 12 warps an SM.
  const int heads = 2 * c.n_kv_heads + (a.q ? c.n_heads : 0);
  const int rows = c.max_new < c.page_size ? c.max_new : c.page_size;
  const bool wide = rows >= 16;
  const int warps = wide ? 16 : 8;
  int split = 1;
  while (split < c.n_kv_heads && rows < warps && 2 * split * warps <= heads * rows &&
         items * split * warps < 12LL * num_sms())
    split *= 2;
  const FastDiv by_page = fast_div((uint32_t)c.page_size);
  const dim3 grid((unsigned)items + 1, (unsigned)split), block((unsigned)(32 * warps));
  return wide ? launch_pdl(rope_append_page_kernel<16, 4>, grid, block, 0, s, 1, a, rope, by_page, lane_bits)
              : launch_pdl(rope_append_page_kernel<8, 2>, grid, block, 0, s, 1, a, rope, by_page, lane_bits);
}

}  // namespace moe
