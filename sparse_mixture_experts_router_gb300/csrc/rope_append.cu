// Rotary positions of the new tokens' queries and keys, and their keys and
// values written into the paged cache: one launch, every input read once and
// every output written once.
//
// Pair i of a head turns by theta = p * base^(-2i/rot_dim), p the token's
// position on the pair's axis (time, height, width). fp32 angles of far
// positions are useless (at p = 2^20 one ulp is 1/16 rad), so the angle is a
// 64-bit fraction of a turn: the host gives each pair's turns per position
// as f_i = 2^64 base^(-2i/rot_dim) / 2 pi, and p * f_i in wrapping integer
// arithmetic is the angle modulo one turn, off by at most p * 2^-53 of f_i's
// rounding. sincospi of that fraction is then fp32-exact to its own bounds.
//
// One block per token. A head is held by a group of lanes (a power of two,
// 8 elements a lane), so the E4M3 scale of a key or value is a shuffle
// reduction inside the group, and both halves of every pair are read by the
// lanes that need them (the second read hits L1) with no staging. The
// token's sines and cosines are computed once, by the block, for all heads.
// One block more checks the lists and writes the status.
// Bound by memory; what it costs beyond that is the latency of one block's
// chain (sequence of the token, its page, the sines, the stores).
#include <cfloat>
#include <cmath>

#include "serve_util.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;  // heads a group holds in registers at a time
constexpr int kMaxPairs = kAttnMaxDim / 2;

struct RopeTable {
  uint64_t turns[kMaxPairs];  // f_i
};

// Eight elements of a row as fp32.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  bf16x2_to_f32(q.x, x[0], x[1]);
  bf16x2_to_f32(q.y, x[2], x[3]);
  bf16x2_to_f32(q.z, x[4], x[5]);
  bf16x2_to_f32(q.w, x[6], x[7]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]),
                 f32x2_to_bf16x2(x[4], x[5]), f32x2_to_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T, bool kE4M3>
__global__ void __launch_bounds__(kThreads)
    rope_append_kernel(const AttnArgs a, const __grid_constant__ RopeTable rope, int lane_bits) {
  __shared__ float2 turn[kMaxPairs];  // (cos, sin) of this token's pairs
  __shared__ int s_at, s_page;
  const moe_attn_config& c = a.c;
  const int t = blockIdx.x, lanes = 1 << lane_bits, groups = kThreads >> lane_bits;
  const int group = threadIdx.x >> lane_bits, gl = threadIdx.x & (lanes - 1);
  const int pairs = c.rot_dim / 2, e0 = gl * 8;
  const bool held = e0 < c.head_dim;
  const int nq = a.q ? c.n_heads : 0, units = nq + 2 * c.n_kv_heads;

  // Element e0 + i turns with its partner: the same vector's neighbour
  // (interleaved), or the element rot_dim/2 away.
  const bool low = e0 < pairs;
  const bool vec_partner = !c.rot_interleaved && pairs % 8 == 0;
  auto source = [&](int u) -> const T* {
    if (u < nq) return static_cast<const T*>(a.q) + (int64_t)t * c.q_stride + u * c.head_dim;
    if (u < nq + c.n_kv_heads)
      return static_cast<const T*>(a.k) + (int64_t)t * c.k_stride + (u - nq) * c.head_dim;
    return static_cast<const T*>(a.v) + (int64_t)t * c.v_stride +
           (u - nq - c.n_kv_heads) * c.head_dim;
  };
  float x[kUnits][8], y[kUnits][8];  // own elements and partners
  auto load = [&](int u0) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int u = u0 + k * groups;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = y[k][i] = 0.f;
      if (u >= units || !held) continue;
      const T* p = source(u);
      load8(p + e0, x[k]);
      if (u >= nq + c.n_kv_heads || e0 >= c.rot_dim) continue;
      if (c.rot_interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[k][i] = x[k][i ^ 1];
      } else if (vec_partner) {
        load8(p + (low ? e0 + pairs : e0 - pairs), y[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i;
          if (e < c.rot_dim) y[k][i] = to_f32(p[e < pairs ? e + pairs : e - pairs]);
        }
      }
    }
  };

  pdl_wait();
  pdl_trigger();
  if (t == c.n_tokens) {
    // a token before the first position has no slot
    check_lists<kThreads>(a, [](const SeqRange& r) { return r.len - r.n; });
    return;
  }
  load(group);  // in flight while the token's place is looked up

  // The token's sequence is found by one comparison a thread (a search would
  // be a chain of reads), and its thread goes on to the page.
  if (threadIdx.x == 0) s_page = -1, s_at = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < c.n_seqs; b += kThreads) {
    const SeqRange r = seq_range(a, b);
    const int j = t - r.row0, p = r.len - r.n + j;
    if (!r.ok || j < 0 || j >= r.n) continue;
    s_at = p;
    if (p >= 0) s_page = page_of(a, b, p);
  }
  __syncthreads();
  const int at = s_at, page = s_page;
  const bool ok = page >= 0 && at >= 0;
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    const int axis = (i >= c.rot_sections[0]) + (i >= c.rot_sections[0] + c.rot_sections[1]);
    const int64_t pos = a.positions ? a.positions[(int64_t)axis * c.n_tokens + t] : at;
    const int64_t angle = (int64_t)((uint64_t)pos * rope.turns[i]);
    float2 cs;
    sincospif((float)angle * 0x1p-63f, &cs.y, &cs.x);
    turn[i] = cs;
  }
  __syncthreads();
  // This lane's elements are the same of every head: factors of the element
  // and of its partner, kept in registers.
  float own[8], other[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = e0 + i;
    own[i] = 1.f, other[i] = 0.f;
    if (e < c.rot_dim) {
      const bool first = c.rot_interleaved ? i % 2 == 0 : e < pairs;
      const float2 cs = turn[c.rot_interleaved ? e / 2 : first ? e : e - pairs];
      own[i] = cs.x;
      other[i] = first ? -cs.y : cs.y;
    }
  }

  const int place = at % c.page_size;
  const int64_t row = (int64_t)page * c.page_stride + (int64_t)place * c.token_stride;
  for (int u0 = group; u0 - group < units; u0 += kUnits * groups) {
    if (u0 != group) load(u0);
    __syncwarp();  // in place: the partners are read before they are overwritten
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int u = u0 + k * groups;
      float o[8];
      const bool turned = u < nq + c.n_kv_heads;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = turned ? x[k][i] * own[i] + y[k][i] * other[i] : x[k][i];
      float amax = 0.f;
      if (kE4M3) {
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(o[i]));
        for (int m = lanes / 2; m > 0; m >>= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
      }
      if (u >= units || !held) continue;
      if (u < nq) {
        store8(static_cast<T*>(a.out) + ((int64_t)t * c.n_heads + u) * c.head_dim + e0, o);
        continue;
      }
      if (!ok) continue;
      const bool key = u < nq + c.n_kv_heads;
      const int h = key ? u - nq : u - nq - c.n_kv_heads;
      const int64_t off = row + h * c.head_stride + e0;
      if (kE4M3) {
        const float inv = amax > 0.f ? fminf(__fdiv_rn(448.f, amax), FLT_MAX) : 0.f;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = e4m3x2(__fmul_rn(o[2 * i], inv), __fmul_rn(o[2 * i + 1], inv));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(key ? a.k_cache : a.v_cache) + off) =
            make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        if (gl == 0)
          (key ? a.k_scale : a.v_scale)[((int64_t)page * c.n_kv_heads + h) * c.page_size + place] =
              __fdiv_rn(amax, 448.f);
      } else {
        store8(static_cast<T*>(key ? a.k_cache : a.v_cache) + off, o);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const AttnArgs& a, cudaStream_t s) {
  if (a.c.n_tokens == 0) return launch_reset_status(a.status, s);
  RopeTable rope = {};
  const double ratio = a.c.rot_dim ? std::pow((double)a.c.rope_base, -2.0 / a.c.rot_dim) : 0.0;
  double f = 18446744073709551616.0 / 6.283185307179586476925;  // one radian, 2^64 a turn
  for (int i = 0; i < a.c.rot_dim / 2; ++i, f *= ratio) rope.turns[i] = (uint64_t)(f + 0.5);
  int lane_bits = 0;
  while ((8 << lane_bits) < a.c.head_dim) ++lane_bits;
  ProfScope p(K_ROPE_APPEND, s);
  const dim3 grid((unsigned)a.c.n_tokens + 1), block(kThreads);
  if (a.c.dtype == MOE_F32)
    return launch_pdl(rope_append_kernel<float, false>, grid, block, 0, s, 1, a, rope, lane_bits);
  if (a.c.cache_dtype == MOE_E4M3)
    return launch_pdl(rope_append_kernel<__nv_bfloat16, true>, grid, block, 0, s, 1, a, rope,
                      lane_bits);
  return launch_pdl(rope_append_kernel<__nv_bfloat16, false>, grid, block, 0, s, 1, a, rope,
                    lane_bits);
}

}  // namespace moe
