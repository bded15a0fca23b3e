// Rotary positions of the new tokens' queries and keys, and their keys and
// values written into the paged cache: one launch, every input read once and
// every output written once.
//
// Pair i of a head turns by theta = p * base^(-2i/rot_dim), p the token's
// position on the pair's axis (time, height, width). fp32 angles of far
// positions are useless (at p = 2^20 one ulp is 1/16 rad), so the angle is a
// 64-bit fraction of a turn: the host gives each pair's turns per position
// as f_i = 2^64 base^(-2i/rot_dim) / 2 pi, rounded (rope_turns.h), and p * f_i in
// wrapping integer arithmetic is the angle modulo one turn, off by p / 2 units:
// 2^-34 of a turn at most. As fp32 half turns for sincospi it is off by up to
// 2^-25 of one, 1.6 x 2^-24 rad, at any position.
//
// One block or one warp per token. A head is held by a group of lanes (a power of two,
// 8 elements a lane), so the E4M3 scale of a key or value is a shuffle
// reduction inside the group, and so is the exchange of the pairs' halves. The
// token's sines and cosines are computed once for all heads.
// One block more checks the lists and writes the status.
// Bound by memory; what it costs beyond that is the latency of one block's
// chain (sequence of the token, its page, the sines, the stores).
#include <cfloat>

#include "rope_turns.h"
#include "serve_util.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = kAttnMaxDim / 2;

struct RopeTable {
  uint64_t turns[kMaxPairs];  // f_i
};

// Eight elements of a row, as stored and as fp32.
template <typename T>
struct alignas(16) Eight {
  T v[8];
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
  Eight<T> r;
  constexpr int n = (int)sizeof(r) / 16;
#pragma unroll
  for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Eight<T>& r) {
  constexpr int n = (int)sizeof(r) / 16;
#pragma unroll
  for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(&r)[i];
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
__device__ __forceinline__ void widen(const Eight<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = r.v[i];
}
__device__ __forceinline__ void widen(const Eight<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) bf16x2_to_f32(w[i], x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The first sequence whose rows end after row t, found by a whole warp in
// steps of 32 comparisons (n_seqs if none).
__device__ __forceinline__ int seq_of_row(const int32_t* cu_new, int n_seqs, int t, int lane) {
  int lo = 0, hi = n_seqs;  // the answer is in lo .. hi
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step - 1;
    const unsigned after = __ballot_sync(0xffffffffu, i >= hi || __ldg(cu_new + i + 1) > t);
    if (!after) return hi;  // only where the list does not ascend
    const int f = __ffs(after) - 1;
    hi = min(hi, lo + (f + 1) * step - 1);
    lo += f * step;
  }
  return lo;
}

// kWarps warps a token (1 or all of the block's).
template <typename T, bool kE4M3, int kWarps>
__global__ void __launch_bounds__(kThreads)
    rope_append_kernel(const AttnArgs a, const __grid_constant__ RopeTable rope, int lane_bits) {
  constexpr int kTokens = kThreads / 32 / kWarps;
  constexpr int kUnits = kWarps == 1 ? 8 : 3;  // heads a group of lanes has in flight
  // (cos, sin) of each token's pairs, padded against bank conflicts
  __shared__ float2 turns[kTokens][kMaxPairs + kMaxPairs / 8];
  const moe_attn_config& c = a.c;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 % kWarps;
  const int slot = threadIdx.x / 32 / kWarps, t = (int)blockIdx.x * kTokens + slot - kTokens;
  const int lanes = 1 << lane_bits, groups = (32 * kWarps) >> lane_bits;
  const int group = (warp * 32 + lane) >> lane_bits, gl = lane & (lanes - 1);
  const int pairs = c.rot_dim / 2, e0 = gl * 8;
  const bool held = e0 < c.head_dim;
  const int nq = a.q ? c.n_heads : 0, nk = c.n_kv_heads, units = nq + 2 * nk;
  float2* turn = turns[slot];

  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) {
    // a token before the first position has no slot
    check_lists<kThreads>(a, [](const SeqRange& r) { return r.len - r.n; });
    return;
  }
  if (kWarps == 1 && t >= c.n_tokens) return;

  const T* qr = static_cast<const T*>(a.q) + (int64_t)t * c.q_stride + e0;
  const T* kr = static_cast<const T*>(a.k) + (int64_t)t * c.k_stride + e0;
  const T* vr = static_cast<const T*>(a.v) + (int64_t)t * c.v_stride + e0;
  auto source = [&](int u) {
    return u < nq        ? qr + u * c.head_dim
           : u < nq + nk ? kr + (u - nq) * c.head_dim
                         : vr + (u - nq - nk) * c.head_dim;
  };
  Eight<T> x[kUnits];
  auto load = [&](int u0) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int u = u0 + k * groups;
      x[k] = {};
      if (u < units && held) x[k] = load8(source(u));
    }
  };
  // Element e0 + i turns with its partner: the same vector's neighbour
  // (interleaved), or the element rot_dim/2 away, which another lane of the
  // group holds (whole vectors away) or which is read again. Zero where an
  // element does not turn, so that whatever it is passes.
  const bool vec_partner = pairs % 8 == 0;
  const int from = lane + (e0 < pairs ? pairs : -pairs) / 8;
  const bool turns_here = e0 < c.rot_dim;
  auto partners = [&](int u, const Eight<T>& x, float (&y)[8]) {
    if (!c.rot_interleaved && vec_partner) {
      Eight<T> z;
      constexpr int n = (int)sizeof(z) / 4;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const uint32_t w =
            __shfl_sync(0xffffffffu, reinterpret_cast<const uint32_t*>(&x)[i], from);
        reinterpret_cast<uint32_t*>(&z)[i] = turns_here ? w : 0u;
      }
      widen(z, y);
    } else {
      const T* p = source(u < units ? u : 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        if (e >= c.rot_dim)
          y[i] = 0.f;
        else if (c.rot_interleaved)
          y[i] = to_f32(x.v[i ^ 1]);
        else
          y[i] = to_f32(p[e < pairs ? i + pairs : i - pairs]);
      }
    }
  };
  load(group);  // in flight while the token's place is looked up

  // The token's sequence, position and page.
  const int b = seq_of_row(a.cu_new, c.n_seqs, t, lane);
  int at = -1, page = -1;
  if (b < c.n_seqs) {
    const SeqRange r = seq_range(a, b);
    const int j = t - r.row0;
    if (r.ok && j >= 0 && j < r.n) at = r.len - r.n + j;
    if (at >= 0) page = page_of(a, b, at);
  }
  for (int i = warp * 32 + lane; i < pairs; i += 32 * kWarps) {
    const int axis = (i >= c.rot_sections[0]) + (i >= c.rot_sections[0] + c.rot_sections[1]);
    const int64_t pos = a.positions ? a.positions[(int64_t)axis * c.n_tokens + t] : at;
    const int64_t angle = (int64_t)((uint64_t)pos * rope.turns[i]);
    float2 cs;
    // the high word is enough: 2^-32 of half a turn
    sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &cs.y, &cs.x);
    turn[i + i / 8] = cs;
  }
  if (kWarps == 1)
    __syncwarp();
  else
    __syncthreads();
  // This lane's elements are the same of every head: factors of the element
  // and of its partner, kept in registers. An element that does not turn is x 1
  // + 0 (-0), which is x for a zero of either sign.
  float own[8], other[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = e0 + i;
    own[i] = 1.f, other[i] = -0.f;
    if (e < c.rot_dim) {
      const bool first = c.rot_interleaved ? i % 2 == 0 : e < pairs;
      const int n = c.rot_interleaved ? e / 2 : first ? e : e - pairs;
      const float2 cs = turn[n + n / 8];
      own[i] = cs.x;
      other[i] = first ? -cs.y : cs.y;
    }
  }

  const int place = page >= 0 ? at % c.page_size : 0;
  const int64_t row = (int64_t)page * c.page_stride + (int64_t)place * c.token_stride + e0;
  T* out = static_cast<T*>(a.out) + (int64_t)t * c.n_heads * c.head_dim + e0;
  for (int u0 = group; u0 - group < units; u0 += kUnits * groups) {
    if (u0 != group) load(u0);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int u = u0 + k * groups;
      if (u - group >= units) break;  // the same for the whole warp
      const bool in = u < units && held;
      const bool turned = u < nq + nk;
      if (!kE4M3 && u - group + ((warp * 32) >> lane_bits) >= nq + nk) {
        // the whole warp has values, and the cache is of their type: as they are
        const int64_t off = row + (u - nq - nk) * c.head_stride;
        if (in && page >= 0) store8(static_cast<T*>(a.v_cache) + off, x[k]);
        continue;
      }
      float o[8], y[8];
      widen(x[k], o);
      partners(u, x[k], y);
      if (turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = o[i] * own[i] + y[i] * other[i];
      }
      __syncwarp();  // in place: the partners are read before they are overwritten
      float amax = 0.f;
      if (kE4M3) {
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(o[i]));
        for (int m = lanes / 2; m > 0; m >>= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
      }
      if (!in) continue;
      if (u < nq) {
        store8(out + u * c.head_dim, o);
        continue;
      }
      if (page < 0) continue;
      const bool key = u < nq + nk;
      const int h = u - nq - (key ? 0 : nk);
      const int64_t off = row + h * c.head_stride;
      if (kE4M3) {
        const float inv = amax > 0.f ? fminf(__fdiv_rn(448.f, amax), FLT_MAX) : 0.f;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = e4m3x2(__fmul_rn(o[2 * i], inv), __fmul_rn(o[2 * i + 1], inv));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(key ? a.k_cache : a.v_cache) + off) =
            make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        if (gl == 0)
          (key ? a.k_scale : a.v_scale)[((int64_t)page * nk + h) * c.page_size + place] =
              __fdiv_rn(amax, 448.f);
      } else {
        store8(static_cast<T*>(key ? a.k_cache : a.v_cache) + off, o);
      }
    }
  }
}

template <typename T, bool kE4M3>
cudaError_t launch(const AttnArgs& a, const RopeTable& rope, int lane_bits, cudaStream_t s) {
  // Few tokens: a block each, for the latency of one; many: a warp each, so
  // that a token's lookups and sines are issued by one warp and not by eight.
  constexpr int kAll = kThreads / 32;
  if (a.c.n_tokens < 8 * num_sms())
    return launch_pdl(rope_append_kernel<T, kE4M3, kAll>, dim3((unsigned)a.c.n_tokens + 1),
                      dim3(kThreads), 0, s, 1, a, rope, lane_bits);
  return launch_pdl(rope_append_kernel<T, kE4M3, 1>,
                    dim3((unsigned)ceil_div(a.c.n_tokens, kAll) + 1), dim3(kThreads), 0, s, 1, a,
                    rope, lane_bits);
}

}  // namespace

cudaError_t launch_rope_append(const AttnArgs& a, cudaStream_t s) {
  if (a.c.n_tokens == 0) return launch_reset_status(a.status, s);
  RopeTable rope = {};
  rope_turns(a.c.rope_base, a.c.rot_dim / 2, rope.turns);
  int lane_bits = 0;
  while ((8 << lane_bits) < a.c.head_dim) ++lane_bits;
  ProfScope p(K_ROPE_APPEND, s);
  if (a.c.dtype == MOE_F32) return launch<float, false>(a, rope, lane_bits, s);
  if (a.c.cache_dtype == MOE_E4M3) return launch<__nv_bfloat16, true>(a, rope, lane_bits, s);
  return launch<__nv_bfloat16, false>(a, rope, lane_bits, s);
}

}  // namespace moe
