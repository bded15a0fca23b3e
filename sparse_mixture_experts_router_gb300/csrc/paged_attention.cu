// Attention of the new tokens over a paged key-value cache.
//
// out = sum_i exp(s_i) v_i / sum_i exp(s_i) over the positions a token sees,
// in one pass over them with the running maximum m, sum l and weighted sum o
// of a softmax (all fp32): a key that raises m scales l and o by
// exp(m_old - m_new). Partial (m, l, o) of disjoint key ranges join the same
// way, so a row's keys are split over the warps of a block.
//
// Simple form: one block per (new token, query head), one key a warp and
// step, the head's elements spread over the lanes.
#include "serve_util.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kPerLane = kAttnMaxDim / 32;

__device__ __forceinline__ float cache_value(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float cache_value(const __nv_bfloat16* p, int64_t i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ float cache_value(const uint8_t* p, int64_t i) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)p[i]));
  float f;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l;}" : "=f"(f) : "r"(h));
  return f;
}

template <typename T, typename C>
__global__ void __launch_bounds__(kWarps * 32) paged_attention_kernel(const AttnArgs a) {
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kAttnMaxDim];
  const moe_attn_config& c = a.c;
  const int j = blockIdx.x, b = blockIdx.y, h = blockIdx.z;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_trigger();
  const SeqRange r = seq_range(a, b);
  if (!r.ok && threadIdx.x == 0) set_status(a.status, status_check());
  if (j >= r.n) return;
  const int t = r.row0 + j, pos = r.len - r.n + j, kh = h / (c.n_heads / c.n_kv_heads);
  const int first = c.window ? max(0, pos - c.window + 1) : 0;
  float q[kPerLane], o[kPerLane] = {}, m = -INFINITY, l = 0.f;
  const T* qp = static_cast<const T*>(a.q) + (int64_t)t * c.q_stride + h * c.head_dim;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    q[i] = e < c.head_dim ? to_f32(qp[e]) * c.scale : 0.f;
  }
  for (int key = first + warp; key <= pos; key += kWarps) {
    const int page = page_of(a, b, key), at = key % c.page_size;
    if (page < 0) {
      if (lane == 0) set_status(a.status, status_check());
      continue;
    }
    const int64_t off =
        (int64_t)page * c.page_stride + (int64_t)at * c.token_stride + kh * c.head_stride;
    float ks = 1.f, vs = 1.f;
    if (a.k_scale) {
      const int64_t si = ((int64_t)page * c.n_kv_heads + kh) * c.page_size + at;
      ks = a.k_scale[si];
      vs = a.v_scale[si];
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 32 * i;
      if (e < c.head_dim) s += q[i] * cache_value(static_cast<const C*>(a.k_cache), off + e);
    }
    s = warp_sum(s) * ks;
    const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : __expf(m - top);
    const float w = s == -INFINITY ? 0.f : __expf(s - top);
    if (top == -INFINITY) continue;
    m = top;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 32 * i;
      if (e < c.head_dim)
        o[i] = o[i] * f + w * vs * cache_value(static_cast<const C*>(a.v_cache), off + e);
    }
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) so[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < kWarps; ++w)
    if (sm[w] != -INFINITY) total += sl[w] * __expf(sm[w] - top);
  for (int e = threadIdx.x; e < c.head_dim; e += kWarps * 32) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (sm[w] != -INFINITY) v += so[w][e] * __expf(sm[w] - top);
    static_cast<T*>(a.out)[((int64_t)t * c.n_heads + h) * c.head_dim + e] =
        from_f32<T>(total > 0.f ? v / total : 0.f);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)t * c.n_heads + h] = total > 0.f ? top + logf(total) : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_attention(const AttnArgs& a, cudaStream_t s) {
  cudaError_t e = launch_reset_status(a.status, s);
  if (e != cudaSuccess || a.c.n_tokens == 0) return e;
  ProfScope p(K_ATTENTION, s);
  const dim3 grid((unsigned)a.c.max_new, (unsigned)a.c.n_seqs, (unsigned)a.c.n_heads);
  const dim3 block(kWarps * 32);
  if (a.c.dtype == MOE_F32)
    return launch_pdl(paged_attention_kernel<float, float>, grid, block, 0, s, 1, a);
  if (a.c.cache_dtype == MOE_E4M3)
    return launch_pdl(paged_attention_kernel<__nv_bfloat16, uint8_t>, grid, block, 0, s, 1, a);
  return launch_pdl(paged_attention_kernel<__nv_bfloat16, __nv_bfloat16>, grid, block, 0, s, 1, a);
}

}  // namespace moe
