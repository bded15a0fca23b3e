// Attention of the new tokens over a paged key-value cache.
//
// out = sum_i exp(s_i) v_i / sum_i exp(s_i) over the positions a token sees,
// in one pass over them with the running maximum m, sum l and weighted sum o
// of a softmax (all fp32): a key that raises m scales l and o by
// exp(m_old - m_new). Partial (m, l, o) of disjoint key ranges join the same
// way, so a row's keys are split over warps, and over the blocks of a cluster.
//
// bf16 and E4M3 caches run on the matrix kernel of paged_attention_mma.cuh.
// fp32 caches run on the kernel below, on the CUDA cores: one block per (new
// token, query head), one key a warp and step, the head's elements spread
// over the lanes.
#include "paged_attention_mma.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kPerLane = kAttnMaxDim / 32;

__global__ void __launch_bounds__(kWarps * 32) f32_kernel(const AttnArgs a) {
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kAttnMaxDim];
  const moe_attn_config& c = a.c;
  const int j = blockIdx.x, b = (int)blockIdx.y - 1, h = blockIdx.z;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_trigger();
  if (b < 0) {
    if (j == 0 && h == 0) check_lists<kWarps * 32>(a, attn::FirstKey{c.window});
    return;
  }
  const SeqRange r = seq_range(a, b);
  if (j >= r.n) return;
  const int t = r.row0 + j, pos = r.len - r.n + j, kh = h / (c.n_heads / c.n_kv_heads);
  const int first = c.window ? max(0, pos - c.window + 1) : 0;
  float q[kPerLane], o[kPerLane] = {}, m = -INFINITY, l = 0.f;
  const float* qp = static_cast<const float*>(a.q) + (int64_t)t * c.q_stride + h * c.head_dim;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    q[i] = e < c.head_dim ? qp[e] * c.scale : 0.f;
  }
  for (int key = first + warp; key <= pos; key += kWarps) {
    const int page = page_of(a, b, key), at = key % c.page_size;
    if (page < 0) continue;
    const int64_t off =
        (int64_t)page * c.page_stride + (int64_t)at * c.token_stride + kh * c.head_stride;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 32 * i;
      if (e < c.head_dim) s += q[i] * static_cast<const float*>(a.k_cache)[off + e];
    }
    s = warp_sum(s);
    const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : __expf(m - top);
    const float w = s == -INFINITY ? 0.f : __expf(s - top);
    if (top == -INFINITY) continue;
    m = top;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 32 * i;
      if (e < c.head_dim)
        o[i] = o[i] * f + w * static_cast<const float*>(a.v_cache)[off + e];
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
    static_cast<float*>(a.out)[((int64_t)t * c.n_heads + h) * c.head_dim + e] =
        total > 0.f ? v / total : 0.f;
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)t * c.n_heads + h] = total > 0.f ? top + logf(total) : -INFINITY;
}

}  // namespace

namespace attn {
cudaError_t launch_bf16(const Params& p, int dim, int nt, unsigned blocks, cudaStream_t s);
cudaError_t launch_e4m3(const Params& p, int dim, int nt, unsigned blocks, cudaStream_t s);
}  // namespace attn

cudaError_t launch_paged_attention(const AttnArgs& a, cudaStream_t s) {
  const moe_attn_config& c = a.c;
  if (c.n_tokens == 0) return launch_reset_status(a.status, s);
  ProfScope p(K_ATTENTION, s);
  if (c.cache_dtype == MOE_F32) {
    const dim3 grid((unsigned)c.max_new, (unsigned)c.n_seqs + 1, (unsigned)c.n_heads);
    return launch_pdl(f32_kernel, grid, dim3(kWarps * 32), 0, s, 1, a);
  }
  // Query rows of a (sequence, head) in blocks of 8 nt.
  const bool f8 = c.cache_dtype == MOE_E4M3;
  const int most = c.head_dim <= 128 ? 4 : 2;
  const int tiles = ceil_div((long long)c.n_heads / c.n_kv_heads * c.max_new, 8);
  attn::Params prm = {};
  prm.a = a;
  prm.page_div = attn::fast_div((uint32_t)c.page_size);
  prm.row_blocks = ceil_div(tiles, most);
  const int nt = ceil_div(tiles, prm.row_blocks);
  const long long items = (long long)c.n_seqs * c.n_kv_heads * prm.row_blocks;
  long long keys = (long long)c.max_pages * c.page_size;
  if (c.window) keys = keys < c.window + c.max_new ? keys : c.window + c.max_new;
  const int key_tiles = ceil_div(keys, f8 ? 32 : 16);
  prm.parts = 1;
  while (prm.parts < 16 && items * prm.parts < 4LL * 2 * num_sms() &&
         key_tiles >= 2 * attn::kWarps * prm.parts)
    prm.parts *= 2;
  const unsigned blocks = (unsigned)((items + 1) * prm.parts);
  return f8 ? attn::launch_e4m3(prm, c.head_dim, nt, blocks, s)
            : attn::launch_bf16(prm, c.head_dim, nt, blocks, s);
}

}  // namespace moe
