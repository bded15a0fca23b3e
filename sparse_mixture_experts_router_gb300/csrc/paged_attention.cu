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
#include <algorithm>

#include "paged_attention.cuh"

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


// Rows whose keys were cut into splits: one warp a row.
constexpr int kJoinWarps = 4;
template <typename Elem>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_kernel(const __grid_constant__ attn::Params prm, int block_rows, int rows) {
  const moe_attn_config& c = prm.a.c;
  const int i = (int)blockIdx.x * kJoinWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_trigger();
  if (i >= rows) return;
  attn::Item it;
  it.index = i / block_rows;
  const int r = i % block_rows, rb = it.index % prm.row_blocks, head = it.index / prm.row_blocks;
  it.kh = head % c.n_kv_heads;
  it.sq = seq_range(prm.a, head / c.n_kv_heads);
  it.G = c.n_heads / c.n_kv_heads;
  it.row0 = rb * block_rows;
  if (it.row0 + r >= it.G * it.sq.n) return;
  const int64_t row0 = (int64_t)it.index * prm.splits * attn::kMaxRows + r;
  const float2 ml = lane < prm.splits ? prm.split_ml[row0 + (int64_t)lane * attn::kMaxRows]
                                      : make_float2(-INFINITY, 0.f);
  float top = ml.x;
#pragma unroll
  for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float f = ptx::ex2(ml.x - top), sum = warp_sum(ml.y * f);
  attn::Params out = prm;
  out.splits = 1;
  const int vecs = c.head_dim / 4;
  for (int v0 = 0; v0 < vecs; v0 += 32) {
    const int v = v0 + lane;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < prm.splits; ++s) {
      const float fs = __shfl_sync(0xffffffffu, f, s);
      if (v >= vecs) continue;
      const float4 y = reinterpret_cast<const float4*>(
          prm.split_o)[(row0 + (int64_t)s * attn::kMaxRows) * vecs + v];
      x.x += y.x * fs, x.y += y.y * fs, x.z += y.z * fs, x.w += y.w * fs;
    }
    if (v < vecs) attn::write_row<Elem>(out, it, r, v, x, top, sum);
  }
}

// How a call is cut; of cfg alone, so that the workspace holds its splits.
struct Plan {
  int nt;  // query rows of an item / 8
  int row_blocks, parts, splits;
  long long items;
};
Plan plan_of(const moe_attn_config& c) {
  Plan p;
  const int tiles = ceil_div((long long)(c.n_heads / c.n_kv_heads) * c.max_new, 8);
  p.row_blocks = ceil_div(tiles, c.head_dim <= 128 ? 4 : 2);
  p.nt = ceil_div(tiles, p.row_blocks);
  p.items = (long long)c.n_seqs * c.n_kv_heads * p.row_blocks;
  long long keys = (long long)c.max_pages * c.page_size;
  if (c.window) keys = std::min(keys, (long long)c.window + c.max_new);
  const long long key_tiles = ceil_div(keys, c.cache_dtype == MOE_E4M3 ? 32 : 16);
  // Parts: four waves of blocks, so that uneven sequences even out, as long
  // as every warp has a tile.
  p.parts = 1;
  while (p.parts < attn::kMaxParts && p.items * p.parts < 4LL * 2 * attn::kPlanSms &&
         key_tiles >= 8 * p.parts)
    p.parts *= 2;
  // Splits: where the largest clusters still leave SMs idle and a warp has 16
  // tiles or more.
  p.splits = 1;
  if (p.parts == attn::kMaxParts && p.items > 0 && c.cache_dtype != MOE_F32)
    p.splits = (int)std::max(1LL, std::min({2LL * attn::kPlanSms / (p.items * p.parts),
                                            key_tiles / (16 * 4 * p.parts),
                                            (long long)attn::kMaxSplits}));
  return p;
}
size_t split_rows(const Plan& p) {
  return p.splits > 1 ? (size_t)p.items * p.splits * attn::kMaxRows : 0;
}

}  // namespace

namespace attn {
cudaError_t launch_bf16(const Params& p, int dim, int nt, unsigned blocks, cudaStream_t s);
cudaError_t launch_e4m3(const Params& p, int dim, int nt, unsigned blocks, cudaStream_t s);
}  // namespace attn

size_t attention_scratch_bytes(const moe_attn_config& c) {
  return split_rows(plan_of(c)) * ((size_t)c.head_dim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_paged_attention(const AttnArgs& a, void* scratch, cudaStream_t s) {
  const moe_attn_config& c = a.c;
  if (c.n_tokens == 0) return launch_reset_status(a.status, s);
  if (c.cache_dtype == MOE_F32) {
    ProfScope p(K_ATTENTION, s);
    const dim3 grid((unsigned)c.max_new, (unsigned)c.n_seqs + 1, (unsigned)c.n_heads);
    return launch_pdl(f32_kernel, grid, dim3(kWarps * 32), 0, s, 1, a);
  }
  const Plan plan = plan_of(c);
  attn::Params prm = {};
  prm.a = a;
  prm.page_div = attn::fast_div((uint32_t)c.page_size);
  prm.parts = plan.parts;
  prm.splits = plan.splits;
  prm.row_blocks = plan.row_blocks;
  prm.split_o = static_cast<float*>(scratch);
  prm.split_ml = reinterpret_cast<float2*>(prm.split_o + split_rows(plan) * c.head_dim);
  const unsigned blocks = (unsigned)((plan.items * plan.splits + 1) * plan.parts);
  cudaError_t e;
  {
    ProfScope p(K_ATTENTION, s);
    e = c.cache_dtype == MOE_E4M3 ? attn::launch_e4m3(prm, c.head_dim, plan.nt, blocks, s)
                                  : attn::launch_bf16(prm, c.head_dim, plan.nt, blocks, s);
  }
  if (e != cudaSuccess || plan.splits == 1) return e;
  ProfScope p(K_ATTENTION_JOIN, s);
  const int rows = (int)(plan.items * 8 * plan.nt);
  return launch_pdl(join_kernel<__nv_bfloat16>, dim3((unsigned)ceil_div(rows, kJoinWarps)),
                    dim3(kJoinWarps * 32), 0, s, 1, prm, 8 * plan.nt, rows);
}

}  // namespace moe
