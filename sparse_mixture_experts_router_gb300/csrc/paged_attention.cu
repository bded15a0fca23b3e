// Attention of the new tokens over a paged key-value cache.
//
// out = sum_i exp(s_i) v_i / sum_i exp(s_i) over the positions a token sees,
// in one pass over them with the running maximum m, sum l and weighted sum o
// of a softmax (all fp32): a key that raises m scales l and o by
// exp(m_old - m_new). Partial (m, l, o) of disjoint key ranges join the same
// way, so a row's keys are split over warps, and over the blocks of a cluster.
//
// Here: how a call is cut, and the join of splits. bf16 and E4M3 caches run on
// the matrix kernel of paged_attention_mma.cuh, above a number of query rows
// (not E4M3 with a scale a token) on the tcgen05 kernels of
// paged_attention_tc.cu and paged_attention_tc_e4m3.cu; fp32 caches on that of
// paged_attention_f32.cu.
#include <algorithm>

#include "paged_attention.cuh"

namespace moe {
namespace {

// Query rows of a bf16 head group above which the tcgen05 kernel runs. us of it
// and of the warp-level kernel's blocks of 16 (8 key-value heads, 8 new tokens):
//                                            48 rows       56 rows
//   32 sequences of 100 to 6000 keys, D 128  137 and 143   139 and 177
//   128 of 30 to 1000, D 128                 115 and 107   118 and 138
//   32 of 100 to 6000, D 64                  112 and  90   114 and 115
//   2 of 20000, D 128                         89 and  52    90 and  98
constexpr int kTcRows = 48;
// The same of an E4M3 cache with a scale a page. us of the warp-level kernel and of the
// tcgen05 kernel (32 sequences of 100 to 12000 keys, 8 key-value heads, 8 new tokens, D 128):
//             48 rows       64            80            128
//   pages of 64  245 and 267   304 and 269   358 and 272   532 and 286
//   pages of 16  255 and 337   315 and 340   369 and 348   547 and 366
// (64 rows were level in both kernels' first form, and with pages of 64 no longer are.)
constexpr int kTcRowsE4m3 = 64;

// Rows whose keys were cut into splits: one warp a row. kRef: E4M3 caches.
constexpr int kJoinWarps = 4;
template <typename Elem, bool kRef>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_kernel(const __grid_constant__ attn::Params prm, int rows) {
  const moe_attn_config& c = prm.a.c;
  const int i = (int)blockIdx.x * kJoinWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_trigger();
  if (i >= rows) return;
  const int block_rows = prm.item_rows;
  attn::Item it;
  it.index = i / block_rows;
  const int r = i % block_rows, rb = it.index % prm.row_blocks, head = it.index / prm.row_blocks;
  it.kh = head % c.n_kv_heads;
  it.sq = seq_range(prm.a, head / c.n_kv_heads);
  it.G = prm.group;
  it.row0 = rb * block_rows;
  if (it.row0 + r >= it.G * it.sq.n) return;
  const int64_t row0 = (int64_t)it.index * prm.splits * block_rows + r;
  const float2 ml = lane < prm.splits ? prm.split_ml[row0 + (int64_t)lane * block_rows]
                                      : make_float2(-INFINITY, 0.f);
  float top = ml.x;
#pragma unroll
  for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  float f = ptx::ex2(ml.x - top), ref = 0.f;
  const float sum = warp_sum(ml.y * f);
  if (kRef) {
    const float own = lane < prm.splits ? prm.split_ref[row0 + (int64_t)lane * block_rows] : -INFINITY;
    ref = own;
#pragma unroll
    for (int x = 16; x > 0; x /= 2) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, x));
    f = ptx::ex2(own - ref);
  }
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
          prm.split_o)[(row0 + (int64_t)s * block_rows) * vecs + v];
      x.x += y.x * fs, x.y += y.y * fs, x.z += y.z * fs, x.w += y.w * fs;
    }
    if (v < vecs) attn::write_row<Elem, kRef>(out, it, r, v, x, top, sum, ref);
  }
}

// How a call is cut; of cfg alone, so that the workspace holds its splits.
struct Plan {
  bool tc;                // the tcgen05 kernel
  int unit, nt;           // query rows of an item: unit * nt
  int row_blocks, parts, splits;
  long long items;
  int rows() const { return unit * nt; }
};
Plan plan_of(const moe_attn_config& c) {
  Plan p;
  const bool f32 = c.cache_dtype == MOE_F32, f8 = is_e4m3(c.cache_dtype);
  const long long all_rows = (long long)(c.n_heads / c.n_kv_heads) * c.max_new;
  p.tc = c.head_dim <= 128 && (c.cache_dtype == MOE_BF16        ? all_rows > kTcRows
                               : c.cache_dtype == MOE_E4M3_PAGE && all_rows > kTcRowsE4m3);
  p.unit = p.tc ? 16 : f32 ? 4 : 8;
  const int units = ceil_div(all_rows, p.unit);
  // Rows of a block: 16 (fp32: 12), although each block of them reads the keys
  // again, most of the time from L2: more take the registers and the shared
  // memory of an SM's third block. Against larger blocks, since removed: bf16,
  // 20 rows: 147 us in one block, 138 in two; E4M3, 28 rows: 282 and 206; fp32,
  // 16 rows: 42.6 and 37.3.
  // The tcgen05 kernels take all that they have lanes of Tensor Memory for: 128,
  // of an E4M3 cache 256 in two streams (as one item and as two of up to 128, the calls
  // above: 136 rows 365 and 427 us, 192: 378 and 437, 256: 398 and 460).
  p.row_blocks = ceil_div(units, p.tc ? (f8 ? 16 : 8) : f32 && c.head_dim <= 128 ? 3 : 2);
  p.nt = ceil_div(units, p.row_blocks);
  p.items = (long long)c.n_seqs * c.n_kv_heads * p.row_blocks;
  long long keys = (long long)c.max_pages * c.page_size;
  if (c.window) keys = std::min(keys, (long long)c.window + c.max_new);
  // A part's unit of work: a tile for each of a block's warps.
  const int warps = p.tc ? 1 : 4;
  const int tile = p.tc ? 128 : f32 ? 8 : attn::keys_of(c.head_dim, f8);
  const long long steps = ceil_div(keys, warps * tile);
  // Parts. A block costs its steps and about kPartCost / 2 more (its start, its
  // turn to join), blocks on all slots share the work, and the longest block
  // ends last: items x (steps + kPartCost / 2 x parts) / slots + steps / parts,
  // least where items x kPartCost / 2 x parts^2 = steps x slots; parts is the
  // power of two nearest to that, and leaves a block two steps. Over 115 drawn
  // calls a cost of 2, 4, 6, 7, 12 steps took 1.03, 0.99, 0.98, 0.97, 0.99 of
  // filling the SMs and then up to three waves of at least eight steps; over
  // 50 of an fp32 cache 7, 10, 14, 20 took 0.92, 0.93, 0.94, 0.95. Clusters of
  // 16 are placed badly unless all run at once: 84 sequences of 8000 keys take
  // 79 us in 16 parts, 65 in eight.
  const int per_sm = p.tc  ? 1
                     : f32 ? attn::f32_blocks_per_sm(c.head_dim, p.nt)
                           : attn::blocks_per_sm(c.head_dim);
  const long long slots = (long long)per_sm * attn::kPlanSms;
  const int most = p.tc ? 8 : attn::kMaxParts;  // 16 whole SMs are more than some GPCs have
  constexpr long long kPartCost = 15;
  p.parts = 1;
  while (p.parts < most && steps >= 2 * p.parts &&
         p.items * p.parts * p.parts * kPartCost <= steps * slots &&
         (p.parts < 8 || 2 * p.items * p.parts <= slots))
    p.parts *= 2;
  // Splits: where the largest clusters still leave SMs idle (their blocks two
  // an SM where they fit) and a block keeps four steps.
  p.splits = 1;
  if (p.parts == most && p.items > 0)
    p.splits = (int)std::max(1LL, std::min({std::min(slots, 2LL * attn::kPlanSms) / (p.items * p.parts),
                                            steps / (4 * p.parts),
                                            (long long)attn::kMaxSplits}));
  return p;
}
size_t split_rows(const Plan& p) {
  return p.splits > 1 ? (size_t)p.items * p.splits * p.rows() : 0;
}

}  // namespace

namespace attn {
cudaError_t launch_bf16(const Params& p, int dim, int nt, unsigned blocks, cudaStream_t s);
cudaError_t launch_e4m3(const Params& p, int dim, int nt, unsigned blocks, cudaStream_t s);
cudaError_t launch_f32(const Params& p, int dim, int nt, unsigned blocks, cudaStream_t s);
cudaError_t launch_tc(const Params& p, int dim, unsigned blocks, cudaStream_t s);
cudaError_t launch_tc_e4m3(const Params& p, int dim, unsigned blocks, cudaStream_t s);
}  // namespace attn

size_t attention_scratch_bytes(const moe_attn_config& c) {
  return split_rows(plan_of(c)) *
         ((size_t)c.head_dim * sizeof(float) + sizeof(float2) + (is_e4m3(c.cache_dtype) ? sizeof(float) : 0));
}

cudaError_t launch_paged_attention(const AttnArgs& a, void* scratch, cudaStream_t s) {
  const moe_attn_config& c = a.c;
  if (c.n_tokens == 0) return launch_reset_status(a.status, s);
  const Plan plan = plan_of(c);
  attn::Params prm = {};
  prm.a = a;
  prm.parts = plan.parts;
  prm.splits = plan.splits;
  prm.row_blocks = plan.row_blocks;
  prm.group = c.n_heads / c.n_kv_heads;
  prm.item_rows = plan.rows();
  // One block looks at 4096 pages in about 5 us; 79 sequences of 440 to 940
  // pages took it 86 us, where the attention takes 15.
  prm.check_in_use = (long long)c.n_seqs * c.max_pages > 4096;
  prm.by_page = fast_div((uint32_t)c.page_size);
  prm.by_group = fast_div((uint32_t)prm.group);
  prm.by_parts = fast_div((uint32_t)prm.parts);
  prm.by_splits = fast_div((uint32_t)prm.splits);
  prm.by_rows = fast_div((uint32_t)prm.row_blocks);
  prm.by_heads = fast_div((uint32_t)c.n_kv_heads);
  prm.by_vecs = fast_div((uint32_t)c.head_dim / 4);
  prm.split_o = static_cast<float*>(scratch);
  prm.split_ml = reinterpret_cast<float2*>(prm.split_o + split_rows(plan) * c.head_dim);
  prm.split_ref = reinterpret_cast<float*>(prm.split_ml + split_rows(plan));
  const unsigned blocks = (unsigned)((plan.items * plan.splits + 1) * plan.parts);
  cudaError_t e = prm.check_in_use ? launch_reset_status(a.status, s) : cudaSuccess;
  if (e != cudaSuccess) return e;
  {
    ProfScope p(K_ATTENTION, s);
    e = plan.tc && is_e4m3(c.cache_dtype) ? attn::launch_tc_e4m3(prm, c.head_dim, blocks, s)
        : plan.tc                   ? attn::launch_tc(prm, c.head_dim, blocks, s)
        : c.cache_dtype == MOE_F32  ? attn::launch_f32(prm, c.head_dim, plan.nt, blocks, s)
        : is_e4m3(c.cache_dtype)    ? attn::launch_e4m3(prm, c.head_dim, plan.nt, blocks, s)
                                    : attn::launch_bf16(prm, c.head_dim, plan.nt, blocks, s);
  }
  if (e != cudaSuccess || plan.splits == 1) return e;
  ProfScope p(K_ATTENTION_JOIN, s);
  const int rows = (int)(plan.items * plan.rows());
  const dim3 grid((unsigned)ceil_div(rows, kJoinWarps)), block(kJoinWarps * 32);
  return c.dtype == MOE_F32       ? launch_pdl(join_kernel<float, false>, grid, block, 0, s, 1, prm, rows)
         : is_e4m3(c.cache_dtype) ? launch_pdl(join_kernel<__nv_bfloat16, true>, grid, block, 0, s, 1, prm, rows)
                                  : launch_pdl(join_kernel<__nv_bfloat16, false>, grid, block, 0, s, 1, prm, rows);
}

}  // namespace moe
