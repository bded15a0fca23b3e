// Verification of drafted tokens.
//
// A draft x with target probability p and draft probability q is accepted
// while u q < p; both sides are products of two 24-bit fractions, exact in
// fp64. Of a sequence's rows only one is then read whole: the target's at
// the first rejection (and the draft model's there), or after the last
// draft. The token drawn from r = max(p - q, 0) is the least i whose running
// sum passes u R. Running sums in floating point depend on the order they
// are taken in, which a split over many threads changes; so every entry is
// held as an integer of 2^-60 units and the sums are exact, whatever the
// split: two passes over the row, one for the sums of segments and one for
// the place inside the segment that holds u R.
//
// Bound by memory for a batch (one or two rows a sequence) and by latency
// for a single sequence.
#include "serve_util.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// A probability: clamped to [0, 1], NaN as 0; and in 2^-60 units.
__device__ __forceinline__ float prob(float x) { return fminf(fmaxf(x, 0.f), 1.f); }
__device__ __forceinline__ uint64_t fixed60(float x) { return __float2ull_rz(prob(x) * 0x1p60f); }
__device__ __forceinline__ uint64_t warp_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ uint64_t residual(const T* p, const T* q, int hot, int i) {
  const uint64_t v = fixed60(to_f32(p[i]));
  const uint64_t w = q ? fixed60(to_f32(q[i])) : i == hot ? 1ull << 60 : 0ull;
  return v > w ? v - w : 0ull;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
  __shared__ uint64_t part[kWarps];
  __shared__ int s_accepted;
  const moe_verify_config& c = a.c;
  const int b = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_trigger();
  const SeqRange r = seq_rows(a.cu_new, b, c.n_seqs, c.n_tokens, c.max_new);
  if (!r.ok && threadIdx.x == 0) set_status(a.status, status_check());
  const T* p = static_cast<const T*>(a.p);
  const T* q = static_cast<const T*>(a.q);
  const int drafts = max(r.n - 1, 0);

  if (warp == 0) {
    int acc = 0;
    for (int j0 = 0; j0 < drafts; j0 += 32) {
      const int j = j0 + lane;
      bool take = true;
      if (j < drafts) {
        const int x = a.tokens[r.row0 + j + 1];
        take = x >= 0 && x < c.vocab;
        if (!take) set_status(a.status, status_check());
        if (take) {
          const int64_t row = r.row0 + j;
          const double px = prob(to_f32(p[row * c.p_stride + x]));
          const double qx = q ? prob(to_f32(q[row * c.q_stride + x])) : 1.f;
          take = (double)a.u_accept[row] * qx < px;
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !take || j >= drafts);
      acc = j0 + (no ? __ffs(no) - 1 : 32);
      if (no) break;
    }
    if (lane == 0) s_accepted = min(acc, drafts);
  }
  __syncthreads();
  const int acc = s_accepted;
  if (threadIdx.x == 0) {
    a.n_accepted[b] = acc;
    if (a.kv_next) a.kv_next[b] = a.kv_len[b] - (drafts - acc);
  }
  if (r.n == 0) return;
  for (int j = threadIdx.x; j < r.n; j += kThreads)
    if (j != acc) a.out_tokens[r.row0 + j] = j < acc ? a.tokens[r.row0 + j + 1] : -1;

  const int64_t row = r.row0 + acc;
  const T* pr = p + row * c.p_stride;
  const bool rejected = acc < drafts;
  const T* qr = rejected && q ? q + row * c.q_stride : nullptr;
  int hot = rejected && !q ? a.tokens[row + 1] : -1;
  const int per = (c.vocab + kWarps - 1) / kWarps, i0 = warp * per, i1 = min(i0 + per, c.vocab);
  uint64_t total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t sum = 0;
    for (int i = i0 + lane; i < i1; i += 32) sum += residual(pr, qr, hot, i);
    sum = warp_sum_u64(sum);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) total += part[w];
    if (total > 0 || !rejected) break;
    qr = nullptr;  // nowhere above the draft model: the target itself
    hot = -1;
    __syncthreads();
  }
  if (total == 0) {
    if (threadIdx.x == 0) a.out_tokens[row] = -1;
    return;
  }
  const float u = fminf(fmaxf(a.u_sample[b], 0.f), 0x1.fffffep-1f);
  const uint64_t mark = __umul64hi(__float2ull_rz(u * 0x1p64f), total);
  uint64_t before = 0;
  for (int w = 0; w < warp; ++w) before += part[w];
  if (mark < before || mark >= before + part[warp]) return;
  for (int i = i0; i < i1; i += 32) {
    uint64_t v = i + lane < i1 ? residual(pr, qr, hot, i + lane) : 0ull;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + v > mark);
    if (hit) {
      if (lane == 0) a.out_tokens[row] = i + __ffs(hit) - 1;
      return;
    }
    before += __shfl_sync(0xffffffffu, v, 31);
  }
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, cudaStream_t s) {
  cudaError_t e = launch_reset_status(a.status, s);
  if (e != cudaSuccess || a.c.n_seqs == 0) return e;
  ProfScope p(K_VERIFY, s);
  const dim3 grid((unsigned)a.c.n_seqs), block(kThreads);
  if (a.c.dtype == MOE_F32) return launch_pdl(verify_kernel<float>, grid, block, 0, s, 1, a);
  return launch_pdl(verify_kernel<__nv_bfloat16>, grid, block, 0, s, 1, a);
}

}  // namespace moe
