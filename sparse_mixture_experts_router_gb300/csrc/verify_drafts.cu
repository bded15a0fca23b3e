// Verification of drafted tokens.
//
// A draft x with target probability p and draft probability q is accepted
// while u q < p; both sides are products of two 24-bit fractions, exact in
// fp64. Of a sequence's rows only one is then read whole: the target's at
// the first rejection (and the draft model's there), or after the last
// draft. The token drawn from r = max(p - q, 0) is the least i whose running
// sum passes u R. Running sums in floating point depend on the order they
// are taken in, which a split over many threads changes; so every entry is
// held as an integer of 2^-60 units (rounded to nearest) and the sums are
// exact, whatever the split: one pass over the row for the sums of segments
// (one a warp), and a second over the one segment that holds u R.
//
// A sequence is a cluster of up to 16 blocks, so that a single row of the
// vocabulary spreads over 16 SMs; the blocks' sums meet in distributed shared
// memory. Every block finds the accepted drafts by itself: that takes the
// same time as being told. The first block's other warps check the lists
// meanwhile and it writes the status, so the call is one launch. Bound by
// memory and by the additions for a batch (one or two rows a sequence), and by
// latency for a single sequence: five dependent
// reads (rows, draft, its probabilities, the row, the segment) and one
// exchange between the blocks.
#include <algorithm>

#include "serve_util.cuh"
#include "serve_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 16;

// A probability: clamped to [0, 1], NaN as 0.
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }

// Sums of max(p - q, 0) in 2^-60 units. A conversion of fp32 to a 64-bit
// integer runs at the FP64 units' rate, 1/64 of fp32's here, and would take
// five times as long as reading the row. Adding a constant whose last bit
// weighs 2^-22 rounds p to such units and leaves them in the sum's own bit
// pattern; what was rounded off is exact, and goes the same way in units of
// 2^-44 and 2^-60. So a pair (p, q) costs seven packed fp32 additions, and the
// three digits are summed as 32-bit integers, the constants' patterns cancelling
// between p and q.
struct Digits {
  int a = 0, b = 0, c = 0;  // units 2^-22, 2^-44, 2^-60
  __device__ __forceinline__ void add(float p, float q) {
    // p and q go through the additions as one pair of fp32; where p <= q it is
    // (q, q), whose digits cancel
    const float y = prob(q);
    const uint64_t v = ptx::f32x2(fmaxf(prob(p), y), y);
    const uint64_t y1 = add2(v, twice(2.f));
    const uint64_t r1 = sub2(v, add2(y1, twice(-2.f)));
    const uint64_t y2 = add2(r1, twice(0x1.8p-21f));
    const uint64_t r2 = sub2(r1, add2(y2, twice(-0x1.8p-21f)));
    const uint64_t y3 = add2(r2, twice(0x1.8p-37f));
    a += (int)(uint32_t)y1 - (int)(uint32_t)(y1 >> 32);
    b += (int)(uint32_t)y2 - (int)(uint32_t)(y2 >> 32);
    c += (int)(uint32_t)y3 - (int)(uint32_t)(y3 >> 32);
  }
  static __device__ __forceinline__ uint64_t twice(float x) { return ptx::f32x2(x, x); }
  static __device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    return ptx::add_f32x2(x, y);
  }
  static __device__ __forceinline__ uint64_t sub2(uint64_t x, uint64_t y) {
    return ptx::fma_f32x2(y, twice(-1.f), x);  // x - y, rounded once
  }
  // At most 256 elements fit the digits.
  __device__ __forceinline__ uint64_t value() const {
    return (uint64_t)(((int64_t)a << 38) + ((int64_t)b << 16) + c);
  }
};

__device__ __forceinline__ uint64_t warp_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan_u64(uint64_t v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// 16 bytes of a row as fp32: 4 fp32 or 8 bf16 elements.
__device__ __forceinline__ void unpack(uint4 v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(uint4 v, float (&x)[8]) {
  bf16x2_to_f32(v.x, x[0], x[1]);
  bf16x2_to_f32(v.y, x[2], x[3]);
  bf16x2_to_f32(v.z, x[4], x[5]);
  bf16x2_to_f32(v.w, x[6], x[7]);
}

// r = max(p - q, 0) of a row in vectors of kE elements on p's 16-byte grid:
// vector v holds elements v kE - shift ... (those outside the row are 0).
template <typename T>
struct Residual {
  static constexpr int kE = 16 / (int)sizeof(T);
  const T* p;
  const T* q;  // null: none, or all of it at `hot`
  int hot, vocab, shift;
  bool q_grid;  // q's 16-byte grid is p's
  __device__ Residual(const T* p_, const T* q_, int hot_, int vocab_)
      : p(p_), q(q_), hot(hot_), vocab(vocab_) {
    shift = (int)((uintptr_t)p % 16) / (int)sizeof(T);
    q_grid = (uintptr_t)p % 16 == (uintptr_t)q % 16;
  }
  __device__ int vectors() const { return (vocab + shift + kE - 1) / kE; }
  __device__ __forceinline__ void row(const T* src, bool grid, int e, float (&x)[kE]) const {
    if (grid && e >= 0 && e + kE <= vocab) {
      unpack(__ldg(reinterpret_cast<const uint4*>(src + e)), x);
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) x[i] = e + i >= 0 && e + i < vocab ? to_f32(src[e + i]) : 0.f;
    }
  }
  __device__ __forceinline__ void load(int v, float (&x)[kE], float (&y)[kE]) const {
    const int e = v * kE - shift;
    row(p, true, e, x);
    if (q) {
      row(q, q_grid, e, y);
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) y[i] = e + i == hot ? 1.f : 0.f;
    }
  }
  // A warp's vectors v .. v + kStep - 1, in flight at once: each lane's sum.
  // The pass is bound by instructions as much as by memory, so a step inside
  // the row has no checks of its own (17.6 us for the batch of 64, with them
  // 18.4; copied ahead through shared memory, more instructions yet, 20.3).
  static constexpr int kU = 16 / kE, kStep = 32 * kU;
  __device__ __forceinline__ uint64_t step(int v, int lane, int end) const {
    float x[kU][kE], y[kU][kE];
    Digits d;
    if (v * kE >= shift && (v + kStep) * kE - shift <= vocab && (!q || q_grid)) {
      const uint4* from = reinterpret_cast<const uint4*>(p + (v + lane) * kE - shift);
#pragma unroll
      for (int k = 0; k < kU; ++k) unpack(__ldg(from + 32 * k), x[k]);
      if (q) {
        from = reinterpret_cast<const uint4*>(q + (v + lane) * kE - shift);
#pragma unroll
        for (int k = 0; k < kU; ++k) unpack(__ldg(from + 32 * k), y[k]);
#pragma unroll
        for (int k = 0; k < kU; ++k)
#pragma unroll
          for (int i = 0; i < kE; ++i) d.add(x[k][i], y[k][i]);
      } else {
        const int at = hot - (v + lane) * kE + shift;
#pragma unroll
        for (int k = 0; k < kU; ++k)
#pragma unroll
          for (int i = 0; i < kE; ++i) d.add(x[k][i], at == 32 * kE * k + i ? 1.f : 0.f);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kU; ++k) load(min(v + lane + 32 * k, end - 1), x[k], y[k]);
#pragma unroll
      for (int k = 0; k < kU; ++k)
        if (v + lane + 32 * k < end) {
#pragma unroll
          for (int i = 0; i < kE; ++i) d.add(x[k][i], y[k][i]);
        }
    }
    return d.value();
  }
};


// Whether the lists are wrong, as far as thread t of n has looked: a few
// threads a sequence.
__device__ bool bad_lists(const VerifyArgs& a, int t, int n) {
  const moe_verify_config& c = a.c;
  const int per = max(1, n / c.n_seqs), sub = t % per;
  bool bad = false;
  for (int b = t / per; b < c.n_seqs && t < n / per * per; b += n / per) {
    const SeqRange r = seq_rows(a.cu_new, b, c.n_seqs, c.n_tokens, c.max_new);
    bad |= !r.ok;
    for (int j = 1 + sub; j < r.n; j += per) {
      const int x = a.tokens[r.row0 + j];
      bad |= x < 0 || x >= c.vocab;
    }
  }
  return bad;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs a, int parts) {
  __shared__ uint64_t warp_part[kWarps];
  __shared__ uint64_t slot_part[kWarps][32];  // a warp's sum, of 32 stretches of its segment
  __shared__ uint64_t block_part[2][kMaxParts];  // every block's sum, of each pass
  __shared__ int s_accepted;
  constexpr int kE = Residual<T>::kE;
  const moe_verify_config& c = a.c;
  const int part = (int)(blockIdx.x % parts), b = (int)(blockIdx.x / parts);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  ptx::cluster_arrive();  // the cluster's blocks have started before any is written to
  pdl_wait();
  pdl_trigger();
  const SeqRange r = seq_rows(a.cu_new, b, c.n_seqs, c.n_tokens, c.max_new);
  const T* p = static_cast<const T*>(a.p);
  const T* q = static_cast<const T*>(a.q);
  const int drafts = max(r.n - 1, 0);

  bool bad = false;
  if (warp == 0) {
    int acc = 0;
    for (int j0 = 0; j0 < drafts; j0 += 32) {
      const int j = j0 + lane;
      bool take = true;
      if (j < drafts) {
        const int x = a.tokens[r.row0 + j + 1];
        take = x >= 0 && x < c.vocab;
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
  } else if (blockIdx.x == 0) {
    bad = bad_lists(a, (int)threadIdx.x - 32, kThreads - 32);
  }
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = bad ? status_check() : MOE_OK;
  const int acc = s_accepted;
  if (part == 0) {
    if (threadIdx.x == 0) {
      a.n_accepted[b] = acc;
      if (a.kv_next) a.kv_next[b] = a.kv_len[b] - (drafts - acc);
    }
    for (int j = threadIdx.x; j < r.n; j += kThreads)
      if (j != acc) a.out_tokens[r.row0 + j] = j < acc ? a.tokens[r.row0 + j + 1] : -1;
  }
  __syncwarp();
  ptx::cluster_wait();
  if (r.n == 0) return;

  const int64_t row = r.row0 + acc;
  const bool rejected = acc < drafts;
  Residual<T> res(p + row * c.p_stride, rejected && q ? q + row * c.q_stride : nullptr,
                  rejected && !q ? a.tokens[row + 1] : -1, c.vocab);
  const float u = fminf(fmaxf(a.u_sample[b], 0.f), 0x1.fffffep-1f);
  // This warp's segment of the row: whole steps, the row's end aside.
  constexpr int kU = Residual<T>::kU, kStep = Residual<T>::kStep;
  const int nv = res.vectors(), segs = parts * kWarps, seg = part * kWarps + warp;
  const int row_steps = (nv + kStep - 1) / kStep;
  const int v0 = (int)((long long)row_steps * seg / segs) * kStep;
  const int v1 = min((int)((long long)row_steps * (seg + 1) / segs) * kStep, nv);
  const int per_slot = (max(v1 - v0, 0) + 32 * kStep - 1) / (32 * kStep);  // steps a stretch
  uint64_t total = 0, before = 0, mine = 0;
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t sum = 0, run = 0;
    slot_part[warp][lane] = 0;
    __syncwarp();
    for (int v = v0, step = 0; v < v1; v += kStep, ++step) {
      run += res.step(v, lane, v1);
      if ((step + 1) % per_slot && v + kStep < v1) continue;
      run = warp_sum_u64(run);
      if (lane == 0) slot_part[warp][step / per_slot] = run;
      sum += run;
      run = 0;
    }
    if (lane == 0) warp_part[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const uint64_t s = warp_sum_u64(lane < kWarps ? warp_part[lane] : 0ull);
      if (lane < parts)
        ptx::st_cluster_u64(ptx::mapa_shared(ptx::smem_addr(&block_part[pass][part]), lane), s);
    }
    ptx::cluster_sync();
    total = before = 0;
    for (int i = 0; i < parts; ++i) {
      const uint64_t s = block_part[pass][i];
      total += s;
      if (i < part) before += s;
    }
    for (int w = 0; w < warp; ++w) before += warp_part[w];
    mine = warp_part[warp];
    if (total > 0 || !rejected) break;
    // nowhere above the draft model: the target itself
    res = Residual<T>(p + row * c.p_stride, nullptr, -1, c.vocab);
    __syncthreads();
  }
  if (total == 0) {
    if (part == 0 && threadIdx.x == 0) a.out_tokens[row] = -1;
    return;
  }
  const uint64_t mark = __umul64hi(__float2ull_rz(u * 0x1p64f), total);
  if (mark < before || mark - before >= mine) return;
  // The segment holds the mark: the stretch that does, then the step (its
  // vectors again in flight all at once), then the vector and the element.
  __syncwarp();
  int first;
  {
    const uint64_t own = slot_part[warp][lane], upto = warp_scan_u64(own, lane);
    const int at = __ffs(__ballot_sync(0xffffffffu, before + upto > mark)) - 1;
    before += __shfl_sync(0xffffffffu, upto - own, at);
    first = v0 + at * per_slot * kStep;
  }
  for (int v = first; v < v1; v += kStep) {
    float x[kU][kE], y[kU][kE];
#pragma unroll
    for (int k = 0; k < kU; ++k) res.load(min(v + 32 * k + lane, v1 - 1), x[k], y[k]);
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      uint64_t e[kE], own = 0;  // running sums of this lane's vector
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        Digits d;
        d.add(x[k][i], y[k][i]);
        if (v + 32 * k + lane < v1) own += d.value();
        e[i] = own;
      }
      const uint64_t upto = warp_scan_u64(own, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, before + upto > mark);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          int n = 0;
#pragma unroll
          for (int i = 0; i < kE - 1; ++i) n += before + (upto - own) + e[i] <= mark;
          a.out_tokens[row] = (v + 32 * k + lane) * kE - res.shift + n;
        }
        return;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, cudaStream_t s) {
  static thread_local int device = -1, room[kMaxParts + 1];  // clusters that run at once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (device != dev) {
    e = cudaFuncSetAttribute(verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    for (int n = 1; n <= kMaxParts; ++n) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(n);
      cfg.blockDim = dim3(kThreads);
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim = {(unsigned)n, 1, 1};
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&room[n], verify_kernel<T>, &cfg);
      if (e != cudaSuccess) return e;
    }
    device = dev;
  }
  // Blocks a sequence: as many as let all sequences run at once, with a vector
  // for half their threads at least (64 sequences of 129280 tokens: 23 us by
  // 4, 18 by 8, 28 by 16; 200 of 50021: 28 by 1, 24 by 2, 27 by 3, of which
  // the GPU's parts hold a few clusters too few). Clusters between 8 and 16
  // leave parts of the GPU empty: 30 us by 9 where 8 take 24.
  const long long fed = ((long long)a.c.vocab * sizeof(T) / 16) / (kThreads / 2);
  int parts = kMaxParts;
  while (parts > 1 && (parts > fed || a.c.n_seqs > room[parts])) parts -= parts > 8 ? 8 : 1;
  return launch_pdl(verify_kernel<T>, dim3((unsigned)a.c.n_seqs * (unsigned)parts), dim3(kThreads),
                    0, s, parts, a, parts);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, cudaStream_t s) {
  if (a.c.n_seqs == 0) return launch_reset_status(a.status, s);
  ProfScope p(K_VERIFY, s);
  return a.c.dtype == MOE_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace moe
