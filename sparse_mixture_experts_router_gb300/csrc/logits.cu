// Penalties, biases and masks on logits, temperature and softmax: one pass, one
// launch.
//
// A row of the vocabulary is a cluster of up to 16 blocks, each with a slice of it.
// A thread has 32 of the slice's logits in registers from the load to the store,
// so a row is read once and written once. What a sequence's history does to a
// token is looked up by token: each block counts the history's tokens that fall
// into its slice in shared memory, one word a token, with integer additions, whose
// order does not matter; then the same words hold the slice's biases. The
// softmax needs the row's maximum and sum: each block takes its own sum relative
// to its own maximum, and the blocks exchange both at once through distributed
// shared memory. A vocabulary of more than 16 slices goes through its slices'
// tiles twice, once for maximum and sum and once more to write.
//
// Bound by memory for many rows; for one, by the latency of its chain (row,
// sequence, history, exchange). One cluster more checks the lists meanwhile and
// writes the status.
#include <cfloat>

#include "rope_append.cuh"
#include "serve_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 32;                  // logits a thread holds
constexpr int kTile = kThreads * kHeld;    // of a block
constexpr int kMaxParts = 16;
constexpr uint32_t kInPrompt = 1u << 31;   // of a token's word; below it: times generated

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
__device__ __forceinline__ void store(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store(float* p, const float (&x)[8]) { store8(p, x); }
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]));
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) { store8(p, x); }

// Entries lo .. hi-1 of b's list of n, clamped; ok: nothing had to be.
struct ListRange {
  int lo, hi;
  bool ok;
};
__device__ __forceinline__ ListRange list_range(const int32_t* cu, int b, int n_seqs, int n) {
  const int lo = cu[b], hi = cu[b + 1];
  ListRange r;
  r.ok = lo >= 0 && hi >= lo && hi <= n && (b > 0 || lo == 0) && (b < n_seqs - 1 || hi == n);
  r.lo = clamp_int(lo, 0, n);
  r.hi = clamp_int(hi, r.lo, n);
  return r;
}

// Whether the lists are wrong, as far as thread t of n has looked.
__device__ bool bad_lists(const LogitsArgs& a, int t, int n) {
  const moe_logits_config& c = a.c;
  bool bad = false;
  for (int i = t; i < c.n_tokens; i += n) {
    if (a.tokens) bad |= (unsigned)a.tokens[i] >= (unsigned)c.vocab;
    if (a.mask_row) bad |= a.mask_row[i] < -1 || a.mask_row[i] >= c.n_masks;
  }
#pragma unroll 4
  for (int i = t; i < c.n_history; i += n) bad |= (unsigned)__ldg(a.history + i) >= (unsigned)c.vocab;
  const int per = max(1, n / max(1, c.n_seqs)), sub = t % per;
  for (int b = t / per; b < c.n_seqs && t < n / per * per; b += n / per) {
    bad |= !seq_rows(a.cu_new, b, c.n_seqs, c.n_tokens, c.max_new).ok;
    if (c.n_history) {
      const ListRange r = list_range(a.cu_history, b, c.n_seqs, c.n_history);
      bad |= !r.ok || a.n_prompt[b] < 0 || a.n_prompt[b] > r.hi - r.lo;
    }
    if (c.n_bias) {
      const ListRange r = list_range(a.cu_bias, b, c.n_seqs, c.n_bias);
      bad |= !r.ok;
      for (int i = r.lo + sub; i < r.hi; i += per) {
        const int x = a.bias_token[i];
        bad |= (unsigned)x >= (unsigned)c.vocab || (i > r.lo && a.bias_token[i - 1] >= x);
      }
    }
    // written so that a NaN is bad
    if (a.repetition) bad |= !(a.repetition[b] > 0.f && a.repetition[b] <= FLT_MAX);
    if (a.presence) bad |= !(fabsf(a.presence[b]) <= FLT_MAX);
    if (a.frequency) bad |= !(fabsf(a.frequency[b]) <= FLT_MAX);
    if (a.temperature) bad |= !(a.temperature[b] >= 0.f && a.temperature[b] <= FLT_MAX);
  }
  return bad;
}

// A block's largest x, the sum of exp of the others relative to it, and the lowest
// index that has it.
struct Part {
  float top, sum;
  int at;
  int pad;
};

template <typename In, typename Out>
__global__ void __launch_bounds__(kThreads, 2) logits_kernel(const LogitsArgs a, int parts, int tiles) {
  constexpr int kE = 16 / (int)sizeof(In), kV = kHeld / kE;
  extern __shared__ uint4 words4[];  // a word for each token of a tile
  uint32_t* words = reinterpret_cast<uint32_t*>(words4);
  __shared__ Part inbox[kMaxParts];
  __shared__ float warp_f[kWarps];
  __shared__ int warp_i[kWarps];
  const moe_logits_config& c = a.c;
  const int part = (int)blockIdx.x % parts, row = (int)blockIdx.x / parts - 1;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, V = c.vocab;

  pdl_wait();
  pdl_trigger();
  ptx::cluster_arrive();  // the cluster's blocks have started before any is written to
  if (row < 0) {
    const bool bad = __syncthreads_or(bad_lists(a, part * kThreads + threadIdx.x, parts * kThreads));
    ptx::cluster_wait();
    if (threadIdx.x == 0)
      ptx::st_cluster_u64(ptx::mapa_shared(ptx::smem_addr(&inbox[part]), 0), bad);
    __syncwarp();
    ptx::cluster_sync();
    if (part == 0 && threadIdx.x == 0) {
      bool any = false;
      for (int i = 0; i < parts; ++i) any |= *reinterpret_cast<volatile uint64_t*>(&inbox[i]) != 0;
      *a.status = any ? status_check() : MOE_OK;
    }
    return;
  }

  // This block's vectors of the row, on the row's 16-byte grid: vector v is elements
  // v kE - shift ...
  const In* x_row = static_cast<const In*>(a.logits) + row * c.logits_stride;
  Out* p_row = static_cast<Out*>(a.p) + row * c.p_stride;
  const int shift = (int)((uintptr_t)x_row % 16) / (int)sizeof(In);
  const bool out_grid = (uintptr_t)(p_row + kE - shift) % (kE * sizeof(Out) < 16 ? kE * sizeof(Out) : 16) == 0;
  const int vectors = (V + shift + kE - 1) / kE;
  const int v_begin = (int)((long long)vectors * part / parts);
  const int v_end = (int)((long long)vectors * (part + 1) / parts);
  constexpr int kTileVecs = kTile / kE;

  // Its sequence and what that asks for.
  const int b = seq_of_row(a.cu_new, c.n_seqs, row, lane);
  SeqRange sq = {0, 0, 0, false};
  ListRange hist = {0, 0, false}, bias = {0, 0, false};
  int generated = 0;  // first entry of the history that was generated
  float rep = 1.f, pres = 0.f, freq = 0.f, temp = 1.f;
  const uint32_t* mask = nullptr;
  if (b < c.n_seqs) {
    sq = seq_rows(a.cu_new, b, c.n_seqs, c.n_tokens, c.max_new);
    if (a.repetition) rep = a.repetition[b];
    if (a.presence) pres = a.presence[b];
    if (a.frequency) freq = a.frequency[b];
    if (a.temperature) temp = a.temperature[b];
    if (c.n_history) {
      hist = list_range(a.cu_history, b, c.n_seqs, c.n_history);
      generated = hist.lo + clamp_int(a.n_prompt[b], 0, hist.hi - hist.lo);
    }
    if (c.n_bias) bias = list_range(a.cu_bias, b, c.n_seqs, c.n_bias);
  }
  if (a.mask_row) {
    const int m = a.mask_row[row];
    if (m >= 0 && m < c.n_masks) mask = a.mask + (int64_t)m * ((V + 31) / 32);
  }
  const int fed = a.tokens && row >= sq.row0 && row < sq.row0 + sq.n ? row + 1 - sq.row0 : 0;
  const bool counts = (rep != 1.f || pres != 0.f || freq != 0.f) && hist.hi - hist.lo + fed > 0;
  const bool biased = bias.hi > bias.lo;
  const bool greedy = temp == 0.f;
  const float inv_t = greedy ? 1.f : __fdiv_rn(1.f, temp);

  float x[kV][kE];
  // The tile's logits as the softmax takes them; -inf outside the row.
  auto take = [&](int v0) {
    const int v1 = max(v0, min(v0 + kTileVecs, v_end)), base = v0 * kE - shift;
    uint4 raw[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const int v = v0 + k * kThreads + threadIdx.x, e = v * kE - shift;
      if (v < v1 && e >= 0 && e + kE <= V) raw[k] = *reinterpret_cast<const uint4*>(x_row + e);
    }
    const int n_words = (v1 - v0) * kE;
    if (counts || biased) {
      __syncthreads();  // the words' last use
      for (int i = threadIdx.x; i < n_words / 4; i += kThreads) words4[i] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
    }
    if (counts) {
      auto count = [&](int token, bool prompt) {
        const int at = token - base;
        if ((unsigned)at >= (unsigned)n_words || (unsigned)token >= (unsigned)V) return;
        if (prompt)
          atomicOr(words + at, kInPrompt);
        else
          atomicAdd(words + at, 1u);
      };
#pragma unroll 4
      for (int i = hist.lo + threadIdx.x; i < hist.hi; i += kThreads)
        count(__ldg(a.history + i), i < generated);
      for (int i = threadIdx.x; i < fed; i += kThreads) count(a.tokens[sq.row0 + i], false);
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const int at = k * kThreads + threadIdx.x, v = v0 + at, e = v * kE - shift;
      if (v < v1 && e >= 0 && e + kE <= V) {
        unpack(raw[k], x[k]);
      } else {
#pragma unroll
        for (int i = 0; i < kE; ++i)
          x[k][i] = v < v1 && e + i >= 0 && e + i < V ? to_f32(x_row[e + i]) : -INFINITY;
      }
      if (counts && v < v1) {
#pragma unroll
        for (int i = 0; i < kE; i += 4) {
          const uint4 w4 = words4[(at * kE + i) / 4];
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          if (!(w[0] | w[1] | w[2] | w[3])) continue;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            if (!w[y]) continue;
            float z = x[k][i + y];
            z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
            const uint32_t n = w[y] & ~kInPrompt;
            if (n) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)n)), pres);
            x[k][i + y] = z;
          }
        }
      }
    }
    if (biased) {
      if (counts) {
        __syncthreads();
        for (int i = threadIdx.x; i < n_words / 4; i += kThreads) words4[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
      }
      for (int i = bias.lo + threadIdx.x; i < bias.hi; i += kThreads) {
        const int token = a.bias_token[i], at = token - base;
        if ((unsigned)at < (unsigned)n_words && (unsigned)token < (unsigned)V)
          words[at] = __float_as_uint(a.bias[i]);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const int at = k * kThreads + threadIdx.x;
        if (v0 + at >= v1) continue;
#pragma unroll
        for (int i = 0; i < kE; i += 4) {
          const uint4 w = words4[(at * kE + i) / 4];
          x[k][i] += __uint_as_float(w.x), x[k][i + 1] += __uint_as_float(w.y);
          x[k][i + 2] += __uint_as_float(w.z), x[k][i + 3] += __uint_as_float(w.w);
        }
      }
    }
    if (mask) {
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const int v = v0 + k * kThreads + threadIdx.x, e = v * kE - shift;
        if (v >= v1) continue;
        const int first = max(e, 0), last = min(e + kE, V) - 1;  // first <= last
        const uint32_t lo = __ldg(mask + first / 32), hi = __ldg(mask + last / 32);
        // bit i: element e + i
        const uint32_t bits = first / 32 == last / 32
                                  ? (e >= 0 ? lo >> (e % 32) : lo << -e)
                                  : __funnelshift_r(lo, hi, (uint32_t)(e % 32));
#pragma unroll
        for (int i = 0; i < kE; ++i)
          if (!(bits >> i & 1)) x[k][i] = -INFINITY;
      }
    }
#pragma unroll
    for (int k = 0; k < kV; ++k)
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (x[k][i] != x[k][i]) x[k][i] = -INFINITY;
  };
  auto write = [&](int v0, auto value) {
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const int v = v0 + k * kThreads + threadIdx.x, e = v * kE - shift;
      if (v >= min(v0 + kTileVecs, v_end)) continue;
      float y[kE];
#pragma unroll
      for (int i = 0; i < kE; ++i) y[i] = value(x[k][i], e + i);
      if (out_grid && e >= 0 && e + kE <= V) {
        store(p_row + e, y);
      } else {
#pragma unroll
        for (int i = 0; i < kE; ++i)
          if (e + i >= 0 && e + i < V) p_row[e + i] = from_f32<Out>(y[i]);
      }
    }
  };

  if (c.out_logits) {
    for (int t = 0; t < tiles; ++t) {
      const int v0 = v_begin + t * kTileVecs;
      take(v0);
      write(v0, [&](float z, int) { return z * inv_t; });
    }
    ptx::cluster_wait();
    return;
  }

  // exp relative to `top`; equal values (infinities too) give 1
  auto weight = [&](float z, float top) {
    return z == top ? 1.f : expf(__fmul_rn(z - top, inv_t));
  };
  Part mine = {-INFINITY, 0.f, 0x7fffffff, 0};
  for (int t = 0; t < tiles; ++t) {
    const int v0 = v_begin + t * kTileVecs;
    take(v0);
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kV; ++k)
#pragma unroll
      for (int i = 0; i < kE; ++i) top = fmaxf(top, x[k][i]);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncthreads();  // the warps' values of the tile before have been read
    if (lane == 0) warp_f[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_f[w]);
    if (top == -INFINITY) continue;  // the same for the whole block
    float sum = 0.f;
    int at = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kV; ++k)
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        if (greedy) {
          if (x[k][i] == top)
            at = min(at, (v0 + k * kThreads + (int)threadIdx.x) * kE - shift + i);
        } else if (tiles == 1) {
          x[k][i] = weight(x[k][i], top);
          sum += x[k][i];
        } else {
          sum += weight(x[k][i], top);
        }
      }
    sum = warp_sum(sum);
    if (greedy) at = __reduce_min_sync(0xffffffffu, at);
    __syncthreads();
    if (lane == 0) warp_f[warp] = sum, warp_i[warp] = at;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += warp_f[w];
      at = min(at, warp_i[w]);
    }
    if (top > mine.top) {
      mine.sum = mine.top == -INFINITY ? sum : mine.sum * weight(mine.top, top) + sum;
      mine.top = top;
      mine.at = at;
    } else {
      mine.sum += sum * weight(top, mine.top);
    }
  }
  ptx::cluster_wait();
  if (threadIdx.x < parts) {
    const uint32_t to = ptx::mapa_shared(ptx::smem_addr(&inbox[part]), threadIdx.x);
    ptx::st_cluster_v2(to, mine.top, mine.sum);
    ptx::st_cluster_v2(to + 8, __int_as_float(mine.at), 0.f);
  }
  __syncwarp();
  ptx::cluster_sync();
  float top = -INFINITY, sum = 0.f;
  int at = 0x7fffffff;
  for (int i = 0; i < parts; ++i) top = fmaxf(top, inbox[i].top);
  for (int i = 0; i < parts; ++i) {
    if (inbox[i].top > -INFINITY) sum += inbox[i].sum * weight(inbox[i].top, top);
    if (inbox[i].top == top) at = min(at, inbox[i].at);
  }
  const bool none = top == -INFINITY;
  const float f = none ? 0.f : __fdiv_rn(1.f, sum);
  if (tiles == 1 && !greedy) {
    // x is relative to this block's maximum
    const float own = mine.top == -INFINITY ? 0.f : f * weight(mine.top, top);
    write(v_begin, [&](float w, int) { return own == 0.f ? 0.f : w * own; });
    return;
  }
  for (int t = 0; t < tiles; ++t) {
    const int v0 = v_begin + t * kTileVecs;
    if (tiles > 1 && !greedy) take(v0);
    write(v0, [&](float z, int e) {
      if (greedy) return !none && e == at ? 1.f : 0.f;
      return none ? 0.f : weight(z, top) * f;
    });
  }
}

template <typename In, typename Out>
cudaError_t launch(const LogitsArgs& a, cudaStream_t s) {
  static thread_local int configured = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured != dev) {
    e = cudaFuncSetAttribute(logits_kernel<In, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTile * 4);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(logits_kernel<In, Out>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured = dev;
  }
  // Blocks a row: as many as a block's registers need, and more while the GPU has
  // slots for them (two blocks an SM) and every thread a vector.
  constexpr int kE = 16 / (int)sizeof(In);
  const int vectors = a.c.vocab / kE + 2;  // at most, wherever a row starts
  int parts = 1;
  while (parts < kMaxParts &&
         (ceil_div(vectors, parts) > kTile / kE ||
          ((long long)a.c.n_tokens * 2 * parts <= 2LL * num_sms() && vectors / (2 * parts) >= kThreads)))
    parts *= 2;
  const int slice = (int)ceil_div(vectors, parts), tiles = (int)ceil_div(slice, kTile / kE);
  const int smem = a.c.n_history || a.c.n_bias || a.tokens ? (tiles > 1 ? kTile : slice * kE) * 4 : 0;
  ProfScope p(K_LOGITS, s);
  return launch_pdl(logits_kernel<In, Out>, dim3((unsigned)(a.c.n_tokens + 1) * (unsigned)parts), dim3(kThreads),
                    (size_t)smem, s, parts, a, parts, tiles);
}

}  // namespace

cudaError_t launch_logits(const LogitsArgs& a, cudaStream_t s) {
  if (a.c.n_tokens == 0) return launch_reset_status(a.status, s);
  if (a.c.dtype == MOE_F32)
    return a.c.out_dtype == MOE_F32 ? launch<float, float>(a, s) : launch<float, __nv_bfloat16>(a, s);
  return a.c.out_dtype == MOE_F32 ? launch<__nv_bfloat16, float>(a, s)
                                  : launch<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace moe
