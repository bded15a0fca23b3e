// Penalties, biases and masks on logits, temperature and softmax: one pass, one
// launch.
//
// A row of the vocabulary is a cluster of up to 16 blocks, each with a slice of it.
// A thread has up to 64 of the slice's logits in registers from the load to the store,
// so a row is read once and written once (96 bytes a thread spill). What a sequence's history does to a
// token is looked up by token: each block counts the history's tokens that fall
// into its slice in shared memory, one word a token, with integer additions, whose
// order does not matter; then the same words hold the slice's biases. The
// softmax needs the row's maximum and sum: each block takes its own sum relative
// to its own maximum, and the blocks exchange both at once through distributed
// shared memory. A vocabulary of more than 16 slices goes through its slices'
// tiles twice, once for maximum and sum and once more to write; its loops hold more than the
// registers do (fp32: 1.9 KB a thread spilled): 64 rows of 524288 take 286 us.
//
// One row of 32000 takes 6.7 us, the latency of its chain (row, sequence, history, maximum
// and sum, exchange). 161 rows of 129280 in fp32 with masks, biases and histories of up to
// 3000 take 75 us, 2.26 TB/s, 0.33 of a copy's rate: a block runs that chain once, 2800
// instructions a warp that nothing repeats, so that they wait for their fetch as much as for
// data, and clusters of eight find 225 of 304 slots. In bf16, with half the bytes and as many
// instructions, 59 us. Blocks of 128, 512 and 1024 threads took
// 78 to 89 us, 32 and 48 logits a thread (below) 78 and 123. One cluster more checks the
// lists meanwhile and writes the status.
#include <cfloat>

#include "rope_append.cuh"
#include "serve_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 16;
constexpr uint32_t kInPrompt = 1u << 31;    // of a token's word; below it: times generated

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
  // 16 bytes a load, eight in flight: one cluster reads every sequence's history
  auto wrong = [&](int token) { return (unsigned)token + 1 > (unsigned)c.vocab; };
  const int vecs = c.n_history / 4;
#pragma unroll 8
  for (int i = t; i < vecs; i += n) {
    const int4 x = __ldg(reinterpret_cast<const int4*>(a.history) + i);
    bad |= wrong(x.x) | wrong(x.y) | wrong(x.z) | wrong(x.w);
  }
  if (t < c.n_history % 4) bad |= wrong(__ldg(a.history + 4 * vecs + t));
  // A bias's token is above the one before it, but where a list starts.
  auto starts = [&](int i) {
    int lo = 0, hi = c.n_seqs;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (__ldg(a.cu_bias + mid) < i)
        lo = mid + 1;
      else
        hi = mid;
    }
    return __ldg(a.cu_bias + lo) == i;
  };
#pragma unroll 4
  for (int i = t; i < c.n_bias; i += n) {
    const int x = __ldg(a.bias_token + i), before = i > 0 ? __ldg(a.bias_token + i - 1) : -1;
    bad |= (unsigned)x >= (unsigned)c.vocab;
    if (before >= x) bad |= !starts(i);
  }
  for (int b = t; b < c.n_seqs; b += n) {
    bad |= !seq_rows(a.cu_new, b, c.n_seqs, c.n_tokens, c.max_new).ok;
    if (c.n_history) {
      const ListRange r = list_range(a.cu_history, b, c.n_seqs, c.n_history);
      bad |= !r.ok || a.n_prompt[b] < 0 || a.n_prompt[b] > r.hi - r.lo;
    }
    if (c.n_bias) bad |= !list_range(a.cu_bias, b, c.n_seqs, c.n_bias).ok;
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
struct alignas(16) Part {
  float top, sum;
  int at;
};

// A vector that lies partly in the row: its elements of the row, NaN elsewhere. Put together word
// by word: an array of elements that is read as one vector has the alignment of an element.
template <typename In>
__device__ __noinline__ uint4 load_edge(const In* row, int e, int V) {
  constexpr int kPer = 4 / (int)sizeof(In);  // elements a word
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int at = e + i * kPer + j;
      if (at < 0 || at >= V) continue;
      if (kPer == 1)
        w[i] = reinterpret_cast<const uint32_t*>(row)[at];
      else
        w[i] = (w[i] & ~(0xffffu << 16 * j)) | (uint32_t)reinterpret_cast<const uint16_t*>(row)[at] << 16 * j;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename Out>
__device__ __noinline__ void store_edge(Out* row, int e, int V, float4 y) {
  if (e >= 0 && e < V) row[e] = from_f32<Out>(y.x);
  if (e + 1 >= 0 && e + 1 < V) row[e + 1] = from_f32<Out>(y.y);
  if (e + 2 >= 0 && e + 2 < V) row[e + 2] = from_f32<Out>(y.z);
  if (e + 3 >= 0 && e + 3 < V) row[e + 3] = from_f32<Out>(y.w);
}

// kHeld: logits a thread holds. kTiles: a block has several tiles of logits and goes through them twice.
template <typename In, typename Out, int kHeld, bool kTiles>
__global__ void __launch_bounds__(kThreads, kHeld > 16 ? 2 : 4)
    logits_kernel(const LogitsArgs a, int part_bits, int tiles) {
  constexpr int kE = 16 / (int)sizeof(In), kV = kHeld / kE;
  constexpr int kTileVecs = kThreads * kV;
  extern __shared__ uint4 words4[];  // a word for each token of a tile
  uint32_t* words = reinterpret_cast<uint32_t*>(words4);
  __shared__ Part inbox[kMaxParts], of_warps[kWarps];
  __shared__ uint32_t masks[kThreads * kHeld / 32 + 2];
  const moe_logits_config& c = a.c;
  const int parts = 1 << part_bits, part = (int)blockIdx.x & (parts - 1);
  const int row = (int)(blockIdx.x >> part_bits) - 1;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, V = c.vocab;

  pdl_wait();
  pdl_trigger();
  // The cluster's blocks have started before any is written to; nothing to release yet.
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
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

  // This block's vectors v_begin .. v_end-1 of the row, on the row's 16-byte grid: vector v
  // is elements v kE - shift ...; only the row's first and last may lie partly outside.
  const In* x_row = static_cast<const In*>(a.logits) + row * c.logits_stride;
  Out* p_row = static_cast<Out*>(a.p) + row * c.p_stride;
  const int shift = (int)((uintptr_t)x_row % 16) / (int)sizeof(In);
  const bool out_grid = (uintptr_t)(p_row + kE - shift) % (kE * sizeof(Out) < 16 ? kE * sizeof(Out) : 16) == 0;
  const int vectors = (V + shift + kE - 1) / kE;  // at most 2^22 + 1, times 16
  const int v_begin = vectors * part >> part_bits, v_end = vectors * (part + 1) >> part_bits;
  const bool edges = v_begin * kE < shift || v_end * kE - shift > V;

  // Of a tile: this thread's vectors are k kThreads + threadIdx.x < n; element e0 + k kStep ..
  constexpr int kStep = kThreads * kE;
  const int t0 = (int)threadIdx.x;
  auto count_of = [&](int v0) { return min(kTileVecs, v_end - v0); };
  auto first_of = [&](int v0) { return (v0 + t0) * kE - shift; };
  auto whole = [&](int e) { return !edges || (e >= 0 && e + kE <= V); };

  uint4 raw[kV];
  auto load = [&](int v0) {
    const int n = count_of(v0), e0 = first_of(v0);
    const uint4* from = reinterpret_cast<const uint4*>(x_row + e0);
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      // outside the row NaN, which counts as -inf
      raw[k] = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
      if (k * kThreads + t0 < n && whole(e0 + k * kStep)) raw[k] = from[k * kThreads];
    }
    if (edges) {
#pragma unroll
      for (int k = 0; k < kV; ++k)
        if (k * kThreads + t0 < n && !whole(e0 + k * kStep)) raw[k] = load_edge(x_row, e0 + k * kStep, V);
    }
  };
  // The row's sequence is counted from the list where the threads hold it, in one round trip.
  const bool by_count = c.n_seqs <= 2 * kThreads;
  const int end0 = by_count && t0 < c.n_seqs ? __ldg(a.cu_new + t0 + 1) : 0x7fffffff;
  const int end1 = by_count && kThreads + t0 < c.n_seqs ? __ldg(a.cu_new + kThreads + t0 + 1) : 0x7fffffff;
  const int mask_row = a.mask_row ? __ldg(a.mask_row + row) : -1;
  load(v_begin);  // in flight meanwhile
  int b;
  if (by_count) {
    b = __syncthreads_count(end0 <= row);
    if (c.n_seqs > kThreads) b += __syncthreads_count(end1 <= row);
  } else {
    b = seq_of_row(a.cu_new, c.n_seqs, row, lane);
  }
  ListRange hist = {0, 0, false}, bias = {0, 0, false};
  int generated = 0;  // first entry of the history that was generated
  float rep = 1.f, pres = 0.f, freq = 0.f, temp = 1.f;
  const uint32_t* mask = nullptr;
  if (b >= c.n_seqs) {  // a row of no sequence, which the check records: left as it was
    ptx::cluster_wait();
    return;
  }
  const SeqRange sq = seq_rows(a.cu_new, b, c.n_seqs, c.n_tokens, c.max_new);
  if (a.repetition) rep = a.repetition[b];
  if (a.presence) pres = a.presence[b];
  if (a.frequency) freq = a.frequency[b];
  if (a.temperature) temp = a.temperature[b];
  if (c.n_history) {
    hist = list_range(a.cu_history, b, c.n_seqs, c.n_history);
    generated = hist.lo + clamp_int(a.n_prompt[b], 0, hist.hi - hist.lo);
  }
  if (c.n_bias) bias = list_range(a.cu_bias, b, c.n_seqs, c.n_bias);
  if (mask_row >= 0 && mask_row < c.n_masks) mask = a.mask + (int64_t)mask_row * ((V + 31) / 32);
  const int fed = a.tokens && row >= sq.row0 && row < sq.row0 + sq.n ? row + 1 - sq.row0 : 0;
  const bool counts = (rep != 1.f || pres != 0.f || freq != 0.f) && hist.hi - hist.lo + fed > 0;
  const bool biased = bias.hi > bias.lo;
  const bool greedy = temp == 0.f;
  const float inv_t = greedy ? 1.f : __fdiv_rn(1.f, temp), inv_rep = __fdiv_rn(1.f, rep);

  // The first entries of the history, in flight with the logits.
  constexpr int kAhead = 8;
  int ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    ahead[i] = -1;
    if (counts && hist.lo + i * kThreads + t0 < hist.hi) ahead[i] = __ldg(a.history + hist.lo + i * kThreads + t0);
  }

  // The mask's words of a tile, from that of its first element on (one before it, unused,
  // where the row starts inside its first vector).
  constexpr int kTile = kTileVecs * kE, kMaskAhead = (kTile / 32 + 2 + kThreads - 1) / kThreads;
  uint32_t mask_ahead[kMaskAhead];
  auto load_mask = [&](int v0) {
    const int first = (v0 * kE - shift) >> 5, last = min((v0 + max(0, count_of(v0))) * kE - shift, V) - 1 >> 5;
#pragma unroll
    for (int i = 0; i < kMaskAhead; ++i) {
      const int w = first + i * kThreads + t0;
      mask_ahead[i] = 0;
      if (mask && w >= 0 && w <= last) mask_ahead[i] = __ldg(mask + w);
    }
  };
  load_mask(v_begin);

  float x[kV][kE];
  // The tile's logits (loaded before) as the softmax takes them; -inf outside the row.
  auto take = [&](int v0) {
    const int n = count_of(v0), e0 = first_of(v0);
    const int base = v0 * kE - shift, n_words = max(0, n) * kE;
    if (counts || biased || mask) {
      __syncthreads();  // the words' last use
      if (counts || biased)
        for (int i = t0; i < n_words / 4; i += kThreads) words4[i] = make_uint4(0u, 0u, 0u, 0u);
      if (mask) {
#pragma unroll
        for (int i = 0; i < kMaskAhead; ++i)
          if (i * kThreads + t0 < kTile / 32 + 2) masks[i * kThreads + t0] = mask_ahead[i];
      }
      __syncthreads();
    }
    if (counts) {
      // (of a vector partly in the row the places outside have words too, and NaN as logits)
      auto count = [&](int token, bool prompt) {
        const unsigned at = (unsigned)token - (unsigned)base;
        if (at >= (unsigned)n_words) return;
        if (prompt)
          atomicOr(words + at, kInPrompt);
        else
          atomicAdd(words + at, 1u);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) count(ahead[i], hist.lo + i * kThreads + t0 < generated);
      // The rest of a long history, most of it 16 bytes a load: 64 sequences of up to 100 000
      // tokens take 147 us; with 4 bytes here and in the check of the lists 499.
      const int rest = hist.lo + kAhead * kThreads, v_first = (rest + 3) / 4, v_last = hist.hi / 4;
      if (rest + t0 < min(4 * v_first, hist.hi)) count(__ldg(a.history + rest + t0), rest + t0 < generated);
#pragma unroll 4
      for (int v = v_first + t0; v < v_last; v += kThreads) {
        const int4 h = __ldg(reinterpret_cast<const int4*>(a.history) + v);
        count(h.x, 4 * v < generated);
        count(h.y, 4 * v + 1 < generated);
        count(h.z, 4 * v + 2 < generated);
        count(h.w, 4 * v + 3 < generated);
      }
      const int last = 4 * max(v_first, v_last) + t0;
      if (last < hist.hi) count(__ldg(a.history + last), last < generated);
      for (int i = t0; i < fed; i += kThreads) count(a.tokens[sq.row0 + i], false);
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kV; ++k) unpack(raw[k], x[k]);
    if (counts) {
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const int at = k * kThreads + t0;
        if (at >= n) continue;
#pragma unroll
        for (int i = 0; i < kE; i += 4) {
          const uint4 w4 = words4[(at * kE + i) / 4];
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          if (!(w[0] | w[1] | w[2] | w[3])) continue;
          if (biased) words4[(at * kE + i) / 4] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float z = x[k][i + y] * (x[k][i + y] > 0.f ? inv_rep : rep);
            const uint32_t made = w[y] & ~kInPrompt;
            const float less = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)made)), pres);
            if (w[y]) x[k][i + y] = made ? less : z;
          }
        }
      }
    }
    if (biased) {
      if (counts) __syncthreads();
#pragma unroll 4
      for (int i = bias.lo + t0; i < bias.hi; i += kThreads) {
        const int token = __ldg(a.bias_token + i), at = token - base;
        if ((unsigned)at < (unsigned)n_words && (unsigned)token < (unsigned)V)
          words[at] = __float_as_uint(__ldg(a.bias + i));
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const int at = k * kThreads + t0;
        if (at >= n) continue;
#pragma unroll
        for (int i = 0; i < kE; i += 4) {
          const uint4 w = words4[(at * kE + i) / 4];
          x[k][i] += __uint_as_float(w.x), x[k][i + 1] += __uint_as_float(w.y);
          x[k][i + 2] += __uint_as_float(w.z), x[k][i + 3] += __uint_as_float(w.w);
        }
      }
    }
    if (mask) {
      // kStep is a multiple of 32: a thread's vectors start at the same bit of their words
      const int bit = e0 & 31;
      const uint32_t* from = masks + (e0 >> 5) - (base >> 5);
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        if (k * kThreads + t0 >= n) continue;
        const uint32_t bits = __funnelshift_r(from[k * (kStep / 32)], from[k * (kStep / 32) + 1], bit);
#pragma unroll
        for (int i = 0; i < kE; ++i)
          if (!(bits >> i & 1)) x[k][i] = -INFINITY;
      }
    }
#pragma unroll
    for (int k = 0; k < kV; ++k)
#pragma unroll
      for (int i = 0; i < kE; ++i) x[k][i] = fmaxf(x[k][i], -INFINITY);  // a NaN too
  };
  // Writes x times f.
  auto write = [&](int v0, float f) {
    const int n = count_of(v0), e0 = first_of(v0);
    const uint64_t by = ptx::f32x2(f, f), minus_zero = ptx::f32x2(-0.f, -0.f);
#pragma unroll
    for (int k = 0; k < kV; ++k)
#pragma unroll
      for (int i = 0; i < kE; i += 2) {
        const uint64_t y = ptx::fma_f32x2(ptx::f32x2(x[k][i], x[k][i + 1]), by, minus_zero);
        x[k][i] = ptx::f32x2_lo(y), x[k][i + 1] = ptx::f32x2_hi(y);
      }
#pragma unroll
    for (int k = 0; k < kV; ++k)
      if (k * kThreads + t0 < n && out_grid && whole(e0 + k * kStep)) store(p_row + e0 + k * kStep, x[k]);
    if (edges || !out_grid) {
#pragma unroll
      for (int k = 0; k < kV; ++k)
        if (k * kThreads + t0 < n && !(out_grid && whole(e0 + k * kStep))) {
#pragma unroll
          for (int i = 0; i < kE; i += 4)
            store_edge(p_row, e0 + k * kStep + i, V, make_float4(x[k][i], x[k][i + 1], x[k][i + 2], x[k][i + 3]));
        }
    }
  };

  if (c.out_logits) {
    for (int t = 0; t < (kTiles ? tiles : 1); ++t) {
      const int v0 = v_begin + t * kTileVecs;
      if (t > 0) load(v0), load_mask(v0);
      take(v0);
      write(v0, fminf(inv_t, FLT_MAX));  // a subnormal temperature's inverse is infinite, by which 0 is NaN
    }
    ptx::cluster_wait();
    return;
  }

  // exp(z / temperature) relative to `top`; equal values (infinities too) give 1
  const float scale = fminf(inv_t, 2.0e38f) * 1.4426950408889634f;
  auto weight = [&](float z, float top) { return z == top ? 1.f : ptx::ex2((z - top) * scale); };
  // The sum of x's weights relative to top (above -inf), x becoming them.
  auto weights = [&](float top) {
    if (top == INFINITY) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kV; ++k)
#pragma unroll
        for (int i = 0; i < kE; ++i) sum += x[k][i] = x[k][i] == INFINITY ? 1.f : 0.f;
      return sum;
    }
    const uint64_t minus = ptx::f32x2(-top, -top), by = ptx::f32x2(scale, scale);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < kV; ++k)
#pragma unroll
      for (int i = 0; i < kE; i += 2) {
        const uint64_t d =
            ptx::fma_f32x2(ptx::add_f32x2(ptx::f32x2(x[k][i], x[k][i + 1]), minus), by, 0ull);
        x[k][i] = ptx::ex2(ptx::f32x2_lo(d));
        x[k][i + 1] = ptx::ex2(ptx::f32x2_hi(d));
        sum[i / 2 % 2] = ptx::add_f32x2(sum[i / 2 % 2], ptx::f32x2(x[k][i], x[k][i + 1]));
      }
    sum[0] = ptx::add_f32x2(sum[0], sum[1]);
    return ptx::f32x2_lo(sum[0]) + ptx::f32x2_hi(sum[0]);
  };
  // Two parts of a row as one.
  auto join = [&](const Part& p, const Part& q) {
    Part r;
    r.top = fmaxf(p.top, q.top);
    r.sum = r.top == -INFINITY ? 0.f : p.sum * weight(p.top, r.top) + q.sum * weight(q.top, r.top);
    r.at = p.top == q.top ? min(p.at, q.at) : p.top > q.top ? p.at : q.at;
    return r;
  };
  // All lanes' parts as one, in an order that is the same each time.
  auto join_lanes = [&](Part p) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      Part q;
      q.top = __shfl_xor_sync(0xffffffffu, p.top, o);
      q.sum = __shfl_xor_sync(0xffffffffu, p.sum, o);
      q.at = __shfl_xor_sync(0xffffffffu, p.at, o);
      p = lane & o ? join(q, p) : join(p, q);
    }
    return p;
  };
  constexpr int kNowhere = 0x7fffffff;

  // A warp's largest, and sum relative to it; x becomes the weights.
  Part mine = {-INFINITY, 0.f, kNowhere};
  for (int t = 0; t < (kTiles ? tiles : 1); ++t) {
    const int v0 = v_begin + t * kTileVecs;
    if (t > 0) load(v0), load_mask(v0);
    take(v0);
    Part p = {-INFINITY, 0.f, kNowhere};
#pragma unroll
    for (int k = 0; k < kV; ++k)
#pragma unroll
      for (int i = 0; i < kE; ++i) p.top = fmaxf(p.top, x[k][i]);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) p.top = fmaxf(p.top, __shfl_xor_sync(0xffffffffu, p.top, o));
    if (p.top > -INFINITY) {
      if (greedy) {
        const int e0 = first_of(v0);
#pragma unroll
        for (int k = kV - 1; k >= 0; --k)
#pragma unroll
          for (int i = kE - 1; i >= 0; --i)
            if (x[k][i] == p.top) p.at = e0 + k * kStep + i;  // the lane's lowest
        p.at = __reduce_min_sync(0xffffffffu, p.at);
      } else {
        p.sum = warp_sum(weights(p.top));
      }
    }
    mine = kTiles ? join(mine, p) : p;
  }
  // The block's warps, then the cluster's blocks.
  if (lane == 0) of_warps[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const Part p = join_lanes(lane < kWarps ? of_warps[lane] : Part{-INFINITY, 0.f, kNowhere});
    ptx::cluster_wait();
    if (lane < parts) {
      const uint32_t to = ptx::mapa_shared(ptx::smem_addr(&inbox[part]), lane);
      ptx::st_cluster_v2(to, p.top, p.sum);
      ptx::st_cluster_v2(to + 8, __int_as_float(p.at), 0.f);
    }
    __syncwarp();
  } else {
    ptx::cluster_wait();
  }
  ptx::cluster_sync();
  const Part all = join_lanes(lane < parts ? inbox[lane] : Part{-INFINITY, 0.f, kNowhere});
  const bool none = all.top == -INFINITY;
  const float f = none ? 0.f : __fdiv_rn(1.f, all.sum);
  for (int t = 0; t < (kTiles ? tiles : 1); ++t) {
    const int v0 = v_begin + t * kTileVecs;
    float own = f;
    if (greedy) {
      const int e0 = first_of(v0);
#pragma unroll
      for (int k = 0; k < kV; ++k)
#pragma unroll
        for (int i = 0; i < kE; ++i) x[k][i] = e0 + k * kStep + i == all.at ? 1.f : 0.f;
      own = 1.f;
    } else if (none || (!kTiles && mine.top == -INFINITY)) {
#pragma unroll
      for (int k = 0; k < kV; ++k)
#pragma unroll
        for (int i = 0; i < kE; ++i) x[k][i] = 0.f;
    } else if (kTiles) {
      load(v0);
      load_mask(v0);
      take(v0);
      weights(all.top);
    } else {
      own = f * weight(mine.top, all.top);  // x is relative to this warp's largest
    }
    write(v0, own);
  }
}

template <typename In, typename Out, int kHeld, bool kTiles>
cudaError_t launch_one(const LogitsArgs& a, int part_bits, int tiles, int smem, cudaStream_t s) {
  static thread_local int configured = -1;
  const auto kernel = logits_kernel<In, Out, kHeld, kTiles>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured != dev) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kThreads * kHeld * 4);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured = dev;
  }
  ProfScope p(K_LOGITS, s);
  return launch_pdl(kernel, dim3((unsigned)(a.c.n_tokens + 1) << part_bits), dim3(kThreads), (size_t)smem, s,
                    1 << part_bits, a, part_bits, tiles);
}

template <typename In, typename Out>
cudaError_t launch(const LogitsArgs& a, cudaStream_t s) {
  constexpr int kE = 16 / (int)sizeof(In);
  // of the row that starts latest on its grid
  const int vectors = ceil_div(a.c.vocab + (a.c.logits_stride % kE ? kE - 1 : 0), kE);
  // 64 logits a thread (two blocks an SM) for the batch: 75 us for 161 rows of 129280, with
  // 32 (four blocks) 78, with 48 (rows in 16 blocks) 123. 16 (four blocks) where those
  // leave the GPU unfilled and 16 blocks hold a row: 1, 16 and 64 rows of 32000 take 6.8,
  // 7.5 and 9.6 us, with 64 logits a thread 7.7, 8.8 and 11.0.
  constexpr int kMany = 64, kFew = 16;
  auto tile = [](int held) { return kThreads * (held / kE); };
  auto blocks = [&](int held) {
    int bits = 0;
    while ((1 << bits) < kMaxParts && ceil_div(vectors, 1 << bits) > tile(held)) ++bits;
    return bits;
  };
  const int held = ((long long)a.c.n_tokens << blocks(kMany)) <= 2 * num_sms() &&
                           vectors <= kMaxParts * tile(kFew)
                       ? kFew
                       : kMany;
  // Blocks a row: as many as its registers need, and more while the GPU has slots for
  // them and every thread a vector.
  int bits = blocks(held);
  while ((1 << bits) < kMaxParts &&
         ((long long)a.c.n_tokens << bits) * 2 <= (held == kFew ? 4 : 2) * num_sms() &&
         vectors >> (bits + 1) >= kThreads)
    ++bits;
  const int slice = ceil_div(vectors, 1 << bits), tiles = ceil_div(slice, tile(held));
  const int smem = a.c.n_history || a.c.n_bias || a.tokens ? (tiles > 1 ? tile(held) : slice) * kE * 4 : 0;
  if (held == kFew) return launch_one<In, Out, kFew, false>(a, bits, tiles, smem, s);
  if (tiles == 1) return launch_one<In, Out, kMany, false>(a, bits, tiles, smem, s);
  return launch_one<In, Out, kMany, true>(a, bits, tiles, smem, s);
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
