// Attention of the new tokens over a paged bf16 or E4M3 cache, on warp-level
// matrix products.
//
// The work is memory-bound: each cached key and value meets only the rows of
// one head group (R = new tokens x heads per key-value head, 8 for an 8-way
// shared head), R multiply-adds an element. So the kernel is a stream of the
// cache through shared memory, and everything else is arranged to stay out of
// that stream's way:
//  - A block of 4 warps (6 for heads above 128) holds one (sequence, key-value
//    head, up to 16 query rows) item, or one of the C parts that its keys are
//    cut into: the parts are a thread-block cluster and join through its
//    distributed shared memory, so one launch and no scratch in global memory.
//  - Each warp streams its own tiles (8 KB: 16 keys of 128 bf16 elements, 32 of
//    E4M3 or of 64 bf16) through its own ring of stages with cp.async and no
//    block-wide synchronisation; the pages of the tile after next are looked up
//    one step ahead.
//  - The products are taken transposed, S^T = K Q^T and O^T = V^T P^T: keys
//    and head elements fill the 16 rows of an m16n8k16 product and query rows
//    its 8 columns, so 8 query rows waste nothing, K and V are read from
//    shared memory once for all rows, and P^T reaches the second product's
//    operand layout by a register transpose (movmatrix).
//  - The running maximum is only raised when a score passes it by more than
//    2^8 (log2 units: 8): until then weights up to 2^8 stand, which costs no
//    precision (fp32 sums; bf16 and fp16 weights keep their relative step)
//    and spares the reduction across lanes and the scaling of O.
// Rounding: scores, maxima, sums and O are fp32. The weights p are rounded to
// the type of the second product: bf16 twice (p = hi + lo, 2^-16 of p, two
// products) for a bf16 cache, whose error one rounding would double; for an E4M3
// cache once, times the value's scale, to fp16 (2^-11). The largest of those is
// kept between 2^7 and 2^15, so that they have fp16's precision down to 2^-21 of
// it and none is off by more than 2^-32 of it, however many keys a row has. The sum
// of weights, which has no scales in it, is relative to the same maximum while the
// scales allow it (from about 2^-53 to 2^80), else to one of its own. E4M3
// elements are exact in fp16. Queries become fp16 too, each row scaled by a power
// of two so that its largest element is at least 2^14: elements down to 2^-31 of
// that are exact, those below it off by 2^-39 of it at most. Scores by E4M3
// products, with queries as sums of two E4M3 terms, took 108 us where these take
// 101 (256 sequences of 1 to 2047 keys, 8 rows). The scales of keys multiply
// scores, those of values multiply weights.
#pragma once
#include <type_traits>

#include "paged_attention.cuh"

namespace moe {
namespace attn {

// Warps of a block: four, three blocks an SM; heads above 128 fill an SM's
// shared memory with one block of six.
constexpr int warps_of(int dim) { return dim > 128 ? 6 : 4; }

template <int kDim, bool kF8>
struct Tile {
  static constexpr int kKeys = keys_of(kDim, kF8);
  static constexpr int kRow = kDim * (kF8 ? 1 : 2);  // bytes of a key in shared memory
  static constexpr int kChunks = kRow / 16;
  static constexpr int kBytes = kKeys * kRow;        // one of K, V
  static constexpr int kStage = 2 * kBytes + (kF8 ? 2 * kKeys * 4 : 0);
  // Stages a warp. Two where that lets three blocks share an SM and not two:
  // more warps hide more than more bytes in flight do (the batch of 64 uneven
  // sequences 175 -> 173 us, 256 short ones in E4M3 130 -> 116 us; four
  // stages, one block an SM: 268 and 221 us).
  static constexpr int kStages = kStage >= 8192 ? 2 : 4;
  // Byte offset of 16-byte chunk c of key k: chunk c of the 8 keys that one
  // matrix load takes falls into 8 different bank groups. Those are 8
  // consecutive keys, and of E4M3 keys also the 8 of 16 that agree in bit 1
  // (see key_of).
  static __host__ __device__ constexpr uint32_t at(int k, int c) {
    if (!kF8) return (uint32_t)(k * kRow + ((c ^ (k & 7)) << 4));
    const int mixed = (k & 5) | (((k >> 1) ^ (k >> 3)) & 1) << 1;
    return (uint32_t)(k * kRow + ((c ^ (kChunks >= 8 ? mixed : mixed >> 1)) << 4));
  }
  // at() is linear over exclusive or, and stages start on multiples of 256
  // bytes (bf16: 1024): one lane's addresses differ by a constant exclusive
  // or (chunks, kChunkBit) or by a constant and one (keys), which is all that
  // a copy or a matrix load then computes.
  static constexpr uint32_t kChunkBit = 16;
  static constexpr uint32_t key_xor(int k) { return at(k, 0) - (uint32_t)(k * kRow); }
  // Row r (0..15) of a score product is this key of its 16. The byte-wise
  // transposed load of values gives a lane 4 consecutive keys, and the second
  // product pairs them with the weights' rows (2q, 2q+1, 2q+8, 2q+9).
  static __host__ __device__ constexpr int key_of(int r) {
    return kF8 ? (r % 8 / 2) * 4 + r / 8 * 2 + r % 2 : r;
  }
};

// Shared memory after the rings, and how the variants differ.
template <int kDim, int kNT, bool kF8>
struct Layout {
  using T = Tile<kDim, kF8>;
  static constexpr int kWarps = warps_of(kDim), kThreads = kWarps * 32, kRows = 8 * kNT;
  // Queries in shared memory where they would take 32 registers a thread and
  // more, which costs more than their reads. 16 rows, 64 sequences of 100 to 4000
  // keys, in registers and in shared memory: bf16 101 and 98 us, E4M3 85 and 81,
  // bf16 heads of 64 61 and 56; 32 sequences, heads of 256, E4M3 (the registers
  // spill) 48 and 38.
  static constexpr bool kSharedQ = kNT >= 2;
  static constexpr int kQRow = kDim * 2 + 16;  // bytes; 16 against bank conflicts
  static constexpr bool kOwnInbox = kNT == 1;  // the others' would cost the third block
  static constexpr int kRing = kWarps * T::kStages * T::kStage;
  static constexpr int kInbox = kOwnInbox ? (int)sizeof(Inbox<kRows, kDim, kF8>) : 0;
  static constexpr int kStat = (kF8 ? 3 : 2) * (kWarps + 1) * kRows * 4;
  static constexpr int kRange = kRows * 8;   // last and first position of a row
  static constexpr int kFactor = kRows * 4;  // of a row's scores
  static constexpr int kQ = kSharedQ ? kRows * kQRow : 0;
  static constexpr int kAll = kRing + kInbox + kStat + kRange + kFactor + kQ;
};

// Two E4M3 codes (the low 16 bits of v) as fp16.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int kDim, int kNT, bool kF8>
__global__ void __launch_bounds__(warps_of(kDim) * 32, blocks_per_sm(kDim))
    mma_kernel(const __grid_constant__ Params prm) {
  using T = Tile<kDim, kF8>;
  using L = Layout<kDim, kNT, kF8>;
  constexpr int kS = T::kStages, kMT = T::kKeys / 16, kDT = kDim / 16;
  constexpr int kRows = L::kRows, kWarps = L::kWarps, kThreads = L::kThreads;
  // Scores as two chains of products, where few warps an SM leave one chain's
  // latency uncovered. Heads of 256, 32 sequences of 100 to 4000 keys, one chain
  // and two: bf16 8 rows 34.4 and 33.9 us, E4M3 16 rows 39.3 and 38.2; smaller
  // heads have more warps: E4M3 heads of 128 81.5 and 83.1, bf16 of 64 56.5 and
  // 57.3 (64 sequences, 16 rows).
  constexpr bool kTwoSums = kDim > 128;
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnArgs& a = prm.a;
  const moe_attn_config& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, quad = lane % 4, oct = lane / 4;
  auto* inbox = reinterpret_cast<Inbox<kRows, kDim, kF8>*>(
      L::kOwnInbox ? smem + L::kRing : smem + kS * T::kStage);
  uint8_t* rest = smem + L::kRing + L::kInbox;
  float* stat = reinterpret_cast<float*>(rest);  // m, l of each warp's rows; E4M3: l's reference
  float* joined = stat + (kF8 ? 3 : 2) * kWarps * kRows;  // l's reference and l of the block's rows; E4M3: m
  float* l_ref = stat + (2 * kWarps + warp) * kRows;      // (E4M3) this warp's
  int2* range = reinterpret_cast<int2*>(rest + L::kStat);
  float* factor = reinterpret_cast<float*>(rest + L::kStat + L::kRange);
  uint8_t* qs = rest + L::kStat + L::kRange + L::kFactor;

  pdl_wait();
  pdl_trigger();
  Item it;
  if (!item_of<kThreads>(prm, kRows, it)) return;
  start_cluster(prm);
  const Range rg = range_of(prm, it, kRows, T::kKeys);
  const int mine = rg.t1 - rg.t0 > warp ? (rg.t1 - rg.t0 - warp - 1) / kWarps + 1 : 0;

  // ---- the stream of tiles ----
  const uint32_t ring = ptx::smem_addr(smem) + warp * kS * T::kStage;
  const uint8_t* kc = static_cast<const uint8_t*>(a.k_cache);
  const uint8_t* vc = static_cast<const uint8_t*>(a.v_cache);
  const int esz = kF8 ? 1 : 2;
  // This lane's part of a key: its chunk, and where that is from the first
  // key of a tile that lies in one page.
  const uint32_t chunk_bytes = (lane % T::kChunks) * 16 < c.head_dim * esz ? 16u : 0u;
  const int64_t token_step = c.token_stride * esz;
  const int64_t lane_off = chunk_bytes ? lane / T::kChunks * token_step + lane % T::kChunks * 16 : 0;
  constexpr int kPer = 32 / T::kChunks;  // keys one instruction copies
  const int64_t step = kPer * token_step;
  const uint32_t copy_at = T::at(lane / T::kChunks, lane % T::kChunks);
  const bool pages_hold_tiles = c.page_size % T::kKeys == 0;
  auto tile_key = [&](int i) { return rg.base + (rg.t0 + warp + kWarps * i) * T::kKeys; };
  auto look_up = [&](int i) {
    Slot slot = {-1, -1};
    if (i < mine) slot = slot_of(prm, it, rg, tile_key(i) + lane % T::kKeys);
    return slot;
  };
  auto load = [&](int i, const Slot& slot) {
    if (i < mine) {
      slot.check(prm);
      const int64_t off = slot.in(c) ? slot.at(c, it.kh) * esz : -1;
      const bool whole =
          pages_hold_tiles && __all_sync(0xffffffffu, off >= 0);  // tiles start on their multiples
      const uint32_t st = ring + (i % kS) * T::kStage;
      if (whole) {  // one page, every key of it: one offset and a step
        const int64_t o = __shfl_sync(0xffffffffu, off, 0) + lane_off;
        const uint8_t *ks = kc + o, *vs = vc + o;
#pragma unroll
        for (int k = 0; k < T::kKeys; k += kPer, ks += step, vs += step) {
          const uint32_t dst = ((st + copy_at) ^ T::key_xor(k)) + k * T::kRow;
          ptx::cp_async16(dst, ks, chunk_bytes);
          ptx::cp_async16(dst + T::kBytes, vs, chunk_bytes);
        }
      } else {
#pragma unroll
        for (int k = 0; k < T::kKeys; k += kPer) {
          const int key = k + lane / T::kChunks;
          const int64_t o = __shfl_sync(0xffffffffu, off, key);
          const uint32_t n = o >= 0 ? chunk_bytes : 0u;
          const int64_t src = n ? o + (lane % T::kChunks) * 16 : 0;
          const uint32_t dst = ((st + copy_at) ^ T::key_xor(k)) + k * T::kRow;
          ptx::cp_async16(dst, kc + src, n);
          ptx::cp_async16(dst + T::kBytes, vc + src, n);
        }
      }
      if (kF8) {
        const int64_t s = off >= 0 ? slot.scale_at(c, it.kh) : 0;
        const uint32_t n = off >= 0 ? 4u : 0u, dst = st + 2 * T::kBytes + lane * 4;
        ptx::cp_async4(dst, a.k_scale + s, n);
        ptx::cp_async4(dst + T::kKeys * 4, a.v_scale + s, n);
      }
    }
    ptx::cp_async_commit();
  };
  Slot ahead[kS];  // of this lane's key of the first tiles
#pragma unroll
  for (int i = 0; i < kS; ++i) ahead[i] = look_up(i);
#pragma unroll
  for (int i = 0; i < kS - 1; ++i) load(i, ahead[i]);
  Slot next = ahead[kS - 1];

  // ---- queries, as the second operand of S^T = K Q^T ----
  // Elements (bf16: 2 quad, + 1 of 8; fp16: 4 quad, .. + 3 of 16, in the order
  // the keys' are read) of row 8 n + oct.
  const float scale = c.scale * 1.4426950408889634f;
  auto query = [&](int n, uint32_t (&q)[kDT][2]) {
    const uint8_t* p = static_cast<const uint8_t*>(a.q) + it.q_at(prm, 8 * n + oct) * 2;
    float f = scale;
    if (!kF8) {
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = 16 * d + 8 * h;  // head_dim is a multiple of 8
          q[d][h] =
              e < c.head_dim ? *reinterpret_cast<const uint32_t*>(p + 2 * (e + 2 * quad)) : 0u;
        }
    } else {
      uint2 raw[kDT];
      float amax = 0.f;
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        raw[d] = make_uint2(0u, 0u);
        if (16 * d < c.head_dim) raw[d] = *reinterpret_cast<const uint2*>(p + 2 * (16 * d + 4 * quad));
        float x, y;
        bf16x2_to_f32(raw[d].x, x, y);
        amax = fmaxf(amax, fmaxf(fabsf(x), fabsf(y)));
        bf16x2_to_f32(raw[d].y, x, y);
        amax = fmaxf(amax, fmaxf(fabsf(x), fabsf(y)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // The row is scaled to [2^14, 2^15) for fp16, by 2^(14 - e) of its largest
      // element (both factors kept normal).
      const int e = clamp_int((int)(__float_as_uint(amax) >> 23) - 127, -112, 128);
      const float down = __uint_as_float((uint32_t)(141 - e) << 23);
      f *= __uint_as_float((uint32_t)(113 + e) << 23);
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        float x, y;
        bf16x2_to_f32(raw[d].x, x, y);
        q[d][0] = pack_f16(x * down, y * down);
        bf16x2_to_f32(raw[d].y, x, y);
        q[d][1] = pack_f16(x * down, y * down);
      }
    }
    return f;
  };
  uint32_t q[L::kSharedQ ? 1 : kNT][kDT][2];
  float sc[kNT][2];  // factor of the scores of this lane's two columns, log2 units
  for (int r = threadIdx.x; r < kRows; r += kThreads) {
    const int last = it.pos(prm, r);
    range[r] = make_int2(last, it.first(last));
  }
  if (L::kSharedQ) {
    if (warp < kNT) {  // a warp a tile of 8 rows
      const float f = query(warp, q[0]);
      if (quad == 0) factor[8 * warp + oct] = f;
      uint8_t* row = qs + (8 * warp + oct) * L::kQRow + 4 * quad;
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<uint32_t*>(row + 32 * d + 16 * h) = q[0][d][h];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) sc[n][j] = kF8 ? factor[8 * n + 2 * quad + j] : scale;
  } else {
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const float f = query(n, q[n]);
      // columns 2 quad and 2 quad + 1 belong to the lanes of those rows
      sc[n][0] = kF8 ? __shfl_sync(0xffffffffu, f, 8 * quad) : scale;
      sc[n][1] = kF8 ? __shfl_sync(0xffffffffu, f, 8 * quad + 4) : scale;
    }
    __syncthreads();
  }
  const uint32_t q_lane = ptx::smem_addr(qs) + lane % 8 * L::kQRow + lane / 8 * 16;
  // Two steps of 16 elements of query tile n.
  auto query_frag = [&](int n, int d, uint32_t (&r)[4]) {
    if (L::kSharedQ) {
      ptx::ldmatrix4<false>(q_lane + 8 * n * L::kQRow + 32 * d, r);
    } else {
      r[0] = q[n][d][0], r[1] = q[n][d][1], r[2] = q[n][d + 1][0], r[3] = q[n][d + 1][1];
    }
  };

  // ---- the pass over the keys ----
  const uint32_t k_lane = T::at(T::key_of(lane % 16), lane / 16);
  const uint32_t v_lane =
      kF8 ? T::at(lane, 0) : T::at(lane % 8 + lane / 16 * 8, lane / 8 % 2);
  float o[kNT][kDT][4], m[kNT][2], l[kNT][2];
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    m[n][0] = m[n][1] = -3.0e38f;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int d = 0; d < kDT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][d][i] = 0.f;
  }
  auto advance = [&](int i) {
    ptx::cp_async_wait_group<kS - 2>();
    __syncwarp();
    load(i + kS - 1, next);  // into the stage that step i - 1 has read
    next = look_up(i + kS);
  };
  // Tile i, which has arrived. False, and nothing is changed, where l and O need references of
  // their own (E4M3; the same for the whole warp), which they have in the instance kApart. That
  // is in a loop of its own and asked for by the scales: in this loop, and asked for by weights
  // that grow too large, it cost every call 1 to 4%, so 40 rows 257 us for 244 (32 sequences of
  // 100 to 12000 keys, heads of 128).
  auto tile = [&](int i, auto instance) __attribute__((always_inline)) {
    constexpr bool kApart = decltype(instance)::value;
    const uint32_t K = ring + (i % kS) * T::kStage, V = K + T::kBytes;
    const uint32_t k_at = K + k_lane, v_at = V + v_lane;
    const int key0 = tile_key(i);

    float s[kMT][kNT][4], s2[kMT][kNT][4];
#pragma unroll
    for (int t = 0; t < kMT; ++t)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[t][n][x] = s2[t][n][x] = 0.f;
#pragma unroll
    for (int d = 0; d < kDT; d += 2) {
      uint32_t k[kMT][2][4];  // two steps of 16 elements of the tile's keys
#pragma unroll
      for (int t = 0; t < kMT; ++t) {
        if (!kF8) {
          ptx::ldmatrix4<false>((k_at ^ 2 * d * T::kChunkBit) + 16 * t * T::kRow, k[t][0]);
          ptx::ldmatrix4<false>((k_at ^ (2 * d + 2) * T::kChunkBit) + 16 * t * T::kRow, k[t][1]);
        } else {
          uint32_t r[4];
          ptx::ldmatrix4<false>((k_at ^ d * T::kChunkBit ^ T::key_xor(16 * t)) + 16 * t * T::kRow, r);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            k[t][h][0] = e4m3x2_f16(r[2 * h]);
            k[t][h][1] = e4m3x2_f16(r[2 * h + 1]);
            k[t][h][2] = e4m3x2_f16(r[2 * h] >> 16);
            k[t][h][3] = e4m3x2_f16(r[2 * h + 1] >> 16);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        uint32_t f[4];
        query_frag(n, d, f);
#pragma unroll
        for (int t = 0; t < kMT; ++t) {
          ptx::mma16816<kF8>(s[t][n], k[t][0], f[0], f[1]);
          ptx::mma16816<kF8>(kTwoSums ? s2[t][n] : s[t][n], k[t][1], f[2], f[3]);
        }
      }
    }
    if (kTwoSums) {
#pragma unroll
      for (int t = 0; t < kMT; ++t)
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[t][n][x] += s2[t][n][x];
    }

    // Scores of keys key0 + 16 t + key_of(oct) (and of oct + 8), columns 2 quad
    // (+ 1).
    float ks[kMT][2], vs[kMT][2];
    if (kF8) {
      const float* f = reinterpret_cast<const float*>(smem + (V + T::kBytes - ptx::smem_addr(smem)));
#pragma unroll
      for (int t = 0; t < kMT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ks[t][h] = f[16 * t + T::key_of(8 * h + oct)];
          vs[t][h] = f[T::kKeys + 16 * t + T::key_of(8 * h + oct)];
        }
    }
    const bool edge = key0 + T::kKeys - 1 > rg.hi_min || key0 < rg.lo_max;
    // Weights against the running maximum; over the bound, the maximum is
    // raised and they are taken again.
    float p[kMT][kNT][4];
    // This lane's largest score of a row, and its largest with the value's scale (an infinite
    // scale aside: the sum of weights does not see values).
    auto tops = [&](int n, int j, float& top, float& top_v) {
      top = top_v = -INFINITY;
#pragma unroll
      for (int t = 0; t < kMT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float v = s[t][n][2 * h + j];
          top = fmaxf(top, v);
          if (kF8 && vs[t][h] > 0.f && vs[t][h] < INFINITY) top_v = fmaxf(top_v, v + __log2f(vs[t][h]));
        }
    };
#pragma unroll
    for (int t = 0; t < kMT; ++t)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[t][n][x] *= sc[n][x % 2];
          if (kF8) s[t][n][x] *= ks[t][x / 2];
        }
    if (edge) {
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int2 seen = range[8 * n + 2 * quad + x % 2];
#pragma unroll
          for (int t = 0; t < kMT; ++t) {
            const int key = key0 + 16 * t + T::key_of(8 * (x / 2) + oct);
            if (key > seen.x || key < seen.y) s[t][n][x] = -INFINITY;
          }
        }
      if (kF8) {  // a key that no row sees has a scale of 0 here
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = key0 + 16 * t + T::key_of(8 * h + oct);
            if (key > rg.hi_max || key < rg.lo_min) vs[t][h] = 1.f;
          }
      }
    }
    // Scales for which l and O can share a reference: where weights are up to 2^15 with them, they
    // are up to 2^68 without, and none that fp32 has flushed to 0 would be above 2^-46 with them.
    // (By their bits, which order positive numbers and leave a NaN above them.)
    uint32_t least = __float_as_uint(1.f), most = least;
    if (kF8) {
#pragma unroll
      for (int t = 0; t < kMT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          least = min(least, __float_as_uint(vs[t][h]));
          most = max(most, __float_as_uint(vs[t][h]));
        }
    }
    const bool far = least < (127u - 53u) << 23 || most > (127u + 80u) << 23;
    bool raise = kApart || far;
#pragma unroll
    for (int t = 0; t < kMT; ++t)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float v = s[t][n][x];
          p[t][n][x] = ptx::ex2(v - m[n][x % 2]);
          if (!kF8)
            raise = raise || v > m[n][x % 2] + 8.f;
          else  // 0 * vs may be a NaN of a key that is not seen
            raise = raise || (v != -INFINITY && !(p[t][n][x] * vs[t][x / 2] <= 0x1p15f));
        }
    if (!kApart && __any_sync(0xffffffffu, raise)) {
      if (kF8 && __any_sync(0xffffffffu, far)) return false;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // E4M3: the largest weight times its value's scale becomes 2^7.
          float top, top_v;
          tops(n, j, top, top_v);
          float up = kF8 ? top_v - 7.f : top;
#pragma unroll
          for (int x = 4; x < 32; x *= 2) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, x));
          up = fmaxf(m[n][j], up);
          const float f = ptx::ex2(m[n][j] - up);
          m[n][j] = up;
          l[n][j] *= f;
#pragma unroll
          for (int d = 0; d < kDT; ++d) {
            o[n][d][j] *= f;
            o[n][d][2 + j] *= f;
          }
#pragma unroll
          for (int t = 0; t < kMT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) p[t][n][2 * h + j] = ptx::ex2(s[t][n][2 * h + j] - up);
        }
    }
    if (kApart) {
      // m follows the scores with their values' scales, l's reference (in shared memory) the
      // scores alone.
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top, top_v;
          tops(n, j, top, top_v);
#pragma unroll
          for (int x = 4; x < 32; x *= 2) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, x));
          }
          float& kept = l_ref[8 * n + 2 * quad + j];
          const float was = kept, ref = top > was + 8.f ? top : was;
          __syncwarp();
          if (oct == 0) kept = ref;
          l[n][j] *= ptx::ex2(was - ref);
          const float up = top_v > m[n][j] + 15.f ? top_v - 7.f : m[n][j], f = ptx::ex2(m[n][j] - up);
          m[n][j] = up;
#pragma unroll
          for (int d = 0; d < kDT; ++d) {
            o[n][d][j] *= f;
            o[n][d][2 + j] *= f;
          }
#pragma unroll
          for (int t = 0; t < kMT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float v = s[t][n][2 * h + j];
              l[n][j] += ptx::ex2(v - ref);
              // 0 for a key that is not seen, whatever its scale
              p[t][n][2 * h + j] = v == -INFINITY ? 0.f : ptx::ex2(v + __log2f(vs[t][h]) - up);
            }
        }
    }
    if (!kApart) {
#pragma unroll
    for (int t = 0; t < kMT; ++t)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          l[n][x % 2] += p[t][n][x];
          if (kF8 && p[t][n][x] > 0.f) p[t][n][x] *= vs[t][x / 2];
        }
    }

    // A key that some rows see and others do not may hold values that are not
    // finite, and 0 times those is not 0: such a tile goes element by element.
    if (edge && rg.hi_min != rg.hi_max) {
      bool wild = false;
#pragma unroll 1
      for (int d = 0; d < T::kChunks / 2 * kMT; ++d) {
        const uint4 v = ptx::ld_shared_v4(V + (d * 32 + lane) * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (kF8)
            wild = wild || (w[x] & 0x7fu) == 0x7fu || (w[x] & 0x7f00u) == 0x7f00u ||
                   (w[x] & 0x7f0000u) == 0x7f0000u || (w[x] & 0x7f000000u) == 0x7f000000u;
          else
            wild = wild || (w[x] & 0x7f80u) == 0x7f80u || (w[x] & 0x7f800000u) == 0x7f800000u;
        }
      }
      if (__any_sync(0xffffffffu, wild)) {
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll 1
            for (int k8 = 0; k8 < 8; ++k8) {
              const int k = 16 * t + T::key_of(8 * h + k8), key = key0 + k;
#pragma unroll
              for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float w = __shfl_sync(0xffffffffu, p[t][n][2 * h + j], 4 * k8 + quad);
                  const int2 seen = range[8 * n + 2 * quad + j];
                  if (key > seen.x || key < seen.y) continue;
#pragma unroll
                  for (int d = 0; d < kDT; ++d)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                      const int e = 16 * d + oct + 8 * r;
                      const uint32_t at = V - ptx::smem_addr(smem) + T::at(k, e * (kF8 ? 1 : 2) / 16);
                      float v;
                      if (kF8) {
                        const uint32_t f = e4m3x2_f16(smem[at + e % 16]);
                        v = __half2float(__ushort_as_half((uint16_t)f));
                      } else {
                        v = __uint_as_float(
                            (uint32_t) * reinterpret_cast<const uint16_t*>(smem + at + e % 8 * 2) << 16);
                      }
                      o[n][d][2 * r + j] += w * v;
                    }
                }
            }
        __syncwarp();
        return true;
      }
    }

    // P^T as the second operand of O^T = V^T P^T.
    uint32_t ph[kMT][kNT][2], pl[kMT][kNT][2];
#pragma unroll
    for (int t = 0; t < kMT; ++t)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = p[t][n][2 * h], y = p[t][n][2 * h + 1];
          if (kF8) {
            ph[t][n][h] = ptx::movmatrix_trans(pack_f16(x, y));
          } else {
            uint32_t hi, lo;
            split_bf16(ptx::f32x2(x, y), hi, lo);
            ph[t][n][h] = ptx::movmatrix_trans(hi);
            pl[t][n][h] = ptx::movmatrix_trans(lo);
          }
        }
#pragma unroll
    for (int d = 0; d < kDT; ++d) {
      uint32_t r[4];
      if (!kF8) {
#pragma unroll
        for (int t = 0; t < kMT; ++t) {
          ptx::ldmatrix4<true>((v_at ^ 2 * d * T::kChunkBit) + 16 * t * T::kRow, r);
#pragma unroll
          for (int n = 0; n < kNT; ++n) ptx::mma16816<false>(o[n][d], r, ph[t][n][0], ph[t][n][1]);
#pragma unroll
          for (int n = 0; n < kNT; ++n) ptx::mma16816<false>(o[n][d], r, pl[t][n][0], pl[t][n][1]);
        }
      } else {
        ptx::ldmatrix2_bytes_trans(v_at ^ d * T::kChunkBit, r);
#pragma unroll
        for (int t = 0; t < kMT; ++t) {
          const uint32_t x = r[2 * t], y = r[2 * t + 1];
          const uint32_t v[4] = {e4m3x2_f16(x), e4m3x2_f16(y), e4m3x2_f16(x >> 16),
                                 e4m3x2_f16(y >> 16)};
#pragma unroll
          for (int n = 0; n < kNT; ++n) ptx::mma16816<true>(o[n][d], v, ph[t][n][0], ph[t][n][1]);
        }
      }
    }
    __syncwarp();  // every lane has read this stage
    return true;
  };
  int i = 0;
  for (; i < mine; ++i) {
    advance(i);
    if (!tile(i, std::false_type{})) break;
  }
  const bool apart = kF8 && i < mine;
  if (apart) {
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (oct == 0) l_ref[8 * n + 2 * quad + j] = m[n][j];
    __syncwarp();
    for (bool here = true; i < mine; ++i, here = false) {
      if (!here) advance(i);
      tile(i, std::true_type{});
    }
  }
  ptx::cp_async_wait_all();

  // ---- join: the warps of the block, then the blocks of the cluster ----
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int x = 4; x < 32; x *= 2) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], x);
      if (oct == 0) {
        stat[warp * kRows + 8 * n + 2 * quad + j] = m[n][j];
        stat[(kWarps + warp) * kRows + 8 * n + 2 * quad + j] = l[n][j];
        if (kF8 && !apart) l_ref[8 * n + 2 * quad + j] = m[n][j];
      }
    }
  __syncthreads();
  // O of each warp, relative to the block's maximum, [row][kDim + 4] floats
  // in the warp's own stages (the pad keeps the stores free of conflicts).
  constexpr int kLd = kDim + 4;
  static_assert(kRows * kLd * 4 <= kS * T::kStage, "the joined rows fit the stages");
  float* mine_o = reinterpret_cast<float*>(smem + warp * kS * T::kStage);
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 8 * n + 2 * quad + j;
      float top = stat[r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, stat[w * kRows + r]);
      const float f = ptx::ex2(m[n][j] - top);
      if (warp == 0 && oct == 0) {
        const float* refs = stat + (kF8 ? 2 * kWarps * kRows : 0) + r;
        float sum = 0.f, ref = refs[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) ref = fmaxf(ref, refs[w * kRows]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          sum += stat[(kWarps + w) * kRows + r] * ptx::ex2(refs[w * kRows] - ref);
        joined[r] = ref;
        joined[kRows + r] = sum;
        if (kF8) joined[2 * kRows + r] = top;
      }
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mine_o[r * kLd + 16 * d + oct + 8 * h] =
              o[n][d][2 * h + j] * f;
    }
  __syncthreads();
  finish<kRows, kDim, kWarps, kThreads, L::kOwnInbox, __nv_bfloat16, kF8>(
      prm, it, reinterpret_cast<float*>(smem), kS * T::kStage / 4, kLd, joined, inbox);
}

template <int kDim, int kNT, bool kF8>
cudaError_t launch_mma(const Params& p, unsigned blocks, cudaStream_t s) {
  static thread_local int configured = -1;
  return launch(mma_kernel<kDim, kNT, kF8>, &configured, p, blocks, warps_of(kDim) * 32,
                Layout<kDim, kNT, kF8>::kAll, s);
}

}  // namespace attn
}  // namespace moe
