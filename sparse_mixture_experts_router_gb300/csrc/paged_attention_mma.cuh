// Attention of the new tokens over a paged bf16 or E4M3 cache, on warp-level
// matrix products.
//
// The work is memory-bound: each cached key and value meets only the rows of
// one head group (R = new tokens x heads per key-value head, 8 for an 8-way
// shared head), R multiply-adds an element. So the kernel is a stream of the
// cache through shared memory, and everything else is arranged to stay out of
// that stream's way:
//  - A block of 4 warps holds one (sequence, key-value head, up to 8 NT query
//    rows) item, or one of the C parts that its keys are cut into: the parts
//    are a thread-block cluster and join through its distributed shared
//    memory, so one launch and no scratch in global memory.
//  - Each warp streams its own tiles (16 keys of bf16, 32 of E4M3) through its
//    own ring of stages with cp.async and no block-wide synchronisation; the
//    pages of the tile after next are looked up one step ahead.
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
// the type of the second product: bf16 twice (p = hi + lo, 2^-17 of p, two
// products) for a bf16 cache, whose error one rounding would double; fp16
// (2^-12) for an E4M3 cache. E4M3 elements and queries become fp16 exactly,
// each query row scaled by a power of two, and the scales of keys multiply
// scores, those of values multiply weights.
#pragma once
#include "serve_util.cuh"
#include "sm103_ptx.cuh"

namespace moe {
namespace attn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

// n / d for 0 <= n < 2^30 and 1 <= d < 2^30 as a multiplication.
struct FastDiv {
  uint64_t mul;
  int shift;
};
inline FastDiv fast_div(uint32_t d) {
  int bits = 0;
  while ((1u << bits) < d) ++bits;
  const int shift = 30 + bits;
  return {((1ull << shift) + d - 1) / d, shift};
}
__device__ __forceinline__ int div(const FastDiv& f, int n) {
  return (int)(((uint64_t)n * f.mul) >> f.shift);
}

template <int kDim, bool kF8>
struct Tile {
  static constexpr int kKeys = kF8 ? 32 : 16;
  static constexpr int kRow = kDim * (kF8 ? 1 : 2);  // bytes of a key in shared memory
  static constexpr int kChunks = kRow / 16;
  static constexpr int kBytes = kKeys * kRow;        // one of K, V
  static constexpr int kStage = 2 * kBytes + (kF8 ? 2 * kKeys * 4 : 0);
  // Stages a warp: about 24 KB in flight, at least 3.
  static constexpr int kStages = kStage >= 16384 ? 3 : kStage >= 8192 ? 3 : 6;
  // Byte offset of 16-byte chunk c of key k: the chunks of 8 consecutive keys
  // fall into different banks.
  static __device__ __forceinline__ uint32_t at(int k, int c) {
    return kChunks >= 8 ? (uint32_t)(k * kRow + ((c ^ (k & 7)) << 4))
                        : (uint32_t)(k * kRow + ((c ^ ((k >> 1) & 3)) << 4));
  }
};

template <int kDim, int kNT, bool kF8>
constexpr int smem_bytes() {
  return kWarps * Tile<kDim, kF8>::kStages * Tile<kDim, kF8>::kStage +
         (2 * kWarps + 2) * 8 * kNT * 4;
}

// The first position that a sequence's new tokens see.
struct FirstKey {
  int window;
  __device__ int operator()(const SeqRange& r) const {
    return window ? max(0, r.len - r.n - window + 1) : 0;
  }
};

struct Params {
  AttnArgs a;
  FastDiv page_div;
  int parts, row_blocks;  // C, blocks of 8 NT query rows a (sequence, head)
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
__global__ void __launch_bounds__(kThreads) mma_kernel(const __grid_constant__ Params prm) {
  using T = Tile<kDim, kF8>;
  constexpr int kS = T::kStages, kMT = T::kKeys / 16, kDT = kDim / 16, kRows = 8 * kNT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnArgs& a = prm.a;
  const moe_attn_config& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, quad = lane % 4, oct = lane / 4;
  float* stat = reinterpret_cast<float*>(smem + kWarps * kS * T::kStage);  // m, l of each warp's rows
  float* joined = stat + 2 * kWarps * kRows;                               // m, l of the block's

  pdl_wait();
  pdl_trigger();
  const int part = (int)(blockIdx.x % prm.parts);
  int item = (int)(blockIdx.x / prm.parts) - 1;
  if (item < 0) {  // the first cluster
    if (part == 0) check_lists<kThreads>(a, FirstKey{c.window});
    return;
  }
  const int rb = item % prm.row_blocks;
  item /= prm.row_blocks;
  const int kh = item % c.n_kv_heads, b = item / c.n_kv_heads;
  const SeqRange sq = seq_range(a, b);
  const int G = c.n_heads / c.n_kv_heads, R = G * sq.n, row0 = rb * kRows;
  if (row0 >= R) return;  // the same for the whole cluster

  // Rows past the last one repeat it and are not written.
  auto row_pos = [&](int r) { return sq.len - sq.n + min(row0 + r, R - 1) / G; };
  auto row_first = [&](int pos) { return c.window ? max(0, pos - c.window + 1) : 0; };
  const int hi_min = row_pos(0), hi_max = row_pos(kRows - 1);
  const int lo_min = row_first(hi_min), lo_max = row_first(hi_max);
  const bool one_range = hi_min == hi_max;  // every row sees the same keys
  const int base = lo_min / T::kKeys * T::kKeys;
  const int tiles = hi_max < 0 ? 0 : (hi_max - base) / T::kKeys + 1;
  const int t0 = (int)((long long)tiles * part / prm.parts);
  const int t1 = (int)((long long)tiles * (part + 1) / prm.parts);
  const int mine = t1 - t0 > warp ? (t1 - t0 - warp - 1) / kWarps + 1 : 0;

  // ---- the stream of tiles ----
  const uint32_t ring = ptx::smem_addr(smem) + warp * kS * T::kStage;
  const uint8_t* kc = static_cast<const uint8_t*>(a.k_cache);
  const uint8_t* vc = static_cast<const uint8_t*>(a.v_cache);
  const int esz = kF8 ? 1 : 2;
  const bool chunk_in = (lane % T::kChunks) * 16 < c.head_dim * esz;
  auto tile_key = [&](int i) { return base + (t0 + warp + kWarps * i) * T::kKeys; };
  // This lane's key of tile i: its page (negative: not a key any row sees, or
  // no page of the cache) and its place in the page.
  int page = -1, place = 0;
  auto look_up = [&](int i) {
    const int key = tile_key(i) + lane % T::kKeys;
    page = -1;
    if (i < mine && key >= lo_min && key <= hi_max) {
      const int n = div(prm.page_div, key);
      place = key - n * c.page_size;
      page = __ldg(a.table + (int64_t)b * c.max_pages + n);
      if (page >= c.n_pages) page = -1;
    }
  };
  auto load = [&](int i) {  // tile i, the lane's page of it at hand
    if (i < mine) {
      int64_t off = -1;
      if (page >= 0)
        off = ((int64_t)page * c.page_stride + (int64_t)place * c.token_stride +
               (int64_t)kh * c.head_stride) * esz;
      const uint32_t st = ring + (i % kS) * T::kStage;
      constexpr int kPer = 32 / T::kChunks;  // keys one instruction copies
#pragma unroll
      for (int k = 0; k < T::kKeys; k += kPer) {
        const int key = k + lane / T::kChunks;
        const int64_t o = __shfl_sync(0xffffffffu, off, key);
        const uint32_t n = o >= 0 && chunk_in ? 16u : 0u;
        const int64_t src = n ? o + (lane % T::kChunks) * 16 : 0;
        const uint32_t dst = st + T::at(key, lane % T::kChunks);
        ptx::cp_async16(dst, kc + src, n);
        ptx::cp_async16(dst + T::kBytes, vc + src, n);
      }
      if (kF8) {
        const int64_t s = page >= 0 ? ((int64_t)page * c.n_kv_heads + kh) * c.page_size + place : 0;
        const uint32_t n = page >= 0 ? 4u : 0u, dst = st + 2 * T::kBytes + lane * 4;
        ptx::cp_async4(dst, a.k_scale + s, n);
        ptx::cp_async4(dst + T::kKeys * 4, a.v_scale + s, n);
      }
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kS - 1; ++i) {
    look_up(i);
    load(i);
  }
  look_up(kS - 1);

  // ---- queries, as the second operand of S^T = K Q^T ----
  uint32_t q[kNT][kDT][2];
  float sc[kNT][2];  // factor of the scores of this lane's two columns, log2 units
  const float scale = c.scale * 1.4426950408889634f;
  auto q_row = [&](int r) {
    r = min(row0 + r, R - 1);
    return static_cast<const uint8_t*>(a.q) +
           ((int64_t)(sq.row0 + r / G) * c.q_stride + (int64_t)(kh * G + r % G) * c.head_dim) * 2;
  };
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    const uint8_t* p = q_row(8 * n + oct);
    sc[n][0] = sc[n][1] = scale;
    if (!kF8) {
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = 16 * d + 8 * h;  // head_dim is a multiple of 8
          q[n][d][h] =
              e < c.head_dim ? *reinterpret_cast<const uint32_t*>(p + 2 * (e + 2 * quad)) : 0u;
        }
    } else {
      // Four consecutive elements a lane: keys are read in the same order, so
      // the products pair up. The row is scaled to [1, 2) for fp16.
      uint2 raw[kDT];
      float amax = 0.f;
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        raw[d] = make_uint2(0u, 0u);
        if (16 * d < c.head_dim)
          raw[d] = *reinterpret_cast<const uint2*>(p + 2 * (16 * d + 4 * quad));
        float x, y;
        bf16x2_to_f32(raw[d].x, x, y);
        amax = fmaxf(amax, fmaxf(fabsf(x), fabsf(y)));
        bf16x2_to_f32(raw[d].y, x, y);
        amax = fmaxf(amax, fmaxf(fabsf(x), fabsf(y)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^-e and 2^e of the row's largest, kept normal
      const int e = clamp_int((int)(__float_as_uint(amax) >> 23) - 127, -126, 126);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        float x, y;
        bf16x2_to_f32(raw[d].x, x, y);
        q[n][d][0] = pack_f16(x * down, y * down);
        bf16x2_to_f32(raw[d].y, x, y);
        q[n][d][1] = pack_f16(x * down, y * down);
      }
      // columns 2 quad and 2 quad + 1 belong to the lanes of those rows
      sc[n][0] *= __shfl_sync(0xffffffffu, up, 8 * quad);
      sc[n][1] *= __shfl_sync(0xffffffffu, up, 8 * quad + 4);
    }
  }
  int hi[kNT][2], lo[kNT][2];
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      hi[n][j] = row_pos(8 * n + 2 * quad + j);
      lo[n][j] = row_first(hi[n][j]);
    }

  // ---- the pass over the keys ----
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
  for (int i = 0; i < mine; ++i) {
    ptx::cp_async_wait_group<kS - 2>();
    __syncwarp();
    load(i + kS - 1);  // into the stage that step i - 1 has read
    look_up(i + kS);
    const uint32_t K = ring + (i % kS) * T::kStage, V = K + T::kBytes;
    const int key0 = tile_key(i);

    float s[kMT][kNT][4];
#pragma unroll
    for (int t = 0; t < kMT; ++t)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[t][n][x] = 0.f;
    if (!kF8) {
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        uint32_t k[4];
        ptx::ldmatrix4<false>(K + T::at(lane % 16, 2 * d + lane / 16), k);
#pragma unroll
        for (int n = 0; n < kNT; ++n) ptx::mma16816<false>(s[0][n], k, q[n][d][0], q[n][d][1]);
      }
    } else {
#pragma unroll
      for (int t = 0; t < kMT; ++t)
#pragma unroll
        for (int d = 0; d < kDT; d += 2) {
          uint32_t r[4];
          ptx::ldmatrix4<false>(K + T::at(16 * t + lane % 16, d + lane / 16), r);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t k[4] = {e4m3x2_f16(r[2 * h]), e4m3x2_f16(r[2 * h + 1]),
                                   e4m3x2_f16(r[2 * h] >> 16), e4m3x2_f16(r[2 * h + 1] >> 16)};
#pragma unroll
            for (int n = 0; n < kNT; ++n)
              ptx::mma16816<true>(s[t][n], k, q[n][d + h][0], q[n][d + h][1]);
          }
        }
    }

    // Scores of keys key0 + 16 t + oct (+ 8), columns 2 quad (+ 1).
    float ks[kMT][2], vs[kMT][2];
    if (kF8) {
      const float* f = reinterpret_cast<const float*>(smem + (V + T::kBytes - ptx::smem_addr(smem)));
#pragma unroll
      for (int t = 0; t < kMT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ks[t][h] = f[16 * t + 8 * h + oct];
          vs[t][h] = f[T::kKeys + 16 * t + 8 * h + oct];
        }
    }
    const bool edge = key0 + T::kKeys - 1 > hi_min || key0 < lo_max;
    bool raise = false;
#pragma unroll
    for (int t = 0; t < kMT; ++t)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float v = s[t][n][x] * sc[n][x % 2];
          if (kF8) v *= ks[t][x / 2];
          if (edge) {
            const int key = key0 + 16 * t + 8 * (x / 2) + oct;
            if (key > hi[n][x % 2] || key < lo[n][x % 2]) v = -INFINITY;
          }
          s[t][n][x] = v;
          if (!kF8) {
            raise = raise || v > m[n][x % 2] + 8.f;
          } else {
            const float p = ptx::ex2(v - m[n][x % 2]);
            raise = raise || !(p <= 0x1p68f && (v == -INFINITY || p * vs[t][x / 2] <= 256.f));
          }
        }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top = m[n][j];
#pragma unroll
          for (int t = 0; t < kMT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v = s[t][n][2 * h + j];
              // E4M3: the largest weight times its value's scale, and no
              // weight itself above 2^60
              if (kF8) v = fmaxf(vs[t][h] > 0.f ? v + __log2f(vs[t][h]) : -INFINITY, v - 60.f);
              top = fmaxf(top, v);
            }
#pragma unroll
          for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float f = ptx::ex2(m[n][j] - top);
          m[n][j] = top;
          l[n][j] *= f;
#pragma unroll
          for (int d = 0; d < kDT; ++d) {
            o[n][d][j] *= f;
            o[n][d][2 + j] *= f;
          }
        }
    }
#pragma unroll
    for (int t = 0; t < kMT; ++t)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float p = ptx::ex2(s[t][n][x] - m[n][x % 2]);
          l[n][x % 2] += p;
          s[t][n][x] = kF8 && p > 0.f ? p * vs[t][x / 2] : p;
        }

    // A key that some rows see and others do not may hold values that are not
    // finite, and 0 times those is not 0: such a tile goes element by element.
    if (edge && !one_range) {
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
              const int k = 16 * t + 8 * h + k8, key = key0 + k;
#pragma unroll
              for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float p = __shfl_sync(0xffffffffu, s[t][n][2 * h + j], 4 * k8 + quad);
                  if (key > hi[n][j] || key < lo[n][j]) continue;
#pragma unroll
                  for (int d = 0; d < kDT; ++d)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                      const int e = kF8 ? 16 * d + 2 * oct + r : 16 * d + oct + 8 * r;
                      const uint32_t at = V - ptx::smem_addr(smem) + T::at(k, e * (kF8 ? 1 : 2) / 16);
                      float v;
                      if (kF8) {
                        const uint32_t f = e4m3x2_f16(smem[at + e % 16]);
                        v = __half2float(__ushort_as_half((uint16_t)f));
                      } else {
                        v = __uint_as_float(
                            (uint32_t) * reinterpret_cast<const uint16_t*>(smem + at + e % 8 * 2) << 16);
                      }
                      o[n][d][2 * r + j] += p * v;
                    }
                }
            }
        __syncwarp();
        continue;
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
          const float x = s[t][n][2 * h], y = s[t][n][2 * h + 1];
          if (kF8) {
            ph[t][n][h] = ptx::movmatrix_trans(pack_f16(x, y));
          } else {
            const uint32_t w = f32x2_to_bf16x2(x, y);
            float xh, yh;
            bf16x2_to_f32(w, xh, yh);
            ph[t][n][h] = ptx::movmatrix_trans(w);
            pl[t][n][h] = ptx::movmatrix_trans(f32x2_to_bf16x2(x - xh, y - yh));
          }
        }
#pragma unroll
    for (int d = 0; d < kDT; ++d) {
      uint32_t r[4];
      if (!kF8) {
        ptx::ldmatrix4<true>(V + T::at(lane % 8 + lane / 16 * 8, 2 * d + lane / 8 % 2), r);
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          ptx::mma16816<false>(o[n][d], r, ph[0][n][0], ph[0][n][1]);
          ptx::mma16816<false>(o[n][d], r, pl[0][n][0], pl[0][n][1]);
        }
      } else {
        // 16-bit units of V are element pairs (2 oct, 2 oct + 1): rows 0-7 of
        // the product take the even elements and rows 8-15 the odd ones.
        ptx::ldmatrix4<true>(V + T::at(lane, d), r);
#pragma unroll
        for (int t = 0; t < kMT; ++t) {
          const uint32_t x = r[2 * t], y = r[2 * t + 1];
          const uint32_t v[4] = {e4m3x2_f16(__byte_perm(x, 0, 0x4420)),
                                 e4m3x2_f16(__byte_perm(x, 0, 0x4431)),
                                 e4m3x2_f16(__byte_perm(y, 0, 0x4420)),
                                 e4m3x2_f16(__byte_perm(y, 0, 0x4431))};
#pragma unroll
          for (int n = 0; n < kNT; ++n) ptx::mma16816<true>(o[n][d], v, ph[t][n][0], ph[t][n][1]);
        }
      }
    }
    __syncwarp();  // every lane has read this stage
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
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          sum += stat[(kWarps + w) * kRows + r] * ptx::ex2(stat[w * kRows + r] - top);
        joined[r] = top;
        joined[kRows + r] = sum;
      }
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mine_o[r * kLd + (kF8 ? 16 * d + 2 * oct + h : 16 * d + oct + 8 * h)] =
              o[n][d][2 * h + j] * f;
    }
  __syncthreads();
  const int rows = min(kRows, R - row0), vecs = c.head_dim / 4;
  const float4* w0 = reinterpret_cast<const float4*>(smem);
  constexpr int kWarpVecs = kS * T::kStage / 16;
  auto block_sum = [&](int r, int v) {
    float4 x = w0[r * (kLd / 4) + v];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 y = w0[w * kWarpVecs + r * (kLd / 4) + v];
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    return x;
  };
  auto write = [&](int r, int v, float4 x, float top, float sum) {
    const float f = sum > 0.f ? 1.f / sum : sum;  // a NaN stays one
    if (sum == 0.f) x = make_float4(0.f, 0.f, 0.f, 0.f);
    else x.x *= f, x.y *= f, x.z *= f, x.w *= f;
    const int g = row0 + r;
    const int64_t at = (int64_t)(sq.row0 + g / G) * c.n_heads + kh * G + g % G;
    reinterpret_cast<uint2*>(a.out)[at * vecs + v] =
        make_uint2(f32x2_to_bf16x2(x.x, x.y), f32x2_to_bf16x2(x.z, x.w));
    if (v == 0 && a.lse)
      a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  };
  if (prm.parts == 1) {
    for (int i = threadIdx.x; i < rows * vecs; i += kThreads) {
      const int r = i / vecs, v = i - r * vecs;
      write(r, v, block_sum(r, v), joined[r], joined[kRows + r]);
    }
    return;
  }
  float4* sum0 = reinterpret_cast<float4*>(smem);  // the block's O, in the first warp's place
  for (int i = threadIdx.x; i < rows * vecs; i += kThreads) {
    const int r = i / vecs, v = i - r * vecs;
    sum0[r * (kLd / 4) + v] = block_sum(r, v);
  }
  ptx::cluster_sync();
  const uint32_t sum_at = ptx::smem_addr(smem), joined_at = ptx::smem_addr(joined);
  for (int i = part * kThreads + threadIdx.x; i < rows * vecs; i += prm.parts * kThreads) {
    const int r = i / vecs, v = i - r * vecs;
    float top = -INFINITY, sum = 0.f;
    for (int p = 0; p < prm.parts; ++p)
      top = fmaxf(top, ptx::ld_cluster_f32(ptx::mapa_shared(joined_at + r * 4, p)));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < prm.parts; ++p) {
      const uint32_t jp = ptx::mapa_shared(joined_at + r * 4, p);
      const float f = ptx::ex2(ptx::ld_cluster_f32(jp) - top);
      const float4 y = ptx::ld_cluster_v4(ptx::mapa_shared(sum_at + (r * kLd + 4 * v) * 4, p));
      sum += ptx::ld_cluster_f32(jp + kRows * 4) * f;
      x.x += y.x * f, x.y += y.y * f, x.z += y.z * f, x.w += y.w * f;
    }
    write(r, v, x, top, sum);
  }
  ptx::cluster_sync();  // no block leaves while another reads its memory
}

// Launches the kernel for n_tiles x 8 query rows.
template <int kDim, int kNT, bool kF8>
cudaError_t launch(const Params& p, unsigned blocks, cudaStream_t s) {
  constexpr int smem = smem_bytes<kDim, kNT, kF8>();
  static thread_local int device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (device != dev) {
    e = cudaFuncSetAttribute(mma_kernel<kDim, kNT, kF8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(mma_kernel<kDim, kNT, kF8>,
                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    device = dev;
  }
  return launch_pdl(mma_kernel<kDim, kNT, kF8>, dim3(blocks), dim3(kThreads), (size_t)smem, s, p.parts,
                    p);
}

}  // namespace attn
}  // namespace moe
