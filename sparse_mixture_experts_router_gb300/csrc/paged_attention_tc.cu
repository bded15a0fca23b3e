// Attention of many query rows over a paged bf16 cache, on tcgen05.
//
// From about 50 query rows of a head group (drafts of a widely shared head) a
// cached element meets enough multiply-adds that warp-level products, 0.6
// PFLOP/s here, bound the kernel and not memory. Here an item has up to 128
// rows, the M of a tcgen05.mma, so the keys are read once for all of them:
//   S (128 x 128) = Q K^T      both from shared memory
//   O (128 x D)  += P V        P from Tensor Memory, V from shared memory
// with S twice, P over the S it came from, and O in Tensor Memory. A row is a
// lane, so a thread has (half) a row of scores in its registers and the softmax
// needs no exchange but one maximum between the two threads of a row. As in
// the other kernels the running maximum is raised only when a score passes it
// by 8 (log2 units); then the row of O is read, scaled and written back.
//
// 13 warps: 8 softmax (two per 32 rows, 64 keys each), one that issues the
// products, 4 that copy keys and values (cp.async, page by page, into the
// 128-byte swizzled layout) through a ring of 32 KB slots in the order they
// are used: K0 K1 V0 K2 V1 ... The products of tile i + 1 run under the softmax
// of tile i.
//
// Keys that some rows of the item see and others do not (at most its new tokens
// at either end) are masked row by row in the first and last tiles. A masked
// weight is 0, and 0 times a value that is not finite is not 0: the block looks
// at those keys' values first, and where one is not finite the products take
// only the keys that every row sees, and the others are added at the end, row
// by row, with fused multiply-adds.
//
// One block an SM. At 128 rows, 32 sequences of 500 to 8000 keys: 185 us, 0.46 of
// measured HBM bandwidth, 385 TFLOP/s (warp-level products, eight blocks of 16
// rows: 404 us). A tile takes about 3000 cycles: 1300 for the exponentials and
// the packing of weights, 550 for reading scores and their maximum, the rest
// waiting for products and copies; what lies outside the tiles (about 10 us a
// block, nothing else on the SM) is the next largest part.
//
// Rounding: as the warp-level kernel: fp32 scores, sums and O, weights as two
// bf16 terms.
#include "paged_attention.cuh"
#include "sm103_wait.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kSoftmax = 256;  // threads 0 .. 255
constexpr int kMmaWarp = 8;
constexpr int kLoadWarps = 4;  // two leave the softmax 168 registers, and take 199 us for 185
constexpr int kEdgeKeys = 8;   // keys that only some rows see, taken at a time
constexpr int kThreads = kSoftmax + 32 + 32 * kLoadWarps;
constexpr int kKeys = 128;
constexpr int kRows = 128;
constexpr uint32_t kTmemCols = 512;  // S and P: 0-127, 128-255; O: from 256
constexpr uint32_t kTmemO = 256;

template <int kDim>
struct Layout {
  static constexpr int kHalves = kDim / 64;            // 128-byte rows of 64 elements
  static constexpr int kHalf = kKeys * 128;            // bytes
  static constexpr int kSlot = kHalves * kHalf;
  static constexpr int kSlots = kDim == 128 ? 5 : 8;
  static constexpr int kRing = kSlots * kSlot;
  static constexpr int kQ = kSlot;                     // 128 rows
  static constexpr int kLd = kDim + 4;
  static constexpr int kO = kRows * kLd * 4;           // over the ring, at the end
  static constexpr int kBars = 256;
  static constexpr int kMax = 4 * kRows * 4;           // of the two threads of a row, two tiles
  static constexpr int kJoined = 2 * kRows * 4;
  static constexpr int kLine = 2 * kDim * 2;           // a key and its value
  static constexpr int kLines = kEdgeKeys * kLine;
  static constexpr int kAll = 1024 + kRing + kQ + kBars + kMax + kJoined + kLines;
  static_assert(kO + (int)sizeof(Inbox<kRows, kDim>) <= kRing, "the join fits the ring");
};

struct Bars {
  uint64_t full[8], empty[8], s_full[2], p_full[2], pv_done, o_full, drained;
  uint32_t tmem;
  int abort_flag;
};

// D (+)= A B with A (M x 16, 16-bit) in Tensor Memory.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory");
}

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(const __grid_constant__ Params prm) {
  using L = Layout<kDim>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - ptx::smem_addr(smem_raw) % 1024) % 1024;
  uint8_t* qs = smem + L::kRing;
  Bars& bars = *reinterpret_cast<Bars*>(qs + L::kQ);
  float* half_max = reinterpret_cast<float*>(qs + L::kQ + L::kBars);
  float* joined = half_max + 4 * kRows;
  uint8_t* lines = reinterpret_cast<uint8_t*>(joined + 2 * kRows);
  const AttnArgs& a = prm.a;
  const moe_attn_config& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  pdl_wait();
  pdl_trigger();
  Item it;
  if (!item_of<kThreads>(prm, prm.item_rows, it)) return;
  start_cluster(prm);
  Range rg = range_of(prm, it, prm.item_rows, kKeys);

  volatile int* abort_flag = &bars.abort_flag;
  // A warp's wait: all lanes go on, or none. After a wait has run out the
  // others return at once, and the softmax warps still meet at their barriers.
  auto warp_wait = [&](uint64_t& bar, uint32_t parity) {
    return __all_sync(0xffffffffu,
                      wait_phase(ptx::smem_addr(&bar), parity, abort_flag, a.status));
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      ptx::mbar_init(ptx::smem_addr(&bars.full[i]), 32 * kLoadWarps);
      ptx::mbar_init(ptx::smem_addr(&bars.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&bars.s_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars.p_full[i]), kSoftmax);
    }
    ptx::mbar_init(ptx::smem_addr(&bars.pv_done), 1);
    ptx::mbar_init(ptx::smem_addr(&bars.o_full), 1);
    ptx::mbar_init(ptx::smem_addr(&bars.drained), 1);
    bars.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_addr(&bars.tmem), kTmemCols);
    ptx::tmem_relinquish();
  }
  // The values of the keys that not every row sees.
  const int low = min(rg.lo_max, rg.hi_max + 1);         // lo_min .. low - 1
  const int after = max(rg.hi_min + 1, rg.lo_max);       // after .. hi_max
  const int below = max(0, low - rg.lo_min), edges = below + max(0, rg.hi_max + 1 - after);
  auto edge_key = [&](int e) { return e < below ? rg.lo_min + e : after + e - below; };
  bool wild = false;
  for (int i = threadIdx.x; i < edges * (kDim / 8); i += kThreads) {
    const Slot s = slot_of(prm, it, rg, edge_key(i / (kDim / 8)));
    s.check(prm);
    const int v = i % (kDim / 8);
    if (!s.in(c) || 8 * v >= c.head_dim) continue;
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v_cache) +
                                                    s.at(c, it.kh) + 8 * v);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int y = 0; y < 4; ++y)
      wild = wild || (w[y] & 0x7f80u) == 0x7f80u || (w[y] & 0x7f800000u) == 0x7f800000u;
  }
  ptx::tc_fence_before();
  wild = __syncthreads_or(wild);  // and the barriers and Tensor Memory are ready
  ptx::tc_fence_after();
  const uint32_t tmem = bars.tmem;
  const uint32_t ring = ptx::smem_addr(smem);

  // The keys of the products, in tiles of kKeys from key0 on.
  Range seen = rg;
  if (wild) seen.lo_min = rg.lo_max, seen.hi_max = rg.hi_min;
  const int key0 = seen.lo_min, keys = max(0, seen.hi_max + 1 - key0);
  {
    const int tiles = (keys + kKeys - 1) / kKeys;
    const int at = it.split * prm.parts + it.part, of = prm.splits * prm.parts;
    const int each = tiles / of, more = tiles - each * of;
    rg.t0 = at * each + min(at, more);
    rg.t1 = rg.t0 + each + (at < more);
  }
  const int n = rg.t1 - rg.t0;
  auto tile_key = [&](int i) { return key0 + (rg.t0 + i) * kKeys; };

  // Queries, in the layout of a K-major operand; negated for a negative scale,
  // so that larger products are larger scores. The copying warps are off
  // already; the warp that issues the products waits for the queries.
  if (warp <= kMmaWarp) {
    constexpr int kFill = kSoftmax + 32, kAll = kRows * kDim / 8;
    const uint32_t flip = c.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int i0 = 0; i0 < kAll; i0 += 4 * kFill) {
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kFill + threadIdx.x, r = i / (kDim / 8), v = i % (kDim / 8);
        x[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i < kAll && 8 * v < c.head_dim)
          x[k] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                 it.q_at(prm, r) + 8 * v);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kFill + threadIdx.x, r = i / (kDim / 8), v = i % (kDim / 8);
        if (i >= kAll) continue;
        x[k].x ^= flip, x[k].y ^= flip, x[k].z ^= flip, x[k].w ^= flip;
        *reinterpret_cast<uint4*>(qs + v / 8 * L::kHalf + r * 128 + ((v % 8 ^ (r & 7)) << 4)) = x[k];
      }
    }
    ptx::fence_proxy_async_smem();
    asm volatile("bar.sync 2, %0;" ::"n"(kFill) : "memory");
  }

  float m = -3.0e38f, l = 0.f;  // of this thread's row (l: of its half of the keys)
  const float scale = fabsf(c.scale) * 1.4426950408889634f;
  const int half = warp / 4, row = warp % 4 * 32 + lane;  // softmax warps
  const bool active = warp < 8 && warp % 4 * 32 < it.rows;
  const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
  constexpr int kCols = kDim / 2;  // columns of O a thread keeps
  const int pos = it.pos(prm, row), first = it.first(pos);

  if (warp < 8) {
    // ------------------------------------------------------------- softmax --
    for (int i = 0; i < n; ++i) {
      const int buf = i & 1;
      const bool go = warp_wait(bars.s_full[buf], (i >> 1) & 1) && active;
      ptx::tc_fence_after();
      const uint32_t s_at = tmem + lanes + buf * kKeys;
      uint32_t w[2][32];
      float top = -INFINITY;
      if (go) {
        ptx::tmem_ld32(s_at + 64 * half, w[0]);
        ptx::tmem_ld32(s_at + 64 * half + 32, w[1]);
        ptx::tmem_ld_wait();
        // columns from .. to - 1 of these 64 are keys that the row sees
        const int at = tile_key(i) + 64 * half;
        const int from = first - at, to = min(pos, seen.hi_max) + 1 - at;
        if (__any_sync(0xffffffffu, from > 0 || to < 64)) {
#pragma unroll
          for (int x = 0; x < 64; ++x)
            if (x < from || x >= to) w[x / 32][x % 32] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int x = 0; x < 64; ++x) top = fmaxf(top, __uint_as_float(w[x / 32][x % 32]));
        top *= scale;
        half_max[max_slot(i, half, row, kRows)] = top;
      }
      softmax_sync();  // and both threads of a row have read its scores
      if (go) {
        top = fmaxf(top, half_max[max_slot(i, half ^ 1, row, kRows)]);
        const bool raise = top > m + 8.f;
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ptx::ex2(m - top) : 1.f;
          if (raise) m = top;
          l *= f;
          if (i > 0) {
            // O is still while P of this tile is not there
            if (warp_wait(bars.pv_done, (i - 1) & 1)) {
              ptx::tc_fence_after();
#pragma unroll
              for (int x = 0; x < kCols; x += 16) {
                uint32_t o[16];
                const uint32_t at = tmem + lanes + kTmemO + half * kCols + x;
                ptx::tmem_ld16(at, o);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                ptx::tmem_st16(at, o);
              }
            }
          }
        }
        // Weights: high terms over S's columns 0-63, low terms over 64-127.
        const uint64_t scale2 = ptx::f32x2(scale, scale), minus_m = ptx::f32x2(-m, -m);
        uint64_t sum = 0;
#pragma unroll
        for (int x = 0; x < 64; x += 32) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const uint64_t v = ptx::fma_f32x2(
                (uint64_t)w[x / 32][2 * y + 1] << 32 | w[x / 32][2 * y], scale2, minus_m);
            const uint64_t p = ptx::f32x2(ptx::ex2(ptx::f32x2_lo(v)), ptx::ex2(ptx::f32x2_hi(v)));
            sum = ptx::add_f32x2(sum, p);
            split_bf16(p, hi[y], lo[y]);
          }
          ptx::tmem_st16(s_at + 32 * half + x / 2, hi);
          ptx::tmem_st16(s_at + 64 + 32 * half + x / 2, lo);
        }
        l += ptx::f32x2_lo(sum) + ptx::f32x2_hi(sum);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
      }
      ptx::mbar_arrive(ptx::smem_addr(&bars.p_full[buf]));
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products --
    if (lane == 0) {
      constexpr uint32_t kQk = ptx::idesc_bf16_f32(kRows, kKeys);
      constexpr uint32_t kPv = ptx::idesc_bf16_f32_mn(kRows, kDim, false);
      const uint32_t q_at = ptx::smem_addr(qs);
      int g = 0;  // slots taken so far
      auto take = [&](uint32_t& at) {  // the next slot's operand, ready to be read
        const int slot = g % L::kSlots;
        if (!wait_phase(ptx::smem_addr(&bars.full[slot]), (g / L::kSlots) & 1, abort_flag, a.status))
          return false;
        ptx::fence_proxy_async_smem();  // the copies were plain writes to shared memory
        at = ring + slot * L::kSlot;
        return true;
      };
      auto give = [&]() { ptx::mma_commit(ptx::smem_addr(&bars.empty[g++ % L::kSlots])); };
      auto scores = [&](int i) {
        uint32_t k_at;
        if (!take(k_at)) return false;
#pragma unroll
        for (int d = 0; d < kDim / 16; ++d) {
          const uint32_t off = d / 4 * L::kHalf + d % 4 * 32;
          ptx::mma_bf16(tmem + (i & 1) * kKeys, ptx::sdesc_k128(q_at + off),
                        ptx::sdesc_k128(k_at + off), kQk, d > 0);
        }
        ptx::mma_commit(ptx::smem_addr(&bars.s_full[i & 1]));
        give();
        return true;
      };
      bool ok = n == 0 || scores(0);
      for (int i = 0; ok && i < n; ++i) {
        if (i + 1 < n) {
          // the scores of tile i + 1 go where the weights of tile i - 1 are
          if (i > 0 && !wait_phase(ptx::smem_addr(&bars.pv_done), (i - 1) & 1, abort_flag, a.status))
            break;
          if (!scores(i + 1)) break;
        }
        uint32_t v_at;
        if (!wait_phase(ptx::smem_addr(&bars.p_full[i & 1]), (i >> 1) & 1, abort_flag, a.status) ||
            !take(v_at))
          break;
        ptx::tc_fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t)  // high terms, low terms
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_bf16_ta(tmem + kTmemO, tmem + (i & 1) * kKeys + 64 * t + 8 * k,
                        ptx::sdesc_mn128(v_at + k * 2048, L::kHalf), kPv, i > 0 || t > 0 || k > 0);
        ptx::mma_commit(ptx::smem_addr(&bars.pv_done));
        if (i + 1 == n) ptx::mma_commit(ptx::smem_addr(&bars.o_full));
        give();
      }
      if (*abort_flag) {  // leave no product in flight
        ptx::mma_commit(ptx::smem_addr(&bars.drained));
        drain_wait(ptx::smem_addr(&bars.drained), 0);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- copies --
    // One instruction copies 128 bytes (a half of 64 elements) of 4 keys.
    const int w = warp - kMmaWarp - 1, chunk = lane % 8;
    // Keys 32 (w + kLoadWarps x) .. + 31 are this warp's, one a lane to look up.
    constexpr int kSets = kKeys / 32 / kLoadWarps;
    struct Keys {
      Slot s[kSets];
    };
    struct Offsets {
      int64_t o[kSets];
    };
    auto look_up = [&](int i) {
      Keys k;
#pragma unroll
      for (int x = 0; x < kSets; ++x) {
        k.s[x] = {-1, -1};
        if (i < n)
          k.s[x] = slot_of(prm, it, seen, tile_key(i) + 32 * (w + kLoadWarps * x) + lane);
      }
      return k;
    };
    auto offsets = [&](const Keys& k) {
      Offsets r;
#pragma unroll
      for (int x = 0; x < kSets; ++x) {
        k.s[x].check(prm);
        r.o[x] = k.s[x].in(c) ? k.s[x].at(c, it.kh) : (int64_t)-1;
      }
      return r;
    };
    int g = 0;
    auto copy = [&](const void* cache, const Offsets& off) {
      const int slot = g % L::kSlots;
      if (!warp_wait(bars.empty[slot], ((g / L::kSlots) & 1) ^ 1)) return false;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(cache);
#pragma unroll
      for (int x = 0; x < kSets; ++x) {
        const int first = 32 * (w + kLoadWarps * x) + lane / 8;
        const uint32_t st = ring + slot * L::kSlot + first * 128;
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const int64_t o = __shfl_sync(0xffffffffu, off.o[x], k + lane / 8);
          const __nv_bfloat16* from = src + (o >= 0 ? o : 0) + 8 * chunk;
          const uint32_t to = st + k * 128 + ((chunk ^ ((first + k) & 7)) << 4);
#pragma unroll
          for (int h = 0; h < L::kHalves; ++h) {
            const bool in = o >= 0 && 64 * h + 8 * chunk < c.head_dim;
            ptx::cp_async16(to + h * L::kHalf, in ? from + 64 * h : src, in ? 16u : 0u);
          }
        }
      }
      ptx::cp_async_mbar_arrive(ptx::smem_addr(&bars.full[slot]));
      ++g;
      return true;
    };
    Offsets off = offsets(look_up(0));
    Keys next = look_up(1);
    bool ok = n == 0 || copy(a.k_cache, off);
    for (int i = 0; ok && i < n; ++i) {
      const Offsets off_v = off;
      if (i + 1 < n) {
        off = offsets(next);
        next = look_up(i + 2);
        if (!copy(a.k_cache, off)) break;
      }
      ok = copy(a.v_cache, off_v);
    }
    ptx::cp_async_wait_all();  // none in flight when the block's memory is used otherwise
  }

  // ---- the rows of O, and the keys that only some rows see ----
  float o[kCols];
#pragma unroll
  for (int x = 0; x < kCols; ++x) o[x] = 0.f;
  if (warp < 8) {
    if (n > 0 && active && warp_wait(bars.o_full, 0)) {
      ptx::tc_fence_after();
#pragma unroll
      for (int x = 0; x < kCols; x += 16) {
        uint32_t t[16];
        ptx::tmem_ld16(tmem + lanes + kTmemO + half * kCols + x, t);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int y = 0; y < 16; ++y) o[x + y] = __uint_as_float(t[y]);
      }
    }
    softmax_sync();
    half_max[half * kRows + row] = l;
    softmax_sync();
    l += half_max[(half ^ 1) * kRows + row];
    if (wild && it.split == 0 && it.part == 0) {
      for (int e0 = 0; e0 < edges; e0 += kEdgeKeys) {
        softmax_sync();  // the lines and half_max are free
        for (int x = threadIdx.x; x < kEdgeKeys * kDim / 4; x += kSoftmax) {
          const int e = e0 + x / (kDim / 4), v = x % (kDim / 8);
          uint4 y = make_uint4(0u, 0u, 0u, 0u);
          if (e < edges && 8 * v < c.head_dim) {
            const Slot s = slot_of(prm, it, rg, edge_key(e));
            if (s.in(c))
              y = *reinterpret_cast<const uint4*>(
                  static_cast<const __nv_bfloat16*>(x / (kDim / 8) % 2 ? a.v_cache : a.k_cache) +
                  s.at(c, it.kh) + 8 * v);
          }
          reinterpret_cast<uint4*>(lines)[x] = y;
        }
        softmax_sync();
        for (int e = e0; e < min(edges, e0 + kEdgeKeys); ++e) {
          const uint4* line = reinterpret_cast<const uint4*>(lines + (e - e0) * L::kLine);
          const int key = edge_key(e);
          float dot = 0.f;
#pragma unroll
          for (int v = 0; v < kCols / 8; ++v) {
            const int chunk = half * kCols / 8 + v;
            const uint4 x = *reinterpret_cast<const uint4*>(
                qs + chunk / 8 * L::kHalf + row * 128 + ((chunk % 8 ^ (row & 7)) << 4));
            const uint4 y = line[chunk];
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              float x0, x1, y0, y1;
              bf16x2_to_f32(xs[z], x0, x1);
              bf16x2_to_f32(ys[z], y0, y1);
              dot = fmaf(x0, y0, fmaf(x1, y1, dot));
            }
          }
          if (e > e0) softmax_sync();  // half_max has been read
          half_max[half * kRows + row] = dot;
          softmax_sync();
          if (key <= pos && key >= first) {
            // both threads of a row add the halves in the same order
            const float v = (half_max[row] + half_max[kRows + row]) * scale;
            const float top = fmaxf(m, v), f = ptx::ex2(m - top), p = ptx::ex2(v - top);
            m = top;
            l = l * f + p;
            const uint32_t* value = reinterpret_cast<const uint32_t*>(line) + kDim / 2 + half * kCols / 2;
#pragma unroll
            for (int x = 0; x < kCols; x += 2) {
              float y0, y1;
              bf16x2_to_f32(value[x / 2], y0, y1);
              o[x] = fmaf(p, y0, o[x] * f);
              o[x + 1] = fmaf(p, y1, o[x + 1] * f);
            }
          }
          __syncwarp();  // the barriers above are the whole warp's
        }
      }
    }
    ptx::tc_fence_before();
  }
  if (prm.parts == 1 && warp < 8 && row < it.rows) {
#pragma unroll
    for (int x = 0; x < kCols; x += 4) {
      const int v = (half * kCols + x) / 4;
      if (4 * v < c.head_dim)
        write_row<__nv_bfloat16>(prm, it, row, v, make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]),
                                 m, l);
    }
  }
  __syncthreads();  // all products and copies are done: the ring is free
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if (prm.parts == 1) return;
  if (warp < 8) {
    float* at = reinterpret_cast<float*>(smem) + row * L::kLd + half * kCols;
#pragma unroll
    for (int x = 0; x < kCols; x += 4)
      *reinterpret_cast<float4*>(at + x) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
    if (half == 0) {
      joined[row] = m;
      joined[kRows + row] = l;
    }
  }
  __syncthreads();
  finish<kRows, kDim, 1, kThreads, false, __nv_bfloat16>(
      prm, it, reinterpret_cast<float*>(smem), 0, L::kLd, joined,
      reinterpret_cast<Inbox<kRows, kDim>*>(smem + L::kO));
}

template <int kDim>
cudaError_t launch_one(const Params& p, unsigned blocks, cudaStream_t s) {
  static thread_local int configured = -1;
  return launch(tc_kernel<kDim>, &configured, p, blocks, kThreads, Layout<kDim>::kAll, s);
}

}  // namespace

cudaError_t launch_tc(const Params& p, int dim, unsigned blocks, cudaStream_t s) {
  return dim <= 64 ? launch_one<64>(p, blocks, s) : launch_one<128>(p, blocks, s);
}

}  // namespace attn
}  // namespace moe
