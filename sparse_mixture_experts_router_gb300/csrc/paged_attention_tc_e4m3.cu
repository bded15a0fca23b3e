// Attention of many query rows over an E4M3 cache with a scale per page and head,
// on tcgen05.
//
// An item has up to 128 rows, the M of a tcgen05.mma, and its keys go by in tiles of
// 128:
//   S (128 x 128) = Q K^T      fp16, both from shared memory
//   O (128 x D)  += P V        fp16, P from Tensor Memory (over the S it came from)
// tcgen05 takes E4M3 only against E4M3, for which queries and weights are too
// coarse; but every E4M3 code is an fp16 number, so the copying warps widen codes on
// their way into shared memory (one conversion for two codes) and leave the scales
// out. A page's scale is one number for all of its tokens, so it costs a thread
// nothing there: with s the score in log2 units and v the value's scale, the weight
// that meets the code is
//   2^s v / 2^M = 2^(s + log2 v - M),
// a fused multiply-add whose factor and addend are constants of 32 keys. (Where pages
// do not hold whole groups of 32, and once a scale outside 2^-40 .. 2^40 has come by, whose
// weights could leave fp32's range, it is 2^(s - M) times v.) M is the running reference of a
// row: when it is raised, the largest weight becomes 2^7, and it stands until one
// passes 2^15, so that fp16 holds weights to 2^-11 of themselves down to 2^-21 of
// the largest and none is off by more than 2^-32 of it. The sum of weights
// is taken without v (the group's sum times 1 / v); no weight without v passes 2^68.
//
// A row is a lane of Tensor Memory and one thread, which reads its scores 32 at a time and
// exchanges nothing; where some of them raise M, O and the tile's weights so far
// are scaled in place. 4 warps of softmax, 8 that widen keys and values (their codes
// loaded a tile ahead into registers), one that issues the products. Two blocks an SM, each with half of Tensor Memory (S 128 columns, O
// 128) and one tile of K and V: one's products run under the other's softmax.
//
// Keys that some rows of the item see and others do not (at most its new tokens at
// either end) are masked row by row; where one of their values is NaN (0 times NaN is
// not 0), those keys are left out of the products and added at the end, row by row.
#include "paged_attention.cuh"
#include "sm103_wait.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kSoftmaxWarps = 4, kCopyWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps + kCopyWarps;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // whole warpgroups
// Registers a thread: 64 at launch, which the warpgroups share out anew (softmax, two
// of copies, products: 104 + 2 x 56 + 40 = 4 x 64).
constexpr int kSoftmaxRegs = 104, kCopyRegs = 56, kMmaRegs = 40;
static_assert(kSoftmaxRegs + 2 * kCopyRegs + kMmaRegs <= 4 * 64, "");
constexpr int kKeys = 128, kRows = 128;
constexpr int kGroup = 32, kGroups = kKeys / kGroup;  // keys that may share a page
constexpr uint32_t kTmemCols = 256, kTmemO = 128;
constexpr int kEdgeKeys = 8;  // keys that only some rows see, taken at a time

template <int kDim>
struct Layout {
  static constexpr int kHalves = kDim / 64;      // 128-byte rows of 64 elements
  static constexpr int kHalf = 128 * 128;        // bytes: of 128 rows
  static constexpr int kTile = kHalves * kHalf;  // Q, K or V
  static constexpr int kInbox = (int)sizeof(Inbox<kRows, kDim>);
  static constexpr int kTiles = 3 * kTile > kInbox ? 3 * kTile : (kInbox + 1023) / 1024 * 1024;
  static constexpr int kBars = 128;
  static constexpr int kScales = 2 * 4 * kKeys * 4;  // of two tiles: of keys; of values; their log2 and inverse
  static constexpr int kLines = kEdgeKeys * (2 * kDim + 16);
  static constexpr int kAll = 1024 + kTiles + kBars + kScales + kLines;
};

struct Bars {
  // K, V of a tile are there; its scores (and K's slot is free); its weights; its
  // part of O (and V's slot and the weights' place are free)
  uint64_t k_full, v_full, s_full, p_full, pv_done, drained;
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 128, "");

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D (+)= A B with A (M x 16, 16-bit) in Tensor Memory.
__device__ __forceinline__ void mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  uint32_t x[16], y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = r[i], y[i] = r[16 + i];
  ptx::tmem_st16(at, x);
  ptx::tmem_st16(at + 16, y);
}
// Waits for this thread's tcgen05.ld; r, loaded by one of them, is not used before.
__device__ __forceinline__ void tmem_ready(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ uint32_t codes_f16(uint32_t v) {  // two codes, the low 16 bits
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v));
  return r;
}
__device__ __forceinline__ bool has_nan(uint32_t codes) {  // any of four
  return (((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
}
__device__ __forceinline__ bool has_nan(const uint4& v) {
  return has_nan(v.x) || has_nan(v.y) || has_nan(v.z) || has_nan(v.w);
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftmaxWarps) : "memory");
}

// kUniform: pages hold whole groups of 32 keys.
template <int kDim, bool kUniform>
__global__ void __launch_bounds__(kThreads, 2) tc_e4m3_kernel(const __grid_constant__ Params prm) {
  using L = Layout<kDim>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - ptx::smem_addr(smem_raw) % 1024) % 1024;
  uint8_t *qs = smem, *k_tile = smem + L::kTile, *v_tile = smem + 2 * L::kTile;
  Bars& bars = *reinterpret_cast<Bars*>(smem + L::kTiles);
  float* scales = reinterpret_cast<float*>(smem + L::kTiles + L::kBars);
  uint8_t* lines = reinterpret_cast<uint8_t*>(scales) + L::kScales;
  const AttnArgs& a = prm.a;
  const moe_attn_config& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  pdl_wait();
  pdl_trigger();
  Item it;
  if (!item_of<kThreads>(prm, prm.item_rows, it)) return;
  Range rg = range_of(prm, it, prm.item_rows, kKeys);

  volatile int* abort_flag = &bars.abort_flag;
  // A warp's wait: all lanes go on, or none. After one has run out the others
  // return at once.
  auto warp_wait = [&](uint64_t& bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_phase(ptx::smem_addr(&bar), parity, abort_flag, a.status));
  };
  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_addr(&bars.k_full), 32 * kCopyWarps);
    ptx::mbar_init(ptx::smem_addr(&bars.v_full), 32 * kCopyWarps);
    ptx::mbar_init(ptx::smem_addr(&bars.s_full), 1);
    ptx::mbar_init(ptx::smem_addr(&bars.p_full), 32 * kSoftmaxWarps);
    ptx::mbar_init(ptx::smem_addr(&bars.pv_done), 1);
    ptx::mbar_init(ptx::smem_addr(&bars.drained), 1);
    bars.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_addr(&bars.tmem), kTmemCols);
    ptx::tmem_relinquish();
  }
  // The values of the keys that not every row sees.
  const uint8_t* k_cache = static_cast<const uint8_t*>(a.k_cache);
  const uint8_t* v_cache = static_cast<const uint8_t*>(a.v_cache);
  const int row_vecs = c.head_dim / 16;
  const int low = min(rg.lo_max, rg.hi_max + 1);    // lo_min .. low - 1
  const int after = max(rg.hi_min + 1, rg.lo_max);  // after .. hi_max
  const int below = max(0, low - rg.lo_min), edges = below + max(0, rg.hi_max + 1 - after);
  auto edge_key = [&](int e) { return e < below ? rg.lo_min + e : after + e - below; };
  bool wild = false;
  for (int i = threadIdx.x; i < edges * 8; i += kThreads) {
    const Slot s = slot_of(prm, it, rg, edge_key(i / 8));
    s.check(prm);
    if (i % 8 >= row_vecs || !s.in(c)) continue;
    wild = wild || has_nan(*reinterpret_cast<const uint4*>(v_cache + s.at(c, it.kh) + i % 8 * 16)) ||
           !(a.v_scale[s.scale_at(c, it.kh)] <= 3.4e38f);
  }
  ptx::tc_fence_before();
  wild = __syncthreads_or(wild);  // and the barriers and Tensor Memory are ready
  ptx::tc_fence_after();
  const uint32_t tmem = bars.tmem;

  // The keys of the products, in tiles of kKeys from key0 on.
  Range seen = rg;
  if (wild) seen.lo_min = rg.lo_max, seen.hi_max = rg.hi_min;
  const int key0 = seen.lo_min / kGroup * kGroup;
  {
    const int tiles = seen.hi_max < seen.lo_min ? 0 : (seen.hi_max - key0) / kKeys + 1;
    const int at = it.split * prm.parts + it.part, of = prm.splits * prm.parts;
    const int each = tiles / of, more = tiles - each * of;
    rg.t0 = at * each + min(at, more);
    rg.t1 = rg.t0 + each + (at < more);
  }
  const int n = rg.t1 - rg.t0;
  auto tile_key = [&](int i) { return key0 + (rg.t0 + i) * kKeys; };

  float m = -3.0e38f, l = 0.f, factor = 0.f;  // of this thread's row; factor of its scores, log2 units
  bool wide = false;                          // scales outside 2^-40 .. 2^40 have come by
  const int row = warp * 32 + lane;
  const bool active = warp < kSoftmaxWarps && warp * 32 < it.rows;
  const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
  const int pos = it.pos(prm, row), first = it.first(pos);

  if (warp < kSoftmaxWarps) {
    more_registers<kSoftmaxRegs>();
    // ------------------------------------------------------------- queries --
    // As fp16, each row scaled by a power of two to [2^14, 2^15) for its largest element
    // (negated for a negative scale, so that larger products are larger scores).
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + it.q_at(prm, row));
    uint4 x[kDim / 8];
#pragma unroll
    for (int v = 0; v < kDim / 8; ++v) {
      x[v] = make_uint4(0u, 0u, 0u, 0u);
      if (8 * v < c.head_dim) x[v] = q[v];
    }
    float amax = 0.f;
#pragma unroll
    for (int v = 0; v < kDim / 8; ++v) {
      const uint32_t w[4] = {x[v].x, x[v].y, x[v].z, x[v].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float lo, hi;
        bf16x2_to_f32(w[y], lo, hi);
        amax = fmaxf(amax, fmaxf(fabsf(lo), fabsf(hi)));
      }
    }
    const int e = clamp_int((int)(__float_as_uint(amax) >> 23) - 127, -112, 128);
    const float down = copysignf(__uint_as_float((uint32_t)(141 - e) << 23), c.scale);
    factor = fabsf(c.scale) * 1.4426950408889634f * __uint_as_float((uint32_t)(113 + e) << 23);
#pragma unroll
    for (int v = 0; v < kDim / 8; ++v) {
      uint32_t w[4] = {x[v].x, x[v].y, x[v].z, x[v].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float lo, hi;
        bf16x2_to_f32(w[y], lo, hi);
        w[y] = pack_f16(lo * down, hi * down);
      }
      *reinterpret_cast<uint4*>(qs + v / 8 * L::kHalf + row * 128 + ((v % 8 ^ (row & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    ptx::fence_proxy_async_smem();
    asm volatile("bar.arrive 2, %0;" ::"n"(32 * kSoftmaxWarps + 32) : "memory");
    // ------------------------------------------------------------- softmax --
    // Weights of keys 32 g .. + 31 of tile i from their scores w, into P.
    auto weights = [&](int i, int g, uint32_t (&w)[32]) {
      const float* fk = scales + (i & 1) * 4 * kKeys;
      const float *fv = fk + kKeys, *ev = fv + kKeys, *iv = ev + kKeys;
      const int at = tile_key(i) + kGroup * g;
      // columns from .. to - 1 are keys that the row sees
      const int from = max(first, seen.lo_min) - at, to = min(pos, seen.hi_max) + 1 - at;
      if (__any_sync(0xffffffffu, from > 0 || to < kGroup)) {
#pragma unroll
        for (int x = 0; x < kGroup; ++x)
          if (x < from || x >= to) w[x] = 0xff800000u;  // -inf
      }
      // the largest score, and the largest with its value's scale
      float top = -INFINITY, top_v = -INFINITY;
      if (kUniform) {
        float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 32; ++x) t[x % 4] = fmaxf(t[x % 4], __uint_as_float(w[x]));
        top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * (factor * fk[g]);
        top_v = top + ev[g];
        wide = wide || !(fabsf(ev[g]) <= 40.f);
      } else {
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float t = __uint_as_float(w[x]) * (factor * fk[kGroup * g + x]);
          top = fmaxf(top, t);
          top_v = fmaxf(top_v, t + ev[kGroup * g + x]);
        }
      }
      const bool raise = top_v > m + 15.f || top > m + 68.f;
      if (__any_sync(0xffffffffu, raise)) {
        const float up = raise ? fmaxf(top_v - 7.f, top - 60.f) : m, f = ptx::ex2(m - up);
        m = up;
        l *= f;
        uint32_t o[16];
        if (i > 0) {  // O is still while P of this tile is not there
#pragma unroll 1
          for (int x = 0; x < kDim; x += 16) {
            ptx::tmem_ld16(tmem + lanes + kTmemO + x, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            ptx::tmem_st16(tmem + lanes + kTmemO + x, o);
          }
        }
#pragma unroll 1
        for (int x = 0; x < g; ++x) {  // this tile's weights so far
          ptx::tmem_st_wait();
          ptx::tmem_ld16(tmem + lanes + 16 * x, o);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const float2 p = unpack_f16(o[y]);
            o[y] = pack_f16(p.x * f, p.y * f);
          }
          ptx::tmem_st16(tmem + lanes + 16 * x, o);
        }
      }
      uint64_t sum[2] = {0, 0};
      uint32_t p[16];
      if (kUniform && !wide) {
        const float f1 = factor * fk[g], a1 = ev[g] - m;
        const uint64_t f2 = ptx::f32x2(f1, f1), a2 = ptx::f32x2(a1, a1);
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const uint64_t v = ptx::fma_f32x2((uint64_t)w[2 * y + 1] << 32 | w[2 * y], f2, a2);
          const float lo = ptx::ex2(ptx::f32x2_lo(v)), hi = ptx::ex2(ptx::f32x2_hi(v));
          sum[y % 2] = ptx::add_f32x2(sum[y % 2], ptx::f32x2(lo, hi));
          p[y] = pack_f16(lo, hi);
        }
        sum[0] = ptx::add_f32x2(sum[0], sum[1]);
        l = fmaf(ptx::f32x2_lo(sum[0]) + ptx::f32x2_hi(sum[0]), iv[g], l);
      } else {
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const int k = kUniform ? g : kGroup * g + 2 * y, k1 = kUniform ? g : k + 1;
          const float lo = ptx::ex2(fmaf(__uint_as_float(w[2 * y]), factor * fk[k], -m));
          const float hi = ptx::ex2(fmaf(__uint_as_float(w[2 * y + 1]), factor * fk[k1], -m));
          sum[y % 2] = ptx::add_f32x2(sum[y % 2], ptx::f32x2(lo, hi));
          p[y] = pack_f16(lo * fv[k], hi * fv[k1]);
        }
        sum[0] = ptx::add_f32x2(sum[0], sum[1]);
        l += ptx::f32x2_lo(sum[0]) + ptx::f32x2_hi(sum[0]);
      }
      ptx::tmem_st16(tmem + lanes + 16 * g, p);  // over scores that have been read
    };
    for (int i = 0; i < n; ++i) {
      if (warp_wait(bars.s_full, i & 1) && active) {
        ptx::tc_fence_after();
#pragma unroll 1
        for (int g = 0; g < kGroups; ++g) {
          uint32_t w[32];
          ptx::tmem_ld32(tmem + lanes + kGroup * g, w);
          tmem_ready(w);
          weights(i, g, w);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
      }
      ptx::mbar_arrive(ptx::smem_addr(&bars.p_full));
    }
  // ---- the keys that only some rows see, where a value is NaN ----
  {
    const bool go = n == 0 || warp_wait(bars.pv_done, (n - 1) & 1);
    ptx::tc_fence_after();
    if (wild && it.split == 0 && it.part == 0 && go) {
      if (n == 0) {
        uint32_t z[32] = {};
#pragma unroll
        for (int x = 0; x < kDim; x += 32) tmem_st32(tmem + lanes + kTmemO + x, z);
        ptx::tmem_st_wait();
      }
      float* line_scale = reinterpret_cast<float*>(lines + kEdgeKeys * 2 * kDim);
      for (int e0 = 0; e0 < edges; e0 += kEdgeKeys) {
        softmax_sync();  // the lines are free
        for (int x = threadIdx.x; x < kEdgeKeys * kDim / 8; x += 32 * kSoftmaxWarps) {
          const int e = e0 + x / (kDim / 8), v = x % (kDim / 8) % (kDim / 16);
          const bool value = x % (kDim / 8) >= kDim / 16;
          uint4 y = make_uint4(0u, 0u, 0u, 0u);
          if (e < edges) {
            const Slot s = slot_of(prm, it, rg, edge_key(e));
            if (s.in(c)) {
              if (v < row_vecs)
                y = *reinterpret_cast<const uint4*>((value ? v_cache : k_cache) + s.at(c, it.kh) + 16 * v);
              if (v == 0)
                line_scale[2 * (e - e0) + value] = (value ? a.v_scale : a.k_scale)[s.scale_at(c, it.kh)];
            }
          }
          reinterpret_cast<uint4*>(lines)[x] = y;
        }
        softmax_sync();
        for (int e = e0; e < min(edges, e0 + kEdgeKeys); ++e) {
          const int key = edge_key(e);
          const uint8_t* line = lines + (e - e0) * 2 * kDim;
          const bool see = key <= pos && key >= first;
          float dot = 0.f;
          for (int v = 0; v < c.head_dim / 8; ++v) {
            const uint4 x = *reinterpret_cast<const uint4*>(qs + v / 8 * L::kHalf + row * 128 +
                                                            ((v % 8 ^ (row & 7)) << 4));
            const uint2 y = *reinterpret_cast<const uint2*>(line + 8 * v);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
            const uint32_t ys[4] = {codes_f16(y.x), codes_f16(y.x >> 16), codes_f16(y.y), codes_f16(y.y >> 16)};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const float2 qx = unpack_f16(xs[z]), kx = unpack_f16(ys[z]);
              dot = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, dot));
            }
          }
          // weight and O relative to the largest of both, in fp32
          const float s = dot * (factor * line_scale[2 * (e - e0)]), vs = line_scale[2 * (e - e0) + 1];
          const float up = see && s > m ? s : m, f = ptx::ex2(m - up), p = see ? ptx::ex2(s - up) : 0.f;
          m = up;
          l = l * f + p;
          for (int x = 0; x < kDim; x += 32) {
            uint32_t o[32];
            ptx::tmem_ld32(tmem + lanes + kTmemO + x, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 32; y += 2) {
              const float2 v = unpack_f16(codes_f16(*reinterpret_cast<const uint16_t*>(line + kDim + x + y)));
              const float o0 = __uint_as_float(o[y]) * f, o1 = __uint_as_float(o[y + 1]) * f;
              o[y] = __float_as_uint(see ? fmaf(p * vs, v.x, o0) : o0);
              o[y + 1] = __float_as_uint(see ? fmaf(p * vs, v.y, o1) : o1);
            }
            tmem_st32(tmem + lanes + kTmemO + x, o);
          }
          ptx::tmem_st_wait();
        }
      }
    }
  }
  const bool any = n > 0 || (wild && it.split == 0 && it.part == 0);  // O is there
  const int vecs = c.head_dim / 4;
  if (prm.parts == 1) {
    if (active) {
#pragma unroll
      for (int x = 0; x < kDim; x += 32) {
        uint32_t o[32];
        ptx::tmem_ld32(tmem + lanes + kTmemO + x, o);
        ptx::tmem_ld_wait();
        if (row < it.rows) {
#pragma unroll
          for (int y = 0; y < 32; y += 4)
            if (x + y < c.head_dim)
              write_row<__nv_bfloat16>(prm, it, row, (x + y) / 4,
                                       any ? make_float4(__uint_as_float(o[y]), __uint_as_float(o[y + 1]),
                                                         __uint_as_float(o[y + 2]), __uint_as_float(o[y + 3]))
                                           : make_float4(0.f, 0.f, 0.f, 0.f),
                                       m, l);
        }
      }
      ptx::tc_fence_before();
    }
  } else {
    // Every block's tiles are free: each sends the others their slices of O.
    auto* inbox = reinterpret_cast<Inbox<kRows, kDim>*>(smem);
    __syncwarp();
    ptx::cluster_sync();
    const int slice = div(prm.by_parts, it.rows * vecs + prm.parts - 1);
    if (active) {
      if (row < it.rows)
        for (int b = 0; b < prm.parts; ++b)
          ptx::st_cluster_v2(ptx::mapa_shared(ptx::smem_addr(&inbox->ml[it.part][row]), b), m, l);
      int i = row * vecs, to = i / slice;
#pragma unroll
      for (int x = 0; x < kDim; x += 32) {
        uint32_t o[32];
        ptx::tmem_ld32(tmem + lanes + kTmemO + x, o);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int y = 0; y < 32; y += 4) {
          if (row >= it.rows || x + y >= c.head_dim) continue;
          if (i >= (to + 1) * slice) ++to;
          ptx::st_cluster_v4(
              ptx::mapa_shared(ptx::smem_addr(&inbox->o[it.part * slice + i - to * slice]), to),
              any ? make_float4(__uint_as_float(o[y]), __uint_as_float(o[y + 1]), __uint_as_float(o[y + 2]),
                                __uint_as_float(o[y + 3]))
                  : make_float4(0.f, 0.f, 0.f, 0.f));
          ++i;
        }
      }
      ptx::tc_fence_before();
    }
    __syncwarp();
    ptx::cluster_sync();
  }
  __syncthreads();
  if (prm.parts > 1)
    join_slices<kRows, kDim, 32 * kSoftmaxWarps, __nv_bfloat16>(prm, it, reinterpret_cast<Inbox<kRows, kDim>*>(smem));
  } else if (warp >= kMmaWarp) {
    fewer_registers<kMmaRegs>();
    // ------------------------------------------------------------ products --
    if (warp == kMmaWarp) {
      asm volatile("bar.sync 2, %0;" ::"n"(32 * kSoftmaxWarps + 32) : "memory");  // the queries
      const bool issues = elect_one();
      const uint32_t qk = idesc_f16(kRows, kKeys, false), pv = idesc_f16(kRows, c.head_dim, true);
      // operands: an offset in bytes is added to the address field, in units of 16
      const uint64_t q_desc = ptx::sdesc_k128(ptx::smem_addr(qs)), k_desc = ptx::sdesc_k128(ptx::smem_addr(k_tile));
      const uint64_t v_desc = ptx::sdesc_mn128(ptx::smem_addr(v_tile), L::kHalf);
      for (int i = 0; i < n; ++i) {
        // K is there; the weights of tile i - 1 have been used
        if (!warp_wait(bars.k_full, i & 1) || (i > 0 && !warp_wait(bars.pv_done, (i - 1) & 1))) break;
        ptx::tc_fence_after();
        if (issues) {
#pragma unroll
          for (int d = 0; d < kDim / 16; ++d) {
            const uint32_t off = (d / 4 * L::kHalf + d % 4 * 32) >> 4;
            if (d < row_vecs) ptx::mma_bf16(tmem, q_desc + off, k_desc + off, qk, d > 0);
          }
          ptx::mma_commit(ptx::smem_addr(&bars.s_full));
        }
        if (!warp_wait(bars.v_full, i & 1) || !warp_wait(bars.p_full, i & 1)) break;
        ptx::tc_fence_after();
        if (issues) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ta(tmem + kTmemO, tmem + 8 * k, v_desc + (k * 2048 >> 4), pv, i > 0 || k > 0);
          ptx::mma_commit(ptx::smem_addr(&bars.pv_done));
        }
      }
      __syncwarp();
      if (issues && *abort_flag) {  // leave no product in flight
        ptx::mma_commit(ptx::smem_addr(&bars.drained));
        drain_wait(ptx::smem_addr(&bars.drained), 0);
      }
      __syncwarp();
    }
    if (prm.parts > 1) {  // with the softmax warps
      ptx::cluster_sync();
      ptx::cluster_sync();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
      ptx::tc_fence_after();
      ptx::tmem_dealloc(tmem, kTmemCols);
    }
  } else {
    fewer_registers<kCopyRegs>();
    // -------------------------------------------------------------- copies --
    // Keys 16 w .. + 15 of a tile are this warp's. One load takes 16 codes a lane, of
    // kPer keys a warp; they become two 16-byte chunks of the key's row.
    constexpr int kMine = kKeys / kCopyWarps, kShare = kGroup / kMine;  // warps of a group
    constexpr int kVecs = kDim / 16, kPer = 32 / kVecs, kLoads = kMine / kPer;
    const int w = warp - kSoftmaxWarps, vec = lane % kVecs, sub = lane / kVecs;
    const bool held = vec < row_vecs;
    auto look_up = [&](int i) {
      Slot s = {-1, -1};
      if (kUniform) {  // the keys of the group
        if (i < n) s = slot_of(prm, it, seen, tile_key(i) + kGroup * (w / kShare) + lane);
      } else if (i < n && lane < kMine) {
        s = slot_of(prm, it, seen, tile_key(i) + kMine * w + lane);
      }
      return s;
    };
    // Of this lane's key; where a group has one page, of the group's first key, whether a
    // row sees it or not.
    struct Place {
      int64_t at;    // -1: none
      float ks, vs;  // its page's scales
      int from;      // the lane that has them
    };
    auto place = [&](const Slot& s) {
      s.check(prm);
      Place p = {-1, 1.f, 1.f, 0};
      if (s.in(c)) {
        p.at = s.at(c, it.kh);
        p.ks = __ldg(a.k_scale + s.scale_at(c, it.kh));
        p.vs = __ldg(a.v_scale + s.scale_at(c, it.kh));
      }
      if (kUniform) {
        p.at -= lane * c.token_stride;
        const unsigned with = __ballot_sync(0xffffffffu, s.in(c));
        p.from = with ? __ffs(with) - 1 : 0;
        p.at = __shfl_sync(0xffffffffu, p.at, p.from);
        if (!with) p.at = INT64_MIN;
      }
      return p;
    };
    const int64_t sub_at = (int64_t)(w % kShare * kMine + sub) * c.token_stride + 16 * vec, step = (int64_t)kPer * c.token_stride;
    uint4 rk[kLoads], rv[kLoads];
    // Codes of tile i, whose place is p.
    auto fetch = [&](const uint8_t* cache, int i, const Place& p, uint4 (&r)[kLoads]) {
      const int key = tile_key(i) + kMine * w + sub;
      const uint8_t* at = cache + p.at + sub_at;
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        r[x] = make_uint4(0u, 0u, 0u, 0u);
        if (kUniform) {
          const int k = key + x * kPer;
          if (held && p.at != INT64_MIN && k >= seen.lo_min && k <= seen.hi_max)
            r[x] = __ldg(reinterpret_cast<const uint4*>(at + x * step));
        } else {
          const int64_t o = __shfl_sync(0xffffffffu, p.at, x * kPer + sub);
          if (o >= 0 && held) r[x] = __ldg(reinterpret_cast<const uint4*>(cache + o) + vec);
        }
      }
    };
    // The two chunks in an order that keeps the eight lanes of a store apart.
    auto widen = [&](uint8_t* tile, const uint4 (&r)[kLoads]) {
      const int half = vec / 4, c0 = 2 * (vec % 4);
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        const int key = kMine * w + x * kPer + sub;
        uint8_t* at = tile + half * L::kHalf + key * 128;
        uint4 lo, hi;
        lo.x = codes_f16(r[x].x), lo.y = codes_f16(r[x].x >> 16);
        lo.z = codes_f16(r[x].y), lo.w = codes_f16(r[x].y >> 16);
        hi.x = codes_f16(r[x].z), hi.y = codes_f16(r[x].z >> 16);
        hi.z = codes_f16(r[x].w), hi.w = codes_f16(r[x].w >> 16);
        if (!held) continue;
        const bool swap = half;
        *reinterpret_cast<uint4*>(at + (((c0 + swap) ^ (key & 7)) << 4)) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(at + (((c0 + !swap) ^ (key & 7)) << 4)) = swap ? lo : hi;
      }
    };
    // K of tile i, with its scales: into the slot that tile i - 1's scores have left.
    auto put_k = [&](int i, const Place& p) {
      widen(k_tile, rk);
      float* fk = scales + (i & 1) * 4 * kKeys;
      if (kUniform ? lane == p.from && w % kShare == 0 : lane < kMine) {
        const int k = kUniform ? w / kShare : kMine * w + lane;
        fk[k] = p.ks;
        fk[kKeys + k] = p.vs;
        fk[2 * kKeys + k] = log2f(p.vs);
        if (kUniform) fk[3 * kKeys + k] = __fdiv_rn(1.f, p.vs);
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_addr(&bars.k_full));
    };
    Place next = place(look_up(0));  // of the tile after the one at work
    Slot after_next = look_up(1);
    if (n > 0) {
      fetch(k_cache, 0, next, rk);
      fetch(v_cache, 0, next, rv);
      put_k(0, next);
      next = place(after_next);
      after_next = look_up(2);
      fetch(k_cache, 1, next, rk);
    }
    for (int i = 0; i < n; ++i) {
      if (i > 0 && !warp_wait(bars.pv_done, (i - 1) & 1)) break;  // V's slot is free
      widen(v_tile, rv);
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_addr(&bars.v_full));
      if (i + 1 == n) break;
      fetch(v_cache, i + 1, next, rv);
      if (!warp_wait(bars.s_full, i & 1)) break;  // K's slot is free
      put_k(i + 1, next);
      next = place(after_next);
      after_next = look_up(i + 3);
      fetch(k_cache, i + 2, next, rk);
    }
    __syncwarp();
    if (prm.parts > 1) {
      ptx::cluster_sync();
      ptx::cluster_sync();
    }
    __syncthreads();
  }
}

template <int kDim, bool kUniform>
cudaError_t launch_one(const Params& p, unsigned blocks, cudaStream_t s) {
  static thread_local int configured = -1;
  return launch(tc_e4m3_kernel<kDim, kUniform>, &configured, p, blocks, kThreads, Layout<kDim>::kAll, s);
}

}  // namespace

cudaError_t launch_tc_e4m3(const Params& p, int dim, unsigned blocks, cudaStream_t s) {
  if (p.a.c.page_size % kGroup == 0)
    return dim <= 64 ? launch_one<64, true>(p, blocks, s) : launch_one<128, true>(p, blocks, s);
  return dim <= 64 ? launch_one<64, false>(p, blocks, s) : launch_one<128, false>(p, blocks, s);
}

}  // namespace attn
}  // namespace moe
