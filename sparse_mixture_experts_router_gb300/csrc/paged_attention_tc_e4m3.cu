// Attention of many query rows over an E4M3 cache with a scale per page and head,
// on tcgen05.
//
// Per tile of 128 keys and 128 rows (the M of a tcgen05.mma):
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
// do not hold whole groups of 32 it is 2^(s - M) times v.) M is the running reference of a
// row: when it is raised, the largest weight becomes 2^7, and it stands until one
// passes 2^15, so that fp16 holds weights to 2^-11 of themselves down to 2^-21 of
// the largest and none is off by more than 2^-32 of it. The sum of weights
// is taken without v (the group's sum times 1 / v), relative to 2^M too: scales of 2^-40 ..
// 2^40 leave all of that in fp32's range. Once another has come by, the sum has a reference
// of its own, which follows the scores without v, and a weight takes two exponentials.
//
// A block has the SM and runs two streams of tiles, each with its S and O in Tensor
// Memory, four warps of softmax and a warp that issues its products, so that one's
// products run under the other's softmax. An item of more than 128 rows (up to 256) is
// two streams of rows that share the tiles of keys; one of up to 128 rows is two
// streams of keys (even tiles and odd ones), joined at the end. A row is a lane of
// Tensor Memory and one thread, which has the tile's 128 scores in registers. 4 warps
// widen keys and values, two tiles of each ahead.
//
// Keys that some rows of the item see and others do not (at most its new tokens at
// either end) are masked row by row; where one of their values is NaN (0 times NaN is
// not 0), those keys are left out of the products and added at the end, row by row.
//
// 4 sequences of 200 to 1024 new tokens over 1500 to 4000 keys, 32/8 heads of 128, pages of
// 64: 150 to 203 us as the lengths fall, 184 to 195 and 500 to 530 TFLOP/s, 0.27 to 0.28 of the
// measured dense rate, for the mean of them (578 us in the warp-level kernel's blocks of 16 rows).
// Pages that do not hold whole groups of 32 keys: 216 to 298 us, as each key has its own lookup
// and each score its own factors. Bound by latency: of a stream's tile about 2800
// cycles were softmax when the first took 205 (a warp alone on its scheduler issues every 5 to 6
// cycles, and has 128 scores to load, compare, exponentiate, round and store), 530 Q K^T and 1000
// P V, and two streams overlap so far that the tensor pipe is busy 29% of the time; and items of
// unequal length, one an SM, leave a last wave that few of them fill. One stream and 16 warps took
// 243 us, two threads a row with two blocks an SM 253 (spills); with 8 warps that widen, 40
// rows of 32 sequences took 292 us for 264. Far scales in the tile's one path, and not in one
// of their own, cost 3 to 8%.
#include <cfloat>

#include "paged_attention.cuh"
#include "sm103_wait.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kSoftmaxWarps = 8, kCopyWarps = 4;  // four a stream; four
constexpr int kMmaWarp = kSoftmaxWarps + kCopyWarps;  // a stream's: + 0, + 1
constexpr int kThreads = 32 * (kMmaWarp + 4);         // whole warpgroups
// Registers a thread: 128 at launch, which the warpgroups share out anew (128 scores and
// their addresses take 184; the copies in flight 104).
constexpr int kSoftmaxRegs = 184, kCopyRegs = 104, kMmaRegs = 40;
static_assert(2 * kSoftmaxRegs + kCopyRegs + kMmaRegs <= 4 * 128, "");
constexpr int kKeys = 128, kTileRows = 128, kRows = 2 * kTileRows;
constexpr int kGroup = 32, kGroups = kKeys / kGroup;  // keys that may share a page
constexpr uint32_t kTmemCols = 512, kTmemO = 256;     // S of each stream, O of each
constexpr int kEdgeKeys = 8;  // keys that only some rows see, taken at a time

template <int kDim>
struct Layout {
  static constexpr int kHalves = kDim / 64;      // 128-byte rows of 64 elements
  static constexpr int kHalf = 128 * 128;        // bytes: of 128 rows
  static constexpr int kTile = kHalves * kHalf;  // 128 rows of Q, K or V
  static constexpr int kK = 2 * kTile, kV = 4 * kTile, kRing = 6 * kTile;
  static constexpr int kLd = kDim + 4;           // floats a row of a stream's O, to be joined
  static constexpr int kInbox = ((int)sizeof(Inbox<kRows, kDim, true>) + 1023) / 1024 * 1024;
  static constexpr int kTiles = kRing > kInbox ? kRing : kInbox;
  static_assert(kTileRows * kLd * 4 <= kRing - kK, "a stream's O fits over K and V");
  static constexpr int kBars = 256;
  // of four tiles: of keys; of values, their log2 and inverse
  static constexpr int kScales = 4 * 4 * kKeys * 4;
  static constexpr int kLines = kEdgeKeys * (2 * kDim + 16);
  static constexpr int kJoin = kTileRows * (16 + 8);
  static constexpr int kAll = 1024 + kTiles + kBars + kScales + kLines + kJoin;
};

struct Bars {
  // of the two slots of K and of V: filled, used by every stream that uses them
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
  // of a stream: a tile's scores are there, its weights, its part of O
  uint64_t s_full[2], p_full[2], pv_done[2], drained[2];
  uint32_t tmem;
  int abort_flag;
  int far_tile;  // the first of the block's tiles with a value's scale outside 2^-40 .. 2^40
};
static_assert(sizeof(Bars) <= 256, "");

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
// Two codes (the low 16 bits of v) as fp16.
__device__ __forceinline__ uint32_t codes_f16(uint32_t v) {
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
// 16 bytes that are read once (not to push other things out of the first-level cache), or
// zeros. One predicated load, so that nothing waits for it before it is used.
__device__ __forceinline__ uint4 ld_once(const void* p, bool there) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)there));
  return v;
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
__global__ void __launch_bounds__(kThreads, 1) tc_e4m3_kernel(const __grid_constant__ Params prm) {
  using L = Layout<kDim>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - ptx::smem_addr(smem_raw) % 1024) % 1024;
  Bars& bars = *reinterpret_cast<Bars*>(smem + L::kTiles);
  float* scales = reinterpret_cast<float*>(smem + L::kTiles + L::kBars);
  uint8_t* lines = reinterpret_cast<uint8_t*>(scales) + L::kScales;
  float4* of_odd = reinterpret_cast<float4*>(lines + L::kLines);  // the odd stream's (M, sum, the sum's reference) of a row
  float* sum_refs = reinterpret_cast<float*>(of_odd + kTileRows);  // of the streams' rows, where that is not M
  const AttnArgs& a = prm.a;
  const moe_attn_config& c = a.c;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;

  pdl_wait();
  pdl_trigger();
  Item it;
  if (!item_of<kThreads>(prm, prm.item_rows, it)) return;
  Range rg = range_of(prm, it, prm.item_rows, kKeys);
  const bool by_rows = prm.item_rows > kTileRows;  // the streams are of rows, else of keys
  // streams that use a tile of keys: both, where the item has rows for both
  const int users = by_rows && it.rows > kTileRows ? 2 : 1;

  volatile int* abort_flag = &bars.abort_flag;
  // A warp's wait: all lanes go on, or none. After one has run out the others
  // return at once.
  auto warp_wait = [&](uint64_t& bar, int phase) {
    return __all_sync(0xffffffffu, wait_phase(ptx::smem_addr(&bar), (uint32_t)phase & 1, abort_flag, a.status));
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&bars.k_full[i]), 32 * kCopyWarps);
      ptx::mbar_init(ptx::smem_addr(&bars.v_full[i]), 32 * kCopyWarps);
      ptx::mbar_init(ptx::smem_addr(&bars.k_free[i]), users);
      ptx::mbar_init(ptx::smem_addr(&bars.v_free[i]), users);
      ptx::mbar_init(ptx::smem_addr(&bars.s_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars.p_full[i]), 32 * kSoftmaxWarps / 2);
      ptx::mbar_init(ptx::smem_addr(&bars.pv_done[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars.drained[i]), 1);
    }
    bars.abort_flag = 0;
    bars.far_tile = 0x7fffffff;
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

  // The keys of the products, in tiles of kKeys from key0 on: this block's n tiles.
  Range seen = rg;
  if (wild) seen.lo_min = rg.lo_max, seen.hi_max = rg.hi_min;
  int key0 = seen.lo_min / kGroup * kGroup, n;
  {
    const int tiles = seen.hi_max < seen.lo_min ? 0 : (seen.hi_max - key0) / kKeys + 1;
    const int at = it.split * prm.parts + it.part, of = prm.splits * prm.parts;
    const int each = tiles / of, more = tiles - each * of;
    key0 += (at * each + min(at, more)) * kKeys;
    n = each + (at < more);
  }
  // Stream st's tiles: all, or every other.
  const int t_step = by_rows ? 1 : 2;
  auto tiles_of = [&](int st) { return by_rows ? (st < users ? n : 0) : (n - st + 1) / 2; };
  auto tile_of = [&](int st, int t) { return by_rows ? t : 2 * t + st; };

  if (warp < kSoftmaxWarps) {
    more_registers<kSoftmaxRegs>();
    const int st = warp / 4, row_in = warp % 4 * 32 + lane, row = by_rows ? st * kTileRows + row_in : row_in;
    const int rows_here = by_rows ? it.rows - st * kTileRows : it.rows;
    const bool active = warp % 4 * 32 < rows_here;
    const int my_tiles = tiles_of(st);
    uint8_t* qs = smem + (by_rows ? st * L::kTile : 0);
    // ------------------------------------------------------------- queries --
    // As fp16, each row scaled by a power of two to [2^14, 2^15) for its largest element
    // (negated for a negative scale, so that larger products are larger scores).
    float factor;  // of the row's scores, log2 units
    {
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
      if (by_rows || st == 0) {
#pragma unroll
        for (int v = 0; v < kDim / 8; ++v) {
          uint32_t w[4] = {x[v].x, x[v].y, x[v].z, x[v].w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float lo, hi;
            bf16x2_to_f32(w[y], lo, hi);
            w[y] = pack_f16(lo * down, hi * down);
          }
          *reinterpret_cast<uint4*>(qs + v / 8 * L::kHalf + row_in * 128 + ((v % 8 ^ (row_in & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    ptx::fence_proxy_async_smem();
    asm volatile("bar.arrive 2, %0;" ::"n"(32 * kSoftmaxWarps + 64) : "memory");
    // ------------------------------------------------------------- softmax --
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t s_at = tmem + lanes + kKeys * st, o_at = tmem + lanes + kTmemO + 128 * st;
    const int pos = it.pos(prm, row), first = it.first(pos);
    float m = -3.0e38f, l = 0.f;
    // A score's factor with its key's scale: never 0 (a query of zeros, a page of zeros), by
    // which -inf would be NaN; products are below 2^33, so the least normal number is 0 to them.
    auto by = [&](float key_scale) { return fmaxf(factor * key_scale, FLT_MIN); };
    sum_refs[threadIdx.x] = -INFINITY;  // not in use
    // of the stream's first tile's columns, from .. to - 1 are keys that the row sees
    int from = max(first, seen.lo_min) - key0 - tile_of(st, 0) * kKeys;
    int to = min(pos, seen.hi_max) + 1 - key0 - tile_of(st, 0) * kKeys;
    for (int t = 0; t < my_tiles; ++t, from -= t_step * kKeys, to -= t_step * kKeys) {
      if (warp_wait(bars.s_full[st], t) && active) {
        ptx::tc_fence_after();
        const float* fk = scales + (tile_of(st, t) & 3) * 4 * kKeys;
        const float *fv = fk + kKeys, *ev = fv + kKeys, *iv = ev + kKeys;
        auto scale_o = [&](float f) {  // O is still while P of this tile is not there
#pragma unroll 1
          for (int x = 0; x < kDim; x += 16) {
            uint32_t o[16];
            ptx::tmem_ld16(o_at + x, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            ptx::tmem_st16(o_at + x, o);
          }
        };
        if (__builtin_expect(tile_of(st, t) >= *const_cast<volatile int*>(&bars.far_tile), 0)) {
          // A scale outside 2^-40 .. 2^40 has come by, in this tile or before (either stream's).
          float top = -INFINITY, top_v = -INFINITY;
          uint32_t s[32];
          auto score = [&](int g, int x) {
            const bool seen_here = kGroup * g + x >= from && kGroup * g + x < to;
            return seen_here ? __uint_as_float(s[x]) * by(fk[kUniform ? g : kGroup * g + x]) : -INFINITY;
          };
#pragma unroll 1
          for (int g = 0; g < kGroups; ++g) {
            ptx::tmem_ld32(s_at + kGroup * g, s);
            tmem_ready(s);
#pragma unroll
            for (int x = 0; x < kGroup; ++x) {
              const float v = score(g, x);
              top = fmaxf(top, v);
              top_v = fmaxf(top_v, v + ev[kUniform ? g : kGroup * g + x]);
            }
          }
          const float was = sum_refs[threadIdx.x] == -INFINITY ? m : sum_refs[threadIdx.x];
          const float ref = top > was + 8.f ? top : was;
          sum_refs[threadIdx.x] = ref;
          l *= ptx::ex2(was - ref);
          const bool raise = top_v > m + 15.f;
          if (__any_sync(0xffffffffu, raise)) {
            const float up = raise ? top_v - 7.f : m, f = ptx::ex2(m - up);
            m = up;
            if (t > 0) scale_o(f);
          }
#pragma unroll 1
          for (int g = 0; g < kGroups; ++g) {
            uint32_t p[16];
            ptx::tmem_ld32(s_at + kGroup * g, s);
            tmem_ready(s);
            auto weight = [&](int x) {
              const float v = score(g, x);
              l += ptx::ex2(v - ref);
              // 0 for a key that is not seen, whatever its scale
              return v == -INFINITY ? 0.f : ptx::ex2(v + (ev[kUniform ? g : kGroup * g + x] - m));
            };
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const float lo = weight(2 * y);
              p[y] = pack_f16(lo, weight(2 * y + 1));
            }
            ptx::tmem_st16(s_at + 16 * g, p);  // over scores of this group or of one before
          }
        } else {
          const bool edge = __any_sync(0xffffffffu, from > 0 || to < kKeys);
          uint32_t w[kGroups][32];
#pragma unroll
          for (int g = 0; g < kGroups; ++g) ptx::tmem_ld32(s_at + kGroup * g, w[g]);
          // the largest score with its value's scale (without it, it is at most 40 more)
          float top_v = -INFINITY;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            tmem_ready(w[g]);
            if (edge) {
#pragma unroll
              for (int x = 0; x < kGroup; ++x)
                if (kGroup * g + x < from || kGroup * g + x >= to) w[g][x] = 0xff800000u;  // -inf
            }
            if (kUniform) {
              float u[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int x = 0; x < 32; ++x) u[x % 4] = fmaxf(u[x % 4], __uint_as_float(w[g][x]));
              top_v = fmaxf(top_v, fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3])) * by(fk[g]) + ev[g]);
            } else {
#pragma unroll
              for (int x = 0; x < 32; ++x)
                top_v = fmaxf(top_v, __uint_as_float(w[g][x]) * by(fk[kGroup * g + x]) + ev[kGroup * g + x]);
            }
          }
          const bool raise = top_v > m + 15.f;
          if (__any_sync(0xffffffffu, raise)) {
            const float up = raise ? top_v - 7.f : m, f = ptx::ex2(m - up);
            m = up;
            l *= f;
            if (t > 0) scale_o(f);
          }
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            uint64_t sum[2] = {0, 0};
            uint32_t p[16];
            if (kUniform) {
              const float f1 = by(fk[g]), a1 = ev[g] - m;
              const uint64_t f2 = ptx::f32x2(f1, f1), a2 = ptx::f32x2(a1, a1);
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                const uint64_t v = ptx::fma_f32x2((uint64_t)w[g][2 * y + 1] << 32 | w[g][2 * y], f2, a2);
                const float lo = ptx::ex2(ptx::f32x2_lo(v)), hi = ptx::ex2(ptx::f32x2_hi(v));
                sum[y % 2] = ptx::add_f32x2(sum[y % 2], ptx::f32x2(lo, hi));
                p[y] = pack_f16(lo, hi);
              }
              sum[0] = ptx::add_f32x2(sum[0], sum[1]);
              l = fmaf(ptx::f32x2_lo(sum[0]) + ptx::f32x2_hi(sum[0]), iv[g], l);
            } else {
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                const int k = kGroup * g + 2 * y, k1 = k + 1;
                const float lo = ptx::ex2(fmaf(__uint_as_float(w[g][2 * y]), by(fk[k]), -m));
                const float hi = ptx::ex2(fmaf(__uint_as_float(w[g][2 * y + 1]), by(fk[k1]), -m));
                sum[y % 2] = ptx::add_f32x2(sum[y % 2], ptx::f32x2(lo, hi));
                p[y] = pack_f16(lo * fv[k], hi * fv[k1]);
              }
              sum[0] = ptx::add_f32x2(sum[0], sum[1]);
              l += ptx::f32x2_lo(sum[0]) + ptx::f32x2_hi(sum[0]);
            }
            ptx::tmem_st16(s_at + 16 * g, p);  // over scores, which are in registers
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
      }
      ptx::mbar_arrive(ptx::smem_addr(&bars.p_full[st]));
    }

    float l_ref = sum_refs[threadIdx.x];
    if (l_ref == -INFINITY) l_ref = m;

    // ---- the keys that only some rows see, where a value is NaN ----
    const bool go = my_tiles == 0 || warp_wait(bars.pv_done[st], my_tiles - 1);
    ptx::tc_fence_after();
    const bool adds = wild && it.split == 0 && it.part == 0 && (by_rows || st == 0) && go;
    if (wild && it.split == 0 && it.part == 0) {
      if (adds && my_tiles == 0) {
        uint32_t z[32] = {};
#pragma unroll
        for (int x = 0; x < kDim; x += 32) tmem_st32(o_at + x, z);
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
        for (int e = e0; adds && e < min(edges, e0 + kEdgeKeys); ++e) {
          const int key = edge_key(e);
          const uint8_t* line = lines + (e - e0) * 2 * kDim;
          const bool see = key <= pos && key >= first;
          float dot = 0.f;
          for (int v = 0; v < c.head_dim / 8; ++v) {
            const uint4 x = *reinterpret_cast<const uint4*>(qs + v / 8 * L::kHalf + row_in * 128 +
                                                            ((v % 8 ^ (row_in & 7)) << 4));
            const uint2 y = *reinterpret_cast<const uint2*>(line + 8 * v);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
            const uint32_t ys[4] = {codes_f16(y.x), codes_f16(y.x >> 16), codes_f16(y.y), codes_f16(y.y >> 16)};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const float2 qx = unpack_f16(xs[z]), kx = unpack_f16(ys[z]);
              dot = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, dot));
            }
          }
          // weight (with its value's scale) and O relative to the largest of both, in fp32; the
          // sum to its own
          const float s = dot * (factor * line_scale[2 * (e - e0)]), vs = line_scale[2 * (e - e0) + 1];
          const bool usual = vs > 0.f && vs < INFINITY;
          const float sv = usual ? s + __log2f(vs) : s;
          const float up = see && sv > m ? sv : m, f = ptx::ex2(m - up);
          const float p = see ? ptx::ex2(sv - up) * (usual ? 1.f : vs) : 0.f;
          m = up;
          const float ref = see && s > l_ref ? s : l_ref;
          l = l * ptx::ex2(l_ref - ref) + (see ? ptx::ex2(s - ref) : 0.f);
          l_ref = ref;
          for (int x = 0; x < kDim; x += 32) {
            uint32_t o[32];
            ptx::tmem_ld32(o_at + x, o);
            tmem_ready(o);
#pragma unroll
            for (int y = 0; y < 32; y += 2) {
              const float2 v = unpack_f16(codes_f16(*reinterpret_cast<const uint16_t*>(line + kDim + x + y)));
              const float o0 = __uint_as_float(o[y]) * f, o1 = __uint_as_float(o[y + 1]) * f;
              o[y] = __float_as_uint(see ? fmaf(p, v.x, o0) : o0);
              o[y + 1] = __float_as_uint(see ? fmaf(p, v.y, o1) : o1);
            }
            tmem_st32(o_at + x, o);
          }
          ptx::tmem_st_wait();
        }
      }
    }
    // ---- the rows of O ----
    const int vecs = c.head_dim / 4;
    bool any = my_tiles > 0 || adds;  // O is there
    float scale_o = 1.f, scale_odd = 0.f;
    float* odd_o = reinterpret_cast<float*>(smem + L::kK) + row_in * L::kLd;  // K and V have been used
    if (!by_rows) {
      // the odd stream leaves its O to the even one
      softmax_sync();  // both streams' products are done
      if (st == 1) {
        of_odd[row_in] = make_float4(m, l, l_ref, 0.f);
        if (active && any) {
#pragma unroll 1
          for (int x = 0; x < kDim; x += 32) {
            uint32_t o[32];
            ptx::tmem_ld32(o_at + x, o);
            tmem_ready(o);
#pragma unroll
            for (int y = 0; y < 32; y += 4)
              *reinterpret_cast<uint4*>(odd_o + x + y) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
          }
        }
      }
      softmax_sync();
      if (st == 0) {
        const float4 odd = of_odd[row_in];
        const float up = fmaxf(m, odd.x), ref = fmaxf(l_ref, odd.z);
        scale_o = ptx::ex2(m - up);
        scale_odd = ptx::ex2(odd.x - up);
        m = up;
        l = l * ptx::ex2(l_ref - ref) + odd.y * ptx::ex2(odd.z - ref);
        l_ref = ref;
      }
    }
    const bool odd_any = !by_rows && tiles_of(1) > 0;
    const bool writes = active && (by_rows || st == 0);
    // 32 elements of this thread's row from x on
    auto row_of = [&](int x, float (&o)[32]) {
      uint32_t r[32];
      ptx::tmem_ld32(o_at + x, r);
      tmem_ready(r);
#pragma unroll
      for (int y = 0; y < 32; ++y) o[y] = any ? __uint_as_float(r[y]) * scale_o : 0.f;
      if (odd_any) {
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = fmaf(odd_o[x + y], scale_odd, o[y]);
      }
    };
    if (prm.parts == 1) {
      if (writes) {
#pragma unroll 1
        for (int x = 0; x < kDim; x += 32) {
          float o[32];
          row_of(x, o);
          if (row < it.rows) {
#pragma unroll
            for (int y = 0; y < 32; y += 4)
              if (x + y < c.head_dim)
                write_row<__nv_bfloat16, true>(prm, it, row, (x + y) / 4,
                                               make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]), l_ref, l, m);
          }
        }
      }
      ptx::tc_fence_before();
      __syncthreads();
    } else {
      // O leaves Tensor Memory before every block's tiles are free for what the others send.
      auto* inbox = reinterpret_cast<Inbox<kRows, kDim, true>*>(smem);
      float o[kDim / 32][32];
      if (writes) {
#pragma unroll
        for (int x = 0; x < kDim / 32; ++x) row_of(32 * x, o[x]);
      }
      ptx::tc_fence_before();
      __syncwarp();
      ptx::cluster_sync();
      const int slice = div(prm.by_parts, it.rows * vecs + prm.parts - 1);
      if (writes && row < it.rows) {
        for (int b = 0; b < prm.parts; ++b) {
          ptx::st_cluster_v2(ptx::mapa_shared(ptx::smem_addr(&inbox->ml[it.part][row]), b), l_ref, l);
          ptx::st_cluster(ptx::mapa_shared(ptx::smem_addr(&inbox->ref[it.part][row]), b), m);
        }
        int i = row * vecs, to_block = i / slice;
#pragma unroll
        for (int x = 0; x < kDim; x += 4) {
          if (x >= c.head_dim) continue;
          if (i >= (to_block + 1) * slice) ++to_block;
          ptx::st_cluster_v4(
              ptx::mapa_shared(ptx::smem_addr(&inbox->o[it.part * slice + i - to_block * slice]), to_block),
              make_float4(o[x / 32][x % 32], o[x / 32][x % 32 + 1], o[x / 32][x % 32 + 2], o[x / 32][x % 32 + 3]));
          ++i;
        }
      }
      __syncwarp();
      ptx::cluster_sync();
      __syncthreads();
      join_slices<kRows, kDim, 32 * kSoftmaxWarps, __nv_bfloat16, true>(prm, it, inbox);
    }
  } else if (warp >= kMmaWarp) {
    fewer_registers<kMmaRegs>();
    // ------------------------------------------------------------ products --
    if (warp < kMmaWarp + 2) {
      const int st = warp - kMmaWarp, my_tiles = tiles_of(st);
      asm volatile("bar.sync 2, %0;" ::"n"(32 * kSoftmaxWarps + 64) : "memory");  // the queries
      const bool issues = elect_one();
      const uint32_t qk = idesc_f16(kTileRows, kKeys, false), pv = idesc_f16(kTileRows, c.head_dim, true);
      // operands: an offset in bytes is added to the address field, in units of 16
      const uint64_t q_desc = ptx::sdesc_k128(ptx::smem_addr(smem) + (by_rows ? st * L::kTile : 0));
      const uint64_t k_desc = ptx::sdesc_k128(ptx::smem_addr(smem) + L::kK);
      const uint64_t v_desc = ptx::sdesc_mn128(ptx::smem_addr(smem) + L::kV, L::kHalf);
      const uint32_t s_at = tmem + kKeys * st, o_at = tmem + kTmemO + 128 * st;
      for (int t = 0; t < my_tiles; ++t) {
        const int j = tile_of(st, t), slot = j & 1;
        // K is there; the weights of the tile before have been used
        if (!warp_wait(bars.k_full[slot], j >> 1) || (t > 0 && !warp_wait(bars.pv_done[st], t - 1))) break;
        // K was written by plain stores; the fence is here, and not in the copying warps, where
        // it would wait for their loads of the next tiles
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_after();
        if (issues) {
#pragma unroll
          for (int d = 0; d < kDim / 16; ++d) {
            const uint32_t off = (d / 4 * L::kHalf + d % 4 * 32) >> 4;
            if (d < row_vecs)
              ptx::mma_bf16(s_at, q_desc + off, k_desc + off + (uint32_t)(slot * L::kTile >> 4), qk, d > 0);
          }
          ptx::mma_commit(ptx::smem_addr(&bars.s_full[st]));
          ptx::mma_commit(ptx::smem_addr(&bars.k_free[slot]));
        }
        if (!warp_wait(bars.v_full[slot], j >> 1) || !warp_wait(bars.p_full[st], t)) break;
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_after();
        if (issues) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ta(o_at, s_at + 8 * k, v_desc + (uint32_t)((slot * L::kTile + k * 2048) >> 4), pv, t > 0 || k > 0);
          ptx::mma_commit(ptx::smem_addr(&bars.pv_done[st]));
          ptx::mma_commit(ptx::smem_addr(&bars.v_free[slot]));
        }
      }
      __syncwarp();
      if (issues && *abort_flag) {  // leave no product in flight
        ptx::mma_commit(ptx::smem_addr(&bars.drained[st]));
        drain_wait(ptx::smem_addr(&bars.drained[st]), 0);
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
    // Keys 32 w .. + 31 of a tile, which may share a page, are this warp's. A load takes 16
    // codes a lane: 8 keys, and 64 bytes of each; they become two 16-byte chunks of a key's
    // row, and the 8 lanes of a store have 8 keys' rows, whose swizzles differ.
    constexpr int kLoads = 4 * kDim / 64;
    const int w = warp - kSoftmaxWarps, vec = lane / 8, sub = lane % 8;
    // Lookups are loads without a condition, of the nearest key that a row sees, so that
    // nothing waits for them a tile ahead of their use.
    const int32_t* table = a.table + (int64_t)it.b * c.max_pages;
    const float *ks_head = a.k_scale + it.kh, *vs_head = a.v_scale + it.kh;
    struct Ahead {
      int key, page, off;  // of this lane's key: clamped; its page; its place there
    };
    auto look_up = [&](int i) {
      Ahead h = {0, 0, 0};
      if (n > 0) {
        const int key = key0 + i * kKeys + kGroup * w + lane;
        h.key = clamp_int(key, seen.lo_min, seen.hi_max);
        const int nth = div(prm.by_page, h.key);
        h.off = key - nth * c.page_size;
        if (h.key != key) h.key = -1;
        h.page = __ldg(table + nth);
      }
      return h;
    };
    // Of this lane's key; where a group has one page, of the group's first key, whether a
    // row sees it or not.
    struct Place {
      int64_t at;    // -1 (INT64_MIN): none
      float ks, vs;  // its page's scales
      int from;      // the lane that has them
      bool in;       // the key is seen, its page in the cache
    };
    auto place = [&](const Ahead& h) {
      const bool known = (unsigned)h.page < (unsigned)c.n_pages;
      if (prm.check_in_use && h.key >= 0 && !known) set_status(a.status, status_check());
      Place p;
      p.in = known && h.key >= 0;
      p.from = lane;
      p.ks = p.vs = 1.f;
      const int64_t id = known ? h.page : 0;
      if (c.n_pages > 0) {
        p.ks = __ldg(ks_head + id * c.n_kv_heads);
        p.vs = __ldg(vs_head + id * c.n_kv_heads);
      }
      p.at = id * c.page_stride + (int64_t)(kUniform ? h.off - lane : h.off) * c.token_stride;
      if (kUniform) {
        const unsigned with = __ballot_sync(0xffffffffu, p.in);
        p.from = with ? __ffs(with) - 1 : 0;
        p.at = __shfl_sync(0xffffffffu, p.at, p.from);
        if (!with) p.at = INT64_MIN;
      } else if (!p.in) {
        p.at = -1;
      }
      return p;
    };
    k_cache += (int64_t)it.kh * c.head_stride;
    v_cache += (int64_t)it.kh * c.head_stride;
    const int64_t sub_at = (int64_t)sub * c.token_stride + 16 * vec, step = 8 * c.token_stride;
    uint4 rk[kLoads], rv[kLoads];
    // Load x is of keys x % 4 * 8 + sub of the group and of their 64 bytes x / 4.
    auto fetch = [&](int i, const Place& p) {
      const int key = key0 + i * kKeys + kGroup * w + sub;
      // keys lo .. hi of the group are seen, from this lane's first on
      const int lo = kUniform && p.at == INT64_MIN ? kGroup : seen.lo_min - key, hi = seen.hi_max - key;
      const uint8_t *k_at = k_cache + p.at + sub_at, *v_at = v_cache + p.at + sub_at;
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        const bool held = 4 * (x / 4) + vec < row_vecs;
        if (kUniform) {
          const bool there = held && x % 4 * 8 >= lo && x % 4 * 8 <= hi;
          rk[x] = ld_once(k_at + x / 4 * 64, there);
          rv[x] = ld_once(v_at + x / 4 * 64, there);
          k_at += x % 4 == 3 ? -3 * step : step;
          v_at += x % 4 == 3 ? -3 * step : step;
        } else {
          const int64_t o = __shfl_sync(0xffffffffu, p.at, x % 4 * 8 + sub);
          rk[x] = ld_once(k_cache + o + x / 4 * 64 + 16 * vec, o >= 0 && held);
          rv[x] = ld_once(v_cache + o + x / 4 * 64 + 16 * vec, o >= 0 && held);
        }
      }
    };
    auto widen = [&](uint8_t* tile, const uint4 (&r)[kLoads]) {
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        uint8_t* at = tile + (kGroup * w + sub) * 128 + x / 4 * L::kHalf + x % 4 * 8 * 128;
        uint4 lo, hi;
        lo.x = codes_f16(r[x].x), lo.y = codes_f16(r[x].x >> 16);
        lo.z = codes_f16(r[x].y), lo.w = codes_f16(r[x].y >> 16);
        hi.x = codes_f16(r[x].z), hi.y = codes_f16(r[x].z >> 16);
        hi.z = codes_f16(r[x].w), hi.w = codes_f16(r[x].w >> 16);
        *reinterpret_cast<uint4*>(at + ((2 * vec ^ sub) << 4)) = lo;
        *reinterpret_cast<uint4*>(at + (((2 * vec + 1) ^ sub) << 4)) = hi;
      }
    };
    Place now = place(look_up(0));
    Ahead ahead = look_up(1);
    if (n > 0) fetch(0, now);
    for (int i = 0; i < n; ++i) {
      const int slot = i & 1;
      // the scores and the values of tile i - 2 have been taken
      if (i > 1 && (!warp_wait(bars.k_free[slot], (i >> 1) - 1) || !warp_wait(bars.v_free[slot], (i >> 1) - 1)))
        break;
      widen(smem + L::kK + slot * L::kTile, rk);
      float* fk = scales + (i & 3) * 4 * kKeys;
      if (!kUniform || lane == now.from) {
        const int k = kUniform ? w : kGroup * w + lane;
        const float ks = now.in ? now.ks : 1.f, vs = now.in ? now.vs : 1.f;
        fk[k] = ks;
        fk[kKeys + k] = vs;
        const float log_vs = __log2f(vs);
        fk[2 * kKeys + k] = log_vs;
        if (!(fabsf(log_vs) <= 40.f)) atomicMin(&bars.far_tile, i);
        if (kUniform) fk[3 * kKeys + k] = __frcp_rn(vs);
      }
      ptx::mbar_arrive(ptx::smem_addr(&bars.k_full[slot]));
      widen(smem + L::kV + slot * L::kTile, rv);
      ptx::mbar_arrive(ptx::smem_addr(&bars.v_full[slot]));
      if (i + 1 == n) break;
      now = place(ahead);
      fetch(i + 1, now);
      ahead = look_up(i + 2);
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
