// Attention of the new tokens over a paged fp32 cache, on the CUDA cores.
//
// Tensor cores have no fp32 products, and an fp32 cache is asked for by who
// wants fp32 results, so the products are fused multiply-adds. Per cached
// element R of them (R query rows of the head group) against 4 bytes: up to
// about four rows memory bounds the kernel, beyond that the instructions a
// warp issues (half of them multiply-adds, a quarter loads of shared memory);
// more than 12 rows go in blocks of up to 12 that read the keys again.
//
// Work, parts and join are those of the other caches. Each warp has one tile
// of 8 keys and one of their values in shared memory, filled by cp.async: the
// next keys are on their way while the weights are taken to the values, the
// next values during the scores. Two of each a warp hid no more latency than
// the warps they cost did: with one, three to eight blocks fit an SM instead
// of one to three, and 58 drawn calls take 8% less time (heads above 128:
// 1486 -> 1020 us for 7 sequences of 20000 to 45000 keys). Scores: lane (key, row group)
// takes the dot products of one key with kR rows, 4 elements at a time, keys
// and queries both from shared memory without bank conflicts. Output: each
// lane owns 4 (8 for heads above 128) elements of every row and takes the
// weights of a key by broadcast reads. The maximum is raised only when a
// score passes it by 8 (log2 units). Scores, weights, sums and O are fp32.
#include "paged_attention.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = 8;

template <int kDim>
struct Tile {
  static constexpr int kChunks = kDim / 4;  // 16-byte chunks of a key
  static constexpr int kBytes = kKeys * kDim * 4;
  static __device__ __forceinline__ uint32_t at(int k, int c) {
    return (uint32_t)(k * kDim * 4 + ((c ^ k) << 4));
  }
};
template <int kDim, int kR>
struct Smem {
  static constexpr int kRows = 4 * kR;
  // A warp's tile of keys and of values, later its rows of the join.
  static constexpr int kWarp = std::max(2 * Tile<kDim>::kBytes, kRows * (kDim + 4) * 4);
  static constexpr int kRing = kWarps * kWarp;
  static constexpr int kQ = kRows * (kDim + 4) * 4;
  static constexpr int kP = kWarps * kKeys * kRows * 4;
  static constexpr int kStat = (2 * kWarps + 2) * kRows * 4;
  static constexpr int kInbox = (int)sizeof(Inbox<kRows, kDim>);
  static constexpr int kAll = kRing + kInbox + kQ + kP + kStat;
  static_assert(f32_blocks_per_sm(kDim, kR) * (kAll + 1024) <= 228 * 1024, "shared memory of an SM");
};

template <int kDim, int kR>
__global__ void __launch_bounds__(kThreads, f32_blocks_per_sm(kDim, kR))
    f32_kernel(const __grid_constant__ Params prm) {
  using T = Tile<kDim>;
  using M = Smem<kDim, kR>;
  constexpr int kRows = M::kRows;
  constexpr int kVecs = kDim > 128 ? kDim / 128 : 1;   // float4s of a row a lane owns
  constexpr int kLanes = T::kChunks / kVecs;           // lanes a key's values take
  constexpr int kGroups = 32 / kLanes;                 // keys taken at once
  // Sums that a score is taken in: in one the roundings of head_dim additions
  // come together. Error of out over 200 to 30000 keys, of its norm, in one, two
  // and four sums: heads of 256 1.1e-6 to 1.8e-6, 0.6 to 1.1, 0.4 to 0.8; of 128
  // 0.8 to 1.1, 0.5 to 0.7, 0.3 to 0.5. Two cost up to 2% (12 rows; most calls
  // nothing). Four in the place of two cost heads of 256 up to 3% from 8 rows on
  // and nothing below, heads of 80 to 128 nothing up to 4 rows and 3 to 4% at 8
  // rows, and heads of 64 3%.
  constexpr int kSums = kDim > 128 || (kDim > 64 && kR == 1) ? 4 : 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnArgs& a = prm.a;
  const moe_attn_config& c = a.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, key8 = lane % 8, rg = lane / 8;
  auto* inbox = reinterpret_cast<Inbox<kRows, kDim>*>(smem + M::kRing);
  uint8_t* rest = smem + M::kRing + M::kInbox;
  float* qs = reinterpret_cast<float*>(rest);
  float* ps = reinterpret_cast<float*>(rest + M::kQ) + warp * kKeys * kRows;
  float* stat = reinterpret_cast<float*>(rest + M::kQ + M::kP);
  float* joined = stat + 2 * kWarps * kRows;

  pdl_wait();
  pdl_trigger();
  Item it;
  if (!item_of<kThreads>(prm, kRows, it)) return;
  start_cluster(prm);
  const Range rg_ = range_of(prm, it, kRows, kKeys);
  const int mine = rg_.t1 - rg_.t0 > warp ? (rg_.t1 - rg_.t0 - warp - 1) / kWarps + 1 : 0;

  // ---- the stream of tiles ----
  uint8_t* const K = smem + warp * M::kWarp;
  uint8_t* const V = K + T::kBytes;
  const uint32_t ring = ptx::smem_addr(K);
  const float* kc = static_cast<const float*>(a.k_cache);
  const float* vc = static_cast<const float*>(a.v_cache);
  auto tile_key = [&](int i) { return rg_.base + (rg_.t0 + warp + kWarps * i) * kKeys; };
  auto look_up = [&](int i) {
    Slot slot = {-1, -1};
    if (i < mine) slot = slot_of(prm, it, rg_, tile_key(i) + key8);
    return slot;
  };
  // Elements to this lane's key, -1 where there is none.
  auto offset = [&](const Slot& slot) -> int64_t {
    slot.check(prm);
    return slot.in(c) ? slot.at(c, it.kh) : -1;
  };
  auto load = [&](const float* cache, uint32_t to, int i, int64_t off) {
    if (i < mine) {
      constexpr int kAll = kKeys * T::kChunks / 32;
#pragma unroll
      for (int x = 0; x < kAll; ++x) {
        const int key = x * 32 / T::kChunks + (T::kChunks < 32 ? lane / T::kChunks : 0);
        const int chunk = (x * 32 + lane) % T::kChunks;
        const int64_t o = __shfl_sync(0xffffffffu, off, key);
        const uint32_t n = o >= 0 && 4 * chunk < c.head_dim ? 16u : 0u;
        ptx::cp_async16(to + T::at(key, chunk), cache + (n ? o + 4 * chunk : 0), n);
      }
    }
    ptx::cp_async_commit();
  };
  int64_t off = offset(look_up(0));
  load(kc, ring, 0, off);
  load(vc, ring + T::kBytes, 0, off);
  Slot next = look_up(1);

  // ---- queries, in log2 units ----
  const float scale = c.scale * 1.4426950408889634f;
  for (int i = threadIdx.x; i < kRows * T::kChunks; i += kThreads) {
    const int r = i / T::kChunks, v = i % T::kChunks;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (4 * v < c.head_dim)
      x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + it.q_at(prm, r) + 4 * v);
    *reinterpret_cast<float4*>(qs + r * (kDim + 4) + 4 * v) = x;
  }
  __syncthreads();
  int hi[kR], lo[kR];  // of this lane's rows rg + 4 i
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    hi[i] = it.pos(prm, rg + 4 * i);
    lo[i] = it.first(hi[i]);
  }

  float o[kRows][4 * kVecs], m[kR], l[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i) m[i] = -3.0e38f, l[i] = 0.f;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int x = 0; x < 4 * kVecs; ++x) o[r][x] = 0.f;

  for (int i = 0; i < mine; ++i) {
    ptx::cp_async_wait_group<1>();
    __syncwarp();
    const int key0 = tile_key(i), key = key0 + key8;

    float part[kR][kSums];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int x = 0; x < kSums; ++x) part[r][x] = 0.f;
#pragma unroll 4
    for (int v = 0; v < c.head_dim / 4; ++v) {
      const float4 k = *reinterpret_cast<const float4*>(K + T::at(key8, v));
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const float4 q = *reinterpret_cast<const float4*>(qs + (rg + 4 * r) * (kDim + 4) + 4 * v);
        float* p = part[r];
        p[kSums - 1] = fmaf(k.w, q.w, p[kSums - 1]);
        p[kSums - 2] = fmaf(k.z, q.z, p[kSums - 2]);
        p[1] = fmaf(k.y, q.y, p[1]);
        p[0] = fmaf(k.x, q.x, p[0]);
      }
    }
    float s[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r)
      s[r] = kSums == 2 ? part[r][0] + part[r][1]
                        : (part[r][0] + part[r][1]) + (part[r][kSums - 2] + part[r][kSums - 1]);
    __syncwarp();  // every lane has read the keys
    off = offset(next);
    load(kc, ring, i + 1, off);
    next = look_up(i + 2);
    const bool edge = key0 + kKeys - 1 > rg_.hi_min || key0 < rg_.lo_max;
    bool raise = false;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      s[r] *= scale;
      if (edge && (key > hi[r] || key < lo[r])) s[r] = -INFINITY;
      raise = raise || s[r] > m[r] + 8.f;
    }
    if (__any_sync(0xffffffffu, raise)) {
      float f[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float top = fmaxf(m[r], s[r]);
#pragma unroll
        for (int x = 1; x < 8; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        f[r] = ptx::ex2(m[r] - top);
        m[r] = top;
        l[r] *= f[r];
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float fr = __shfl_sync(0xffffffffu, f[r / 4], r % 4 * 8);
#pragma unroll
        for (int x = 0; x < 4 * kVecs; ++x) o[r][x] *= fr;
      }
    }
    // A weight of -1 stands for a key its row does not see, where rows differ:
    // the value may not be finite.
    const bool mixed = edge && rg_.hi_min != rg_.hi_max;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const float p = ptx::ex2(s[r] - m[r]);
      l[r] += p;
      ps[key8 * kRows + rg + 4 * r] = mixed && (key > hi[r] || key < lo[r]) ? -1.f : p;
    }
    ptx::cp_async_wait_group<1>();
    __syncwarp();
#pragma unroll
    for (int k0 = 0; k0 < kKeys; k0 += kGroups) {
      const int k = k0 + (kGroups > 1 ? lane / kLanes : 0);
      float4 v[kVecs];
#pragma unroll
      for (int x = 0; x < kVecs; ++x)
        v[x] = *reinterpret_cast<const float4*>(V + T::at(k, lane % kLanes + kLanes * x));
#pragma unroll
      for (int r4 = 0; r4 < kR; ++r4) {
        const float4 p4 = *reinterpret_cast<const float4*>(ps + k * kRows + 4 * r4);
        const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (mixed && p[j] == -1.f) continue;
          float* w = o[4 * r4 + j];
#pragma unroll
          for (int x = 0; x < kVecs; ++x) {
            w[4 * x] = fmaf(p[j], v[x].x, w[4 * x]);
            w[4 * x + 1] = fmaf(p[j], v[x].y, w[4 * x + 1]);
            w[4 * x + 2] = fmaf(p[j], v[x].z, w[4 * x + 2]);
            w[4 * x + 3] = fmaf(p[j], v[x].w, w[4 * x + 3]);
          }
        }
      }
    }
    __syncwarp();  // every lane has read the values and the weights
    load(vc, ring + T::kBytes, i + 1, off);
  }
  ptx::cp_async_wait_all();

  // ---- join ----
#pragma unroll
  for (int r = 0; r < kR; ++r) {
#pragma unroll
    for (int x = 1; x < 8; x *= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
    if (key8 == 0) {
      stat[warp * kRows + rg + 4 * r] = m[r];
      stat[(kWarps + warp) * kRows + rg + 4 * r] = l[r];
    }
  }
  __syncthreads();
  constexpr int kLd = kDim + 4;
  float* mine_o = reinterpret_cast<float*>(K);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float top = stat[r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, stat[w * kRows + r]);
    const float f = ptx::ex2(stat[warp * kRows + r] - top);
    if (threadIdx.x == 0) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        sum += stat[(kWarps + w) * kRows + r] * ptx::ex2(stat[w * kRows + r] - top);
      joined[r] = top;
      joined[kRows + r] = sum;
    }
#pragma unroll
    for (int x = 0; x < kVecs; ++x) {
      float4 v = make_float4(o[r][4 * x], o[r][4 * x + 1], o[r][4 * x + 2], o[r][4 * x + 3]);
      if (kGroups > 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, 16);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, 16);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, 16);
      }
      v.x *= f, v.y *= f, v.z *= f, v.w *= f;
      *reinterpret_cast<float4*>(mine_o + r * kLd + 4 * (lane % kLanes + kLanes * x)) = v;
    }
  }
  __syncthreads();
  finish<kRows, kDim, kWarps, kThreads, true, float>(prm, it, reinterpret_cast<float*>(smem),
                                                     M::kWarp / 4, kLd, joined, inbox);
}

template <int kDim, int kR>
cudaError_t launch_one(const Params& p, unsigned blocks, cudaStream_t s) {
  static thread_local int configured = -1;
  return launch(f32_kernel<kDim, kR>, &configured, p, blocks, kThreads, Smem<kDim, kR>::kAll, s);
}

}  // namespace

cudaError_t launch_f32(const Params& p, int dim, int nt, unsigned blocks, cudaStream_t s) {
  if (dim <= 64) {
    if (nt == 1) return launch_one<64, 1>(p, blocks, s);
    if (nt == 2) return launch_one<64, 2>(p, blocks, s);
    return launch_one<64, 3>(p, blocks, s);
  }
  if (dim <= 128) {
    if (nt == 1) return launch_one<128, 1>(p, blocks, s);
    if (nt == 2) return launch_one<128, 2>(p, blocks, s);
    return launch_one<128, 3>(p, blocks, s);
  }
  if (nt == 1) return launch_one<256, 1>(p, blocks, s);
  return launch_one<256, 2>(p, blocks, s);
}

}  // namespace attn
}  // namespace moe
