// What the two append kernels share (rope_append.cu: a scale per token and head,
// or none; rope_append_page.cu: a scale per page and head): vectors of eight
// elements, the table of turns and the search for a row's sequence.
#pragma once
#include "rope_turns.h"
#include "serve_util.cuh"

namespace moe {

constexpr int kMaxPairs = kAttnMaxDim / 2;

struct RopeTable {
  uint64_t turns[kMaxPairs];  // f_i
};

// Eight elements of a row, as stored and as fp32.
template <typename T>
struct alignas(16) Eight {
  T v[8];
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
  Eight<T> r;
  constexpr int n = (int)sizeof(r) / 16;
#pragma unroll
  for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Eight<T>& r) {
  constexpr int n = (int)sizeof(r) / 16;
#pragma unroll
  for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(&r)[i];
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]),
                 f32x2_to_bf16x2(x[4], x[5]), f32x2_to_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void widen(const Eight<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = r.v[i];
}
__device__ __forceinline__ void widen(const Eight<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) bf16x2_to_f32(w[i], x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The first sequence whose rows end after row t, found by a whole warp in
// steps of 32 comparisons (n_seqs if none).
__device__ __forceinline__ int seq_of_row(const int32_t* cu_new, int n_seqs, int t, int lane) {
  int lo = 0, hi = n_seqs;  // the answer is in lo .. hi
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step - 1;
    const unsigned after = __ballot_sync(0xffffffffu, i >= hi || __ldg(cu_new + i + 1) > t);
    if (!after) return hi;  // only where the list does not ascend
    const int f = __ffs(after) - 1;
    hi = min(hi, lo + (f + 1) * step - 1);
    lo += f * step;
  }
  return lo;
}

// Appends to a cache with a scale per page and head (rope_append_page.cu). A
// head is 1 << lane_bits lanes of eight elements.
cudaError_t launch_rope_append_page(const AttnArgs& a, const RopeTable& rope, int lane_bits,
                                    cudaStream_t s);

}  // namespace moe
