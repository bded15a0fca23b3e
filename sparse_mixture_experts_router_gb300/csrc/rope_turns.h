// The turns per position of a head's rotary pairs, as 64-bit fractions of a
// turn. Host code without CUDA.
//
// f_i = 2^64 base^(-2i/rot_dim) / 2 pi has up to 62 bits before the point, and a
// position multiplies its error by up to 2^31: a double's 53 bits, and a product
// that runs over the pairs, would be off by up to 11 x 2^-24 rad there. So the
// factors are pairs of doubles (hi + lo, an unevaluated sum; products with the
// rounding error taken by fma, Dekker 1971), and f_i is off by half a unit: half
// of 2^-33 of a turn at the farthest position.
#pragma once
#include <cmath>
#include <cstdint>

namespace moe {

struct Double2 {
  double hi, lo;
};
inline Double2 operator*(Double2 x, Double2 y) {
  const double p = x.hi * y.hi;
  const double e = std::fma(x.hi, y.hi, -p) + (x.hi * y.lo + x.lo * y.hi);
  const double s = p + e;
  return {s, e - (s - p)};
}

// f_0 .. f_{pairs-1} (and what follows up to a multiple of 8); base >= 1.
inline void rope_turns(float base, int pairs, uint64_t* turns) {
  if (pairs == 0) return;
  // The ratio of neighbours, base^(-1/pairs): pow's, and one Newton step for
  // what its pairs-th power times base is off 1.
  Double2 ratio = {std::pow((double)base, -1.0 / pairs), 0.0}, x = {(double)base, 0.0}, square = ratio;
  for (int n = pairs; n > 0; n /= 2) {
    if (n % 2) x = x * square;
    square = square * square;
  }
  ratio.lo = ratio.hi * (((1.0 - x.hi) - x.lo) / pairs);
  // eight products in flight, each eight pairs on
  const Double2 two = ratio * ratio, four = two * two, eight = four * four;
  const Double2 one_radian = {0x1.45f306dc9c883p+61, -0x1.6b01ec5417056p+7};  // 2^64 / 2 pi
  Double2 f[8] = {one_radian, one_radian * ratio, one_radian * two, one_radian * (two * ratio)};
  for (int k = 4; k < 8; ++k) f[k] = f[k - 4] * four;
  for (int i = 0; i < pairs; i += 8)
    for (int k = 0; k < 8; ++k) {
      // to nearest; 0 < hi < 2^62 and |lo| < 2^9
      const int64_t whole = (int64_t)f[k].hi;
      const double rest = (f[k].hi - (double)whole) + f[k].lo;
      turns[i + k] = (uint64_t)(whole - 1024 + (int64_t)(rest + 1024.5));
      f[k] = f[k] * eight;
    }
}

}  // namespace moe
