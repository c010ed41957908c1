// Rounding to the FP4 main-KV format (E2M1 codes, one E4M3 scale per 16
// channels), shared by the pack kernel and the cache append: every decision is
// an exact f32 comparison.
#pragma once

#include <stdint.h>

namespace csa2 {
namespace fp4 {

// E4M3 ("fn" variant, bias 7, no inf) code -> value, codes 0..126 only.
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  const uint32_t e = c >> 3, m = c & 7u;
  if (e == 0) return static_cast<float>(m) * 0x1p-9f;
  return __uint_as_float(((e + 120u) << 23) | (m << 20));  // (1 + m/8) * 2^(e-7)
}

// Scale code: the E4M3 value nearest amax/6, ties to the even code, saturating
// at 448 (code 126).  Division-free: binary search for the largest code whose
// 6x value is <= amax, then compare amax with 6x the midpoint to the next
// code.  6x an E4M3 value or midpoint has at most 7 significant bits, so every
// product and comparison is exact in f32.
__device__ __forceinline__ uint32_t scale_code_for(float amax) {
  uint32_t lo = 0, hi = 126;  // invariant: 6*v(lo) <= amax (v(0) = 0)
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    if (6.0f * e4m3_value(mid) <= amax) lo = mid; else hi = mid - 1;
  }
  if (lo == 126) return 126;
  const float six_mid = 3.0f * (e4m3_value(lo) + e4m3_value(lo + 1));
  if (amax > six_mid) return lo + 1;
  if (amax < six_mid) return lo;
  return (lo & 1u) ? lo + 1 : lo;  // tie: even code
}

// E2M1 magnitude code (0..7) nearest |x|/s with s > 0, ties to the even code,
// saturating at 6.  Thresholds are the grid midpoints times s (exact).
__device__ __forceinline__ uint32_t e2m1_code(float ax, float s) {
  const float mids[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f};
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const float t = mids[i] * s;
    // passing threshold i moves from code i to i+1; at equality only if i+1 is even
    if (ax > t || (ax == t && ((i + 1) & 1) == 0)) c = i + 1;
  }
  return c;
}

}  // namespace fp4
}  // namespace csa2
