// Score modifications shared by the attention kernels: the tanh cap and the
// depth of a drafted token.
#pragma once

#include "ptx.cuh"

#include <stdint.h>

namespace zl {

// tanh(y) to about 1e-7 of max(|tanh|, 1): 1 - 2 / (e^(2y) + 1) away from zero,
// where e^(2y) overflowing to infinity gives 1 and underflowing to 0 gives -1.
// Near zero that difference cancels, so |y| < 0.25 takes the odd Taylor series
// y - y^3/3 + 2 y^5/15 - 17 y^7/315 + 62 y^9/2835 (first term left out: below
// 3e-9 of y). A score is c * tanh(s / c) and enters an exponent: what counts
// is its absolute error, c times this one.
__device__ __forceinline__ float cap_tanh(float y) {
  const float y2 = y * y;
  float t = fmaf(y2, 62.f / 2835.f, -17.f / 315.f);
  t = fmaf(t, y2, 2.f / 15.f);
  t = fmaf(t, y2, -1.f / 3.f);
  t = fmaf(t * y2, y, y);
  const float e = ex2_approx(y * 2.8853900817779268f);
  const float far = 1.f - __fdividef(2.f, e + 1.f);
  return fabsf(y) < 0.25f ? t : far;
}

// Depth of a drafted token below the context's last position plus one: its
// ancestors among the drafted tokens, itself not counted. (A token whose mask
// is empty counts as a root.)
__device__ __forceinline__ int tree_depth(const uint32_t* bits, int words) {
  int n = 0;
  for (int w = 0; w < words; ++w) n += __popc(__ldg(bits + w));
  return n > 0 ? n - 1 : 0;
}

}  // namespace zl
