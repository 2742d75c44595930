// Score modifications shared by the attention kernels: the tanh cap and the
// depth of a drafted token.
#pragma once

#include "ptx.cuh"

#include <stdint.h>

namespace zl {

// tanh(y) / y for z = y^2 in [0, 1]: the degree-6 polynomial that interpolates
// it at the 7 Chebyshev nodes of the interval. Within 5.2e-8 of tanh(y) / y;
// 1.6e-7 evaluated in 32 bits. (tanh(sqrt z) / sqrt z has its nearest pole at z
// = -(pi / 2)^2, so each further degree gains a factor of about 12.)
constexpr float kTanh0 = 0.999999949f, kTanh1 = -0.33332828f, kTanh2 = 0.133250761f,
                kTanh3 = -0.0534516464f, kTanh4 = 0.0202797083f, kTanh5 = -0.00619432483f,
                kTanh6 = 0.0010380251f;

// tanh(y) for |y| > 1 as 1 - 2 / (e^(2y) + 1), where e^(2y) overflowing to
// infinity gives 1 and underflowing to 0 gives -1.
__device__ __forceinline__ float tanh_far(float y) {
  const float e = ex2_approx(y * 2.8853900817779268f);
  return 1.f - __fdividef(2.f, e + 1.f);
}

// tanh(y) to about 2e-7 of max(|tanh y|, ..): the polynomial up to |y| = 1 and
// tanh_far beyond (its difference cancels near zero). A score is c * tanh(s / c)
// and enters an exponent: what counts is its absolute error.
__device__ __forceinline__ float cap_tanh(float y) {
  const float z = y * y;
  float t = fmaf(z, kTanh6, kTanh5);
  t = fmaf(t, z, kTanh4);
  t = fmaf(t, z, kTanh3);
  t = fmaf(t, z, kTanh2);
  t = fmaf(t, z, kTanh1);
  t = fmaf(t, z, kTanh0);
  return fabsf(y) <= 1.f ? t * y : tanh_far(y);
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
