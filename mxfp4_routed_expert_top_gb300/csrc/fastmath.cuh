// fastmath.cuh — functions whose cost shows in the operators without a handle:
// branch-free, in fp32, with the error that each names (U = 2^-24, half a unit of
// fp32). Arguments of the exponential are rounded to fp32, so that its relative
// error grows by U of their size.
#pragma once

#include <stdint.h>

namespace dfm {

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// 2^x, within 2 units of the last place; below 2^-126: 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + exp(-z)): within (10 + |z|) U of it.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + exp2_fast(-z * kLog2e)); }

// The normal distribution function Phi(z), and exp(-z^2 / 2). With x = |z| /
// sqrt(2), (1 + 2 x) exp(x^2) erfc(x) is a smooth function of t = (x - 2) / (x + 2)
// all the way to infinity (Shepherd and Laframboise, Mathematics of Computation
// 36, 1981, take it and a t of that kind); the polynomial of degree 9 was fitted
// to half of it for x <= 10, and is off by 1.4e-8 of it at most. Phi(z) is within 14
// U for z >= -4, 46 for z >= -8, 128 to where it underflows.
__device__ __forceinline__ float normal_cdf(float z, float* density) {
  const float x = fminf(fabsf(z) * 0.707106781f, 10.f), a = x + 2.f, b = fmaf(2.f, x, 1.f);
  const float r = __fdividef(1.f, a * b), t = (x - 2.f) * b * r;
  float v = -1.99723407e-4f;
  v = fmaf(v, t, -6.139994948e-4f);
  v = fmaf(v, t, 6.566536031e-4f);
  v = fmaf(v, t, 4.315047059e-3f);
  v = fmaf(v, t, -4.030071199e-3f);
  v = fmaf(v, t, -2.710194141e-2f);
  v = fmaf(v, t, 8.202771097e-2f);
  v = fmaf(v, t, -8.301573247e-2f);
  v = fmaf(v, t, -4.638199136e-2f);
  v = fmaf(v, t, 6.384891868e-1f);
  *density = exp2_fast(z * z * (-0.5f * kLog2e));
  const float half = v * *density * (a * r);
  return z < 0.f ? half : 1.f - half;
}

}  // namespace dfm
