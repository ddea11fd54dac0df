// fastmath.cuh — functions whose cost shows in the operators without a handle:
// branch-free, in fp32, with the error that each names (U = 2^-24, half a unit of
// fp32). Arguments of the exponential are rounded to fp32, so that its relative
// error grows by U of their size.
#pragma once

#include <stdint.h>

namespace dfm {

// Two fp32 values in a register pair, which one instruction takes.
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(Pair p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair both(float x) { return pair(x, x); }

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// 2^x, within 2 units of the last place; below 2^-126: 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + exp(-z)): within (10 + |z|) U of it; 0 below z = -87.3, where it is
// under 2^-126 (the quotient by more than 2^126 is 0).
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + exp2_fast(-z * kLog2e)); }

// 1 / x for 2^-126 <= x <= 2^126, within 1 unit of the last place.
__device__ __forceinline__ float recip_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The normal distribution function Phi of two values, and exp(-z^2 / 2). With x =
// |z| / sqrt(2), (1 + 2 x) exp(x^2) erfc(x) is a smooth function of t = (x - 2) /
// (x + 2) all the way to infinity (Shepherd and Laframboise, Mathematics of
// Computation 36, 1981, take it and a t of that kind). The polynomial of degree 9 is
// fitted to half of it on x <= 10, t from -1 to 2/3, by relative error: 1.4e-8 at most
// before its coefficients were rounded to fp32 (a linear program over 3000 Chebyshev
// points gives the least that the degree has, 1.3e-8), 3.7e-8 as they stand. Phi(z) is
// within 14 U for z >= -4, 46 for z >= -8, 128 to where it underflows.
__device__ __forceinline__ Pair normal_cdf(Pair z, Pair* density) {
  const float2 f = halves(z);
  const Pair x = pair(fminf(fabsf(f.x) * 0.707106781f, 10.f), fminf(fabsf(f.y) * 0.707106781f, 10.f));
  const Pair a = add2(x, both(2.f)), b = fma2(x, both(2.f), both(1.f));
  const float2 ab = halves(mul2(a, b));
  const Pair r = pair(recip_fast(ab.x), recip_fast(ab.y)), t = mul2(mul2(add2(x, both(-2.f)), b), r);
  Pair v = both(-1.99723407e-4f);
  v = fma2(v, t, both(-6.139994948e-4f));
  v = fma2(v, t, both(6.566536031e-4f));
  v = fma2(v, t, both(4.315047059e-3f));
  v = fma2(v, t, both(-4.030071199e-3f));
  v = fma2(v, t, both(-2.710194141e-2f));
  v = fma2(v, t, both(8.202771097e-2f));
  v = fma2(v, t, both(-8.301573247e-2f));
  v = fma2(v, t, both(-4.638199136e-2f));
  v = fma2(v, t, both(6.384891868e-1f));
  const float2 e = halves(mul2(mul2(z, z), both(-0.5f * kLog2e)));
  *density = pair(exp2_fast(e.x), exp2_fast(e.y));
  const Pair half = mul2(mul2(v, *density), mul2(a, r));
  const float2 low = halves(half), high = halves(fma2(half, both(-1.f), both(1.f)));
  return pair(f.x < 0.f ? low.x : high.x, f.y < 0.f ? low.y : high.y);
}

}  // namespace dfm
