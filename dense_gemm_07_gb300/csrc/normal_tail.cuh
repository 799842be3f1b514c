// normal_tail.cuh -- the normal distribution's tail, for GELU and its slope.
#pragma once

namespace g07 {

// Phi(-|x|), the lower tail of the normal distribution, times 2, and
// exp(-x^2 / 2): Abramowitz and Stegun, "Handbook of Mathematical Functions",
// 7.1.26, erfc(z) = (a1 t + .. + a5 t^5) exp(-z^2), t = 1 / (1 + p z), at
// z = |x| / sqrt 2, within 1.5e-7 absolute.  GELU and its slope share the
// exponential; 12 instructions where erff and expf take about 50, which bound
// these kernels (2048 x 11008 pack and gradient: 185 us).  In FP32 with the
// approximate exponential and quotient GELU is at most 4.2e-7 off (0.5 x (1 + erf)
// in FP32: 4.4e-7) and its slope, measured, 2.9e-7 (with erf and exp in FP32:
// 0.95e-7), which the FP32 bias gradient takes over; below x = -5 GELU's error is
// above half a unit of BF16 of its value, which is less than 1.5e-6 there.
__device__ __forceinline__ float normal_tail2(float x, float* exp_part) {
  const float t = __fdividef(1.0f, fmaf(0.3275911f * 0.70710678f, fabsf(x), 1.0f));
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * x * -0.72134752f));  // log2(e) / 2
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(t, p, 1.421413741f);
  p = fmaf(t, p, -0.284496736f);
  p = fmaf(t, p, 0.254829592f);
  *exp_part = e;
  return p * t * e;
}

}  // namespace g07
