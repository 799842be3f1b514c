// ckpt8.cuh -- the scale of a run of the 8-bit checkpoint (ckpt8.cu).
#pragma once

#include <cstdint>

namespace g07 {

// Scale byte for a run whose largest magnitude has the FP32 bits `top`
// (magnitudes order as integers): e + 127 for the smallest e >= -126 with
// top <= 127 * 2^e.  top = m 2^k with 1 <= m < 2 gives e = k - 6 when
// m <= 127 / 64 (mantissa bits at most 0x7E0000), else k - 5.  e stops at 121:
// the next step's 64 would be 2^128, so the last few numbers below 2^128 are
// kept as 127 * 2^121.  255: not finite.
__host__ __device__ __forceinline__ uint32_t ckpt8_code(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  const int code =
      static_cast<int>(top >> 23) - 6 + ((top & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return code < 1 ? 1u : code > 248 ? 248u : static_cast<uint32_t>(code);
}
#ifdef __CUDACC__
// 2^-e: exponent bits 254 - code (6 .. 253), so always a normal number; zero
// for a run kept as NaN (its q are then 0 or undefined, and never used).
__device__ __forceinline__ float ckpt8_inverse_step(uint32_t code) {
  return __uint_as_float((code == 255u ? 0u : 254u - code) << 23);
}
// 2^e (a normal number), or NaN.
__device__ __forceinline__ float ckpt8_step(uint32_t code) {
  return __uint_as_float(code == 255u ? 0x7FC00000u : code << 23);
}
// round(v / step), at most 127 in magnitude (only e = 121 reaches past it).
__device__ __forceinline__ int ckpt8_round(float v, float inverse_step) {
  const int q = __float2int_rn(v * inverse_step);
  return q > 127 ? 127 : q < -127 ? -127 : q;
}
#endif

}  // namespace g07
