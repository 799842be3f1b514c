// fp8.cuh -- device code shared by the 8-bit product kernels: the MMA of 8-bit
// codes, packed FP32 arithmetic, and where the rows of a unit of work lie.
#pragma once

#include <cstdint>

#include "sm103_ptx.cuh"

namespace g07 {

// Instruction descriptor of kind::f8f6f4 with E4M3 A and B (K-major) and FP32 D:
// the fields of idesc_bf16_f32 with both formats 0.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem], 32 k of 8-bit codes.
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- two FP32 values in one 64-bit register
__device__ __forceinline__ uint64_t pack2u(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return pack2u(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float half_of(uint64_t v, int high) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return __uint_as_float(high ? hi : lo);
}

// Rows first .. first + count - 1 of one expert.
struct Fp8Rows {
  int expert, first, count;
};

// Unit `unit` of the rows sorted by expert, each expert's rows in units of at most
// `size`; count 0 past the last one.  A warp's work.  Offsets are held to 0 .. M and
// to their running maximum, so whatever they hold, every row belongs to one expert
// at most.
__device__ __forceinline__ Fp8Rows fp8_expert_rows(const int* offsets, int E, int M, int size,
                                                   int unit) {
  const int lane = threadIdx.x & 31;
  auto held = [&](int v) { return v < 0 ? 0 : v > M ? M : v; };
  int last = held(__ldg(offsets)), units = 0;
  for (int base = 0; base < E; base += 32) {
    const int e = base + lane;
    int end = e < E ? held(__ldg(offsets + e + 1)) : 0;
    end = end > last ? end : last;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, end, d);
      if (lane >= d && v > end) end = v;
    }
    int start = __shfl_up_sync(0xFFFFFFFFu, end, 1);
    if (lane == 0) start = last;
    const int n = (end - start + size - 1) / size;
    int upto = n;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += v;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, units + upto > unit);
    if (past != 0) {
      const int at = __ffs(past) - 1;
      Fp8Rows r;
      r.expert = base + at;
      const int i = unit - units - __shfl_sync(0xFFFFFFFFu, upto - n, at);
      r.first = __shfl_sync(0xFFFFFFFFu, start, at) + i * size;
      const int left = __shfl_sync(0xFFFFFFFFu, end, at) - r.first;
      r.count = left < size ? left : size;
      return r;
    }
    units += __shfl_sync(0xFFFFFFFFu, upto, 31);
    last = __shfl_sync(0xFFFFFFFFu, end, 31);
  }
  return Fp8Rows{0, 0, 0};
}

}  // namespace g07
