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

// As mbar_wait, for waits that are over soon: the timer, whose reading takes longer than
// most of them, is left alone for the first 256 polls.
__device__ __forceinline__ bool wait_soon(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns) {
  const uint32_t a = smem_u32(bar);
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(a, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort) return false;
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > limit_ns) return false;
    }
  }
}

// ---- scales on their way to shared memory: copies of one float each (any alignment of
// 4), and an arrival on `bar` when all copies of this thread so far have landed.  A
// block of K takes less time than a load does, so the copies of several are under way.
__device__ __forceinline__ void copy_scale(float* dst, const float* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ void arrive_when_copied(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
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
// c += {lo, hi} * b, for lo and hi that a tensor-memory load is to deliver: volatile, so
// that it stays behind the wait for it.
__device__ __forceinline__ void fma2_loaded(uint64_t& c, uint32_t lo, uint32_t hi, uint64_t b) {
  asm volatile(
      "{\n\t.reg .b64 t;\n\t"
      "mov.b64 t, {%1, %2};\n\t"
      "fma.rn.f32x2 %0, t, %3, %0;\n\t}"
      : "+l"(c)
      : "r"(lo), "r"(hi), "l"(b));
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

// 16 lanes (from the address's lane on) by 32 columns of tensor memory: thread t
// receives, for i = 0 .. 3, columns 8 i + 2 (t % 4) and the next of lane t / 4
// (r[4 i], r[4 i + 1]) and of lane t / 4 + 8 (r[4 i + 2], r[4 i + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
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

// The first row of each expert and the units of at most `size` rows before it, E + 1
// of each; the number of all units.  A warp's work; offsets as above.
__device__ __forceinline__ int fp8_expert_table(const int* offsets, int E, int M, int size,
                                                int* start, int* before) {
  const int lane = threadIdx.x & 31;
  auto held = [&](int v) { return v < 0 ? 0 : v > M ? M : v; };
  int last = held(__ldg(offsets)), units = 0;
  if (lane == 0) {
    start[0] = last;
    before[0] = 0;
  }
  for (int base = 0; base < E; base += 32) {
    const int e = base + lane;
    int end = e < E ? held(__ldg(offsets + e + 1)) : 0;
    end = end > last ? end : last;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, end, d);
      if (lane >= d && v > end) end = v;
    }
    int from = __shfl_up_sync(0xFFFFFFFFu, end, 1);
    if (lane == 0) from = last;
    int upto = (end - from + size - 1) / size;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += v;
    }
    if (e < E) {
      start[e + 1] = end;
      before[e + 1] = units + upto;
    }
    units += __shfl_sync(0xFFFFFFFFu, upto, 31);
    last = __shfl_sync(0xFFFFFFFFu, end, 31);
  }
  return units;
}

}  // namespace g07
