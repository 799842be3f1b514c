// fp8_quantize.cu -- matrices in 8-bit floating point (E4M3) with a scale for each
// 128 values of a row (activations, gradients) or each 128 x 128 (weights).
//
// The scale is the smallest power of two 2^e (e >= -126) that brings the block to
// 448 at most, the largest code, so that dividing by it is exact and the only
// rounding is to the nearest code: the result does not depend on how it is computed.
// A power of two costs no precision, since the codes are themselves floating-point
// numbers: all it gives away is part of the last power of two of their range.  A
// block with a value that is not finite is kept as NaN throughout.
//
// Each value is read once and one byte written.  16384 rows picked from 4096 x 4096
// BF16 take 27 us, 101 MB at 3.9 TB/s: the conversions' instructions (90 for 8 values a
// lane) fill two thirds of the issue slots.
#include <type_traits>

#include "experts.h"
#include "kernels.h"

namespace g07 {
namespace {

constexpr int B = kFp8Block;
constexpr int kThreads = 256;

// What a block is divided by, from the largest magnitude's bits.
struct Scale {
  float step, inverse;
  bool finite;
};
__device__ __forceinline__ Scale scale_of(uint32_t top) {
  Scale s;
  s.finite = top < 0x7F800000u;
  // 448 = 1.75 * 2^8: a mantissa above 1.75 needs the next power
  int e = static_cast<int>(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < 1 ? 1 : e;
  s.step = s.finite ? __uint_as_float(static_cast<uint32_t>(e) << 23) : 1.0f;
  s.inverse = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  return s;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Two codes, the first one in the low byte.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t codes4(const float* v, const Scale& s) {
  const uint32_t c = codes2(v[0] * s.inverse, v[1] * s.inverse) |
                     codes2(v[2] * s.inverse, v[3] * s.inverse) << 16;
  return s.finite ? c : 0x7F7F7F7Fu;
}

// Eight consecutive elements p[0 .. 7] of a row, of which the first `n` exist.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
  if (VEC && n >= 8) {
    load_vec<8>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}
// Eight codes; p on 8 bytes.
__device__ __forceinline__ void store8(uint8_t* p, int n, uint2 c) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// ---- a scale for each 128 values of a row.  16 lanes hold a block, 8 values
// each; the two halves of a warp and the warps of a block take 16 rows, and each
// takes GROUP blocks of its row at once, so that their loads are on their way
// together.
constexpr int kRowsPerBlock = kThreads / 16;
constexpr int kGroup = 4;

// Eight elements as loaded, their largest magnitude in a lane's form (the FP32 bits, or
// two BF16 magnitudes side by side), and that of 16 lanes as FP32 bits.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float v[8];
  template <bool VEC>
  __device__ __forceinline__ void load(const float* p, int n) { load8<VEC>(p, n, v); }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = larger(t, magnitude(v[i]));
    return t;
  }
  static __device__ __forceinline__ uint32_t top_of(uint32_t a, uint32_t b) { return larger(a, b); }
  static __device__ __forceinline__ uint32_t bits(uint32_t t) { return t; }
  __device__ __forceinline__ uint2 codes(const Scale& s) const {
    return make_uint2(codes4(v, s), codes4(v + 4, s));
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint32_t w[4];
  template <bool VEC>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n) {
    if (VEC && n >= 8) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (2 * i < n ? q[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(q[2 * i + 1]) : 0u) << 16;
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) t = __vmaxu2(t, w[i] & 0x7FFF7FFFu);
    return t;
  }
  static __device__ __forceinline__ uint32_t top_of(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
  static __device__ __forceinline__ uint32_t bits(uint32_t t) {
    return larger(t << 16, t & 0xFFFF0000u);
  }
  __device__ __forceinline__ uint2 codes(const Scale& s) const {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
    return make_uint2(codes4(v, s), codes4(v + 4, s));
  }
};

// ALL: every block of 128 is whole and there are groups of kGroup of them.
template <typename T, bool VEC, bool ALL>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(Fp8QuantArgs a, int kbs,
                                                                 int groups) {
  grid_dependency_wait();
  grid_dependents_go();
  const int l = threadIdx.x & 15;
  const int r = static_cast<int>(blockIdx.x / groups) * kRowsPerBlock + (threadIdx.x >> 4);
  const int kb0 = static_cast<int>(blockIdx.x % groups) * kGroup;
  const bool live = r < a.rows;
  int from = r;
  if (live && a.index) from = __ldg(a.index + r);
  const bool zero = !live || from < 0 || from >= a.T;
  const int col0 = kb0 * B + l * 8;
  const T* x = static_cast<const T*>(a.x) + (zero ? 0 : from * a.ldx + col0);
  Eight<T> v[kGroup];
#pragma unroll
  for (int g = 0; g < kGroup; ++g)
    v[g].template load<VEC>(x + g * B, zero ? 0 : ALL ? 8 : a.C - col0 - g * B);
  uint8_t* codes = a.codes + r * a.ld + col0;
  float* scales = a.scales + kb0 * a.ld_scales + r;
#pragma unroll
  for (int g = 0; g < kGroup; ++g) {
    uint32_t top = v[g].top();
#pragma unroll
    for (int d = 8; d; d >>= 1)
      top = Eight<T>::top_of(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    if (!live || (!ALL && kb0 + g >= kbs)) continue;
    const Scale s = scale_of(Eight<T>::bits(top));
    if (l == 0) scales[g * a.ld_scales] = s.step;
    store8(codes + g * B, ALL ? 8 : a.C - col0 - g * B, v[g].codes(s));
  }
}

// ---- the transposed matrix: row c of the codes is column c of X.  A block takes
// 128 rows of X by 64 columns through shared memory; a thread then holds 32 values
// of a column.
constexpr int kTransCols = 64;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_transposed_kernel(Fp8QuantArgs a, int tiles_c) {
  __shared__ T tile[B][kTransCols + (sizeof(T) == 4 ? 1 : 2)];
  __shared__ uint32_t tops[4][kTransCols];
  grid_dependency_wait();
  grid_dependents_go();
  const int c0 = static_cast<int>(blockIdx.x % tiles_c) * kTransCols;
  const int kb = static_cast<int>(blockIdx.x / tiles_c), t0 = kb * B;
  const T* x = static_cast<const T*>(a.x);
  if (VEC) {
    const int col = (threadIdx.x & 7) * 8;
#pragma unroll
    for (int i = 0; i < B / 32; ++i) {
      const int t = i * 32 + (threadIdx.x >> 3);
      float v[8];
      load8<true>(x + (t0 + t) * a.ldx + c0 + col, t0 + t < a.T ? a.C - c0 - col : 0, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) tile[t][col + j] = from_f32<T>(v[j]);
    }
  } else {
    const int col = threadIdx.x & 63;
#pragma unroll 8
    for (int i = 0; i < B / 4; ++i) {
      const int t = i * 4 + (threadIdx.x >> 6);
      tile[t][col] = t0 + t < a.T && c0 + col < a.C ? x[(t0 + t) * a.ldx + c0 + col]
                                                    : from_f32<T>(0.0f);
    }
  }
  __syncthreads();
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  float v[32];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = to_f32(tile[q * 32 + i][c]);
    top = larger(top, magnitude(v[i]));
  }
  tops[q][c] = top;
  __syncthreads();
  if (c0 + c >= a.C) return;
  top = larger(larger(tops[0][c], tops[1][c]), larger(tops[2][c], tops[3][c]));
  const Scale s = scale_of(top);
  if (q == 0) a.scales[kb * a.ld_scales + c0 + c] = s.step;
  const int t = t0 + q * 32;
  uint8_t* out = a.codes + (c0 + c) * a.ld + t;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    store8(out + 8 * i, a.T - t - 8 * i,
           make_uint2(codes4(v + 8 * i, s), codes4(v + 8 * i + 4, s)));
}

// ---- a scale for each 128 x 128: a block of threads holds the square in
// registers between finding its largest value and dividing by the scale.
template <typename T, bool VEC, bool TRANSPOSE>
__global__ void __launch_bounds__(kThreads) quantize_square_kernel(Fp8QuantArgs a, int tiles_c) {
  __shared__ uint32_t tops[kThreads / 32];
  __shared__ __align__(16) uint8_t turned[TRANSPOSE ? B : 1][TRANSPOSE ? B + 16 : 16];
  grid_dependency_wait();
  grid_dependents_go();
  const int tc = static_cast<int>(blockIdx.x % tiles_c), tr = static_cast<int>(blockIdx.x / tiles_c);
  const int l = threadIdx.x & 15, h = threadIdx.x >> 4;
  const int col = tc * B + l * 8;
  const T* x = static_cast<const T*>(a.x) + blockIdx.y * a.x_step;
  uint8_t* codes = a.codes + blockIdx.y * a.codes_step;
  float* scales = a.scales + blockIdx.y * a.scales_step;
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = tr * B + i * 16 + h;
    load8<VEC>(x + row * a.ldx + col, row < a.T ? a.C - col : 0, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = larger(top, magnitude(v[i][j]));
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) top = larger(top, tops[i]);
  const Scale s = scale_of(top);
  if (threadIdx.x == 0)
    scales[TRANSPOSE ? tc * a.ld_scales + tr : tr * a.ld_scales + tc] = s.step;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = tr * B + i * 16 + h;
    const uint2 c = make_uint2(codes4(v[i], s), codes4(v[i] + 4, s));
    if (!TRANSPOSE) {
      if (row < a.T) store8(codes + row * a.ld + col, a.C - col, c);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        turned[l * 8 + j][i * 16 + h] = static_cast<uint8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
    }
  }
  if (TRANSPOSE) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 16 + h, row = tr * B + l * 8;  // row c of the codes' tile
      if (tc * B + c < a.C)
        store8(codes + (tc * B + c) * a.ld + row, a.T - row,
               *reinterpret_cast<const uint2*>(&turned[c][l * 8]));
    }
  }
}

// Rows that start on 16 bytes, with strides that keep them there.
bool wide_rows(const Fp8QuantArgs& a) {
  const int per = a.x_bf16 ? 8 : 4;
  return (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ldx % per == 0 && a.x_step % per == 0;
}

// Calls f with the element type and whether rows are wide.
template <typename F>
cudaError_t by_type(const Fp8QuantArgs& a, F f) {
  using Wide = std::true_type;
  using Narrow = std::false_type;
  const bool w = wide_rows(a);
  const cudaError_t e = a.x_bf16 ? (w ? f(__nv_bfloat16(), Wide()) : f(__nv_bfloat16(), Narrow()))
                                 : (w ? f(float(), Wide()) : f(float(), Narrow()));
  if (e == cudaSuccess) note_launches(1);
  return e;
}

int64_t blocks_of(int64_t n, int64_t size) { return (n + size - 1) / size; }

}  // namespace

cudaError_t launch_fp8_quantize_rows(const Fp8QuantArgs& a, cudaStream_t stream) {
  const int kbs = static_cast<int>(blocks_of(a.C, B)), groups = static_cast<int>(blocks_of(kbs, kGroup));
  const int64_t grid = blocks_of(a.rows, kRowsPerBlock) * groups;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const bool all = a.C % (kGroup * B) == 0;
  return by_type(a, [&](auto t, auto wide) {
    using T = decltype(t);
    constexpr bool kWide = decltype(wide)::value;
    return launch_pdl(all ? quantize_rows_kernel<T, kWide, true> : quantize_rows_kernel<T, kWide, false>,
                      dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a, kbs, groups);
  });
}

cudaError_t launch_fp8_quantize_transposed(const Fp8QuantArgs& a, cudaStream_t stream) {
  const int64_t tiles_c = blocks_of(a.C, kTransCols), grid = tiles_c * blocks_of(a.T, B);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return by_type(a, [&](auto t, auto wide) {
    return launch_pdl(quantize_transposed_kernel<decltype(t), decltype(wide)::value>,
                      dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a,
                      static_cast<int>(tiles_c));
  });
}

cudaError_t launch_fp8_quantize_square(const Fp8QuantArgs& a, bool transpose, cudaStream_t stream) {
  const int64_t tiles_c = blocks_of(a.C, B), grid = tiles_c * blocks_of(a.T, B);
  if (grid > 0x7FFFFFFF || a.batch > 65535) return cudaErrorInvalidValue;
  return by_type(a, [&](auto t, auto wide) {
    using T = decltype(t);
    constexpr bool kWide = decltype(wide)::value;
    return launch_pdl(transpose ? quantize_square_kernel<T, kWide, true>
                                : quantize_square_kernel<T, kWide, false>,
                      dim3(static_cast<unsigned>(grid), static_cast<unsigned>(a.batch)),
                      dim3(kThreads), 0, stream, a, static_cast<int>(tiles_c));
  });
}

}  // namespace g07
