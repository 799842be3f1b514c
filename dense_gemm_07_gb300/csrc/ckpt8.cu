// ckpt8.cu -- activations kept in 8 bits for the backward pass.  A run of 32
// rows (tokens) of a column shares a power-of-two step 2^e, the smallest (at
// least 2^-126) with max|x| <= 127 * 2^e, and holds q = round(x / 2^e), ties to
// even, in -127..127: the value kept, q * 2^e, is at most half a step off, is
// an exact BF16 number, and both directions are exact arithmetic besides the
// one rounding.  A run with a value that is not finite is kept as NaN.
//
// The runs go down the columns because a channel's size is steady over tokens
// while channels differ, and because the weight gradient sums over tokens: one
// scale then covers 32 steps of that sum for a row of X^T.
//
// Layout: q[panel][half][column][16], panel = 32 rows, half = 16 of them; the
// step of (panel, column) as the byte e + 127 (255: NaN).  A thread that owns a
// column of a panel holds a whole run in registers, so neither direction needs
// shared memory; rows past T are kept as zeros.  Memory bounds these kernels.
// Measured at 2048 x 11008, FP32 in, GELU: pack with its activations 27.8 us,
// gradient with its column sums 36.5 us.
#include <cuda_bf16.h>

#include "ckpt8.cuh"
#include "kernels.h"
#include "layer.h"
#include "normal_tail.cuh"

namespace g07 {
namespace {

constexpr int kThreads = 128;

// x Phi(x), and its slope Phi(x) + x phi(x).
template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if (ACT == 1) return fmaxf(v, 0.0f);
  if (ACT == 2) {
    float e;
    const float tail = 0.5f * normal_tail2(v, &e);
    return v * (v > 0.0f ? 1.0f - tail : tail);
  }
  return v;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float v) {
  if (ACT == 1) return v > 0.0f ? 1.0f : (v == v ? 0.0f : v);
  if (ACT == 2) {
    float e;
    const float tail = 0.5f * normal_tail2(v, &e);
    return fmaf(v * 0.39894228f, e, v > 0.0f ? 1.0f - tail : tail);
  }
  return 1.0f;
}

// C adjacent elements (C = 1, or 2 on a boundary of two) of a row.
template <int C>
__device__ __forceinline__ void load_cols(const float* p, float (&v)[C]) {
  if constexpr (C == 2) {
    const float2 a = *reinterpret_cast<const float2*>(p);
    v[0] = a.x;
    v[1] = a.y;
  } else {
    v[0] = *p;
  }
}
template <int C>
__device__ __forceinline__ void load_cols(const __nv_bfloat16* p, float (&v)[C]) {
  if constexpr (C == 2) {
    const uint32_t a = *reinterpret_cast<const uint32_t*>(p);
    v[0] = bf16_lo(a);
    v[1] = bf16_hi(a);
  } else {
    v[0] = __bfloat162float(*p);
  }
}
template <int C>
__device__ __forceinline__ void store_cols(__nv_bfloat16* p, const float (&v)[C]) {
  if constexpr (C == 2)
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(v[0], v[1]);
  else
    *p = __float2bfloat16_rn(v[0]);
}

// The low byte of the FP32 bits of v + 1.5 * 2^23 is round(v), ties to even, in
// two's complement (|v| <= 127).
__device__ __forceinline__ uint32_t round_byte(float v, float inverse_step) {
  return __float_as_uint(fmaf(v, inverse_step, 12582912.0f));
}
__device__ __forceinline__ uint32_t four_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A thread owns C adjacent columns of a panel; a warp's loads of a row are
// contiguous.  OUT: also write act(x).
template <typename X, int C, int ACT, bool OUT>
__global__ void __launch_bounds__(kThreads) ckpt8_pack_kernel(CkptArgs p) {
  grid_dependency_wait();
  grid_dependents_go();
  const int c = (blockIdx.x * kThreads + threadIdx.x) * C;
  if (c >= p.N) return;
  const int panels = (p.T + kCkptRun - 1) / kCkptRun;
  for (int panel = blockIdx.y; panel < panels; panel += gridDim.y) {
    const int t0 = panel * kCkptRun;
    const int rows = min(kCkptRun, p.T - t0);
    const X* x = static_cast<const X*>(p.x) + t0 * p.ldx + c;
    float v[kCkptRun][C];
    if (rows == kCkptRun) {
#pragma unroll
      for (int i = 0; i < kCkptRun; ++i) load_cols<C>(x + i * p.ldx, v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kCkptRun; ++i) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[i][j] = 0.0f;
        if (i < rows) load_cols<C>(x + i * p.ldx, v[i]);
      }
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      uint32_t top = 0;  // magnitudes compare as integers; above 0x7F800000: NaN
#pragma unroll
      for (int i = 0; i < kCkptRun; ++i) top = max(top, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
      const uint32_t code = ckpt8_code(top);
      const float inv = ckpt8_inverse_step(code);
      uint32_t w[8];
      if (code < 248u) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i] = four_bytes(round_byte(v[4 * i][j], inv), round_byte(v[4 * i + 1][j], inv),
                            round_byte(v[4 * i + 2][j], inv), round_byte(v[4 * i + 3][j], inv));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i] = four_bytes(ckpt8_round(v[4 * i][j], inv), ckpt8_round(v[4 * i + 1][j], inv),
                            ckpt8_round(v[4 * i + 2][j], inv), ckpt8_round(v[4 * i + 3][j], inv));
      }
      uint4* q = reinterpret_cast<uint4*>(p.q) + (static_cast<int64_t>(panel) * 2) * p.N + c + j;
      q[0] = make_uint4(w[0], w[1], w[2], w[3]);
      q[p.N] = make_uint4(w[4], w[5], w[6], w[7]);
      p.scales[static_cast<int64_t>(panel) * p.N + c + j] = static_cast<uint8_t>(code);
    }
    if constexpr (OUT) {
      __nv_bfloat16* o = p.out + t0 * p.ld_out + c;
#pragma unroll
      for (int i = 0; i < kCkptRun; ++i)
        if (i < rows) {
          float a[C];
#pragma unroll
          for (int j = 0; j < C; ++j) a[j] = act_value<ACT>(v[i][j]);
          store_cols<C>(o + i * p.ld_out, a);
        }
    }
  }
}

// A column's run of 32 kept values: words and step.
struct Run {
  uint32_t w[8];
  float step;
  __device__ __forceinline__ float at(int i) const {
    return static_cast<float>(static_cast<int8_t>(w[i / 4] >> (8 * (i % 4)))) * step;
  }
};
__device__ __forceinline__ Run load_run(const uint8_t* q, const uint8_t* scales, int panel, int N,
                                        int c) {
  const uint4* src = reinterpret_cast<const uint4*>(q) + (static_cast<int64_t>(panel) * 2) * N + c;
  const uint4 a = src[0], b = src[N];
  return Run{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w},
             ckpt8_step(scales[static_cast<int64_t>(panel) * N + c])};
}

template <typename O>
__global__ void __launch_bounds__(kThreads)
ckpt8_unpack_kernel(int T, int N, const uint8_t* __restrict__ q,
                    const uint8_t* __restrict__ scales, O* __restrict__ out, int64_t ld) {
  grid_dependency_wait();
  grid_dependents_go();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= N) return;
  const int panels = (T + kCkptRun - 1) / kCkptRun;
  for (int panel = blockIdx.y; panel < panels; panel += gridDim.y) {
    const Run r = load_run(q, scales, panel, N, c);
    O* o = out + static_cast<int64_t>(panel) * kCkptRun * ld + c;
#pragma unroll
    for (int i = 0; i < kCkptRun; ++i)
      if (panel * kCkptRun + i < T) o[i * ld] = from_f32<O>(r.at(i));
  }
}

// dz = g * act'(kept z), and the column sums of dz before its rounding: each
// block leaves its own in partial[blockIdx.y][N] and counts itself at its
// columns' counter; the last one to do so adds all of them in the order of the
// rows and puts the counter back to zero.  (A launch of its own for these sums
// cost 4 of 21 us at 127 x 1000.)
template <typename X, int C, int ACT>
__global__ void __launch_bounds__(kThreads) ckpt8_act_grad_kernel(CkptArgs p, ColumnTotals sums) {
  grid_dependency_wait();
  grid_dependents_go();
  const int c = (blockIdx.x * kThreads + threadIdx.x) * C;
  const int panels = c < p.N ? (p.T + kCkptRun - 1) / kCkptRun : 0;
  float sum[C] = {};
  for (int panel = blockIdx.y; panel < panels; panel += gridDim.y) {
    const int t0 = panel * kCkptRun;
    const int rows = min(kCkptRun, p.T - t0);
    const X* x = static_cast<const X*>(p.x) + t0 * p.ldx + c;
    float g[kCkptRun][C];
    if (rows == kCkptRun) {
#pragma unroll
      for (int i = 0; i < kCkptRun; ++i) load_cols<C>(x + i * p.ldx, g[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kCkptRun; ++i) {
#pragma unroll
        for (int j = 0; j < C; ++j) g[i][j] = 0.0f;
        if (i < rows) load_cols<C>(x + i * p.ldx, g[i]);
      }
    }
    Run r[C];
#pragma unroll
    for (int j = 0; j < C; ++j) r[j] = load_run(p.q, p.scales, panel, p.N, c + j);
    __nv_bfloat16* o = p.out + t0 * p.ld_out + c;
#pragma unroll
    for (int i = 0; i < kCkptRun; ++i)
      if (i < rows) {
        float dz[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
          dz[j] = g[i][j] * act_slope<ACT>(r[j].at(i));
          sum[j] += dz[j];
        }
        store_cols<C>(o + i * p.ld_out, dz);
      }
  }
  if (sums.out == nullptr) return;
  if (gridDim.y == 1) {
    if (c < p.N)
#pragma unroll
      for (int j = 0; j < C; ++j) sums.out[c + j] = sum[j];
    return;
  }
  if (c < p.N)
#pragma unroll
    for (int j = 0; j < C; ++j)
      sums.partial[static_cast<int64_t>(blockIdx.y) * p.N + c + j] = sum[j];
  __threadfence();
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(sums.counters + blockIdx.x, 1u) + 1 == gridDim.y;
    if (last) sums.counters[blockIdx.x] = 0u;  // for the next launch
  }
  __syncthreads();
  if (!last || c >= p.N) return;
  __threadfence();
#pragma unroll
  for (int j = 0; j < C; ++j) sum[j] = 0.0f;
#pragma unroll 16
  for (int y = 0; y < static_cast<int>(gridDim.y); ++y)
#pragma unroll
    for (int j = 0; j < C; ++j)
      sum[j] += __ldcg(sums.partial + static_cast<int64_t>(y) * p.N + c + j);
#pragma unroll
  for (int j = 0; j < C; ++j) sums.out[c + j] = sum[j];
}

dim3 panel_grid(int T, int N) {
  const int panels = (T + kCkptRun - 1) / kCkptRun;
  return dim3((N + kThreads - 1) / kThreads, panels < 65535 ? panels : 65535);
}

}  // namespace

// Two columns a thread when every row starts on a boundary of two elements
// (8-byte loads of FP32, 4-byte loads and stores of BF16), else one.
static bool pairs_ok(const CkptArgs& a) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.x), o = reinterpret_cast<uintptr_t>(a.out);
  return a.N % 2 == 0 && a.ldx % 2 == 0 && x % (a.x_bf16 ? 4 : 8) == 0 &&
         (a.out == nullptr || (a.ld_out % 2 == 0 && o % 4 == 0));
}
static unsigned column_blocks(int N, int columns) {
  return static_cast<unsigned>((N + kThreads * columns - 1) / (kThreads * columns));
}

template <typename X, int C>
static cudaError_t pack(const CkptArgs& a, cudaStream_t st) {
  const dim3 grid(column_blocks(a.N, C), panel_grid(a.T, a.N).y), block(kThreads);
  if (a.out == nullptr) return launch_pdl(ckpt8_pack_kernel<X, C, 0, false>, grid, block, 0, st, a);
  if (a.act == 0) return launch_pdl(ckpt8_pack_kernel<X, C, 0, true>, grid, block, 0, st, a);
  if (a.act == 1) return launch_pdl(ckpt8_pack_kernel<X, C, 1, true>, grid, block, 0, st, a);
  return launch_pdl(ckpt8_pack_kernel<X, C, 2, true>, grid, block, 0, st, a);
}

template <typename X, int C>
static cudaError_t act_grad(const CkptArgs& a, const ColumnTotals& sums, int slots,
                            cudaStream_t st) {
  const dim3 grid(column_blocks(a.N, C), slots), block(kThreads);
  if (a.act == 0) return launch_pdl(ckpt8_act_grad_kernel<X, C, 0>, grid, block, 0, st, a, sums);
  if (a.act == 1) return launch_pdl(ckpt8_act_grad_kernel<X, C, 1>, grid, block, 0, st, a, sums);
  return launch_pdl(ckpt8_act_grad_kernel<X, C, 2>, grid, block, 0, st, a, sums);
}

cudaError_t launch_ckpt8_pack(const CkptArgs& a, cudaStream_t stream) {
  using B = __nv_bfloat16;
  const bool two = pairs_ok(a);
  const cudaError_t e = a.x_bf16 ? (two ? pack<B, 2>(a, stream) : pack<B, 1>(a, stream))
                                 : (two ? pack<float, 2>(a, stream) : pack<float, 1>(a, stream));
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_ckpt8_unpack(int T, int N, const uint8_t* q, const uint8_t* scales, void* out,
                                int64_t ld, bool out_bf16, cudaStream_t stream) {
  const dim3 grid = panel_grid(T, N), block(kThreads);
  const cudaError_t e =
      out_bf16 ? launch_pdl(ckpt8_unpack_kernel<__nv_bfloat16>, grid, block, 0, stream, T, N, q,
                            scales, static_cast<__nv_bfloat16*>(out), ld)
               : launch_pdl(ckpt8_unpack_kernel<float>, grid, block, 0, stream, T, N, q, scales,
                            static_cast<float*>(out), ld);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

// The blocks of a column block: each walks the same number of panels, with at
// most about 8 blocks an SM.  (8 fit with 64 registers a thread, one column; the
// forms of two columns take up to 106, so that 4 fit: 2048 x 11008 runs as 946
// blocks on 608 places.)
int ckpt8_act_grad_slots(int T, int N, const LayerDevice& dev) {
  const int64_t panels = (T + kCkptRun - 1) / kCkptRun;
  const int64_t each = panels * column_blocks(N, 2) / (static_cast<int64_t>(dev.sms) * 8) + 1;
  return static_cast<int>((panels + each - 1) / each);
}

int64_t ckpt8_act_grad_counters(int N) { return column_blocks(N, 1); }

cudaError_t launch_ckpt8_act_grad(const CkptArgs& a, const ColumnTotals& sums, int slots,
                                  cudaStream_t stream) {
  using B = __nv_bfloat16;
  const bool two = pairs_ok(a);
  const cudaError_t e = a.x_bf16 ? (two ? act_grad<B, 2>(a, sums, slots, stream)
                                        : act_grad<B, 1>(a, sums, slots, stream))
                                 : (two ? act_grad<float, 2>(a, sums, slots, stream)
                                        : act_grad<float, 1>(a, sums, slots, stream));
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace g07
