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
#include <cuda_bf16.h>

#include "ckpt8.cuh"
#include "kernels.h"
#include "layer.h"

namespace g07 {
namespace {

constexpr int kThreads = 128;

// x * Phi(x) as the GEMM's epilogue computes it, and its slope
// Phi(x) + x phi(x).
__device__ __forceinline__ float act_value(float v, int act) {
  return epi_apply(EpiParams{1.0f, 0.0f, nullptr, act}, v, 0.0f, 0.0f);
}
__device__ __forceinline__ float act_slope(float v, int act) {
  if (act == 1) return v > 0.0f ? 1.0f : (v == v ? 0.0f : v);
  if (act == 2)
    return 0.5f * (1.0f + erff(v * 0.70710678118654752f)) +
           v * expf(-0.5f * v * v) * 0.39894228040143268f;
  return 1.0f;
}

template <typename X>
__global__ void __launch_bounds__(kThreads) ckpt8_pack_kernel(CkptArgs p) {
  grid_dependency_wait();
  grid_dependents_go();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.N) return;
  const int panels = (p.T + kCkptRun - 1) / kCkptRun;
  for (int panel = blockIdx.y; panel < panels; panel += gridDim.y) {
    const int t0 = panel * kCkptRun;
    const int rows = min(kCkptRun, p.T - t0);
    const X* x = static_cast<const X*>(p.x) + t0 * p.ldx + c;
    float v[kCkptRun];
#pragma unroll
    for (int i = 0; i < kCkptRun; ++i) v[i] = i < rows ? to_f32(x[i * p.ldx]) : 0.0f;
    uint32_t top = 0;  // magnitudes compare as integers; above 0x7F800000: NaN
#pragma unroll
    for (int i = 0; i < kCkptRun; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const uint32_t code = ckpt8_code(top);
    const float inv = ckpt8_inverse_step(code);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        w[i] |= (static_cast<uint32_t>(ckpt8_round(v[4 * i + b], inv)) & 0xFFu) << (8 * b);
    }
    uint4* q = reinterpret_cast<uint4*>(p.q) + (static_cast<int64_t>(panel) * 2) * p.N + c;
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[p.N] = make_uint4(w[4], w[5], w[6], w[7]);
    p.scales[static_cast<int64_t>(panel) * p.N + c] = static_cast<uint8_t>(code);
    if (p.out) {
      __nv_bfloat16* o = p.out + t0 * p.ld_out + c;
#pragma unroll
      for (int i = 0; i < kCkptRun; ++i)
        if (i < rows) o[i * p.ld_out] = __float2bfloat16_rn(act_value(v[i], p.act));
    }
  }
}

// A column's run of 32 kept values.
__device__ __forceinline__ void load_run(const uint8_t* q, const uint8_t* scales, int panel, int N,
                                         int c, float (&v)[kCkptRun]) {
  const uint4* src = reinterpret_cast<const uint4*>(q) + (static_cast<int64_t>(panel) * 2) * N + c;
  const uint4 a = src[0], b = src[N];
  const float step = ckpt8_step(scales[static_cast<int64_t>(panel) * N + c]);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < kCkptRun; ++i)
    v[i] = static_cast<float>(static_cast<int8_t>(w[i / 4] >> (8 * (i % 4)))) * step;
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
    float v[kCkptRun];
    load_run(q, scales, panel, N, c, v);
    O* o = out + static_cast<int64_t>(panel) * kCkptRun * ld + c;
#pragma unroll
    for (int i = 0; i < kCkptRun; ++i)
      if (panel * kCkptRun + i < T) o[i * ld] = from_f32<O>(v[i]);
  }
}

// dz = g * act'(kept z) and the block's column sums of dz (before rounding),
// to partial[blockIdx.y][N].
template <typename X>
__global__ void __launch_bounds__(kThreads) ckpt8_act_grad_kernel(CkptArgs p, float* partial) {
  grid_dependency_wait();
  grid_dependents_go();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.N) return;
  const int panels = (p.T + kCkptRun - 1) / kCkptRun;
  float sum = 0.0f;
  for (int panel = blockIdx.y; panel < panels; panel += gridDim.y) {
    const int t0 = panel * kCkptRun;
    const int rows = min(kCkptRun, p.T - t0);
    const X* x = static_cast<const X*>(p.x) + t0 * p.ldx + c;
    float g[kCkptRun], v[kCkptRun];
#pragma unroll
    for (int i = 0; i < kCkptRun; ++i) g[i] = i < rows ? to_f32(x[i * p.ldx]) : 0.0f;
    load_run(p.q, p.scales, panel, p.N, c, v);
    __nv_bfloat16* o = p.out + t0 * p.ld_out + c;
#pragma unroll
    for (int i = 0; i < kCkptRun; ++i)
      if (i < rows) {
        const float dz = g[i] * act_slope(v[i], p.act);
        sum += dz;
        o[i * p.ld_out] = __float2bfloat16_rn(dz);
      }
  }
  if (partial) partial[static_cast<int64_t>(blockIdx.y) * p.N + c] = sum;
}

__global__ void __launch_bounds__(kThreads)
ckpt8_transposed_kernel(int T, int N, const uint8_t* __restrict__ q,
                        const uint8_t* __restrict__ scales, __nv_bfloat16* __restrict__ out,
                        int64_t ld) {
  grid_dependency_wait();
  grid_dependents_go();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= N) return;
  const int panels = (T + kCkptRun - 1) / kCkptRun;
  for (int panel = blockIdx.y; panel < panels; panel += gridDim.y) {
    float v[kCkptRun];
    load_run(q, scales, panel, N, c, v);
    uint4* o = reinterpret_cast<uint4*>(out + c * ld + panel * kCkptRun);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                        pack_bf16(v[8 * i + 4], v[8 * i + 5]),
                        pack_bf16(v[8 * i + 6], v[8 * i + 7]));
  }
}

dim3 panel_grid(int T, int N) {
  const int panels = (T + kCkptRun - 1) / kCkptRun;
  return dim3((N + kThreads - 1) / kThreads, panels < 65535 ? panels : 65535);
}

}  // namespace

cudaError_t launch_ckpt8_pack(const CkptArgs& a, cudaStream_t stream) {
  const dim3 grid = panel_grid(a.T, a.N), block(kThreads);
  const cudaError_t e =
      a.x_bf16 ? launch_pdl(ckpt8_pack_kernel<__nv_bfloat16>, grid, block, 0, stream, a)
               : launch_pdl(ckpt8_pack_kernel<float>, grid, block, 0, stream, a);
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

int ckpt8_act_grad_slots(int T, int N, const LayerDevice& dev) {
  const int64_t panels = (T + kCkptRun - 1) / kCkptRun;
  const int64_t cols = (N + kThreads - 1) / kThreads;
  int64_t s = (static_cast<int64_t>(dev.sms) * 16 + cols - 1) / cols;
  if (s > panels) s = panels;
  return static_cast<int>(s < 1 ? 1 : s);
}

cudaError_t launch_ckpt8_act_grad(const CkptArgs& a, int slots, float* partial,
                                  cudaStream_t stream) {
  const dim3 grid((a.N + kThreads - 1) / kThreads, slots), block(kThreads);
  const cudaError_t e =
      a.x_bf16 ? launch_pdl(ckpt8_act_grad_kernel<__nv_bfloat16>, grid, block, 0, stream, a, partial)
               : launch_pdl(ckpt8_act_grad_kernel<float>, grid, block, 0, stream, a, partial);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_ckpt8_transposed(int T, int N, const uint8_t* q, const uint8_t* scales,
                                    __nv_bfloat16* out, int64_t ld, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(ckpt8_transposed_kernel, panel_grid(T, N), dim3(kThreads), 0,
                                   stream, T, N, q, scales, out, ld);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace g07
