// layer.h -- internal launch interface of the operators that stand beside the
// GEMM in a transformer layer (4-bit weights, norms with gate and residual,
// 8-bit checkpoints): between their C-ABI layer (api_layer.cu) and the kernel
// translation units.  Not installed; not part of the ABI.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/gemm07.h"
#include "epilogue.cuh"
#include "stream_k.cuh"

namespace g07 {

// ---- services of api.cu used by api_layer.cu
struct LayerDevice {
  int sms = 0;
  unsigned int* status = nullptr;  // device status word (kernels.h)
};
// The current device, checked once (GEMM_ERR_UNSUPPORTED_DEVICE otherwise).
gemm_status_t layer_device(LayerDevice* out);
// Scratch for work queued on `stream` (contents undefined); the block is kept
// for the stream's next call unless `owned`, and handed back with
// layer_scratch_done() once the work that uses it has been queued.
struct LayerScratch {
  void* ptr = nullptr;
  bool owned = false;
};
gemm_status_t layer_scratch(cudaStream_t stream, int64_t bytes, LayerScratch* out);
// Scratch of another kind that starts with kLayerCounterBytes of counters: zero
// when the block is new, and put back to zero by whoever uses them.
constexpr int64_t kLayerCounterBytes = 64 << 10;
gemm_status_t layer_counted_scratch(cudaStream_t stream, int64_t bytes, LayerScratch* out);
void layer_scratch_done(const LayerScratch& s, cudaStream_t stream);
gemm_status_t layer_epilogue(const gemm_epilogue_t* e, EpiParams* out);
gemm_status_t layer_from_cuda(cudaError_t e);
// dW := X^T dY + beta dW with X kept in 8 bits (T > 0, sizes checked).
gemm_status_t layer_ckpt8_wgrad(int64_t T, int64_t K, int64_t N, const uint8_t* q,
                                const uint8_t* scales, const uint16_t* dY, int64_t ld_dy,
                                float* dW, int64_t ldw, float beta, cudaStream_t stream);

// Lets `kernel` ask for up to `most` bytes of dynamic shared memory on the current
// device.  The limit belongs to the kernel, not to a launch: it is set once, to the
// largest size of any call, and never lowered under another thread's launch.
// `done`: a bit per device (api.cu admits 64), one word per kernel.
template <typename... P>
cudaError_t allow_shared(void (*kernel)(P...), size_t most, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(most));
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

// ---- element access shared by the kernels
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// N consecutive elements as FP32: N = 8 is one 16-byte (BF16) or two 16-byte
// (FP32) accesses on a 16-byte boundary, N = 1 one element.
template <int N>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[N]) {
  if constexpr (N == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    v[0] = *p;
  }
}
template <int N>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[N]) {
  if constexpr (N == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
  } else {
    v[0] = __bfloat162float(*p);
  }
}
template <int N>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[N]) {
  if constexpr (N == 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}
template <int N>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[N]) {
  if constexpr (N == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}

// ---- asynchronous copies global -> shared of one thread.  The thread that
// issues a copy is the one that reads it, after cp_async_wait: no barrier.
__device__ __forceinline__ uint32_t shared_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes, both addresses on 16 bytes; only the first `bytes` are read, the
// rest of the 16 are zeros.
__device__ __forceinline__ void cp_async_16(void* dst, const void* src, uint32_t bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(shared_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// At most N of this thread's groups are still on their way.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- 4-bit weights (w4.cu)
constexpr int kW4TileN = 16;    // columns of a packed tile
constexpr int kW4TileK = 128;   // rows of a packed tile
constexpr int kW4TileBytes = 1024;
constexpr int kW4MaxRows = 65535 * 8;  // grid rows of 8 rows of A at least
struct W4Args {
  int M = 0, N = 0, K = 0;
  const __nv_bfloat16* A = nullptr;
  int64_t lda = 0;
  const uint8_t* packed = nullptr;
  const __nv_bfloat16* scales = nullptr;
  int64_t ld_scales = 0;
  const uint8_t* zeros = nullptr;
  int64_t ld_zeros = 0;
  int group = 0;
  void* C = nullptr;
  int64_t ldc = 0;
  int c_bf16 = 0;
  EpiParams epi;
};
cudaError_t launch_w4(const W4Args& a, const LayerDevice& dev, cudaStream_t stream);
cudaError_t launch_w4_pack(int K, int N, const uint8_t* codes, int64_t ld, uint8_t* packed,
                           cudaStream_t stream);
cudaError_t launch_w4_quantize(int K, int N, int group, const void* B, int64_t ldb, bool b_bf16,
                               uint8_t* packed, __nv_bfloat16* scales, int64_t ld_scales,
                               uint8_t* zeros, int64_t ld_zeros, cudaStream_t stream);
cudaError_t launch_w4_unpack(int K, int N, int group, const uint8_t* packed,
                             const __nv_bfloat16* scales, int64_t ld_scales, const uint8_t* zeros,
                             int64_t ld_zeros, __nv_bfloat16* B, int64_t ldb, cudaStream_t stream);

// ---- norms with gate and residual (norm_gate.cu)
constexpr int kNormMaxWidth = 16384;
struct NormArgs {
  int T = 0, D = 0;
  const void* x = nullptr;       // T x D, x_bf16 or FP32
  int64_t ldx = 0;
  const void* y = nullptr;       // T x D, y_bf16 or FP32, or null
  int64_t ldy = 0;
  bool x_bf16 = false, y_bf16 = false;
  const float* w_post = nullptr;  // D or null
  const float* gate = nullptr;    // gate[t * gate_row + d * gate_col], or null
  int64_t gate_row = 0;
  int gate_col = 0;
  const float* w_pre = nullptr;   // D or null
  float alpha = 1.0f, eps = 0.0f;
  // forward
  void* x_out = nullptr;          // type of x, or null
  int64_t ld_x_out = 0;
  __nv_bfloat16* h = nullptr;     // T x D (with w_pre)
  int64_t ldh = 0;
  // backward
  const void* d_x_out = nullptr;  // type of x, or null
  int64_t ld_d_x_out = 0;
  const void* dh = nullptr;       // dh_bf16 or FP32 (with w_pre)
  int64_t ld_dh = 0;
  bool dh_bf16 = false;
  void* dx = nullptr;             // type of x
  int64_t ld_dx = 0;
  __nv_bfloat16* dy = nullptr;    // with y
  int64_t ld_dy = 0;
  float* dgate = nullptr;         // laid out as gate
  float* dw_post = nullptr;
  float* dw_pre = nullptr;
};
cudaError_t launch_norm_gate(const NormArgs& a, cudaStream_t stream);
// How the gradient runs: `slots` clusters of `parts` blocks walk the rows, a
// block with part_cols columns of them; its column sums leave slots x 3 x D
// floats in `partial` (null: none are wanted).
struct NormBwdPlan {
  int parts = 0, part_cols = 0, threads = 0, stages = 0, stage_bytes = 0, slots = 0;
};
cudaError_t norm_gate_bwd_plan(const NormArgs& a, const LayerDevice& dev, NormBwdPlan* plan);
cudaError_t launch_norm_gate_bwd(const NormArgs& a, const NormBwdPlan& plan, float* partial,
                                 cudaStream_t stream);

// ---- column sums: out[c] = sum over s = 0 .. slots - 1, in that order, of
// partial[s * ld + c], for `count` vectors of n columns (vector v starts at
// column v * n of the partial rows; a null out skips it).
struct ColumnSums {
  const float* partial = nullptr;
  int64_t ld = 0;
  int slots = 0, n = 0, count = 0;
  float* out[3] = {nullptr, nullptr, nullptr};
};
cudaError_t launch_column_sums(const ColumnSums& s, cudaStream_t stream);

// ---- 8-bit checkpoints (ckpt8.cu)
constexpr int kCkptRun = 32;  // rows that share a scale
struct CkptArgs {
  int T = 0, N = 0;
  const void* x = nullptr;  // pack: the values; act_grad: the gradient
  int64_t ldx = 0;
  bool x_bf16 = false;
  uint8_t* q = nullptr;
  uint8_t* scales = nullptr;
  int act = 0;
  __nv_bfloat16* out = nullptr;  // pack: activations or null; act_grad: dz
  int64_t ld_out = 0;
};
cudaError_t launch_ckpt8_pack(const CkptArgs& a, cudaStream_t stream);
cudaError_t launch_ckpt8_unpack(int T, int N, const uint8_t* q, const uint8_t* scales, void* out,
                                int64_t ld, bool out_bf16, cudaStream_t stream);
// Where act_grad's column sums go (a null out: nowhere).  partial: slots x N
// floats; counters: ckpt8_act_grad_counters(N), zero before and after.
struct ColumnTotals {
  float* out = nullptr;
  float* partial = nullptr;
  unsigned int* counters = nullptr;
};
int ckpt8_act_grad_slots(int T, int N, const LayerDevice& dev);
int64_t ckpt8_act_grad_counters(int N);
cudaError_t launch_ckpt8_act_grad(const CkptArgs& a, const ColumnTotals& sums, int slots,
                                  cudaStream_t stream);

// ---- weight gradient from an 8-bit checkpoint (ckpt8_wgrad.cu)
// SM pairs that can be resident at once (0: the kernel cannot run here).
int ckpt8_wgrad_pairs();
PairSchedule ckpt8_wgrad_schedule(int64_t T, int64_t K, int64_t N, int max_pairs);
int64_t ckpt8_wgrad_partial_bytes(const PairSchedule& s);
int64_t ckpt8_wgrad_counters(const PairSchedule& s);
constexpr int kCkptStageRows = 128;  // rows of X and dY per stage
// tmY: dY, box {64, kCkptStageRows}, 128-byte swizzle; tmW: dW as FP32 boxes {32, 32},
// 128-byte swizzle, or null to store rows; counters: ckpt8_wgrad_counters(s)
// words, zero before and after; partial: ckpt8_wgrad_partial_bytes(s).
cudaError_t launch_ckpt8_wgrad(const CUtensorMap& tmY, const CUtensorMap* tmW,
                               const PairSchedule& s, int T, int K, int N, const uint8_t* q,
                               const uint8_t* scales, float* dW, int64_t ldw, float beta,
                               float* partial, unsigned int* counters, unsigned int* status,
                               cudaStream_t stream);

}  // namespace g07
