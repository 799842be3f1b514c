// experts.h -- internal launch interface of the 8-bit floating-point products and
// of the operators of a layer of experts (routing, the experts' products,
// combining): between their C-ABI layer (api_experts.cu) and the kernel
// translation units.  Not installed; not part of the ABI.
#pragma once

#include "layer.h"

namespace g07 {

// Tensor map over rows of bytes: dims {inner, outer}, row stride ld, boxes of 128
// bytes by `box_rows` rows, 128-byte swizzle, zero fill (api.cu).
gemm_status_t layer_map_bytes(CUtensorMap* map, const void* base, int64_t inner, int64_t outer,
                              int64_t ld, uint32_t box_rows);

// ---- 8-bit floating point (fp8_quantize.cu)
constexpr int kFp8Block = 128;  // values that share a scale, rows of a square block
struct Fp8QuantArgs {
  int T = 0, C = 0;       // X: batch matrices of T x C
  int batch = 1;
  const void* x = nullptr;
  int64_t ldx = 0, x_step = 0;  // x_step: elements from one matrix to the next
  bool x_bf16 = false;
  const int* index = nullptr;  // rows of X to take, or null: all (batch 1, not transposed)
  int rows = 0;                // of the codes: T, C when transposed, or the length of index
  uint8_t* codes = nullptr;
  int64_t ld = 0, codes_step = 0;
  float* scales = nullptr;
  int64_t ld_scales = 0, scales_step = 0;
};
cudaError_t launch_fp8_quantize_rows(const Fp8QuantArgs& a, cudaStream_t stream);
cudaError_t launch_fp8_quantize_transposed(const Fp8QuantArgs& a, cudaStream_t stream);
cudaError_t launch_fp8_quantize_square(const Fp8QuantArgs& a, bool transpose, cudaStream_t stream);

// ---- 8-bit products (fp8_few.cu): C[m][n] = sum over k blocks of
// sa[kb][m] * sb * (sum over the block's k of a[m][k] * b[n][k]), dense (E = 0)
// or with rows sorted by expert.
struct Fp8GemmArgs {
  int M = 0, N = 0, K = 0;
  int E = 0;                    // experts, or 0: dense
  const int* offsets = nullptr;  // E + 1 rows, clamped to 0 .. M and made non-decreasing
  const float* sa = nullptr;    // sa[kb * ld_sa + m]
  int64_t ld_sa = 0;
  const float* sb = nullptr;    // square: sb[(e * ceil(N / 128) + n / 128) * ld_sb + kb]
  int64_t ld_sb = 0;            // rows: sb[kb * ld_sb + n]
  bool b_square = false;
  void* C = nullptr;
  int64_t ldc = 0;
  int c_bf16 = 0;
  EpiParams epi;                // bias of expert e at bias + e * N
};
// How a product runs on 128 x `cols` tiles, each by a cluster of `split` blocks
// that share K.
struct Fp8FewPlan {
  int cols = 0, split = 0, stages = 0;
  int64_t tiles = 0;
};
cudaError_t fp8_few_plan(const Fp8GemmArgs& a, const LayerDevice& dev, Fp8FewPlan* plan);
// tmA: boxes of plan.cols rows; tmB: boxes of 128 rows.
cudaError_t launch_fp8_few(const CUtensorMap& tmA, const CUtensorMap& tmB, const Fp8GemmArgs& a,
                           const Fp8FewPlan& plan, unsigned int* status, cudaStream_t stream);

// ---- the same on tiles of 128 rows by 256 columns, with square scales (fp8_wide.cu).
// tmA: boxes of kFp8WideRows rows; tmB: boxes of kFp8WideCols.  K > 0.
// Whether a product runs there.
bool fp8_takes_wide(const Fp8GemmArgs& a, const LayerDevice& dev);
constexpr int kFp8WideRows = 128, kFp8WideCols = 256;
cudaError_t launch_fp8_wide(const CUtensorMap& tmA, const CUtensorMap& tmB, const Fp8GemmArgs& a,
                            const LayerDevice& dev, cudaStream_t stream);
// cudaErrorInvalidConfiguration unless `kernel` is launched with at least `most`
// registers a block, which its roles' shares (setmaxnreg) are drawn from: a larger
// share would be waited for for ever.  `done` as in allow_shared.
template <typename... P>
cudaError_t check_registers(void (*kernel)(P...), int most, int threads,
                            std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess && fa.numRegs * threads < most) e = cudaErrorInvalidConfiguration;
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

// ---- routing (route.cu)
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxChosen = 32;
constexpr int kRouteMaxGroups = 32;
constexpr int kRouteChunk = 128;  // tokens of a block: their count for an expert is a byte
__host__ __device__ inline int route_count_stride(int E) { return (E + 3) & ~3; }
struct RouteArgs {
  int T = 0, E = 0, k = 0;
  const void* logits = nullptr;
  int64_t ld = 0;
  bool bf16 = false;
  bool sigmoid = false;
  const float* bias = nullptr;
  int groups = 1, kept = 1, group_top = 1;
  bool renorm = false;
  float scale = 1.0f;
  int* index = nullptr;
  float* weight = nullptr;
  int* slot = nullptr;
  int* source = nullptr;
  int* offsets = nullptr;
  uint8_t* counts = nullptr;  // chunks x route_count_stride(E), with more than one chunk
  // gradient
  const int* chosen = nullptr;
  const float* d_weight = nullptr;
  void* d_logits = nullptr;
  int64_t ld_d = 0;
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_route_bwd(const RouteArgs& a, cudaStream_t stream);

// ---- combining (combine.cu)
constexpr int kCombineMaxChosen = 32;
struct CombineArgs {
  int T = 0, D = 0, k = 0, R = 0;
  const void* rows = nullptr;  // R x D
  int64_t ld_rows = 0;
  bool rows_bf16 = false;
  const int* slot = nullptr;   // T x k
  const float* weight = nullptr;
  const void* x = nullptr;     // T x D, or null
  int64_t ldx = 0;
  bool x_bf16 = false;
  void* out = nullptr;         // forward: T x D; gradient: the gradient of it
  int64_t ld_out = 0;
  bool out_bf16 = false;
  void* d_rows = nullptr;      // type of rows
  int64_t ld_d_rows = 0;
  float* d_weight = nullptr;
};
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream);
cudaError_t launch_combine_bwd(const CombineArgs& a, cudaStream_t stream);

}  // namespace g07
