// api_experts.cu -- the C ABI of the 8-bit floating-point products and of a layer of
// experts (include/gemm07.h): argument checks and launches.
#include <cstring>

#include <cuda_runtime.h>

#include "../../include/gemm07.h"
#include "experts.h"

namespace g07 {
namespace {

constexpr int64_t kMaxSize = int64_t(1) << 30;  // indices rounded up to whole tiles fit 32 bits

bool size_ok(int64_t v) { return v >= 0 && v <= kMaxSize; }
// A rows x cols matrix with row stride ld, spanning at most 2^60 elements.
bool matrix_ok(int64_t rows, int64_t cols, int64_t ld) {
  if (ld < (cols > 1 ? cols : 1)) return false;
  return rows == 0 || ld <= (int64_t(1) << 60) / rows;
}
bool type_ok(int32_t t) { return t == GEMM_TYPE_F32 || t == GEMM_TYPE_BF16; }
bool flag_ok(int32_t v) { return v == 0 || v == 1; }
bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

// The copy engine's strides are below 2^40 bytes.
bool codes_ok(int64_t rows, int64_t K, int64_t ld) {
  return matrix_ok(rows, K, ld) && ld % 16 == 0 && ld < (int64_t(1) << 40);
}
bool scales_ok(int64_t rows, int64_t K, int64_t ld, bool square) {
  return square ? matrix_ok(blocks(rows), blocks(K), ld) : matrix_ok(blocks(K), rows, ld);
}
bool fp8_ok(int64_t rows, int64_t K, const gemm_fp8_t* m) {
  if (m == nullptr || !flag_ok(m->square) || !codes_ok(rows, K, m->ld) ||
      !scales_ok(rows, K, m->ld_scales, m->square != 0))
    return false;
  return rows == 0 || K == 0 || (m->codes != nullptr && at16(m->codes) && m->scales != nullptr);
}

// gemm_fp8 and, with E > 0, gemm_fp8_experts.
gemm_status_t product(int64_t E, int64_t M, int64_t N, int64_t K, const gemm_fp8_t* A,
                      const gemm_fp8_t* B, const int32_t* offsets, void* C, int64_t ldc,
                      int32_t c_type, const gemm_epilogue_t* epilogue, cudaStream_t stream) {
  Fp8GemmArgs a;
  const int64_t b_rows = E > 0 ? E * N : N;
  if (!size_ok(M) || !size_ok(N) || !size_ok(K) || !size_ok(b_rows) || !matrix_ok(M, N, ldc) ||
      !type_ok(c_type) || !fp8_ok(M, K, A) || A->square)
    return GEMM_ERR_INVALID_ARG;
  if (E > 0) {
    // (every expert's scales start on a row of their own)
    if (B == nullptr || B->square != 1 || !codes_ok(b_rows, K, B->ld) ||
        !matrix_ok(E * blocks(N), blocks(K), B->ld_scales))
      return GEMM_ERR_INVALID_ARG;
    if (b_rows > 0 && K > 0 && (B->codes == nullptr || !at16(B->codes) || B->scales == nullptr))
      return GEMM_ERR_INVALID_ARG;
  } else if (!fp8_ok(N, K, B)) {
    return GEMM_ERR_INVALID_ARG;
  }
  gemm_status_t s = layer_epilogue(epilogue, &a.epi);
  if (s != GEMM_OK) return s;
  if (M == 0 || N == 0) return GEMM_OK;
  if (C == nullptr || (E > 0 && offsets == nullptr)) return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.E = static_cast<int>(E);
  a.offsets = offsets;
  a.sa = A->scales;
  a.ld_sa = A->ld_scales;
  a.sb = B->scales;
  a.ld_sb = B->ld_scales;
  a.b_square = B->square != 0;
  a.C = C;
  a.ldc = ldc;
  a.c_bf16 = c_type == GEMM_TYPE_BF16 ? 1 : 0;
  CUtensorMap tmA, tmB;
  if (fp8_takes_wide(a, dev)) {
    s = layer_map_bytes(&tmA, A->codes, K, M, A->ld, kFp8WideRows);
    if (s == GEMM_OK) s = layer_map_bytes(&tmB, B->codes, K, b_rows, B->ld, kFp8WideCols);
    if (s != GEMM_OK) return s;
    return layer_from_cuda(launch_fp8_wide(tmA, tmB, a, dev, stream));
  }
  Fp8FewPlan plan;
  s = layer_from_cuda(fp8_few_plan(a, dev, &plan));
  if (s != GEMM_OK) return s;
  std::memset(&tmA, 0, sizeof(tmA));
  std::memset(&tmB, 0, sizeof(tmB));
  if (K > 0) {
    s = layer_map_bytes(&tmA, A->codes, K, M, A->ld, static_cast<uint32_t>(plan.cols));
    if (s == GEMM_OK) s = layer_map_bytes(&tmB, B->codes, K, b_rows, B->ld, 128);
    if (s != GEMM_OK) return s;
  }
  return layer_from_cuda(launch_fp8_few(tmA, tmB, a, plan, dev.status, stream));
}

bool route_ok(const gemm_route_args_t* a, RouteArgs* r) {
  if (a == nullptr || !size_ok(a->T) || a->E < 1 || a->E > kRouteMaxExperts || a->k < 1 ||
      a->k > kRouteMaxChosen || a->T * a->k > 0x7FFFFFFF || !type_ok(a->type) ||
      !matrix_ok(a->T, a->E, a->ld) || (a->T > 0 && a->logits == nullptr))
    return false;
  if (a->score != GEMM_ROUTE_SOFTMAX && a->score != GEMM_ROUTE_SIGMOID) return false;
  if (!flag_ok(a->renormalize)) return false;
  r->T = static_cast<int>(a->T);
  r->E = static_cast<int>(a->E);
  r->k = static_cast<int>(a->k);
  r->logits = a->logits;
  r->ld = a->ld;
  r->bf16 = a->type == GEMM_TYPE_BF16;
  r->sigmoid = a->score == GEMM_ROUTE_SIGMOID;
  r->bias = a->bias;
  r->groups = a->groups;
  r->kept = a->groups_kept;
  r->group_top = a->group_top;
  r->renorm = a->renormalize != 0;
  r->scale = a->scale;
  return true;
}

bool combine_ok(const gemm_combine_args_t* a, CombineArgs* c) {
  if (a == nullptr || !size_ok(a->T) || !size_ok(a->D) || !size_ok(a->R) || a->k < 0 ||
      a->k > kCombineMaxChosen || a->T * a->k > 0x7FFFFFFF || !type_ok(a->rows_type) ||
      !matrix_ok(a->R, a->D, a->ld_rows))
    return false;
  if (a->x != nullptr && (!type_ok(a->x_type) || !matrix_ok(a->T, a->D, a->ldx))) return false;
  if (a->T > 0 && a->k > 0 && (a->slot == nullptr || a->weight == nullptr)) return false;
  if (a->R > 0 && a->D > 0 && a->rows == nullptr) return false;
  c->T = static_cast<int>(a->T);
  c->D = static_cast<int>(a->D);
  c->k = static_cast<int>(a->k);
  c->R = static_cast<int>(a->R);
  c->rows = a->rows;
  c->ld_rows = a->ld_rows;
  c->rows_bf16 = a->rows_type == GEMM_TYPE_BF16;
  c->slot = a->slot;
  c->weight = a->weight;
  c->x = a->x;
  c->ldx = a->ldx;
  c->x_bf16 = a->x_type == GEMM_TYPE_BF16;
  return true;
}

}  // namespace
}  // namespace g07

using namespace g07;

extern "C" {

gemm_status_t gemm_fp8_quantize(const gemm_fp8_quantize_args_t* args, void* stream) {
  if (args == nullptr) return GEMM_ERR_INVALID_ARG;
  const gemm_fp8_quantize_args_t& q = *args;
  if (!size_ok(q.T) || !size_ok(q.C) || !type_ok(q.x_type) || !matrix_ok(q.T, q.C, q.ldx) ||
      !flag_ok(q.square) || !flag_ok(q.transpose) || q.batch < 0 || q.batch > 65535)
    return GEMM_ERR_INVALID_ARG;
  if (q.index != nullptr && (q.square || q.transpose || !size_ok(q.rows)))
    return GEMM_ERR_INVALID_ARG;
  const int64_t rows = q.index != nullptr ? q.rows : q.transpose ? q.C : q.T;
  const int64_t cols = q.transpose ? q.T : q.C;
  if (!codes_ok(rows, cols, q.ld) || !scales_ok(rows, cols, q.ld_scales, q.square != 0))
    return GEMM_ERR_INVALID_ARG;
  const int64_t far = int64_t(1) << 60;
  if (q.batch != 1 &&
      (!q.square || q.x_step < 0 || q.codes_step < 0 || q.scales_step < 0 ||
       (q.batch > 0 && (q.x_step > far / q.batch || q.codes_step > far / q.batch ||
                        q.scales_step > far / q.batch || q.codes_step % 16 != 0))))
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0 || q.batch == 0) return GEMM_OK;
  if ((q.T > 0 && q.x == nullptr) || q.codes == nullptr || !at16(q.codes) || q.scales == nullptr)
    return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  Fp8QuantArgs a;
  a.T = static_cast<int>(q.T);
  a.C = static_cast<int>(q.C);
  a.batch = static_cast<int>(q.batch);
  a.x = q.x;
  a.ldx = q.ldx;
  a.x_step = q.batch > 1 ? q.x_step : 0;
  a.x_bf16 = q.x_type == GEMM_TYPE_BF16;
  a.index = q.index;
  a.rows = static_cast<int>(rows);
  a.codes = static_cast<uint8_t*>(q.codes);
  a.ld = q.ld;
  a.codes_step = q.batch > 1 ? q.codes_step : 0;
  a.scales = q.scales;
  a.ld_scales = q.ld_scales;
  a.scales_step = q.batch > 1 ? q.scales_step : 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return layer_from_cuda(q.square      ? launch_fp8_quantize_square(a, q.transpose != 0, st)
                         : q.transpose ? launch_fp8_quantize_transposed(a, st)
                                       : launch_fp8_quantize_rows(a, st));
}

gemm_status_t gemm_fp8(int64_t M, int64_t N, int64_t K, const gemm_fp8_t* A, const gemm_fp8_t* B,
                       void* C, int64_t ldc, int32_t c_type, const gemm_epilogue_t* epilogue,
                       void* stream) {
  return product(0, M, N, K, A, B, nullptr, C, ldc, c_type, epilogue,
                 static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_fp8_experts(int64_t E, int64_t M, int64_t N, int64_t K, const gemm_fp8_t* A,
                               const gemm_fp8_t* B, const int32_t* offsets, void* C, int64_t ldc,
                               int32_t c_type, const gemm_epilogue_t* epilogue, void* stream) {
  if (E < 1 || E > kRouteMaxExperts) return GEMM_ERR_INVALID_ARG;
  return product(E, M, N, K, A, B, offsets, C, ldc, c_type, epilogue,
                 static_cast<cudaStream_t>(stream));
}

int64_t gemm_route_workspace_bytes(int64_t T, int64_t E) {
  if (!size_ok(T) || E < 1 || E > kRouteMaxExperts) return -1;
  const int64_t chunks = (T + kRouteChunk - 1) / kRouteChunk;
  return chunks > 1 ? chunks * route_count_stride(static_cast<int>(E)) : 0;
}

gemm_status_t gemm_route(const gemm_route_args_t* args, int32_t* index, float* weight,
                         int32_t* slot, int32_t* source, int32_t* offsets, void* workspace,
                         void* stream) {
  RouteArgs a;
  if (!route_ok(args, &a) || args->groups < 1 || args->groups > kRouteMaxGroups ||
      args->E % args->groups != 0 || args->groups_kept < 1 || args->groups_kept > args->groups ||
      (args->group_top != 1 && args->group_top != 2) ||
      args->k > args->groups_kept * (args->E / args->groups))
    return GEMM_ERR_INVALID_ARG;
  if (offsets == nullptr ||
      (a.T > 0 && (index == nullptr || weight == nullptr || slot == nullptr || source == nullptr)))
    return GEMM_ERR_INVALID_ARG;
  if (gemm_route_workspace_bytes(a.T, a.E) > 0 &&
      (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 3u) != 0))
    return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  a.index = index;
  a.weight = weight;
  a.slot = slot;
  a.source = source;
  a.offsets = offsets;
  a.counts = static_cast<uint8_t*>(workspace);
  return layer_from_cuda(launch_route(a, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_route_bwd(const gemm_route_args_t* args, const int32_t* index,
                             const float* d_weight, void* d_logits, int64_t ld_d, void* stream) {
  RouteArgs a;
  if (!route_ok(args, &a) || !matrix_ok(a.T, a.E, ld_d)) return GEMM_ERR_INVALID_ARG;
  if (a.T == 0) return GEMM_OK;
  if (index == nullptr || d_weight == nullptr || d_logits == nullptr) return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  a.chosen = index;
  a.d_weight = d_weight;
  a.d_logits = d_logits;
  a.ld_d = ld_d;
  return layer_from_cuda(launch_route_bwd(a, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_combine(const gemm_combine_args_t* args, void* out, int64_t ld_out,
                           int32_t out_type, void* stream) {
  CombineArgs a;
  if (!combine_ok(args, &a) || !type_ok(out_type) || !matrix_ok(a.T, a.D, ld_out))
    return GEMM_ERR_INVALID_ARG;
  if (a.T == 0 || a.D == 0) return GEMM_OK;
  if (out == nullptr) return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  a.out = out;
  a.ld_out = ld_out;
  a.out_bf16 = out_type == GEMM_TYPE_BF16;
  return layer_from_cuda(launch_combine(a, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_combine_bwd(const gemm_combine_args_t* args, const void* d_out,
                               int64_t ld_d_out, int32_t d_out_type, void* d_rows,
                               int64_t ld_d_rows, float* d_weight, void* stream) {
  CombineArgs a;
  if (!combine_ok(args, &a) || !type_ok(d_out_type) || !matrix_ok(a.T, a.D, ld_d_out) ||
      !matrix_ok(a.R, a.D, ld_d_rows))
    return GEMM_ERR_INVALID_ARG;
  if (a.T == 0 || a.k == 0) return GEMM_OK;
  if (d_weight == nullptr || (a.D > 0 && d_out == nullptr) ||
      (a.R > 0 && a.D > 0 && d_rows == nullptr))
    return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  a.out = const_cast<void*>(d_out);
  a.ld_out = ld_d_out;
  a.out_bf16 = d_out_type == GEMM_TYPE_BF16;
  a.d_rows = d_rows;
  a.ld_d_rows = ld_d_rows;
  a.d_weight = d_weight;
  return layer_from_cuda(launch_combine_bwd(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
