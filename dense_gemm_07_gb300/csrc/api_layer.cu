// api_layer.cu -- the C ABI of the operators around the GEMM in a transformer
// layer (include/gemm07.h): argument checks, scratch and launches.
#include <cuda_runtime.h>

#include "../../include/gemm07.h"
#include "kernels.h"
#include "layer.h"

namespace g07 {
namespace {

constexpr int64_t kMaxSize = 0x7FFFFFFF - 255;  // sizes round up to whole tiles in 32 bits

bool size_ok(int64_t v) { return v >= 0 && v <= kMaxSize; }
// A rows x cols matrix with row stride ld, spanning at most 2^60 elements.
bool matrix_ok(int64_t rows, int64_t cols, int64_t ld) {
  if (ld < (cols > 1 ? cols : 1)) return false;
  return rows == 0 || ld <= (int64_t(1) << 60) / rows;
}
bool type_ok(int32_t t) { return t == GEMM_TYPE_F32 || t == GEMM_TYPE_BF16; }
bool act_ok(int32_t a) {
  return a == GEMM_ACT_NONE || a == GEMM_ACT_RELU || a == GEMM_ACT_GELU;
}
bool group_ok(int32_t g) { return g == 32 || g == 64 || g == 128; }
bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t w4_packed_bytes(int64_t K, int64_t N) {
  return (K + kW4TileK - 1) / kW4TileK * ((N + kW4TileN - 1) / kW4TileN) * kW4TileBytes;
}

bool w4_ok(int64_t K, int64_t N, const gemm_w4_t* W) {
  if (W == nullptr || !group_ok(W->group)) return false;
  const int64_t G = (K + W->group - 1) / W->group;
  if (!matrix_ok(G, N, W->ld_scales)) return false;
  if (W->zeros != nullptr && !matrix_ok(G, N, W->ld_zeros)) return false;
  if (K == 0 || N == 0) return true;
  return W->packed != nullptr && at16(W->packed) && W->scales != nullptr;
}

const __nv_bfloat16* as_bf16(const uint16_t* p) {
  return reinterpret_cast<const __nv_bfloat16*>(p);
}
__nv_bfloat16* as_bf16(uint16_t* p) { return reinterpret_cast<__nv_bfloat16*>(p); }

// The arguments shared by gemm_norm_gate and its gradient.
bool norm_args(const gemm_norm_gate_args_t* a, NormArgs* n) {
  if (a == nullptr || !size_ok(a->T) || a->D < 1 || a->D > kNormMaxWidth) return false;
  if (!type_ok(a->x_type) || !matrix_ok(a->T, a->D, a->ldx)) return false;
  if (a->T > 0 && a->x == nullptr) return false;
  if (a->y != nullptr) {
    if (!type_ok(a->y_type) || !matrix_ok(a->T, a->D, a->ldy)) return false;
  } else if (a->T > 0 &&
             (a->w_post != nullptr || a->gate != nullptr || a->gate_mode != GEMM_GATE_NONE)) {
    return false;
  }
  if (a->gate_mode < GEMM_GATE_NONE || a->gate_mode > GEMM_GATE_FULL) return false;
  const bool no_gate_values = a->gate_mode == GEMM_GATE_NONE ||
                              (a->T == 0 && a->gate_mode != GEMM_GATE_CHANNEL);
  if (no_gate_values ? a->gate_mode == GEMM_GATE_NONE && a->gate != nullptr : a->gate == nullptr)
    return false;
  if (a->gate_mode == GEMM_GATE_FULL && !matrix_ok(a->T, a->D, a->ld_gate)) return false;
  if (!(a->eps >= 0.0f)) return false;
  n->T = static_cast<int>(a->T);
  n->D = static_cast<int>(a->D);
  n->x = a->x;
  n->ldx = a->ldx;
  n->x_bf16 = a->x_type == GEMM_TYPE_BF16;
  n->y = a->y;
  n->ldy = a->ldy;
  n->y_bf16 = a->y_type == GEMM_TYPE_BF16;
  n->w_post = a->w_post;
  n->gate = a->gate;
  n->gate_row = a->gate_mode == GEMM_GATE_FULL ? a->ld_gate : a->gate_mode == GEMM_GATE_ROW ? 1 : 0;
  n->gate_col = a->gate_mode == GEMM_GATE_CHANNEL || a->gate_mode == GEMM_GATE_FULL ? 1 : 0;
  n->w_pre = a->w_pre;
  n->alpha = a->alpha;
  n->eps = a->eps;
  return true;
}

}  // namespace
}  // namespace g07

using namespace g07;

extern "C" {

int64_t gemm_w4_packed_bytes(int64_t K, int64_t N) {
  return size_ok(K) && size_ok(N) ? w4_packed_bytes(K, N) : -1;
}

gemm_status_t gemm_w4(int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda,
                      const gemm_w4_t* W, void* C, int64_t ldc, int32_t c_type,
                      const gemm_epilogue_t* epilogue, void* stream) {
  W4Args a;
  if (!size_ok(M) || M > kW4MaxRows || !size_ok(N) || !size_ok(K) || !matrix_ok(M, K, lda) ||
      !matrix_ok(M, N, ldc) || !type_ok(c_type) || !w4_ok(K, N, W))
    return GEMM_ERR_INVALID_ARG;
  gemm_status_t s = layer_epilogue(epilogue, &a.epi);
  if (s != GEMM_OK) return s;
  if (M == 0 || N == 0) return GEMM_OK;
  if (C == nullptr || (K > 0 && A == nullptr)) return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.A = as_bf16(A);
  a.lda = lda;
  a.packed = static_cast<const uint8_t*>(W->packed);
  a.scales = as_bf16(W->scales);
  a.ld_scales = W->ld_scales;
  a.zeros = W->zeros;
  a.ld_zeros = W->ld_zeros;
  a.group = W->group;
  a.C = C;
  a.ldc = ldc;
  a.c_bf16 = c_type == GEMM_TYPE_BF16 ? 1 : 0;
  return layer_from_cuda(launch_w4(a, dev, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_w4_pack(int64_t K, int64_t N, const uint8_t* codes, int64_t ld, void* packed,
                           void* stream) {
  if (!size_ok(K) || !size_ok(N) || !matrix_ok(K, N, ld)) return GEMM_ERR_INVALID_ARG;
  if (K == 0 || N == 0) return GEMM_OK;
  if (codes == nullptr || packed == nullptr || !at16(packed)) return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  return layer_from_cuda(launch_w4_pack(static_cast<int>(K), static_cast<int>(N), codes, ld,
                                        static_cast<uint8_t*>(packed),
                                        static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_w4_quantize(int64_t K, int64_t N, int32_t group, const void* B, int64_t ldb,
                               int32_t b_type, void* packed, uint16_t* scales, int64_t ld_scales,
                               uint8_t* zeros, int64_t ld_zeros, void* stream) {
  const gemm_w4_t w = {packed, scales, ld_scales, zeros, ld_zeros, group};
  if (!size_ok(K) || !size_ok(N) || !type_ok(b_type) || !matrix_ok(K, N, ldb) || !w4_ok(K, N, &w))
    return GEMM_ERR_INVALID_ARG;
  if (K == 0 || N == 0) return GEMM_OK;
  if (B == nullptr) return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  return layer_from_cuda(launch_w4_quantize(
      static_cast<int>(K), static_cast<int>(N), group, B, ldb, b_type == GEMM_TYPE_BF16,
      static_cast<uint8_t*>(packed), as_bf16(scales), ld_scales, zeros, ld_zeros,
      static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_w4_unpack(int64_t K, int64_t N, const gemm_w4_t* W, uint16_t* B, int64_t ldb,
                             void* stream) {
  if (!size_ok(K) || !size_ok(N) || !matrix_ok(K, N, ldb) || !w4_ok(K, N, W))
    return GEMM_ERR_INVALID_ARG;
  if (K == 0 || N == 0) return GEMM_OK;
  if (B == nullptr) return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  return layer_from_cuda(launch_w4_unpack(
      static_cast<int>(K), static_cast<int>(N), W->group, static_cast<const uint8_t*>(W->packed),
      as_bf16(W->scales), W->ld_scales, W->zeros, W->ld_zeros, as_bf16(B), ldb,
      static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_norm_gate(const gemm_norm_gate_args_t* args, void* x_out, int64_t ld_x_out,
                             uint16_t* h, int64_t ldh, void* stream) {
  NormArgs n;
  if (!norm_args(args, &n)) return GEMM_ERR_INVALID_ARG;
  if (x_out != nullptr && !matrix_ok(n.T, n.D, ld_x_out)) return GEMM_ERR_INVALID_ARG;
  if (n.T > 0 && (h == nullptr) != (n.w_pre == nullptr)) return GEMM_ERR_INVALID_ARG;
  if (h != nullptr && !matrix_ok(n.T, n.D, ldh)) return GEMM_ERR_INVALID_ARG;
  if (n.T == 0) return GEMM_OK;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  n.x_out = x_out;
  n.ld_x_out = ld_x_out;
  n.h = as_bf16(h);
  n.ldh = ldh;
  return layer_from_cuda(launch_norm_gate(n, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_norm_gate_bwd(const gemm_norm_gate_args_t* args,
                                 const gemm_norm_gate_grads_t* grads, void* stream) {
  NormArgs n;
  if (!norm_args(args, &n) || grads == nullptr) return GEMM_ERR_INVALID_ARG;
  const gemm_norm_gate_grads_t& g = *grads;
  if (n.T > 0 && ((g.dh == nullptr) != (n.w_pre == nullptr) || g.dx == nullptr ||
                  (g.dy == nullptr) != (n.y == nullptr)))
    return GEMM_ERR_INVALID_ARG;
  if ((g.dgate == nullptr) != (n.gate == nullptr) ||
      (g.dw_post == nullptr) != (n.w_post == nullptr) ||
      (g.dw_pre == nullptr) != (n.w_pre == nullptr))
    return GEMM_ERR_INVALID_ARG;
  if ((g.d_x_out != nullptr && !matrix_ok(n.T, n.D, g.ld_d_x_out)) ||
      (g.dh != nullptr && (!type_ok(g.dh_type) || !matrix_ok(n.T, n.D, g.ld_dh))) ||
      !matrix_ok(n.T, n.D, g.ld_dx) || (g.dy != nullptr && !matrix_ok(n.T, n.D, g.ld_dy)))
    return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  n.d_x_out = g.d_x_out;
  n.ld_d_x_out = g.ld_d_x_out;
  n.dh = g.dh;
  n.ld_dh = g.ld_dh;
  n.dh_bf16 = g.dh_type == GEMM_TYPE_BF16;
  n.dx = g.dx;
  n.ld_dx = g.ld_dx;
  n.dy = as_bf16(g.dy);
  n.ld_dy = g.ld_dy;
  n.dgate = g.dgate;
  n.dw_post = g.dw_post;
  n.dw_pre = g.dw_pre;
  const bool gate_sums = n.gate != nullptr && n.gate_col != 0 && n.gate_row == 0;
  const bool sums = n.w_post != nullptr || n.w_pre != nullptr || gate_sums;
  LayerScratch ws;
  NormBwdPlan plan;
  if (n.T > 0) {
    s = layer_from_cuda(norm_gate_bwd_plan(n, dev, &plan));
    if (s != GEMM_OK) return s;
  }
  const int slots = plan.slots;
  ColumnSums c;
  if (sums) {
    s = layer_scratch(st, static_cast<int64_t>(slots) * 3 * n.D * 4, &ws);
    if (s != GEMM_OK) return s;
    c.partial = static_cast<const float*>(ws.ptr);
    c.ld = 3 * static_cast<int64_t>(n.D);
    c.slots = slots;
    c.n = n.D;
    c.count = 3;
    c.out[0] = n.dw_post;
    c.out[1] = n.dw_pre;
    c.out[2] = gate_sums ? n.dgate : nullptr;
  }
  if (n.T > 0)
    s = layer_from_cuda(launch_norm_gate_bwd(n, plan, static_cast<float*>(ws.ptr), st));
  if (s == GEMM_OK && sums) s = layer_from_cuda(launch_column_sums(c, st));
  layer_scratch_done(ws, st);
  return s;
}

int64_t gemm_ckpt8_bytes(int64_t T, int64_t N) {
  if (!size_ok(T) || !size_ok(N)) return -1;
  return (T + kCkptRun - 1) / kCkptRun * kCkptRun * N;
}

gemm_status_t gemm_ckpt8_pack(int64_t T, int64_t N, const void* X, int64_t ldx, int32_t x_type,
                              void* q, uint8_t* scales, int32_t activation, uint16_t* act_out,
                              int64_t ld_act, void* stream) {
  if (!size_ok(T) || !size_ok(N) || !matrix_ok(T, N, ldx) || !type_ok(x_type) ||
      !act_ok(activation) || (act_out != nullptr && !matrix_ok(T, N, ld_act)))
    return GEMM_ERR_INVALID_ARG;
  if (T == 0 || N == 0) return GEMM_OK;
  if (X == nullptr || q == nullptr || !at16(q) || scales == nullptr) return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  CkptArgs a;
  a.T = static_cast<int>(T);
  a.N = static_cast<int>(N);
  a.x = X;
  a.ldx = ldx;
  a.x_bf16 = x_type == GEMM_TYPE_BF16;
  a.q = static_cast<uint8_t*>(q);
  a.scales = scales;
  a.act = activation;
  a.out = as_bf16(act_out);
  a.ld_out = ld_act;
  return layer_from_cuda(launch_ckpt8_pack(a, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_ckpt8_unpack(int64_t T, int64_t N, const void* q, const uint8_t* scales,
                                void* out, int64_t ld, int32_t out_type, void* stream) {
  if (!size_ok(T) || !size_ok(N) || !matrix_ok(T, N, ld) || !type_ok(out_type))
    return GEMM_ERR_INVALID_ARG;
  if (T == 0 || N == 0) return GEMM_OK;
  if (out == nullptr || q == nullptr || !at16(q) || scales == nullptr)
    return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  const gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  return layer_from_cuda(launch_ckpt8_unpack(
      static_cast<int>(T), static_cast<int>(N), static_cast<const uint8_t*>(q), scales, out, ld,
      out_type == GEMM_TYPE_BF16, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_ckpt8_act_grad(int64_t T, int64_t N, const void* G, int64_t ldg,
                                  int32_t g_type, const void* q, const uint8_t* scales,
                                  int32_t activation, uint16_t* dZ, int64_t ld_dz, float* dbias,
                                  void* stream) {
  if (!size_ok(T) || !size_ok(N) || !matrix_ok(T, N, ldg) || !type_ok(g_type) ||
      !act_ok(activation) || !matrix_ok(T, N, ld_dz))
    return GEMM_ERR_INVALID_ARG;
  if (N == 0 || (T == 0 && dbias == nullptr)) return GEMM_OK;
  if (T > 0 && (G == nullptr || q == nullptr || !at16(q) || scales == nullptr || dZ == nullptr))
    return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  CkptArgs a;
  a.T = static_cast<int>(T);
  a.N = static_cast<int>(N);
  a.x = G;
  a.ldx = ldg;
  a.x_bf16 = g_type == GEMM_TYPE_BF16;
  a.q = const_cast<uint8_t*>(static_cast<const uint8_t*>(q));
  a.scales = const_cast<uint8_t*>(scales);
  a.act = activation;
  a.out = as_bf16(dZ);
  a.ld_out = ld_dz;
  if (T == 0) {  // the empty sum
    return layer_from_cuda(launch_zero_fill_f32(dbias, N, 1, a.N, epi_identity(), st));
  }
  int slots = ckpt8_act_grad_slots(a.T, a.N, dev);
  LayerScratch ws;
  ColumnTotals sums;
  if (dbias != nullptr) {
    sums.out = dbias;
    // (very wide rows have more column blocks than counters: one block a column
    // block walks all rows then)
    if (ckpt8_act_grad_counters(a.N) * 4 > kLayerCounterBytes) slots = 1;
    if (slots > 1) {
      s = layer_counted_scratch(st, static_cast<int64_t>(slots) * N * 4, &ws);
      if (s != GEMM_OK) return s;
      sums.counters = static_cast<unsigned int*>(ws.ptr);
      sums.partial =
          reinterpret_cast<float*>(static_cast<uint8_t*>(ws.ptr) + kLayerCounterBytes);
    }
  }
  s = layer_from_cuda(launch_ckpt8_act_grad(a, sums, slots, st));
  layer_scratch_done(ws, st);
  return s;
}

gemm_status_t gemm_ckpt8_wgrad(int64_t T, int64_t K, int64_t N, const void* q,
                               const uint8_t* scales, const uint16_t* dY, int64_t ld_dy,
                               float* dW, int64_t ldw, float beta, void* stream) {
  if (!size_ok(T) || !size_ok(K) || !size_ok(N) || !matrix_ok(T, N, ld_dy) ||
      !matrix_ok(K, N, ldw))
    return GEMM_ERR_INVALID_ARG;
  if (K == 0 || N == 0) return GEMM_OK;
  if (dW == nullptr || (T > 0 && (q == nullptr || !at16(q) || scales == nullptr || dY == nullptr)))
    return GEMM_ERR_INVALID_ARG;
  LayerDevice dev;
  gemm_status_t s = layer_device(&dev);
  if (s != GEMM_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    EpiParams epi = epi_identity();
    epi.beta = beta;
    return layer_from_cuda(launch_zero_fill_f32(dW, ldw, static_cast<int>(K),
                                                static_cast<int>(N), epi, st));
  }
  return layer_ckpt8_wgrad(T, K, N, static_cast<const uint8_t*>(q), scales, dY, ld_dy, dW, ldw,
                           beta, st);
}

}  // extern "C"
