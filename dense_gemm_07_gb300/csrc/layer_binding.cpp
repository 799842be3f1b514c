// layer_binding.cpp -- the Python binding of the layer operators (and of the 8-bit
// products, routing and combining of a layer of experts): checks torch
// tensors and passes their sizes, addresses and strides to the C entry points
// of include/gemm07.h.  Compiled code, because at the sizes of a decode step a
// call's own time is the operator's: marshalling a call in Python took 7 to 18
// us of a 12 to 23 us call (gemm_w4 at 1 x 4096 x 4096, gemm_norm_gate at
// 1 x 4096).
//
// A refused argument raises ValueError or TypeError, a status of the library
// GemmError, as in the rest of the package.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/utils/pybind.h>

#include <initializer_list>
#include <limits>
#include <optional>
#include <string>
#include <tuple>

#include "../../include/gemm07.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;

std::string text(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

std::string text(int64_t v) { return std::to_string(v); }

[[noreturn]] void bad_value(const std::string& what) { throw py::value_error(what); }
[[noreturn]] void bad_type(const std::string& what) { throw py::type_error(what); }

void check_status(gemm_status_t s, const char* where) {
  if (s == GEMM_OK) return;
  py::object cls = py::module_::import("dense_gemm_07_gb300._errors").attr("GemmError");
  py::object e = cls(static_cast<int>(s), where);
  PyErr_SetObject(cls.ptr(), e.ptr());
  throw py::error_already_set();
}

at::Device cuda_device(const Tensor& t, const char* name) {
  if (!t.is_cuda()) bad_value(std::string(name) + " must be a CUDA tensor");
  return t.device();
}

// Row stride of a 2-D tensor, after its checks.
int64_t matrix(const Tensor& t, const char* name, std::initializer_list<at::ScalarType> types,
               at::Device device, int64_t rows = -1, int64_t cols = -1) {
  const std::string n = name;
  if (t.dim() != 2) bad_value(n + " must be 2-D");
  bool known = false;
  for (at::ScalarType s : types) known |= t.scalar_type() == s;
  if (!known) {
    std::string list;
    for (at::ScalarType s : types) list += (list.empty() ? "" : " or ") + text(s);
    bad_type(n + " must be " + list);
  }
  if (t.device() != device) bad_value(n + " must be on " + device.str());
  const int64_t r = t.size(0), c = t.size(1);
  if ((rows >= 0 && r != rows) || (cols >= 0 && c != cols))
    bad_value(n + " must be " + text(rows >= 0 ? rows : r) + " x " + text(cols >= 0 ? cols : c) +
              ", not " + text(r) + " x " + text(c));
  const int64_t rs = t.stride(0), cs = t.stride(1);
  if (c > 1 && cs != 1) bad_value(n + ": rows must be contiguous (stride(1) == 1)");
  if (r > 1 && c > 0 && rs < c) bad_value(n + ": rows must not overlap (stride(0) >= columns)");
  const int64_t ld = r > 1 ? rs : c;
  return ld > c ? ld : c > 1 ? c : 1;
}

void vector(const Tensor& t, const char* name, at::Device device, int64_t n) {
  if (t.dim() != 1 || t.size(0) != n || t.scalar_type() != at::kFloat || t.device() != device ||
      (n > 1 && t.stride(0) != 1))
    bad_value(std::string(name) + " must be a contiguous torch.float32 vector of " + text(n) +
              " elements on " + device.str());
}

void bytes16(const Tensor& t, const char* name, int64_t n, at::Device device) {
  if (t.scalar_type() != at::kByte || t.device() != device || !t.is_contiguous() || t.numel() != n)
    bad_value(std::string(name) + " must be " + text(n) + " contiguous uint8 elements on " +
              device.str());
  if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16)
    bad_value(std::string(name) + " must start on a 16-byte boundary");
}

template <typename T = void>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.numel() ? t.data_ptr() : nullptr);
}
template <typename T = void>
T* ptr(const Maybe& t) {
  return t ? ptr<T>(*t) : nullptr;
}

int32_t type_of(const Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? GEMM_TYPE_BF16 : GEMM_TYPE_F32;
}

// Runs work of torch's own on the stream that the call runs on.
template <typename F>
void on_stream(at::Device device, const std::optional<int64_t>& stream, F work) {
  c10::cuda::OptionalCUDAStreamGuard guard;
  if (stream)
    guard.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(*stream),
                                                        device.index()));
  work();
}

// New tensors come straight from the allocator, past torch's dispatcher, which takes most
// of the time of at::empty.  Where torch does more than to allocate, it is still done:
// dispatch modes see the call, and in deterministic mode memory that nothing may be
// written to is filled, on the stream of the call (work there could run before a fill on
// the current stream, which is at::empty's: with both, modes do not see the call).
bool fills() {
  const at::Context& torch = at::globalContext();
  return torch.deterministicAlgorithms() && torch.deterministicFillUninitializedMemory();
}
template <typename Seen, typename Plain>
Tensor fresh(at::Device device, const std::optional<int64_t>& stream, Seen seen, Plain plain) {
  const bool fill = fills();
  if (!(fill && stream) && c10::impl::TorchDispatchModeTLS::any_modes_set()) return seen();
  Tensor t = plain();
  if (fill && t.numel() > 0)
    on_stream(device, stream, [&] {  // (as torch does: NaN, or the largest whole number)
      if (t.is_floating_point())
        t.fill_(std::numeric_limits<double>::quiet_NaN());
      else
        t.fill_(255);  // bytes
    });
  return t;
}

Tensor empty(at::IntArrayRef size, at::ScalarType type, at::Device device,
             const std::optional<int64_t>& stream) {
  return fresh(
      device, stream,
      [&] { return at::empty(size, at::TensorOptions().dtype(type).device(device)); },
      [&] { return Tensor(at::detail::empty_cuda(size, type, device, std::nullopt)); });
}

Tensor empty_strided(at::IntArrayRef size, at::IntArrayRef strides, at::ScalarType type,
                     at::Device device, const std::optional<int64_t>& stream) {
  return fresh(
      device, stream,
      [&] {
        return at::empty_strided(size, strides, at::TensorOptions().dtype(type).device(device));
      },
      [&] { return Tensor(at::detail::empty_strided_cuda(size, strides, type, device)); });
}

// A contiguous tensor of its own over part of a block of bytes (`at` bytes in, a multiple
// of the type's size): several outputs of a call come from one allocation, which takes as
// long as each of them would.
Tensor part(const Tensor& block, at::ScalarType type, at::IntArrayRef size, int64_t at) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(block.storage()), block.key_set(), c10::scalarTypeToTypeMeta(type));
  c10::TensorImpl* impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(type)));
  impl->set_sizes_contiguous(size);
  return t;
}

// `out` after its checks, or a new rows x cols tensor; its row stride in *ld.
Tensor output(const Maybe& out, const char* name, int64_t rows, int64_t cols, at::ScalarType type,
              at::Device device, int64_t* ld, const std::optional<int64_t>& stream) {
  if (out) {
    *ld = matrix(*out, name, {type}, device, rows, cols);
    return *out;
  }
  *ld = cols > 1 ? cols : 1;
  return empty({rows, cols}, type, device, stream);
}

int32_t activation(const std::string& name) {
  if (name == "none") return GEMM_ACT_NONE;
  if (name == "relu") return GEMM_ACT_RELU;
  if (name == "gelu") return GEMM_ACT_GELU;
  bad_value("activation must be one of ['gelu', 'none', 'relu']");
}

// Runs a C entry point with the device current, on the stream given or the
// current one.
template <typename F>
void run(const char* where, at::Device device, const std::optional<int64_t>& stream, F call) {
  const c10::DeviceIndex index = device.index();
  void* s = stream ? reinterpret_cast<void*>(*stream)
                   : static_cast<void*>(c10::cuda::getCurrentCUDAStream(index).stream());
  const c10::DeviceIndex before = c10::cuda::current_device();
  if (before != index) c10::cuda::set_device(index);
  const gemm_status_t status = call(s);
  if (before != index) c10::cuda::set_device(before);
  check_status(status, where);
}

// ---------------------------------------------------------- 4-bit weights

int64_t packed_bytes(int64_t K, int64_t N) {
  const int64_t n = gemm_w4_packed_bytes(K, N);
  if (n < 0) bad_value("no packed matrix of " + text(K) + " x " + text(N));
  return n;
}

int64_t groups_of(int64_t K, int64_t group) {
  if (group != 32 && group != 64 && group != 128) bad_value("group must be 32, 64 or 128");
  return (K + group - 1) / group;
}

gemm_w4_t weights(const Tensor& packed, const Tensor& scales, const Maybe& zeros, int64_t group,
                  int64_t K, at::Device device, int64_t* N) {
  const int64_t G = groups_of(K, group);
  const int64_t ld = matrix(scales, "scales", {at::kBFloat16}, device, G);
  *N = scales.size(1);
  const int64_t ldz = zeros ? matrix(*zeros, "zeros", {at::kByte}, device, G, *N) : *N > 1 ? *N : 1;
  bytes16(packed, "packed", packed_bytes(K, *N), device);
  return gemm_w4_t{ptr(packed), ptr<uint16_t>(scales), ld, ptr<uint8_t>(zeros), ldz,
                   static_cast<int32_t>(group)};
}

Tensor w4(const Tensor& A, const Tensor& packed, const Tensor& scales, const Maybe& zeros,
          int64_t group, const Maybe& out_, double alpha, double beta, const Maybe& bias,
          const std::string& act, const std::optional<at::ScalarType>& out_dtype,
          const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(A, "A");
  const int64_t lda = matrix(A, "A", {at::kBFloat16}, device);
  const int64_t M = A.size(0), K = A.size(1);
  int64_t N = 0;
  const gemm_w4_t w = weights(packed, scales, zeros, group, K, device, &N);
  if (beta != 0.0 && !out_) bad_value("beta != 0 reads C: pass its prior contents as `out`");
  const at::ScalarType type = out_dtype ? *out_dtype : out_ ? out_->scalar_type() : at::kFloat;
  if (type != at::kFloat && type != at::kBFloat16)
    bad_type("out_dtype must be torch.float32 or torch.bfloat16");
  int64_t ldc = 0;
  Tensor out = output(out_, "out", M, N, type, device, &ldc, stream);
  if (bias) vector(*bias, "bias", device, N);
  const gemm_epilogue_t epi = {static_cast<float>(alpha), static_cast<float>(beta),
                               ptr<float>(bias), activation(act)};
  run("gemm_w4", device, stream, [&](void* s) {
    return gemm_w4(M, N, K, ptr<uint16_t>(A), lda, &w, ptr(out), ldc,
                   type == at::kBFloat16 ? GEMM_TYPE_BF16 : GEMM_TYPE_F32, &epi, s);
  });
  return out;
}

Tensor w4_pack(const Tensor& codes, const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(codes, "codes");
  const int64_t ld = matrix(codes, "codes", {at::kByte}, device);
  const int64_t K = codes.size(0), N = codes.size(1);
  Tensor packed = empty({packed_bytes(K, N)}, at::kByte, device, stream);
  run("gemm_w4_pack", device, stream, [&](void* s) {
    return gemm_w4_pack(K, N, ptr<uint8_t>(codes), ld, ptr(packed), s);
  });
  return packed;
}

std::tuple<Tensor, Tensor, Maybe> w4_quantize(const Tensor& B, int64_t group, bool symmetric,
                                              const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(B, "B");
  const int64_t ldb = matrix(B, "B", {at::kFloat, at::kBFloat16}, device);
  const int64_t K = B.size(0), N = B.size(1), G = groups_of(K, group);
  Tensor packed = empty({packed_bytes(K, N)}, at::kByte, device, stream);
  Tensor scales = empty({G, N}, at::kBFloat16, device, stream);
  Maybe zeros;
  if (!symmetric) zeros = empty({G, N}, at::kByte, device, stream);
  const int64_t ld = N > 1 ? N : 1;
  run("gemm_w4_quantize", device, stream, [&](void* s) {
    return gemm_w4_quantize(K, N, static_cast<int32_t>(group), ptr(B), ldb, type_of(B), ptr(packed),
                            ptr<uint16_t>(scales), ld, ptr<uint8_t>(zeros), ld, s);
  });
  return {packed, scales, zeros};
}

Tensor w4_unpack(const Tensor& packed, const Tensor& scales, const Maybe& zeros, int64_t group,
                 const std::optional<int64_t>& rows, const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(packed, "packed");
  if (scales.dim() != 2) bad_value("scales must be 2-D");
  const int64_t K = rows ? *rows : scales.size(0) * group;
  int64_t N = 0;
  const gemm_w4_t w = weights(packed, scales, zeros, group, K, device, &N);
  Tensor out = empty({K, N}, at::kBFloat16, device, stream);
  run("gemm_w4_unpack", device, stream, [&](void* s) {
    return gemm_w4_unpack(K, N, &w, ptr<uint16_t>(out), N > 1 ? N : 1, s);
  });
  return out;
}

// ------------------------------------------------- norms, gate, residual

constexpr int64_t kNormMaxWidth = 16384;

gemm_norm_gate_args_t norm_args(const Tensor& x, const Maybe& y, const Maybe& weight_post,
                                const Maybe& gate, const Maybe& weight_pre, double scale,
                                double eps, at::Device device) {
  gemm_norm_gate_args_t a = {};
  a.ldx = matrix(x, "x", {at::kFloat, at::kBFloat16}, device);
  const int64_t T = x.size(0), D = x.size(1);
  if (D < 1 || D > kNormMaxWidth)
    bad_value("rows must have 1 to " + text(kNormMaxWidth) + " elements");
  a.T = T;
  a.D = D;
  a.x = ptr(x);
  a.x_type = type_of(x);
  a.ldy = D;
  if (y) {
    a.ldy = matrix(*y, "y", {at::kFloat, at::kBFloat16}, device, T, D);
    a.y = ptr(*y);
    a.y_type = type_of(*y);
  } else if (weight_post || gate) {
    bad_value("weight_post and gate need y");
  }
  if (weight_post) vector(*weight_post, "weight_post", device, D);
  if (weight_pre) vector(*weight_pre, "weight_pre", device, D);
  a.w_post = ptr<float>(weight_post);
  a.w_pre = ptr<float>(weight_pre);
  a.ld_gate = D;
  a.gate_mode = GEMM_GATE_NONE;
  if (gate) {
    const auto size = gate->sizes();
    if (size.size() == 2 && size[0] == T && size[1] == D)
      a.gate_mode = GEMM_GATE_FULL;
    else if (size.size() == 2 && size[0] == T && size[1] == 1)
      a.gate_mode = GEMM_GATE_ROW;
    else if (size.size() == 1 && size[0] == D)
      a.gate_mode = GEMM_GATE_CHANNEL;
    else
      bad_value("gate must be D values, T x 1 or T x D");
    if (gate->scalar_type() != at::kFloat || gate->device() != device)
      bad_value("gate must be float32 on " + device.str());
    if (a.gate_mode == GEMM_GATE_FULL)
      a.ld_gate = matrix(*gate, "gate", {at::kFloat}, device);
    else if (!gate->is_contiguous())
      bad_value("a gate per channel or per row must be contiguous");
    a.gate = ptr<float>(*gate);
  }
  a.alpha = static_cast<float>(scale);
  a.eps = static_cast<float>(eps);
  return a;
}

std::tuple<Tensor, Maybe> norm_gate(const Tensor& x, const Maybe& y, const Maybe& weight_post,
                                    const Maybe& gate, const Maybe& weight_pre, double scale,
                                    double eps, const Maybe& x_out_, const Maybe& h_,
                                    const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(x, "x");
  const gemm_norm_gate_args_t a =
      norm_args(x, y, weight_post, gate, weight_pre, scale, eps, device);
  int64_t ld_o = 0, ldh = a.D;
  Tensor x_out = output(x_out_, "x_out", a.T, a.D, x.scalar_type(), device, &ld_o, stream);
  Maybe h;
  if (weight_pre)
    h = output(h_, "h", a.T, a.D, at::kBFloat16, device, &ldh, stream);
  else if (h_)
    bad_value("h needs weight_pre");
  run("gemm_norm_gate", device, stream, [&](void* s) {
    return gemm_norm_gate(&a, ptr(x_out), ld_o, ptr<uint16_t>(h), ldh, s);
  });
  return {x_out, h};
}

std::tuple<Tensor, Maybe, Maybe, Maybe, Maybe> norm_gate_bwd(
    const Tensor& x, const Maybe& y, const Maybe& d_x_out, const Maybe& d_h,
    const Maybe& weight_post, const Maybe& gate, const Maybe& weight_pre, double scale, double eps,
    const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(x, "x");
  const gemm_norm_gate_args_t a =
      norm_args(x, y, weight_post, gate, weight_pre, scale, eps, device);
  if (d_h.has_value() != weight_pre.has_value()) bad_value("d_h goes with weight_pre");
  gemm_norm_gate_grads_t g = {};
  g.ld_d_x_out = g.ld_dh = g.ld_dx = g.ld_dy = a.D;
  if (d_x_out) g.ld_d_x_out = matrix(*d_x_out, "d_x_out", {x.scalar_type()}, device, a.T, a.D);
  g.d_x_out = ptr(d_x_out);
  if (d_h) {
    g.ld_dh = matrix(*d_h, "d_h", {at::kFloat, at::kBFloat16}, device, a.T, a.D);
    g.dh_type = type_of(*d_h);
  }
  g.dh = ptr(d_h);
  Tensor dx = empty({a.T, a.D}, x.scalar_type(), device, stream);
  Maybe dy, dw_post, dgate, dw_pre;
  if (y) dy = empty({a.T, a.D}, at::kBFloat16, device, stream);
  if (weight_post) dw_post = empty({a.D}, at::kFloat, device, stream);
  if (gate) dgate = empty(gate->sizes(), at::kFloat, device, stream);
  if (a.gate_mode == GEMM_GATE_FULL && a.ld_gate > a.D)  // dgate has the gate's row stride
    dgate = empty({a.T, a.ld_gate}, at::kFloat, device, stream).narrow(1, 0, a.D);
  if (weight_pre) dw_pre = empty({a.D}, at::kFloat, device, stream);
  g.dx = ptr(dx);
  g.dy = ptr<uint16_t>(dy);
  g.dgate = ptr<float>(dgate);
  g.dw_post = ptr<float>(dw_post);
  g.dw_pre = ptr<float>(dw_pre);
  run("gemm_norm_gate_bwd", device, stream,
      [&](void* s) { return gemm_norm_gate_bwd(&a, &g, s); });
  return {dx, dy, dw_post, dgate, dw_pre};
}

// --------------------------------------------------- 8-bit checkpoints

constexpr int64_t kRun = 32;

void kept(const Tensor& q, const Tensor& scales, int64_t T, int64_t N, at::Device device) {
  const int64_t runs = (T + kRun - 1) / kRun;
  bytes16(q, "kept.q", runs * kRun * N, device);
  if (scales.scalar_type() != at::kByte || scales.device() != device || !scales.is_contiguous() ||
      scales.dim() != 2 || scales.size(0) != runs || scales.size(1) != N)
    bad_value("kept.scales must be contiguous uint8, ceil(rows / 32) x cols");
}

std::tuple<Tensor, Tensor, Maybe> ckpt8_pack(const Tensor& X, const std::optional<std::string>& act,
                                             const Maybe& act_out_,
                                             const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(X, "X");
  const int64_t ldx = matrix(X, "X", {at::kFloat, at::kBFloat16}, device);
  const int64_t T = X.size(0), N = X.size(1), runs = (T + kRun - 1) / kRun;
  const int32_t kind = act ? activation(*act) : GEMM_ACT_NONE;
  int64_t ld = N > 1 ? N : 1;
  Maybe act_out;
  if (act)
    act_out = output(act_out_, "act_out", T, N, at::kBFloat16, device, &ld, stream);
  else if (act_out_)
    bad_value("act_out needs an activation");
  Tensor q = empty({runs * kRun * N}, at::kByte, device, stream);
  Tensor scales = empty({runs, N}, at::kByte, device, stream);
  run("gemm_ckpt8_pack", device, stream, [&](void* s) {
    return gemm_ckpt8_pack(T, N, ptr(X), ldx, type_of(X), ptr(q), ptr<uint8_t>(scales), kind,
                           ptr<uint16_t>(act_out), ld, s);
  });
  return {q, scales, act_out};
}

Tensor ckpt8_unpack(const Tensor& q, const Tensor& scales, int64_t T, int64_t N,
                    at::ScalarType type, const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(q, "kept.q");
  kept(q, scales, T, N, device);
  if (type != at::kFloat && type != at::kBFloat16)
    bad_type("dtype must be torch.float32 or torch.bfloat16");
  Tensor out = empty({T, N}, type, device, stream);
  run("gemm_ckpt8_unpack", device, stream, [&](void* s) {
    return gemm_ckpt8_unpack(T, N, ptr(q), ptr<uint8_t>(scales), ptr(out), N > 1 ? N : 1,
                             type_of(out), s);
  });
  return out;
}

std::tuple<Tensor, Maybe> ckpt8_act_grad(const Tensor& grad, const Tensor& q, const Tensor& scales,
                                         int64_t T, int64_t N, const std::string& act,
                                         bool bias_grad, const Maybe& out_,
                                         const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(q, "kept.q");
  kept(q, scales, T, N, device);
  const int64_t ldg = matrix(grad, "grad", {at::kFloat, at::kBFloat16}, device, T, N);
  const int32_t kind = activation(act);
  int64_t ld = 0;
  Tensor out = output(out_, "out", T, N, at::kBFloat16, device, &ld, stream);
  Maybe dbias;
  if (bias_grad) dbias = empty({N}, at::kFloat, device, stream);
  run("gemm_ckpt8_act_grad", device, stream, [&](void* s) {
    return gemm_ckpt8_act_grad(T, N, ptr(grad), ldg, type_of(grad), ptr(q), ptr<uint8_t>(scales),
                               kind, ptr<uint16_t>(out), ld, ptr<float>(dbias), s);
  });
  return {out, dbias};
}

Tensor ckpt8_wgrad(const Tensor& q, const Tensor& scales, int64_t T, int64_t K, const Tensor& dY,
                   const Maybe& out_, double beta, const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(q, "kept.q");
  kept(q, scales, T, K, device);
  const int64_t ld = matrix(dY, "dY", {at::kBFloat16}, device);
  if (dY.size(0) != T) bad_value("dY must have the " + text(T) + " rows that were kept");
  const int64_t N = dY.size(1);
  if (beta != 0.0 && !out_) bad_value("beta != 0 reads dW: pass its prior contents as `out`");
  int64_t ldw = 0;
  Tensor out = output(out_, "out", K, N, at::kFloat, device, &ldw, stream);
  run("gemm_ckpt8_wgrad", device, stream, [&](void* s) {
    return gemm_ckpt8_wgrad(T, K, N, ptr(q), ptr<uint8_t>(scales), ptr<uint16_t>(dY), ld,
                            ptr<float>(out), ldw, static_cast<float>(beta), s);
  });
  return out;
}

// ------------------------------------------- 8-bit floating-point products

constexpr int64_t kBlock = 128;

int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

void code_rows(const Tensor& codes, const char* name, at::Device device) {
  const std::string n = name;
  if (codes.scalar_type() != at::kFloat8_e4m3fn) bad_type(n + " must be torch.float8_e4m3fn");
  if (codes.device() != device) bad_value(n + " must be on " + device.str());
  if (codes.size(-1) > 1 && codes.stride(-1) != 1)
    bad_value(n + ": rows must be contiguous (stride(-1) == 1)");
  if (reinterpret_cast<uintptr_t>(codes.data_ptr()) % 16)
    bad_value(n + " must start on a 16-byte boundary");
}

// The row stride of codes (rows x K); a single row has one of its own.
int64_t code_stride(int64_t rows, int64_t K, int64_t stride, const char* name) {
  if (rows <= 1 || K == 0) return (K > 1 ? K + 15 : 16) / 16 * 16;
  if (stride < K || stride % 16)
    bad_value(std::string(name) + ": rows must be a multiple of 16 bytes apart (gemm_fp8_quantize "
                                  "makes them so)");
  return stride > 16 ? stride : 16;
}

// A rows x K matrix in 8 bits, after its checks.
gemm_fp8_t fp8_matrix(const Tensor& codes, const Tensor& scales, bool square, const char* name,
                      at::Device device) {
  const std::string n = name;
  if (codes.dim() != 2) bad_value(n + ".codes must be 2-D");
  code_rows(codes, (n + ".codes").c_str(), device);
  const int64_t R = codes.size(0), K = codes.size(1);
  const int64_t ld_s = square ? matrix(scales, (n + ".scales").c_str(), {at::kFloat}, device,
                                       blocks(R), blocks(K))
                              : matrix(scales, (n + ".scales").c_str(), {at::kFloat}, device,
                                       blocks(K), R);
  return gemm_fp8_t{ptr(codes), code_stride(R, K, codes.stride(0), name), ptr<float>(scales), ld_s,
                    square ? 1 : 0};
}

at::ScalarType product_type(const std::optional<at::ScalarType>& wanted, const Maybe& out) {
  const at::ScalarType type = wanted ? *wanted : out ? out->scalar_type() : at::kFloat;
  if (type != at::kFloat && type != at::kBFloat16)
    bad_type("out_dtype must be torch.float32 or torch.bfloat16");
  return type;
}

int32_t abi_type(at::ScalarType t) { return t == at::kBFloat16 ? GEMM_TYPE_BF16 : GEMM_TYPE_F32; }

std::tuple<Tensor, Tensor> fp8_quantize(const Tensor& X, bool square, bool transpose,
                                        const Maybe& index, const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(X, "X");
  gemm_fp8_quantize_args_t q = {};
  q.batch = 1;
  if (X.dim() == 3) {
    if (!square) bad_value("X must be 2-D (3-D only with square)");
    if (X.scalar_type() != at::kFloat && X.scalar_type() != at::kBFloat16)
      bad_type("X must be torch.float32 or torch.bfloat16");
    q.batch = X.size(0);
    const int64_t T = X.size(1), C = X.size(2);
    if (X.numel() > 0) {
      if (C > 1 && X.stride(2) != 1) bad_value("X: rows must be contiguous (stride(-1) == 1)");
      if (T > 1 && X.stride(1) < C) bad_value("X: rows must not overlap");
      if (q.batch > 1 && X.stride(0) < 0) bad_value("X: matrices must not go backwards");
    }
    q.T = T;
    q.C = C;
    q.ldx = T > 1 && X.numel() > 0 ? X.stride(1) : C > 1 ? C : 1;
    q.x_step = q.batch > 1 ? X.stride(0) : 0;
  } else {
    q.ldx = matrix(X, "X", {at::kFloat, at::kBFloat16}, device);
    q.T = X.size(0);
    q.C = X.size(1);
  }
  q.x = ptr(X);
  q.x_type = type_of(X);
  q.square = square;
  q.transpose = transpose;
  int64_t R = transpose ? q.C : q.T;
  const int64_t K = transpose ? q.T : q.C;
  if (index) {
    if (square || transpose) bad_value("index goes without square and transpose");
    if (index->dim() != 1 || index->scalar_type() != at::kInt || index->device() != device ||
        !index->is_contiguous())
      bad_value("index must be a contiguous int32 vector on " + device.str());
    R = q.rows = index->size(0);
    // (an empty index is no index, and has no rows)
    q.index = ptr<int32_t>(*index);
  }
  // rows start on 128 bytes: a block is one line
  const int64_t ld = K > 0 ? blocks(K) * kBlock : kBlock;
  Tensor codes, scales;
  if (X.dim() == 3) {
    codes = empty_strided({q.batch, R, K}, {R * ld, ld, 1}, at::kFloat8_e4m3fn, device, stream);
    scales = empty({q.batch, blocks(R), blocks(K)}, at::kFloat, device, stream);
    q.codes_step = R * ld;
    q.scales_step = blocks(R) * blocks(K);
  } else {
    codes = empty_strided({R, K}, {ld, 1}, at::kFloat8_e4m3fn, device, stream);
    scales = square ? empty({blocks(R), blocks(K)}, at::kFloat, device, stream)
                    : empty({blocks(K), R}, at::kFloat, device, stream);
  }
  if (codes.numel() == 0) return {codes, scales};
  q.codes = ptr(codes);
  q.ld = ld;
  q.scales = ptr<float>(scales);
  q.ld_scales = scales.size(-1) > 1 ? scales.size(-1) : 1;
  run("gemm_fp8_quantize", device, stream, [&](void* s) { return gemm_fp8_quantize(&q, s); });
  return {codes, scales};
}

Tensor fp8(const Tensor& a_codes, const Tensor& a_scales, bool a_square, const Tensor& b_codes,
           const Tensor& b_scales, bool b_square, const Maybe& out_, double alpha, double beta,
           const Maybe& bias, const std::string& act,
           const std::optional<at::ScalarType>& out_dtype, const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(a_codes, "a.codes");
  if (a_square) bad_value("a must have a scale for each 128 values of a row (square=False)");
  const gemm_fp8_t a = fp8_matrix(a_codes, a_scales, false, "a", device);
  const gemm_fp8_t b = fp8_matrix(b_codes, b_scales, b_square, "b", device);
  const int64_t M = a_codes.size(0), K = a_codes.size(1), N = b_codes.size(0);
  if (b_codes.size(1) != K)
    bad_value("inner sizes differ: a is " + text(M) + " x " + text(K) + ", b is " + text(N) +
              " x " + text(b_codes.size(1)));
  if (beta != 0.0 && !out_) bad_value("beta != 0 reads C: pass its prior contents as `out`");
  const at::ScalarType type = product_type(out_dtype, out_);
  int64_t ldc = 0;
  Tensor out = output(out_, "out", M, N, type, device, &ldc, stream);
  if (bias) vector(*bias, "bias", device, N);
  const gemm_epilogue_t epi = {static_cast<float>(alpha), static_cast<float>(beta),
                               ptr<float>(bias), activation(act)};
  run("gemm_fp8", device, stream, [&](void* s) {
    return gemm_fp8(M, N, K, &a, &b, ptr(out), ldc, abi_type(type), &epi, s);
  });
  return out;
}

Tensor fp8_experts(const Tensor& a_codes, const Tensor& a_scales, bool a_square,
                   const Tensor& b_codes, const Tensor& b_scales, bool b_square,
                   const Tensor& offsets, const Maybe& out_, double alpha, double beta,
                   const Maybe& bias, const std::string& act,
                   const std::optional<at::ScalarType>& out_dtype,
                   const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(a_codes, "a.codes");
  if (a_square) bad_value("a must have a scale for each 128 values of a row (square=False)");
  const gemm_fp8_t a = fp8_matrix(a_codes, a_scales, false, "a", device);
  const int64_t M = a_codes.size(0), K = a_codes.size(1);
  if (!b_square || b_codes.dim() != 3)
    bad_value("b must be E matrices with square scales: codes E x N x K");
  code_rows(b_codes, "b.codes", device);
  const int64_t E = b_codes.size(0), N = b_codes.size(1);
  if (b_codes.size(2) != K)
    bad_value("inner sizes differ: a is " + text(M) + " x " + text(K) + ", b holds " + text(N) +
              " x " + text(b_codes.size(2)));
  const int64_t ld = code_stride(E * N, K, N > 1 ? b_codes.stride(1) : b_codes.stride(0), "b");
  if (E > 1 && N > 0 && K > 0 && b_codes.stride(0) != N * ld)
    bad_value("b.codes: the matrices must follow each other (stride(0) == N * stride(1))");
  if (b_scales.scalar_type() != at::kFloat || b_scales.device() != device ||
      b_scales.dim() != 3 || b_scales.size(0) != E || b_scales.size(1) != blocks(N) ||
      b_scales.size(2) != blocks(K) || !b_scales.is_contiguous())
    bad_value("b.scales must be contiguous float32, E x ceil(N / 128) x ceil(K / 128), on " +
              device.str());
  if (offsets.dim() != 1 || offsets.size(0) != E + 1 || offsets.scalar_type() != at::kInt ||
      offsets.device() != device || !offsets.is_contiguous())
    bad_value("offsets must be a contiguous int32 vector of " + text(E + 1) + " elements on " +
              device.str());
  if (beta != 0.0 && !out_) bad_value("beta != 0 reads C: pass its prior contents as `out`");
  const at::ScalarType type = product_type(out_dtype, out_);
  int64_t ldc = 0;
  Tensor out = output(out_, "out", M, N, type, device, &ldc, stream);
  if (bias && (bias->scalar_type() != at::kFloat || bias->device() != device || bias->dim() != 2 ||
               bias->size(0) != E || bias->size(1) != N || !bias->is_contiguous()))
    bad_value("bias must be contiguous float32, " + text(E) + " x " + text(N) + ", on " +
              device.str());
  const gemm_fp8_t b = {ptr(b_codes), ld, ptr<float>(b_scales), blocks(K) > 1 ? blocks(K) : 1, 1};
  const gemm_epilogue_t epi = {static_cast<float>(alpha), static_cast<float>(beta),
                               ptr<float>(bias), activation(act)};
  run("gemm_fp8_experts", device, stream, [&](void* s) {
    return gemm_fp8_experts(E, M, N, K, &a, &b, ptr<int32_t>(offsets), ptr(out), ldc,
                            abi_type(type), &epi, s);
  });
  return out;
}

// ------------------------------------------------------------ experts

int32_t score_of(const std::string& name) {
  if (name == "softmax") return GEMM_ROUTE_SOFTMAX;
  if (name == "sigmoid") return GEMM_ROUTE_SIGMOID;
  bad_value("score must be 'softmax' or 'sigmoid'");
}

void pairs(const Tensor& t, const char* name, at::ScalarType type, at::Device device, int64_t T,
           int64_t k) {
  if (t.scalar_type() != type || t.device() != device || t.dim() != 2 || t.size(0) != T ||
      t.size(1) != k || !t.is_contiguous())
    bad_value(std::string(name) + " must be contiguous " + (type == at::kInt ? "int32" : "float32") +
              ", " + text(T) + " x " + text(k) + ", on " + device.str());
}

gemm_route_args_t route_args(const Tensor& logits, int64_t k, const std::string& score,
                             bool renormalize, double scale, at::Device device) {
  gemm_route_args_t a = {};
  a.ld = matrix(logits, "logits", {at::kFloat, at::kBFloat16}, device);
  a.T = logits.size(0);
  a.E = logits.size(1);
  a.k = k;
  a.logits = ptr(logits);
  a.type = type_of(logits);
  a.score = score_of(score);
  a.groups = a.groups_kept = a.group_top = 1;
  a.renormalize = renormalize;
  a.scale = static_cast<float>(scale);
  if (a.E < 1 || a.E > 1024) bad_value("there must be 1 to 1024 experts");
  if (k < 1 || k > 32 || k > a.E) bad_value("k must be 1 to 32 of the experts");
  return a;
}

std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor> route(
    const Tensor& logits, int64_t k, const std::string& score, const Maybe& bias, int64_t groups,
    int64_t groups_kept, int64_t group_top, bool renormalize, double scale,
    const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(logits, "logits");
  gemm_route_args_t a = route_args(logits, k, score, renormalize, scale, device);
  if (groups < 1 || groups > 32 || a.E % groups)
    bad_value("groups must be 1 to 32 and divide the experts");
  if (groups_kept < 1 || groups_kept > groups) bad_value("groups_kept must be 1 to groups");
  if (group_top != 1 && group_top != 2) bad_value("group_top must be 1 or 2");
  if (k > groups_kept * (a.E / groups)) bad_value("k is more than the experts of the groups kept");
  if (bias) vector(*bias, "bias", device, a.E);
  a.bias = ptr<float>(bias);
  a.groups = static_cast<int32_t>(groups);
  a.groups_kept = static_cast<int32_t>(groups_kept);
  a.group_top = static_cast<int32_t>(group_top);
  // All outputs and the workspace are one block, which lives as long as any of them: also
  // until the work of another stream than the current one has finished, as the outputs
  // have to.
  const int64_t bytes = gemm_route_workspace_bytes(a.T, a.E), n = a.T * k * 4;
  Tensor block = empty({4 * n + (a.E + 1) * 4 + (bytes > 0 ? bytes : 0)}, at::kByte, device, stream);
  Tensor index = part(block, at::kInt, {a.T, k}, 0);
  Tensor weight = part(block, at::kFloat, {a.T, k}, n);
  Tensor slot = part(block, at::kInt, {a.T, k}, 2 * n);
  Tensor source = part(block, at::kInt, {a.T * k}, 3 * n);
  Tensor offsets = part(block, at::kInt, {a.E + 1}, 4 * n);
  void* workspace =
      bytes > 0 ? static_cast<uint8_t*>(block.data_ptr()) + 4 * n + (a.E + 1) * 4 : nullptr;
  run("gemm_route", device, stream, [&](void* s) {
    return gemm_route(&a, ptr<int32_t>(index), ptr<float>(weight), ptr<int32_t>(slot),
                      ptr<int32_t>(source), ptr<int32_t>(offsets), workspace, s);
  });
  return {index, weight, slot, source, offsets};
}

Tensor route_bwd(const Tensor& logits, const Tensor& index, const Tensor& d_weight,
                 const std::string& score, bool renormalize, double scale, const Maybe& out_,
                 const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(logits, "logits");
  if (index.dim() != 2) bad_value("index must be 2-D");
  const int64_t k = index.size(1);
  const gemm_route_args_t a = route_args(logits, k, score, renormalize, scale, device);
  pairs(index, "index", at::kInt, device, a.T, k);
  pairs(d_weight, "d_weight", at::kFloat, device, a.T, k);
  int64_t ld = 0;
  Tensor out = output(out_, "out", a.T, a.E, logits.scalar_type(), device, &ld, stream);
  run("gemm_route_bwd", device, stream, [&](void* s) {
    return gemm_route_bwd(&a, ptr<int32_t>(index), ptr<float>(d_weight), ptr(out), ld, s);
  });
  return out;
}

gemm_combine_args_t combine_args(const Tensor& rows, const Tensor& slot, const Tensor& weight,
                                 at::Device device) {
  gemm_combine_args_t a = {};
  a.ld_rows = matrix(rows, "rows", {at::kFloat, at::kBFloat16}, device);
  if (slot.dim() != 2) bad_value("slot must be 2-D");
  a.T = slot.size(0);
  a.k = slot.size(1);
  if (a.k > 32) bad_value("a token has at most 32 rows");
  a.D = rows.size(1);
  a.R = rows.size(0);
  pairs(slot, "slot", at::kInt, device, a.T, a.k);
  pairs(weight, "weight", at::kFloat, device, a.T, a.k);
  a.rows = ptr(rows);
  a.rows_type = type_of(rows);
  a.slot = ptr<int32_t>(slot);
  a.weight = ptr<float>(weight);
  a.ldx = a.D > 1 ? a.D : 1;
  return a;
}

Tensor combine(const Tensor& rows, const Tensor& slot, const Tensor& weight, const Maybe& x,
               const Maybe& out_, const std::optional<at::ScalarType>& out_dtype,
               const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(rows, "rows");
  gemm_combine_args_t a = combine_args(rows, slot, weight, device);
  if (x) {
    a.ldx = matrix(*x, "x", {at::kFloat, at::kBFloat16}, device, a.T, a.D);
    a.x = ptr(*x);
    a.x_type = type_of(*x);
  }
  const at::ScalarType type =
      product_type(out_dtype ? out_dtype
                             : out_ ? std::optional<at::ScalarType>(out_->scalar_type())
                                    : std::optional<at::ScalarType>(
                                          x ? x->scalar_type() : rows.scalar_type()),
                   out_);
  int64_t ld = 0;
  Tensor out = output(out_, "out", a.T, a.D, type, device, &ld, stream);
  run("gemm_combine", device, stream,
      [&](void* s) { return gemm_combine(&a, ptr(out), ld, abi_type(type), s); });
  return out;
}

std::tuple<Tensor, Tensor> combine_bwd(const Tensor& d_out, const Tensor& rows, const Tensor& slot,
                                       const Tensor& weight, const Maybe& d_rows_,
                                       const std::optional<int64_t>& stream) {
  const at::Device device = cuda_device(rows, "rows");
  const gemm_combine_args_t a = combine_args(rows, slot, weight, device);
  const int64_t ld_d =
      matrix(d_out, "d_out", {at::kFloat, at::kBFloat16}, device, a.T, a.D);
  int64_t ld = 0;
  Tensor d_rows = output(d_rows_, "d_rows", a.R, a.D, rows.scalar_type(), device, &ld, stream);
  Tensor d_weight = empty({a.T, a.k}, at::kFloat, device, stream);
  run("gemm_combine_bwd", device, stream, [&](void* s) {
    // Only the device knows which rows no slot names: theirs is the gradient of nothing.
    // (Tensor::zero_ takes 5 us more of the host's time.)
    if (!d_rows_ && d_rows.numel() > 0 &&
        cudaMemsetAsync(d_rows.data_ptr(), 0, d_rows.nbytes(), static_cast<cudaStream_t>(s)) !=
            cudaSuccess)
      return GEMM_ERR_LAUNCH;
    return gemm_combine_bwd(&a, ptr(d_out), ld_d, type_of(d_out), ptr(d_rows), ld,
                            ptr<float>(d_weight), s);
  });
  return {d_rows, d_weight};
}

}  // namespace

PYBIND11_MODULE(layer_binding, m) {
  m.def("w4", &w4);
  m.def("w4_pack", &w4_pack);
  m.def("w4_quantize", &w4_quantize);
  m.def("w4_unpack", &w4_unpack);
  m.def("norm_gate", &norm_gate);
  m.def("norm_gate_bwd", &norm_gate_bwd);
  m.def("ckpt8_pack", &ckpt8_pack);
  m.def("ckpt8_unpack", &ckpt8_unpack);
  m.def("ckpt8_act_grad", &ckpt8_act_grad);
  m.def("ckpt8_wgrad", &ckpt8_wgrad);
  m.def("fp8_quantize", &fp8_quantize);
  m.def("fp8", &fp8);
  m.def("fp8_experts", &fp8_experts);
  m.def("route", &route);
  m.def("route_bwd", &route_bwd);
  m.def("combine", &combine);
  m.def("combine_bwd", &combine_bwd);
}
