// layer_binding.cpp -- the Python binding of the layer operators: checks torch
// tensors and passes their sizes, addresses and strides to the C entry points
// of include/gemm07.h.  Compiled code, because at the sizes of a decode step a
// call's own time is the operator's: marshalling a call in Python took 7 to 18
// us of a 12 to 23 us call (gemm_w4 at 1 x 4096 x 4096, gemm_norm_gate at
// 1 x 4096).
//
// A refused argument raises ValueError or TypeError, a status of the library
// GemmError, as in the rest of the package.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <initializer_list>
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

Tensor empty(at::IntArrayRef size, at::ScalarType type, at::Device device) {
  return at::empty(size, at::TensorOptions().dtype(type).device(device));
}

// `out` after its checks, or a new rows x cols tensor; its row stride in *ld.
Tensor output(const Maybe& out, const char* name, int64_t rows, int64_t cols, at::ScalarType type,
              at::Device device, int64_t* ld) {
  if (out) {
    *ld = matrix(*out, name, {type}, device, rows, cols);
    return *out;
  }
  *ld = cols > 1 ? cols : 1;
  return empty({rows, cols}, type, device);
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
  Tensor out = output(out_, "out", M, N, type, device, &ldc);
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
  Tensor packed = empty({packed_bytes(K, N)}, at::kByte, device);
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
  Tensor packed = empty({packed_bytes(K, N)}, at::kByte, device);
  Tensor scales = empty({G, N}, at::kBFloat16, device);
  Maybe zeros;
  if (!symmetric) zeros = empty({G, N}, at::kByte, device);
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
  Tensor out = empty({K, N}, at::kBFloat16, device);
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
  Tensor x_out = output(x_out_, "x_out", a.T, a.D, x.scalar_type(), device, &ld_o);
  Maybe h;
  if (weight_pre)
    h = output(h_, "h", a.T, a.D, at::kBFloat16, device, &ldh);
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
  Tensor dx = empty({a.T, a.D}, x.scalar_type(), device);
  Maybe dy, dw_post, dgate, dw_pre;
  if (y) dy = empty({a.T, a.D}, at::kBFloat16, device);
  if (weight_post) dw_post = empty({a.D}, at::kFloat, device);
  if (gate) dgate = empty(gate->sizes(), at::kFloat, device);
  if (a.gate_mode == GEMM_GATE_FULL && a.ld_gate > a.D)  // dgate has the gate's row stride
    dgate = empty({a.T, a.ld_gate}, at::kFloat, device).narrow(1, 0, a.D);
  if (weight_pre) dw_pre = empty({a.D}, at::kFloat, device);
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
    act_out = output(act_out_, "act_out", T, N, at::kBFloat16, device, &ld);
  else if (act_out_)
    bad_value("act_out needs an activation");
  Tensor q = empty({runs * kRun * N}, at::kByte, device);
  Tensor scales = empty({runs, N}, at::kByte, device);
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
  Tensor out = empty({T, N}, type, device);
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
  Tensor out = output(out_, "out", T, N, at::kBFloat16, device, &ld);
  Maybe dbias;
  if (bias_grad) dbias = empty({N}, at::kFloat, device);
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
  Tensor out = output(out_, "out", K, N, at::kFloat, device, &ldw);
  run("gemm_ckpt8_wgrad", device, stream, [&](void* s) {
    return gemm_ckpt8_wgrad(T, K, N, ptr(q), ptr<uint8_t>(scales), ptr<uint16_t>(dY), ld,
                            ptr<float>(out), ldw, static_cast<float>(beta), s);
  });
  return out;
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
}
