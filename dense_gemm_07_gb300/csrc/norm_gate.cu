// norm_gate.cu -- RMS norms after and before a block, fused with the block's
// gate and the scaled residual, and the gradient.  Per row (token), with x
// the residual stream and y the block's output:
//   r2 = 1 / sqrt(mean(y^2) + eps),  n = y r2,  p = n w_post   (p = y without
//                                                               w_post)
//   u  = alpha x + gate p                                 -> x_out
//   r1 = 1 / sqrt(mean(u^2) + eps),  h = u r1 w_pre       -> h, the next GEMM's A
// and backward, from d_x_out and dh, with x and y read again:
//   du = d_x_out + r1 (dh w_pre - u r1^2 mean(dh w_pre u))
//   dx = alpha du,  dgate = du p,  dp = gate du
//   dy = r2 (dp w_post - n mean(dp w_post n))
//   dw_pre = sum over rows of dh u r1,  dw_post = sum over rows of dp n.
// All of it in FP32 from the values as loaded; each output is rounded once to
// its type.  h uses u before x_out's rounding, and the gradient is that of
// these formulas (rounding passes gradients unchanged).
//
// Memory bounds both: a row is read once into registers, and its sums are
// taken over the block while it stays there.
#include "kernels.h"
#include "layer.h"

namespace g07 {
namespace {

// Sums of N values over the block, in every thread, in warp order.  `buf`
// holds 16 * N floats; one barrier.  Callers use a buffer again only after the
// barrier of a later call, so no thread overwrites what another still reads.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[warp * N + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += buf[w * N + i];
}

// Elements of a row: thread `tid` holds runs of VEC elements at
// (i * blockDim.x + tid) * VEC, i < VPT.
template <typename X, typename Y, int VEC, int VPT>
__global__ void __launch_bounds__(512) norm_gate_kernel(NormArgs p) {
  __shared__ float buf[2][16];
  grid_dependency_wait();
  grid_dependents_go();
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(p.x) + row * p.ldx;
  const Y* y = static_cast<const Y*>(p.y) + row * p.ldy;
  const bool has_y = p.y != nullptr;
  float u[VPT][VEC], yv[VPT][VEC];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int d = (i * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[i][e] = yv[i][e] = 0.0f;
    if (d < p.D) {
      load_vec(x + d, u[i]);
      if (has_y) load_vec(y + d, yv[i]);
    }
  }
  float r2 = 1.0f;
  if (p.w_post) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] = fmaf(yv[i][e], yv[i][e], s[0]);
    block_sums(s, buf[0]);
    r2 = rsqrtf(s[0] / p.D + p.eps);
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int d = (i * blockDim.x + threadIdx.x) * VEC;
    if (d >= p.D) continue;
    float w[VEC], g[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = g[e] = 1.0f;
    if (p.w_post) load_vec(p.w_post + d, w);
    if (p.gate) {
      const float* gp = p.gate + row * p.gate_row;
      if (p.gate_col) {
        load_vec(gp + d, g);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[e] = *gp;
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float pe = yv[i][e] * r2 * w[e];
      u[i][e] = has_y ? fmaf(p.alpha, u[i][e], g[e] * pe) : p.alpha * u[i][e];
      s[0] = fmaf(u[i][e], u[i][e], s[0]);
    }
    if (p.x_out) store_vec(static_cast<X*>(p.x_out) + row * p.ld_x_out + d, u[i]);
  }
  if (p.h == nullptr) return;
  block_sums(s, buf[1]);
  const float r1 = rsqrtf(s[0] / p.D + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int d = (i * blockDim.x + threadIdx.x) * VEC;
    if (d >= p.D) continue;
    float w[VEC];
    load_vec(p.w_pre + d, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] *= u[i][e] * r1;
    store_vec(p.h + row * p.ldh + d, w);
  }
}

// Blocks walk the rows; the column sums (dw_post, dw_pre, dgate) of a block's
// rows gather in shared memory, each element by the one thread that owns its
// column, and go to `partial` (slot blockIdx.x, 3 x D) at the end.
template <typename X, typename Y, typename H, int VEC, int VPT>
__global__ void __launch_bounds__(512) norm_gate_bwd_kernel(NormArgs p, float* partial) {
  extern __shared__ float sums[];  // [3][D]
  __shared__ float row_buf[2][3][32];  // alternate from row to row
  const bool has_y = p.y != nullptr, has_h = p.dh != nullptr;
  const bool row_gate = p.gate != nullptr && p.gate_col == 0;
  const bool col_gate = p.gate != nullptr && p.gate_col != 0 && p.gate_row == 0;
  const bool full_gate = p.gate != nullptr && p.gate_col != 0 && p.gate_row != 0;
  for (int i = threadIdx.x; i < 3 * p.D; i += blockDim.x) sums[i] = 0.0f;
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_go();
  const float inv_d = 1.0f / p.D;
  int odd = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, odd ^= 1) {
    float(*buf)[32] = row_buf[odd];
    const X* x = static_cast<const X*>(p.x) + row * p.ldx;
    const Y* y = static_cast<const Y*>(p.y) + row * p.ldy;
    const X* dxo = static_cast<const X*>(p.d_x_out) + row * p.ld_d_x_out;
    const H* dh = static_cast<const H*>(p.dh) + row * p.ld_dh;
    float u[VPT][VEC], yv[VPT][VEC], du[VPT][VEC], hv[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int d = (i * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[i][e] = yv[i][e] = du[i][e] = hv[i][e] = 0.0f;
      if (d < p.D) {
        load_vec(x + d, u[i]);
        if (has_y) load_vec(y + d, yv[i]);
        if (p.d_x_out) load_vec(dxo + d, du[i]);
        if (has_h) load_vec(dh + d, hv[i]);
      }
    }
    float r2 = 1.0f;
    if (p.w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[0] = fmaf(yv[i][e], yv[i][e], s[0]);
      block_sums(s, buf[0]);
      r2 = rsqrtf(s[0] * inv_d + p.eps);
    }
    auto gate_at = [&](int d, float (&g)[VEC]) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[e] = 1.0f;
      if (p.gate) {
        const float* gp = p.gate + row * p.gate_row;
        if (p.gate_col) {
          load_vec(gp + d, g);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) g[e] = *gp;
        }
      }
    };
    auto vec_at = [&](const float* v, int d, float (&w)[VEC]) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = 1.0f;
      if (v) load_vec(v + d, w);
    };
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int d = (i * blockDim.x + threadIdx.x) * VEC;
      if (d >= p.D) continue;
      float w2[VEC], w1[VEC], g[VEC];
      vec_at(p.w_post, d, w2);
      vec_at(p.w_pre, d, w1);
      gate_at(d, g);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float pe = yv[i][e] * r2 * w2[e];
        u[i][e] = has_y ? fmaf(p.alpha, u[i][e], g[e] * pe) : p.alpha * u[i][e];
        s[0] = fmaf(u[i][e], u[i][e], s[0]);
        s[1] = fmaf(hv[i][e] * w1[e], u[i][e], s[1]);
      }
    }
    float r1 = 0.0f, c1 = 0.0f;
    if (has_h) {
      block_sums(s, buf[1]);
      r1 = rsqrtf(s[0] * inv_d + p.eps);
      c1 = r1 * r1 * (s[1] * inv_d);
    }
    float t[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int d = (i * blockDim.x + threadIdx.x) * VEC;
      if (d >= p.D) continue;
      float w2[VEC], w1[VEC], g[VEC], o[VEC];
      vec_at(p.w_post, d, w2);
      vec_at(p.w_pre, d, w1);
      gate_at(d, g);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (has_h) {
          sums[p.D + d + e] += hv[i][e] * u[i][e] * r1;
          du[i][e] = fmaf(r1, fmaf(hv[i][e], w1[e], -u[i][e] * c1), du[i][e]);
        }
        o[e] = p.alpha * du[i][e];
        const float n = yv[i][e] * r2;
        const float dp = g[e] * du[i][e];
        if (p.w_post) sums[d + e] += dp * n;
        if (col_gate) sums[2 * p.D + d + e] += du[i][e] * (n * w2[e]);
        t[0] = fmaf(dp * w2[e], n, t[0]);
        t[1] = fmaf(du[i][e], n * w2[e], t[1]);
      }
      store_vec(static_cast<X*>(p.dx) + row * p.ld_dx + d, o);
      if (full_gate) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = du[i][e] * (yv[i][e] * r2 * w2[e]);
        store_vec(p.dgate + row * p.gate_row + d, o);
      }
    }
    if (!has_y) continue;
    float c2 = 0.0f;
    if (p.w_post || row_gate) {
      block_sums(t, buf[2]);
      if (p.w_post) c2 = t[0] * inv_d;
      if (row_gate && threadIdx.x == 0) p.dgate[row * p.gate_row] = t[1];
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int d = (i * blockDim.x + threadIdx.x) * VEC;
      if (d >= p.D) continue;
      float w2[VEC], g[VEC], o[VEC];
      vec_at(p.w_post, d, w2);
      gate_at(d, g);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        o[e] = r2 * (g[e] * du[i][e] * w2[e] - yv[i][e] * r2 * c2);
      store_vec(p.dy + row * p.ld_dy + d, o);
    }
  }
  if (partial == nullptr) return;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 3 * p.D;
  // every element was added to by the thread that owns its column
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int d = (i * blockDim.x + threadIdx.x) * VEC;
    if (d >= p.D) continue;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      for (int k = 0; k < 3; ++k) out[k * p.D + d + e] = sums[k * p.D + d + e];
  }
}

// 32 columns per block; the slots are cut into 8 runs, one per warp, whose
// sums are added in run order.
__global__ void __launch_bounds__(256) column_sums_kernel(ColumnSums s) {
  __shared__ float part[8][32];
  grid_dependency_wait();
  grid_dependents_go();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = blockIdx.y;
  float* out = which == 0 ? s.out[0] : which == 1 ? s.out[1] : s.out[2];
  if (out == nullptr) return;
  const int c = blockIdx.x * 32 + lane;
  const int per = (s.slots + 7) / 8;
  const int s0 = warp * per, s1 = min(s0 + per, s.slots);
  float v = 0.0f;
  if (c < s.n) {
    const float* p = s.partial + static_cast<int64_t>(which) * s.n + c;
#pragma unroll 8
    for (int i = s0; i < s1; ++i) v += p[i * s.ld];
  }
  part[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < s.n) {
    v = 0.0f;
    for (int w = 0; w < 8; ++w) v += part[w][lane];
    out[c] = v;
  }
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every row of every operand starts on 16 bytes and holds whole 8-element runs.
bool vector_rows(const NormArgs& a) {
  auto rows = [](const void* p, int64_t ld) { return p == nullptr || (at16(p) && ld % 8 == 0); };
  return a.D % 8 == 0 && rows(a.x, a.ldx) && rows(a.y, a.ldy) && rows(a.x_out, a.ld_x_out) &&
         rows(a.h, a.ldh) && rows(a.d_x_out, a.ld_d_x_out) && rows(a.dh, a.ld_dh) &&
         rows(a.dx, a.ld_dx) && rows(a.dy, a.ld_dy) && at16(a.w_post) && at16(a.w_pre) &&
         (a.gate_col == 0 || (rows(a.gate, a.gate_row) && rows(a.dgate, a.gate_row)));
}

int threads_for(int D, int per_thread) {
  const int t = (D + per_thread - 1) / per_thread;
  return t < 32 ? 32 : (t + 31) / 32 * 32;
}

struct Shape {
  int vec, vpt, threads;
};
Shape shape_for(const NormArgs& a) {
  if (!vector_rows(a)) {
    const int vpt = a.D <= 4096 ? 8 : 32;
    return {1, vpt, threads_for(a.D, vpt)};
  }
  const int vpt = a.D <= 4096 ? 1 : a.D <= 8192 ? 2 : 4;
  return {8, vpt, threads_for(a.D, 8 * vpt)};
}

template <typename X, typename Y>
cudaError_t forward(const NormArgs& a, cudaStream_t st) {
  const Shape s = shape_for(a);
  const dim3 grid(static_cast<unsigned>(a.T)), block(s.threads);
  if (s.vec == 1)
    return s.vpt == 8 ? launch_pdl(norm_gate_kernel<X, Y, 1, 8>, grid, block, 0, st, a)
                      : launch_pdl(norm_gate_kernel<X, Y, 1, 32>, grid, block, 0, st, a);
  if (s.vpt == 1) return launch_pdl(norm_gate_kernel<X, Y, 8, 1>, grid, block, 0, st, a);
  if (s.vpt == 2) return launch_pdl(norm_gate_kernel<X, Y, 8, 2>, grid, block, 0, st, a);
  return launch_pdl(norm_gate_kernel<X, Y, 8, 4>, grid, block, 0, st, a);
}

template <typename K>
cudaError_t launch_bwd(K kernel, const NormArgs& a, const Shape& s, int slots, float* partial,
                       cudaStream_t st) {
  const size_t smem = 3 * sizeof(float) * a.D;
  if (smem > 40 * 1024) {  // 48 KB with the kernel's own arrays needs the opt-in
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(slots), dim3(s.threads), smem, st, a, partial);
}

template <typename X, typename Y, typename H>
cudaError_t backward(const NormArgs& a, int slots, float* partial, cudaStream_t st) {
  const Shape s = shape_for(a);
  if (s.vec == 1)
    return s.vpt == 8
               ? launch_bwd(norm_gate_bwd_kernel<X, Y, H, 1, 8>, a, s, slots, partial, st)
               : launch_bwd(norm_gate_bwd_kernel<X, Y, H, 1, 32>, a, s, slots, partial, st);
  if (s.vpt == 1)
    return launch_bwd(norm_gate_bwd_kernel<X, Y, H, 8, 1>, a, s, slots, partial, st);
  if (s.vpt == 2)
    return launch_bwd(norm_gate_bwd_kernel<X, Y, H, 8, 2>, a, s, slots, partial, st);
  return launch_bwd(norm_gate_bwd_kernel<X, Y, H, 8, 4>, a, s, slots, partial, st);
}

}  // namespace

cudaError_t launch_norm_gate(const NormArgs& a, cudaStream_t stream) {
  using B = __nv_bfloat16;
  const cudaError_t e = a.x_bf16 ? (a.y_bf16 ? forward<B, B>(a, stream) : forward<B, float>(a, stream))
                                 : (a.y_bf16 ? forward<float, B>(a, stream)
                                             : forward<float, float>(a, stream));
  if (e == cudaSuccess) note_launches(1);
  return e;
}

int norm_gate_bwd_slots(const NormArgs& a, const LayerDevice& dev) {
  const int64_t most = static_cast<int64_t>(dev.sms) * (a.D <= 1024 ? 8 : a.D <= 4096 ? 2 : 1);
  return static_cast<int>(a.T < most ? a.T : most);
}

cudaError_t launch_norm_gate_bwd(const NormArgs& a, int slots, float* partial,
                                 cudaStream_t stream) {
  using B = __nv_bfloat16;
  cudaError_t e;
  if (a.x_bf16)
    e = a.y_bf16 ? (a.dh_bf16 ? backward<B, B, B>(a, slots, partial, stream)
                              : backward<B, B, float>(a, slots, partial, stream))
                 : (a.dh_bf16 ? backward<B, float, B>(a, slots, partial, stream)
                              : backward<B, float, float>(a, slots, partial, stream));
  else
    e = a.y_bf16 ? (a.dh_bf16 ? backward<float, B, B>(a, slots, partial, stream)
                              : backward<float, B, float>(a, slots, partial, stream))
                 : (a.dh_bf16 ? backward<float, float, B>(a, slots, partial, stream)
                              : backward<float, float, float>(a, slots, partial, stream));
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_column_sums(const ColumnSums& s, cudaStream_t stream) {
  const dim3 grid((s.n + 31) / 32, s.count);
  const cudaError_t e = launch_pdl(column_sums_kernel, grid, dim3(256), 0, stream, s);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace g07
