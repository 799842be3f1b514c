// combine.cu -- the experts' rows back to their tokens, and the gradient:
//   out[t] = x[t] + sum_j weight[t][j] * rows[slot[t][j]]           (slot -1: no row)
//   d_rows[slot[t][j]] = weight[t][j] * d_out[t]
//   d_weight[t][j]     = sum over columns of d_out[t] * rows[slot[t][j]]
// in FP32, j in order.  Every row is read once and every output written once: memory
// bounds both.  A slot outside 0 .. R - 1 has no row: its weight's finite value does
// not matter, but one that is not finite shows (0 * weight is added).
#include "experts.h"
#include "kernels.h"

namespace g07 {
namespace {

constexpr int kThreads = 128;

// A block takes kThreads * N columns of a token.
template <typename TR, typename TX, typename TO, int N>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a, int parts) {
  grid_dependency_wait();
  grid_dependents_go();
  const int t = static_cast<int>(blockIdx.x / parts);
  const int c = (static_cast<int>(blockIdx.x % parts) * kThreads + static_cast<int>(threadIdx.x)) * N;
  if (c >= a.D) return;
  const int* slot = a.slot + static_cast<int64_t>(t) * a.k;
  const float* weight = a.weight + static_cast<int64_t>(t) * a.k;
  const TR* rows = static_cast<const TR*>(a.rows) + c;
  float sum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < a.k; ++j) {
    const int s = __ldg(slot + j);
    const float w = __ldg(weight + j);
    const bool on = s >= 0 && s < a.R;
    float v[N];
    if (on) load_vec<N>(rows + s * a.ld_rows, v);
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = fmaf(w, on ? v[i] : 0.0f, sum[i]);
  }
  if (a.x) {
    float v[N];
    load_vec<N>(static_cast<const TX*>(a.x) + t * a.ldx + c, v);
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] += v[i];
  }
  store_vec<N>(static_cast<TO*>(a.out) + t * a.ld_out + c, sum);
}

// A block takes a token: its gradient is read once for each 8 experts.
constexpr int kBwdThreads = 256;
constexpr int kAtOnce = 8;

template <typename TR, typename TO, int N>
__global__ void __launch_bounds__(kBwdThreads) combine_bwd_kernel(CombineArgs a) {
  __shared__ float part[kAtOnce][kBwdThreads / 32];
  grid_dependency_wait();
  grid_dependents_go();
  const int t = static_cast<int>(blockIdx.x);
  const int64_t first = static_cast<int64_t>(t) * a.k;
  const TR* rows = static_cast<const TR*>(a.rows);
  TR* d_rows = static_cast<TR*>(a.d_rows);
  const TO* d_out = static_cast<const TO*>(a.out) + t * a.ld_out;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
    float dot[kAtOnce];
    int s[kAtOnce];
    float w[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      dot[j] = 0.0f;
      s[j] = j0 + j < a.k ? __ldg(a.slot + first + j0 + j) : -1;
      if (s[j] >= a.R) s[j] = -1;
      w[j] = s[j] >= 0 ? __ldg(a.weight + first + j0 + j) : 0.0f;
    }
    for (int c = static_cast<int>(threadIdx.x) * N; c < a.D; c += kBwdThreads * N) {
      float d[N];
      load_vec<N>(d_out + c, d);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (s[j] < 0) continue;
        float v[N], g[N];
        load_vec<N>(rows + s[j] * a.ld_rows + c, v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dot[j] = fmaf(d[i], v[i], dot[j]);
          g[i] = w[j] * d[i];
        }
        store_vec<N>(d_rows + s[j] * a.ld_d_rows + c, g);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
      for (int i = 16; i; i >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], i);
      if (lane == 0) part[j][warp] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kAtOnce && j0 + static_cast<int>(threadIdx.x) < a.k) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kBwdThreads / 32; ++i) v += part[threadIdx.x][i];
      a.d_weight[first + j0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

bool wide(const void* p, int64_t ld) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0);
}

// Calls f with a value of the type.
template <typename F>
cudaError_t by(bool bf16, F f) {
  return bf16 ? f(__nv_bfloat16()) : f(float());
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream) {
  const bool vec = a.D % 8 == 0 && wide(a.rows, a.ld_rows) && wide(a.x, a.ldx) && wide(a.out, a.ld_out);
  const int parts = (a.D + kThreads * (vec ? 8 : 1) - 1) / (kThreads * (vec ? 8 : 1));
  const int64_t grid = static_cast<int64_t>(a.T) * parts;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const cudaError_t e = by(a.rows_bf16, [&](auto r) {
    return by(a.x_bf16, [&](auto x) {
      return by(a.out_bf16, [&](auto o) {
        using R = decltype(r);
        using X = decltype(x);
        using O = decltype(o);
        return launch_pdl(vec ? combine_kernel<R, X, O, 8> : combine_kernel<R, X, O, 1>,
                          dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a, parts);
      });
    });
  });
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_combine_bwd(const CombineArgs& a, cudaStream_t stream) {
  const bool vec = a.D % 8 == 0 && wide(a.rows, a.ld_rows) && wide(a.out, a.ld_out) &&
                   wide(a.d_rows, a.ld_d_rows);
  const cudaError_t e = by(a.rows_bf16, [&](auto r) {
    return by(a.out_bf16, [&](auto o) {
      using R = decltype(r);
      using O = decltype(o);
      return launch_pdl(vec ? combine_bwd_kernel<R, O, 8> : combine_bwd_kernel<R, O, 1>,
                        dim3(static_cast<unsigned>(a.T)), dim3(kBwdThreads), 0, stream, a);
    });
  });
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace g07
