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
constexpr int kCols = 8;    // columns of a thread
// Rows on their way together (4096 tokens, 8 rows of 4096 BF16 each: 4 68 us, 8 74, with
// an L2 flush; 55 at the measured bandwidth.  1000 tokens, 5 rows of 3001: 21, 23).
constexpr int kAtOnce = 4;

// A thread's 8 columns of a row, as loaded: VEC: c, c + 1, ... (16-byte accesses); else
// every THREADS-th from c on, so that a warp's accesses are adjacent whatever the rows'
// alignment.  Rows are read once: they need not stay in the caches.
template <typename T, bool VEC, int THREADS>
struct Cols {
  static constexpr int kWords = VEC ? static_cast<int>(sizeof(T)) * kCols / 16 : 1;
  uint4 q[kWords];
  T e[VEC ? 1 : kCols];
  __device__ __forceinline__ void load(const T* row, int c, int D) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) q[i] = __ldcs(reinterpret_cast<const uint4*>(row + c) + i);
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        e[i] = c + i * THREADS < D ? row[c + i * THREADS] : from_f32<T>(0.0f);
    }
  }
  __device__ __forceinline__ void clear() {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) q[i] = make_uint4(0u, 0u, 0u, 0u);
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i) e[i] = from_f32<T>(0.0f);
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (!VEC) {
      return to_f32(e[i]);
    } else if constexpr (sizeof(T) == 4) {
      const uint4& a = q[i / 4];
      return __uint_as_float(i % 4 == 0 ? a.x : i % 4 == 1 ? a.y : i % 4 == 2 ? a.z : a.w);
    } else {
      const uint32_t w = i / 2 == 0 ? q[0].x : i / 2 == 1 ? q[0].y : i / 2 == 2 ? q[0].z : q[0].w;
      return i % 2 ? bf16_hi(w) : bf16_lo(w);
    }
  }
};
template <bool VEC, int THREADS, typename T>
__device__ __forceinline__ void store_cols(T* row, int c, int D, const float (&v)[kCols]) {
  if (VEC) {
    store_vec<8>(row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (c + i * THREADS < D) row[c + i * THREADS] = from_f32<T>(v[i]);
  }
}

// A block takes kThreads * kCols columns of a token.
template <typename TR, typename TX, typename TO, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a, int parts) {
  grid_dependency_wait();
  grid_dependents_go();
  const int t = static_cast<int>(blockIdx.x / parts);
  const int c = static_cast<int>(blockIdx.x % parts) * (kThreads * kCols) +
                static_cast<int>(threadIdx.x) * (VEC ? kCols : 1);
  if (c >= a.D) return;
  const int* slot = a.slot + static_cast<int64_t>(t) * a.k;
  const float* weight = a.weight + static_cast<int64_t>(t) * a.k;
  const TR* rows = static_cast<const TR*>(a.rows);
  float sum[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) sum[i] = 0.0f;
  for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
    Cols<TR, VEC, kThreads> v[kAtOnce];
    float w[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const bool in = j0 + j < a.k;
      const int s = in ? __ldg(slot + j0 + j) : -1;
      w[j] = in ? __ldg(weight + j0 + j) : 0.0f;
      if (s >= 0 && s < a.R)
        v[j].load(rows + s * a.ld_rows, c, a.D);
      else
        v[j].clear();
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
      for (int i = 0; i < kCols; ++i) sum[i] = fmaf(w[j], v[j].at(i), sum[i]);
  }
  if (a.x) {
    Cols<TX, VEC, kThreads> x;
    x.load(static_cast<const TX*>(a.x) + t * a.ldx, c, a.D);
#pragma unroll
    for (int i = 0; i < kCols; ++i) sum[i] += x.at(i);
  }
  store_cols<VEC, kThreads>(static_cast<TO*>(a.out) + t * a.ld_out, c, a.D, sum);
}

// A block takes a token: its gradient is read once for each AT_ONCE of its rows, which
// are all loaded before the first is stored, so that their loads are on their way
// together (4096 tokens, 8 rows of 4096 BF16 each, 570 MB: one row after the other 133
// us, 4 at once 99, 8 at once 93, with an L2 flush; 84 at the measured bandwidth.  8192
// tokens, 4 rows of 1024: 36 and 48 with room for 8).
constexpr int kBwdThreads = 256;

template <typename TR, typename TO, bool VEC, int AT_ONCE>
__global__ void __launch_bounds__(kBwdThreads) combine_bwd_kernel(CombineArgs a) {
  __shared__ float part[AT_ONCE][kBwdThreads / 32];
  grid_dependency_wait();
  grid_dependents_go();
  const int t = static_cast<int>(blockIdx.x);
  const int64_t first = static_cast<int64_t>(t) * a.k;
  const TR* rows = static_cast<const TR*>(a.rows);
  TR* d_rows = static_cast<TR*>(a.d_rows);
  const TO* d_out = static_cast<const TO*>(a.out) + t * a.ld_out;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j0 = 0; j0 < a.k; j0 += AT_ONCE) {
    float dot[AT_ONCE], w[AT_ONCE];
    int s[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      dot[j] = 0.0f;
      s[j] = j0 + j < a.k ? __ldg(a.slot + first + j0 + j) : -1;
      if (s[j] >= a.R) s[j] = -1;
      w[j] = s[j] >= 0 ? __ldg(a.weight + first + j0 + j) : 0.0f;
    }
    for (int c0 = 0; c0 < a.D; c0 += kBwdThreads * kCols) {
      const int c = c0 + static_cast<int>(threadIdx.x) * (VEC ? kCols : 1);
      if (c >= a.D) break;
      Cols<TO, VEC, kBwdThreads> d;
      Cols<TR, VEC, kBwdThreads> v[AT_ONCE];
      d.load(d_out, c, a.D);
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
        if (s[j] >= 0) v[j].load(rows + s[j] * a.ld_rows, c, a.D);
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        if (s[j] < 0) continue;
        float g[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          dot[j] = fmaf(d.at(i), v[j].at(i), dot[j]);
          g[i] = w[j] * d.at(i);
        }
        store_cols<VEC, kBwdThreads>(d_rows + s[j] * a.ld_d_rows, c, a.D, g);
      }
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
#pragma unroll
      for (int i = 16; i; i >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], i);
      if (lane == 0) part[j][warp] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < AT_ONCE && j0 + static_cast<int>(threadIdx.x) < a.k) {
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
  const int parts = (a.D + kThreads * kCols - 1) / (kThreads * kCols);
  const int64_t grid = static_cast<int64_t>(a.T) * parts;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const cudaError_t e = by(a.rows_bf16, [&](auto r) {
    return by(a.x_bf16, [&](auto x) {
      return by(a.out_bf16, [&](auto o) {
        using R = decltype(r);
        using X = decltype(x);
        using O = decltype(o);
        return launch_pdl(vec ? combine_kernel<R, X, O, true> : combine_kernel<R, X, O, false>,
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
      const auto kernel =
          a.k > 4 ? (vec ? combine_bwd_kernel<R, O, true, 8> : combine_bwd_kernel<R, O, false, 8>)
                  : (vec ? combine_bwd_kernel<R, O, true, 4> : combine_bwd_kernel<R, O, false, 4>);
      return launch_pdl(kernel,
                        dim3(static_cast<unsigned>(a.T)), dim3(kBwdThreads), 0, stream, a);
    });
  });
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace g07
