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

// ------------------------------------------------- gradient, rows by copies
//
// The gradient for rows of at most 4096 elements: one block per SM or more
// walks the rows, and each thread copies its own 8 columns of the next rows
// into a ring in shared memory (cp.async) while the block works on the present
// one, so the row's three sums, each a barrier, cost no memory time.  A
// thread's columns are its own for all its rows: their weights and their three
// column sums stay in registers.

constexpr int kRingWidth = 4096;
constexpr int kRingStages = 3;
constexpr int kRingBytes = 220 * 1024;

// Sums over the block as block_sums, with 16 warps' entries always read (those
// of absent warps stay zero).
template <int N>
__device__ __forceinline__ void block_sums16(float (&v)[N], float (*buf)[16]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i][threadIdx.x >> 5] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float4* b = reinterpret_cast<const float4*>(buf[i]);
    const float4 a = b[0], c = b[1], d = b[2], e = b[3];
    v[i] = (((a.x + a.y) + (a.z + a.w)) + ((c.x + c.y) + (c.z + c.w))) +
           (((d.x + d.y) + (d.z + d.w)) + ((e.x + e.y) + (e.z + e.w)));
  }
}

// This thread's 8 columns: adjacent (VEC, rows on 16 bytes) or blockDim.x apart.
template <bool VEC>
__device__ __forceinline__ int own_col(int e) {
  const int t = static_cast<int>(threadIdx.x);
  return VEC ? t * 8 + e : e * static_cast<int>(blockDim.x) + t;
}
template <bool VEC, typename T>
__device__ __forceinline__ void own_load(const T* row, int D, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  if constexpr (VEC) {
    if (own_col<VEC>(0) < D) load_vec(row + own_col<VEC>(0), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (own_col<VEC>(e) < D) v[e] = to_f32(row[own_col<VEC>(e)]);
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void own_store(T* row, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    if (own_col<VEC>(0) < D) store_vec(row + own_col<VEC>(0), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (own_col<VEC>(e) < D) row[own_col<VEC>(e)] = from_f32<T>(v[e]);
  }
}

// Whether rows of T go through the ring (2-byte elements off the 16-byte grid
// are below the smallest asynchronous copy, and are loaded when used).
template <typename T, bool VEC>
constexpr bool kRinged = VEC || sizeof(T) == 4;

// Bytes of a row in the ring.  Adjacent columns: 16-byte pieces, piece i of
// thread t at (i * blockDim.x + t) * 16; else element e of t at
// (e * blockDim.x + t) * 4.
template <typename T, bool VEC>
__host__ __device__ constexpr int ring_row_bytes(int threads) {
  return kRinged<T, VEC> ? threads * 8 * static_cast<int>(sizeof(T)) : 0;
}
template <bool VEC, typename T>
__device__ __forceinline__ void ring_copy(uint8_t* slot, const T* row, int D) {
  if constexpr (VEC) {
    if (own_col<VEC>(0) < D)
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        cp_async_16(slot + (i * blockDim.x + threadIdx.x) * 16,
                    row + own_col<VEC>(0) + i * (16 / sizeof(T)));
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (own_col<VEC>(e) < D)
        cp_async_4(slot + (e * blockDim.x + threadIdx.x) * 4, row + own_col<VEC>(e));
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void ring_read(const uint8_t* slot, const T* row, int D,
                                          float (&v)[8]) {
  if constexpr (!kRinged<T, VEC>) {
    own_load<VEC>(row, D, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    if constexpr (!VEC) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (own_col<VEC>(e) < D)
          v[e] = *reinterpret_cast<const float*>(slot + (e * blockDim.x + threadIdx.x) * 4);
    } else if (own_col<VEC>(0) < D) {
      const uint4 a = *reinterpret_cast<const uint4*>(slot + threadIdx.x * 16);
      if constexpr (sizeof(T) == 2) {
        v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
        v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
      } else {
        const uint4 b = *reinterpret_cast<const uint4*>(slot + (blockDim.x + threadIdx.x) * 16);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
        v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
      }
    }
  }
}

// Offsets of the operands in a stage of the ring, x, y, d_x_out, dh, gate.
struct RingLayout {
  int y, d_x_out, dh, gate, bytes;
};
template <typename X, typename Y, typename H, bool VEC>
__host__ __device__ RingLayout ring_layout(int threads, bool has_y, bool has_dxo, bool has_h,
                                           bool full_gate) {
  RingLayout l;
  l.y = ring_row_bytes<X, VEC>(threads);
  l.d_x_out = l.y + (has_y ? ring_row_bytes<Y, VEC>(threads) : 0);
  l.dh = l.d_x_out + (has_dxo ? ring_row_bytes<X, VEC>(threads) : 0);
  l.gate = l.dh + (has_h ? ring_row_bytes<H, VEC>(threads) : 0);
  l.bytes = l.gate + (full_gate ? ring_row_bytes<float, VEC>(threads) : 0);
  return l;
}

template <typename X, typename Y, typename H, bool VEC, int STAGES>
__global__ void __launch_bounds__(512, 1)
norm_gate_bwd_ring_kernel(NormArgs p, float* partial) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float sums[2][3][2][16];  // alternate from row to row
  const int D = p.D;
  const bool has_y = p.y != nullptr, has_h = p.dh != nullptr, has_dxo = p.d_x_out != nullptr;
  const bool row_gate = p.gate != nullptr && p.gate_col == 0;
  const bool col_gate = p.gate != nullptr && p.gate_col != 0 && p.gate_row == 0;
  const bool full_gate = p.gate != nullptr && p.gate_col != 0 && p.gate_row != 0;
  const RingLayout lay = ring_layout<X, Y, H, VEC>(blockDim.x, has_y, has_dxo, has_h, full_gate);
  for (int i = threadIdx.x; i < 2 * 3 * 2 * 16; i += blockDim.x) (&sums[0][0][0][0])[i] = 0.0f;
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_go();

  auto x_row = [&](int64_t r) { return static_cast<const X*>(p.x) + r * p.ldx; };
  auto y_row = [&](int64_t r) { return static_cast<const Y*>(p.y) + r * p.ldy; };
  auto o_row = [&](int64_t r) { return static_cast<const X*>(p.d_x_out) + r * p.ld_d_x_out; };
  auto h_row = [&](int64_t r) { return static_cast<const H*>(p.dh) + r * p.ld_dh; };
  auto issue = [&](int64_t r, uint8_t* st) {
    if (r < p.T) {
      ring_copy<VEC>(st, x_row(r), D);
      if (has_y) ring_copy<VEC>(st + lay.y, y_row(r), D);
      if (has_dxo) ring_copy<VEC>(st + lay.d_x_out, o_row(r), D);
      if (has_h) ring_copy<VEC>(st + lay.dh, h_row(r), D);
      if (full_gate) ring_copy<VEC>(st + lay.gate, p.gate + r * p.gate_row, D);
    }
    cp_async_commit();
  };
  const int64_t step = gridDim.x;
  int64_t row = blockIdx.x;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(row + s * step, ring + s * lay.bytes);

  float w2[8], w1[8], g[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w2[e] = w1[e] = g[e] = 1.0f;
  if (p.w_post) own_load<VEC>(p.w_post, D, w2);
  if (p.w_pre) own_load<VEC>(p.w_pre, D, w1);
  if (col_gate) own_load<VEC>(p.gate, D, g);
  float next_gate = row_gate && row < p.T ? p.gate[row * p.gate_row] : 1.0f;
  float sum_post[8] = {}, sum_pre[8] = {}, sum_gate[8] = {};
  const float inv_d = 1.0f / D;
  int s = 0, odd = 0;
  for (; row < p.T; row += step, odd ^= 1) {
    // the stage that this thread read one row ago takes the row after the
    // ring's others
    issue(row + (STAGES - 1) * step, ring + (s == 0 ? STAGES - 1 : s - 1) * lay.bytes);
    cp_async_wait<STAGES - 1>();
    const uint8_t* st = ring + s * lay.bytes;
    if (++s == STAGES) s = 0;
    float y[8], u[8], du[8], h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = du[e] = h[e] = 0.0f;
    ring_read<VEC>(st, x_row(row), D, u);
    if (has_y) ring_read<VEC>(st + lay.y, y_row(row), D, y);
    if (has_dxo) ring_read<VEC>(st + lay.d_x_out, o_row(row), D, du);
    if (has_h) ring_read<VEC>(st + lay.dh, h_row(row), D, h);
    if (full_gate) ring_read<VEC>(st + lay.gate, p.gate + row * p.gate_row, D, g);
    if (row_gate) {
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = next_gate;
      if (row + step < p.T) next_gate = p.gate[(row + step) * p.gate_row];
    }
    float r2 = 1.0f;
    if (p.w_post) {
      float a[1] = {0.0f};
#pragma unroll
      for (int e = 0; e < 8; ++e) a[0] = fmaf(y[e], y[e], a[0]);
      block_sums16(a, sums[odd][0]);
      r2 = rsqrtf(a[0] * inv_d + p.eps);
    }
    float b[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] *= r2;  // n from here on
      u[e] = has_y ? fmaf(p.alpha, u[e], g[e] * (y[e] * w2[e])) : p.alpha * u[e];
      b[0] = fmaf(u[e], u[e], b[0]);
      b[1] = fmaf(h[e] * w1[e], u[e], b[1]);
    }
    float r1 = 0.0f, c1 = 0.0f;
    if (has_h) {
      block_sums16(b, sums[odd][1]);
      r1 = rsqrtf(b[0] * inv_d + p.eps);
      c1 = r1 * r1 * (b[1] * inv_d);
    }
    float t[2] = {0.0f, 0.0f}, o[8], dg[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (has_h) {
        sum_pre[e] = fmaf(h[e] * u[e], r1, sum_pre[e]);
        du[e] = fmaf(r1, fmaf(h[e], w1[e], -u[e] * c1), du[e]);
      }
      o[e] = p.alpha * du[e];
      const float dp = g[e] * du[e];
      sum_post[e] = fmaf(dp, y[e], sum_post[e]);
      dg[e] = du[e] * (y[e] * w2[e]);
      sum_gate[e] += dg[e];
      u[e] = dp * w2[e];
      t[0] = fmaf(u[e], y[e], t[0]);
      t[1] += dg[e];
    }
    own_store<VEC>(static_cast<X*>(p.dx) + row * p.ld_dx, D, o);
    if (!has_y) continue;
    if (full_gate) own_store<VEC>(p.dgate + row * p.gate_row, D, dg);
    float c2 = 0.0f;
    if (p.w_post || row_gate) {
      block_sums16(t, sums[odd][2]);
      if (p.w_post) c2 = t[0] * inv_d;
      if (row_gate && threadIdx.x == 0) p.dgate[row * p.gate_row] = t[1];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = r2 * (u[e] - y[e] * c2);
    own_store<VEC>(p.dy + row * p.ld_dy, D, o);
  }
  if (partial == nullptr) return;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 3 * D;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (own_col<VEC>(e) < D) {
      const int c = own_col<VEC>(e);
      out[c] = sum_post[e];
      out[D + c] = sum_pre[e];
      out[2 * D + c] = sum_gate[e];
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

// The ring kernel's launch; with `slots` null only its block count per SM is
// taken: by shared memory, and by 512 threads an SM of at most 128 registers.
template <typename X, typename Y, typename H, bool VEC>
cudaError_t backward_ring(const NormArgs& a, int slots, float* partial, cudaStream_t st,
                          int* per_sm) {
  const int threads = threads_for(a.D, 8);
  const bool full = a.gate != nullptr && a.gate_col != 0 && a.gate_row != 0;
  const int stage = ring_layout<X, Y, H, VEC>(threads, a.y != nullptr, a.d_x_out != nullptr,
                                              a.dh != nullptr, full).bytes;
  // (five FP32 operands of 4096 columns take 80 KB a stage)
  const bool three = kRingStages * stage <= kRingBytes;
  const int smem = (three ? kRingStages : 2) * stage;
  if (per_sm) {
    const int by_smem = kRingBytes / (smem + 2048), by_threads = 512 / threads;
    *per_sm = by_smem < by_threads ? by_smem : by_threads;
    if (*per_sm < 1) *per_sm = 1;
    return cudaSuccess;
  }
  void (*kernel)(NormArgs, float*) = three ? norm_gate_bwd_ring_kernel<X, Y, H, VEC, kRingStages>
                                           : norm_gate_bwd_ring_kernel<X, Y, H, VEC, 2>;
  if (smem > 40 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(slots), dim3(threads), smem, st, a, partial);
}

template <typename X, typename Y, typename H>
cudaError_t backward(const NormArgs& a, int slots, float* partial, cudaStream_t st, int* per_sm) {
  const Shape s = shape_for(a);
  if (a.D <= kRingWidth)
    return s.vec == 8 ? backward_ring<X, Y, H, true>(a, slots, partial, st, per_sm)
                      : backward_ring<X, Y, H, false>(a, slots, partial, st, per_sm);
  if (per_sm) {
    *per_sm = 1;
    return cudaSuccess;
  }
  if (s.vec == 1)
    return launch_bwd(norm_gate_bwd_kernel<X, Y, H, 1, 32>, a, s, slots, partial, st);
  if (s.vpt == 2)
    return launch_bwd(norm_gate_bwd_kernel<X, Y, H, 8, 2>, a, s, slots, partial, st);
  return launch_bwd(norm_gate_bwd_kernel<X, Y, H, 8, 4>, a, s, slots, partial, st);
}

cudaError_t backward_typed(const NormArgs& a, int slots, float* partial, cudaStream_t st,
                           int* per_sm) {
  using B = __nv_bfloat16;
  if (a.x_bf16)
    return a.y_bf16 ? (a.dh_bf16 ? backward<B, B, B>(a, slots, partial, st, per_sm)
                                 : backward<B, B, float>(a, slots, partial, st, per_sm))
                    : (a.dh_bf16 ? backward<B, float, B>(a, slots, partial, st, per_sm)
                                 : backward<B, float, float>(a, slots, partial, st, per_sm));
  return a.y_bf16 ? (a.dh_bf16 ? backward<float, B, B>(a, slots, partial, st, per_sm)
                               : backward<float, B, float>(a, slots, partial, st, per_sm))
                  : (a.dh_bf16 ? backward<float, float, B>(a, slots, partial, st, per_sm)
                               : backward<float, float, float>(a, slots, partial, st, per_sm));
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

// As many blocks as are resident at once, so that a block's rows follow one
// another through its ring.
int norm_gate_bwd_slots(const NormArgs& a, const LayerDevice& dev) {
  int per_sm = 1;
  backward_typed(a, 0, nullptr, nullptr, &per_sm);
  const int64_t most = static_cast<int64_t>(dev.sms) * per_sm;
  return static_cast<int>(a.T < most ? a.T : most);
}

cudaError_t launch_norm_gate_bwd(const NormArgs& a, int slots, float* partial,
                                 cudaStream_t stream) {
  const cudaError_t e = backward_typed(a, slots, partial, stream, nullptr);
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
