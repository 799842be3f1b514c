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
// A row is read once, and its sums are taken over the block while it stays on
// the chip, so memory should bound both; it bounds the forward pass.  Measured:
// forward 2047 x 4096 27.5 us (5.5 TB/s, 81 % of the measured copy rate); gradient
// 8192 x 4096, BF16 stream, 130 us (4.1 TB/s, 61 %), 1000 x 3001, FP32, 28 us
// (2.3 TB/s), 4096 x 8192 over clusters, BF16 stream, 217 us (2.5 TB/s).
#include "kernels.h"
#include "layer.h"
#include "sm103_ptx.cuh"

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

// ------------------------------------------------- gradient, rows by copies
//
// The gradient: one block per SM or more walks the rows, and each thread copies
// its own 8 columns of the next rows into a ring in shared memory (cp.async)
// while the block works on the present one, so the row's sums, each a barrier,
// cost no memory time.  Two barriers a row: the last sums of a row and the first
// of the next one, sum(y^2), go through one.  Rows of more than 4096 elements
// (or of more bytes than three stages hold) are shared by the blocks of a
// cluster, which exchange their sums through distributed shared memory.  A
// thread's columns are its own for all its rows: their weights and their three
// column sums stay in registers.  Arithmetic in pairs (one instruction for two
// FP32 operations).
//
// One row at a time by plain loads took 372 us at 8192 x 4096, this ring 147, and
// 130 with the usual operands in code of their own.  The build of 147 us took 105
// without its copies and 101 without its stores as well.  So the block's own work
// sets most of the time, and it is waiting (4096 x 4096, counters: 1.3 of 4
// instructions a cycle, most stalls on shared memory, then on loads).

constexpr int kRingWidth = 4096;  // columns of a block
constexpr int kMaxParts = 8;      // blocks of a cluster
constexpr int kRingBytes = 220 * 1024;

// Two FP32 numbers in one 64-bit register.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ Pair both(float v) { return pair(v, v); }
__device__ __forceinline__ void unpair(Pair v, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum2(const Pair (&v)[2]) {
  float a, b, c, d;
  unpair(v[0], &a, &b);
  unpair(v[1], &c, &d);
  return (a + b) + (c + d);
}
__device__ __forceinline__ void pairs_of(const float (&v)[8], Pair (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pair(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void floats_of(const Pair (&p)[4], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(p[i], &v[2 * i], &v[2 * i + 1]);
}

// Sums of 2 (or 4) values over the block, in every thread, in a fixed order.
// The values share the butterfly: a step sends the half of them that the other
// lane keeps.  buf: 32 (64) floats; entries of absent warps stay zero.
__device__ __forceinline__ void block_sums2(float (&v)[2], float* buf) {
  const int lane = threadIdx.x & 31;
  float a = lane & 16 ? v[1] : v[0];
  a += __shfl_xor_sync(0xFFFFFFFFu, lane & 16 ? v[0] : v[1], 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  if ((lane & 15) == 0) buf[lane + (threadIdx.x >> 5)] = a;  // [value][16 warps]
  __syncthreads();
  a = buf[lane];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  v[0] = __shfl_sync(0xFFFFFFFFu, a, 0);
  v[1] = __shfl_sync(0xFFFFFFFFu, a, 16);
}
__device__ __forceinline__ void block_sums3(float (&v)[3], float* buf) {
  const int lane = threadIdx.x & 31;
  float a = lane & 16 ? v[2] : v[0], b = lane & 16 ? 0.0f : v[1];
  a += __shfl_xor_sync(0xFFFFFFFFu, lane & 16 ? v[0] : v[2], 16);
  b += __shfl_xor_sync(0xFFFFFFFFu, lane & 16 ? v[1] : 0.0f, 16);
  const float keep = lane & 8 ? b : a, send = lane & 8 ? a : b;
  a = keep + __shfl_xor_sync(0xFFFFFFFFu, send, 8);  // lanes 0, 8, 16: values 0, 1, 2
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  if ((lane & 7) == 0) buf[2 * lane + (threadIdx.x >> 5)] = a;  // [value][16 warps]
  __syncthreads();
  const float2 w = *reinterpret_cast<const float2*>(buf + 2 * lane);
  a = w.x + w.y;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  v[0] = __shfl_sync(0xFFFFFFFFu, a, 0);
  v[1] = __shfl_sync(0xFFFFFFFFu, a, 8);
  v[2] = __shfl_sync(0xFFFFFFFFu, a, 16);
}

// Sums of the blocks' sums over the cluster, by rank: each block leaves its own
// in every block's `box` ([rank][4 values]).  Boxes alternate like the buffers.
template <int N>
__device__ __forceinline__ void cluster_sums(float (&v)[N], float* box, int parts, uint32_t rank) {
  if (parts == 1) return;
  if (threadIdx.x < static_cast<unsigned>(parts)) {
    const uint32_t to = map_to_rank(smem_u32(box + rank * 4), threadIdx.x);
#pragma unroll
    for (int i = 0; i < N; ++i) st_cluster_u32(to + 4 * i, __float_as_uint(v[i]));
  }
  __syncwarp();
  cluster_sync();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int r = 0; r < parts; ++r)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += box[r * 4 + i];
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

// One operand's rows in the ring.  VEC: a thread copies what it reads itself,
// 16-byte piece i at (i * blockDim.x + t) * 16.  Else rows start anywhere: the
// 16-byte granules that hold the row are copied by the block and read from the
// row's offset in its first granule (each granule holds bytes of the row).
template <typename T, bool VEC>
struct RingRows {
  const uint8_t* next;    // the next row to copy (of this thread's first piece, VEC)
  int64_t stride;         // bytes from a row of this block to its next one
  int slot;               // offset in a stage
  uint32_t low, ld_low;   // low address bits of row 0, bytes from row to row

  static __host__ __device__ constexpr int bytes(int threads) {
    return threads * 8 * static_cast<int>(sizeof(T)) + (VEC ? 0 : 32);
  }
  // Rows first, first + step, .. of a matrix, from column col0.
  __device__ __forceinline__ void init(const void* base, int64_t ld, int col0, int first, int step,
                                       int at) {
    const T* row0 = static_cast<const T*>(base) + col0;
    const T* start = row0 + first * ld;
    next = reinterpret_cast<const uint8_t*>(VEC ? start + own_col<true>(0) : start);
    stride = ld * static_cast<int64_t>(sizeof(T)) * step;
    slot = at;
    low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row0));
    ld_low = static_cast<uint32_t>(ld * sizeof(T));
  }
  __device__ __forceinline__ void copy(uint8_t* stage, int D) const {
    if constexpr (VEC) {
      if (own_col<true>(0) < D) {
        uint8_t* to = stage + slot + threadIdx.x * 16;
        cp_async_16(to, next);
        if constexpr (sizeof(T) == 4) cp_async_16(to + blockDim.x * 16, next + 16);
      }
    } else {
      const uintptr_t a = reinterpret_cast<uintptr_t>(next);
      const uintptr_t end = a + D * static_cast<int>(sizeof(T));
#pragma unroll
      for (int i = 0; i <= static_cast<int>(sizeof(T)) / 2; ++i) {
        const int at = (i * blockDim.x + threadIdx.x) * 16;
        const uintptr_t from = (a & ~static_cast<uintptr_t>(15)) + at;
        if (from < end) cp_async_16(stage + slot + at, reinterpret_cast<const void*>(from));
      }
    }
  }
  __device__ __forceinline__ void read(const uint8_t* stage, uint32_t row, int D,
                                       Pair (&p)[4]) const {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    if constexpr (!VEC) {
      const T* r = reinterpret_cast<const T*>(stage + slot + ((low + row * ld_low) & 15u));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (own_col<false>(e) < D) v[e] = to_f32(r[own_col<false>(e)]);
    } else if (own_col<true>(0) < D) {
      const uint4 a = *reinterpret_cast<const uint4*>(stage + slot + threadIdx.x * 16);
      if constexpr (sizeof(T) == 2) {
        v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
        v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
      } else {
        const uint4 b = *reinterpret_cast<const uint4*>(stage + slot +
                                                        (blockDim.x + threadIdx.x) * 16);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
        v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
      }
    }
    pairs_of(v, p);
  }
};

template <typename X, typename Y, typename H, bool VEC>
int ring_stage_bytes(int threads, bool has_y, bool has_dxo, bool has_h, bool full_gate) {
  return RingRows<X, VEC>::bytes(threads) * (has_dxo ? 2 : 1) +
         (has_y ? RingRows<Y, VEC>::bytes(threads) : 0) +
         (has_h ? RingRows<H, VEC>::bytes(threads) : 0) +
         (full_gate ? RingRows<float, VEC>::bytes(threads) : 0);
}

// ALL: every operand and both norms are there, and no gate or one value per
// column: the row's work is then one straight piece of code (8192 x 4096, BF16
// stream: 130 us, in the general form 147).  Everything else takes the general
// form: without a post norm 141 to 144 us at that size.
template <typename X, typename Y, typename H, bool VEC, bool ALL>
__global__ void __launch_bounds__(512, 1)
norm_gate_bwd_kernel(NormArgs p, int parts, int part_cols, int stages, int stage_bytes,
                     float* partial) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float sums[2][32 + 64];  // alternate from row to row
  __shared__ __align__(16) float boxes[2][2][kMaxParts * 4];
  // this block's columns: D of them from col0
  const uint32_t rank = parts > 1 ? cluster_ctarank() : 0u;
  const int col0 = static_cast<int>(rank) * part_cols;
  const int D = min(part_cols, p.D - col0), T = p.T;
  const int slot = static_cast<int>(blockIdx.x) / parts;
  const bool has_y = ALL || p.y != nullptr, has_h = ALL || p.dh != nullptr;
  const bool has_dxo = ALL || p.d_x_out != nullptr, post = ALL || p.w_post != nullptr;
  const bool row_gate = !ALL && p.gate != nullptr && p.gate_col == 0;
  const bool col_gate = p.gate != nullptr && p.gate_col != 0 && p.gate_row == 0;
  const bool full_gate = !ALL && p.gate != nullptr && p.gate_col != 0 && p.gate_row != 0;
  for (int i = threadIdx.x; i < 2 * 96; i += blockDim.x) (&sums[0][0])[i] = 0.0f;
  __syncthreads();
  if (parts > 1) cluster_sync();  // every block of the cluster runs
  grid_dependency_wait();
  grid_dependents_go();

  const int threads = blockDim.x;
  const int step = static_cast<int>(gridDim.x) / parts;
  int row = slot, ahead = row;
  RingRows<X, VEC> rx, ro;
  RingRows<Y, VEC> ry;
  RingRows<H, VEC> rh;
  RingRows<float, VEC> rg;
  int at = 0;
  rx.init(p.x, p.ldx, col0, row, step, at);
  at += rx.bytes(threads);
  ry.init(p.y, p.ldy, col0, row, step, at);
  at += has_y ? ry.bytes(threads) : 0;
  ro.init(p.d_x_out, p.ld_d_x_out, col0, row, step, at);
  at += has_dxo ? ro.bytes(threads) : 0;
  rh.init(p.dh, p.ld_dh, col0, row, step, at);
  at += has_h ? rh.bytes(threads) : 0;
  rg.init(p.gate, p.gate_row, col0, row, step, at);

  uint8_t* fill = ring;  // the stage of row `ahead`
  uint8_t* const ring_end = ring + stages * stage_bytes;
  // A row's copies in three parts, started at different places of an earlier
  // row's work: all at once they fill the load queue and stop the block.
  auto issue_block = [&]() {
    if (ahead < T) {
      if (has_y) ry.copy(fill, D);
      rx.copy(fill, D);
    }
  };
  auto issue_grads = [&]() {
    if (ahead < T && has_h) rh.copy(fill, D);
  };
  auto issue_rest = [&]() {
    if (ahead < T) {
      if (has_dxo) ro.copy(fill, D);
      if (full_gate) rg.copy(fill, D);
    }
    cp_async_commit();
    ahead = ahead < T - step ? ahead + step : T;  // (row numbers stay in 32 bits)
    rx.next += rx.stride;
    ry.next += ry.stride;
    ro.next += ro.stride;
    rh.next += rh.stride;
    rg.next += rg.stride;
    fill += stage_bytes;
    if (fill == ring_end) fill = ring;
  };
  for (int s = 0; s < stages - 1; ++s) {
    issue_block();
    issue_grads();
    issue_rest();
  }

  // The gate and w_post act on a column as one factor, gw = gate * w_post.
  // Without a gate, or with one value per column, both column sums come from
  // sum(du n): dw_post = gate * that, dgate = w_post * that.
  float v[8];
  Pair w2[4], w1[4], g[4], gw[4];
  auto weights = [&](const float* src, Pair (&w)[4]) {
    if (src)
      own_load<VEC>(src, D, v);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 1.0f;
    pairs_of(v, w);
  };
  weights(p.w_post ? p.w_post + col0 : nullptr, w2);
  weights(p.w_pre ? p.w_pre + col0 : nullptr, w1);
  weights(col_gate ? p.gate + col0 : nullptr, g);
#pragma unroll
  for (int i = 0; i < 4; ++i) gw[i] = mul2(g[i], w2[i]);
  float next_gate = row_gate && row < T ? p.gate[row * p.gate_row] : 1.0f;
  Pair sum_post[4] = {}, sum_pre[4] = {};
  const float inv_d = 1.0f / p.D;
  const Pair alpha = both(p.alpha);
  auto squares = [&](const Pair (&q)[4]) {
    Pair a[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i & 1] = fma2(q[i], q[i], a[i & 1]);
    return sum2(a);
  };
  auto scale_of = [&](float sum) { return post ? rsqrtf(sum * inv_d + p.eps) : 1.0f; };
  // The row after the present one has landed (its copies were all started one
  // row ago or, with four stages, two).
  auto landed = [&]() {
    if (stages == 4)
      cp_async_wait<1>();
    else
      cp_async_wait<0>();
  };

  const uint8_t* st = ring;
  Pair y[4] = {}, y_next[4] = {};
  landed();
  __syncthreads();  // (other threads' copies, for rows off the 16-byte grid)
  if (has_y) ry.read(st, row, D, y);
  float first[2] = {squares(y), 0.0f};
  block_sums2(first, sums[1]);
  cluster_sums(first, boxes[1][0], parts, rank);
  float r2 = scale_of(first[0]);

  for (int odd = 0; row < T; odd ^= 1) {
    // the stage of the row before this one takes the row after the ring's others
    issue_block();
    Pair u[4], du[4] = {}, h[4] = {};
    rx.read(st, row, D, u);
    if (has_h) rh.read(st, row, D, h);
    if (full_gate) rg.read(st, row, D, g);
    const bool more = row < T - step;
    if (row_gate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = both(next_gate);
      if (more) next_gate = p.gate[static_cast<int64_t>(row + step) * p.gate_row];
    }
    if (row_gate || full_gate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) gw[i] = mul2(g[i], w2[i]);
    }
    const Pair r2p = both(r2);
    Pair b0[2] = {0, 0}, b1[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = mul2(y[i], r2p);  // n from here on
      u[i] = mul2(alpha, u[i]);
      if (has_y) u[i] = fma2(gw[i], y[i], u[i]);
      b0[i & 1] = fma2(u[i], u[i], b0[i & 1]);
      b1[i & 1] = fma2(mul2(h[i], w1[i]), u[i], b1[i & 1]);
    }
    if (has_dxo) ro.read(st, row, D, du);
    landed();  // the next row, before the barrier that lets others read it
    float b[2] = {sum2(b0), sum2(b1)};
    block_sums2(b, sums[odd]);
    cluster_sums(b, boxes[odd][0], parts, rank);
    issue_grads();
    float r1 = 0.0f, c1 = 0.0f;
    if (has_h) {
      r1 = rsqrtf(b[0] * inv_d + p.eps);
      c1 = r1 * (b[1] * inv_d);
    }
    const Pair r1p = both(r1), c1p = both(-c1);
    Pair t0[2] = {0, 0}, t1[2] = {0, 0}, o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (has_h) {
        u[i] = mul2(u[i], r1p);
        sum_pre[i] = fma2(h[i], u[i], sum_pre[i]);
        du[i] = fma2(mul2(h[i], w1[i]), r1p, du[i]);
        du[i] = fma2(mul2(u[i], r1p), c1p, du[i]);
      }
      o[i] = mul2(alpha, du[i]);
      u[i] = mul2(du[i], gw[i]);
      t0[i & 1] = fma2(u[i], y[i], t0[i & 1]);
    }
    floats_of(o, v);
    own_store<VEC>(static_cast<X*>(p.dx) + row * p.ld_dx + col0, D, v);
    issue_rest();
    if (!row_gate && !full_gate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum_post[i] = fma2(du[i], y[i], sum_post[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum_post[i] = fma2(mul2(g[i], du[i]), y[i], sum_post[i]);
        o[i] = mul2(du[i], mul2(y[i], w2[i]));
        t1[i & 1] = fma2(du[i], mul2(y[i], w2[i]), t1[i & 1]);
      }
      if (full_gate) {
        floats_of(o, v);
        own_store<VEC>(p.dgate + row * p.gate_row + col0, D, v);
      }
    }
    st += stage_bytes;
    if (st == ring_end) st = ring;
    if (has_y && more) ry.read(st, row + step, D, y_next);
    // always: the barrier also says that this row's stage has been read
    float t[3] = {sum2(t0), sum2(t1), squares(y_next)};
    block_sums3(t, sums[odd] + 32);
    cluster_sums(t, boxes[odd][1], parts, rank);
    if (has_y) {
      if (row_gate && threadIdx.x == 0 && rank == 0) p.dgate[row * p.gate_row] = t[1];
      const Pair c2p = both(-(t[0] * inv_d) * r2);
#pragma unroll
      for (int i = 0; i < 4; ++i)  // without w_post dy = gate du: 0 times y need not be 0
        o[i] = post ? fma2(y[i], c2p, mul2(u[i], r2p)) : u[i];
      floats_of(o, v);
      own_store<VEC>(p.dy + row * p.ld_dy + col0, D, v);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = y_next[i];
    r2 = scale_of(t[2]);
    row = more ? row + step : T;
  }
  if (parts > 1) cluster_sync();  // no block leaves while others write its boxes
  if (partial == nullptr) return;
  float* out = partial + static_cast<int64_t>(slot) * 3 * p.D + col0;
  auto leave = [&](const Pair (&sum)[4], float* to) {
    floats_of(sum, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (own_col<VEC>(e) < D) to[own_col<VEC>(e)] = v[e];
  };
  leave(sum_pre, out + p.D);
  if (col_gate) {
    Pair t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[i] = mul2(sum_post[i], w2[i]);
      sum_post[i] = mul2(sum_post[i], g[i]);
    }
    leave(t, out + 2 * p.D);
  }
  leave(sum_post, out);
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

// Calls f<X, Y, H, VEC>() for the operands' types and alignment.
template <bool VEC, typename F>
auto by_types(const NormArgs& a, F f) {
  using B = __nv_bfloat16;
  if (a.x_bf16)
    return a.y_bf16 ? (a.dh_bf16 ? f.template go<B, B, B, VEC>() : f.template go<B, B, float, VEC>())
                    : (a.dh_bf16 ? f.template go<B, float, B, VEC>()
                                 : f.template go<B, float, float, VEC>());
  return a.y_bf16 ? (a.dh_bf16 ? f.template go<float, B, B, VEC>()
                               : f.template go<float, B, float, VEC>())
                  : (a.dh_bf16 ? f.template go<float, float, B, VEC>()
                               : f.template go<float, float, float, VEC>());
}
template <typename F>
auto by_types(const NormArgs& a, F f) {
  return vector_rows(a) ? by_types<true>(a, f) : by_types<false>(a, f);
}

void bwd_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, const NormBwdPlan& b,
                cudaStream_t st) {
  *cfg = cudaLaunchConfig_t{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(b.parts);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg->gridDim = dim3(static_cast<unsigned>(b.slots * b.parts));
  cfg->blockDim = dim3(static_cast<unsigned>(b.threads));
  cfg->dynamicSmemBytes = static_cast<size_t>(b.stages) * b.stage_bytes;
  cfg->stream = st;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

using BwdFunction = void (*)(NormArgs, int, int, int, int, float*);
// The kernel for these operands, with leave to use the whole ring.
struct BwdKernel {
  const NormArgs& a;
  BwdFunction* kernel;
  template <typename X, typename Y, typename H, bool VEC>
  cudaError_t go() const {
    const bool all = a.y != nullptr && a.dh != nullptr && a.d_x_out != nullptr &&
                     a.w_post != nullptr && (a.gate == nullptr || a.gate_row == 0);
    static std::atomic<uint64_t> allowed[2] = {};
    *kernel = VEC && all ? norm_gate_bwd_kernel<X, Y, H, VEC, VEC>
                         : norm_gate_bwd_kernel<X, Y, H, VEC, false>;
    return allow_shared(*kernel, kRingBytes, &allowed[VEC && all]);
  }
};
struct BwdStage {
  const NormArgs& a;
  int threads;
  template <typename X, typename Y, typename H, bool VEC>
  int go() const {
    const bool full = a.gate != nullptr && a.gate_col != 0 && a.gate_row != 0;
    return ring_stage_bytes<X, Y, H, VEC>(threads, a.y != nullptr, a.d_x_out != nullptr,
                                          a.dh != nullptr, full);
  }
};

}  // namespace

cudaError_t launch_norm_gate(const NormArgs& a, cudaStream_t stream) {
  using B = __nv_bfloat16;
  const cudaError_t e = a.x_bf16 ? (a.y_bf16 ? forward<B, B>(a, stream) : forward<B, float>(a, stream))
                                 : (a.y_bf16 ? forward<float, B>(a, stream)
                                             : forward<float, float>(a, stream));
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t norm_gate_bwd_plan(const NormArgs& a, const LayerDevice& dev, NormBwdPlan* plan) {
  NormBwdPlan& b = *plan;
  // The fewest blocks to a row whose columns fit their registers and whose
  // ring holds three rows (five FP32 operands of 4096 columns take 80 KB).
  for (int parts = (a.D + kRingWidth - 1) / kRingWidth;; ++parts) {
    if (parts > kMaxParts) return cudaErrorInvalidValue;
    b.part_cols = ((a.D + parts - 1) / parts + 7) / 8 * 8;
    b.parts = (a.D + b.part_cols - 1) / b.part_cols;  // (no block without columns)
    b.threads = threads_for(b.part_cols, 8);
    b.stage_bytes = by_types(a, BwdStage{a, b.threads});
    if (3 * b.stage_bytes <= kRingBytes) break;
  }
  b.stages = 4 * b.stage_bytes <= kRingBytes ? 4 : 3;
  // As many as are resident at once, so that a block's rows follow one another
  // through its ring: by shared memory, and by 512 threads an SM of at most 128
  // registers; clusters as the occupancy calculator says.
  const int smem = b.stages * b.stage_bytes;
  const int by_smem = kRingBytes / (smem + 2048), by_threads = 512 / b.threads;
  int per_sm = by_smem < by_threads ? by_smem : by_threads;
  if (per_sm < 1) per_sm = 1;
  int slots = dev.sms / b.parts * per_sm;
  b.slots = slots;
  if (b.parts > 1) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    bwd_config(&cfg, attr, b, nullptr);
    cfg.numAttrs = 1;
    int clusters = 0;
    BwdFunction kernel = nullptr;
    cudaError_t e = by_types(a, BwdKernel{a, &kernel});
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    if (clusters < slots) slots = clusters;
  }
  b.slots = a.T < slots ? a.T : slots;
  return cudaSuccess;
}

cudaError_t launch_norm_gate_bwd(const NormArgs& a, const NormBwdPlan& plan, float* partial,
                                 cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  bwd_config(&cfg, attr, plan, stream);
  if (plan.parts == 1) {
    attr[0] = attr[1];  // no cluster
    cfg.numAttrs = 1;
  }
  BwdFunction kernel = nullptr;
  cudaError_t e = by_types(a, BwdKernel{a, &kernel});
  if (e == cudaSuccess)
    e = cudaLaunchKernelEx(&cfg, kernel, a, plan.parts, plan.part_cols, plan.stages,
                           plan.stage_bytes, partial);
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
