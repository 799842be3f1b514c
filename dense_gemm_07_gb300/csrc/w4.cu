// w4.cu -- C = act(alpha * A * W + beta * C + bias) for a few rows of A and a
// matrix W of 4-bit codes:
//   W[k][n] = (q[k][n] - z[g][n]) * s[g][n],  g = k / group,
// q and z whole numbers 0..15 (z = 8 without zero points), s BF16.  Also the
// kernels that bring codes into the packed order, quantise a matrix, and write
// W back as BF16.
//
// The product reads K * N / 2 bytes of codes once and does 2 M K N operations
// on them, so at M <= 16 memory bounds it.  Each weight is turned into the
// exact BF16 whole number q - z and multiplied on the tensor cores
// (mma.sync m16n8k16: 16 columns of W by 8 rows of A, FP32 sums), and the
// scale is applied to a group's FP32 sum, so nothing is rounded to fewer bits
// than 32 between the codes and the result.  mma.sync, not tcgen05: an operand
// decoded in registers would have to be stored to tensor memory or shared
// memory first, and at 16 rows the products are a small part of the time.
#include <cuda_bf16.h>

#include "kernels.h"
#include "layer.h"
#include "sm103_ptx.cuh"

namespace g07 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

// Packed order: tiles of 16 columns x 128 rows, 1 KB each, tile (nt, kt) at
// (nt * KT + kt) * 1 KB.  In a tile, word [half][column c][quarter t][block j]
// (32 bits, in that order) holds column 8 * half + c, rows 32 j + 8 t + e,
// e = 0..7; code e sits at bits 4 * (e / 2 + 4 * (e % 2)).  So lane 4c + t of a
// warp reads 16 bytes per half: its share of four 32-row blocks, and
// (word >> 4i) & 0x000F000F is the pair of rows 2i, 2i + 1.
__host__ __device__ __forceinline__ int nibble_shift(int e) { return 4 * (e / 2 + 4 * (e % 2)); }

// The codes at pair i of a word, as two BF16 whole numbers 128 + q: the bits
// 0x4300 | q are exactly 128 + q.
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, int i) {
  return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
}
// Exact: both operands are whole numbers of at most 8 bits.
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight consecutive elements of a row of A from k, zero past K.
__device__ __forceinline__ uint4 load_a8(const __nv_bfloat16* row, int k, int K, bool vec) {
  if (vec && k + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo =
        k + 2 * i < K ? *reinterpret_cast<const uint16_t*>(row + k + 2 * i) : 0u;
    const uint32_t hi =
        k + 2 * i + 1 < K ? *reinterpret_cast<const uint16_t*>(row + k + 2 * i + 1) : 0u;
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One cluster computes CT tiles of 16 columns by up to 8 * NT rows of A; the
// 128-row tiles of K go round over the warps of its blocks.  A warp copies the
// packed tiles of its next steps into a ring in shared memory (cp.async; each
// lane copies the 16-byte pieces that it decodes, so no barrier is needed), STAGES
// - 1 steps ahead.  Every step's groups (GPT of them in 128 rows) come as one
// 32-bit word per column, scale above 128 + z, held by one lane and handed
// round by shuffles.  The warps' sums are added in warp order, the blocks' in
// rank order.
template <int CT, int NT, int GPT, int STAGES>
__global__ void __launch_bounds__(kThreads, 2) w4_kernel(W4Args p, int vec_a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int RED = 8 * NT + 1;             // row of the sums' exchange
  constexpr int MREGS = GPT == 4 ? 2 : 1;     // two groups of 16 columns a register
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int KT = (p.K + kW4TileK - 1) / kW4TileK;
  const int NTILES = (p.N + kW4TileN - 1) / kW4TileN;
  const int G = (p.K + p.group - 1) / p.group;
  const int blocks = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);
  const int nt0 = blockIdx.x * CT;
  const int m0 = blockIdx.y * 8 * NT;
  const int first = rank * kWarps + warp, step = blocks * kWarps;
  grid_dependency_wait();
  grid_dependents_go();

  uint8_t* ring = smem + warp * (STAGES * CT * kW4TileBytes) + lane * 16;
  const uint8_t* tiles =
      p.packed + static_cast<int64_t>(nt0) * KT * kW4TileBytes + lane * 16;
  auto issue = [&](int kt, int s) {
    if (kt < KT) {
#pragma unroll
      for (int c = 0; c < CT; ++c)
        if (c == 0 || nt0 + c < NTILES) {
          const uint8_t* src = tiles + (static_cast<int64_t>(c) * KT + kt) * kW4TileBytes;
          uint8_t* dst = ring + (s * CT + c) * kW4TileBytes;
          cp_async_16(dst, src);
          cp_async_16(dst + 512, src + 512);
        }
    }
    cp_async_commit();
  };
  // This lane's group word of each tile for step kt: column lane % 16, group
  // lane / 16 (+ 2).
  auto load_meta = [&](int kt, uint32_t (&m)[CT][MREGS]) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int r = 0; r < MREGS; ++r) {
        const int grp = kt * GPT + (lane >> 4) + 2 * r;
        const int n = (nt0 + c) * 16 + (lane & 15);
        uint32_t v = 0x4308u;
        if (kt < KT && grp < G && n < p.N && (GPT > 1 || lane < 16)) {
          const uint32_t z = p.zeros ? p.zeros[grp * p.ld_zeros + n] : 8u;
          v = 0x4300u | z |
              (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(
                   p.scales + grp * p.ld_scales + n))
               << 16);
        }
        m[c][r] = v;
      }
  };
  auto load_a = [&](int kt, uint4 (&a)[NT][4]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int m = m0 + i * 8 + g;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[i][j] = m < p.M && kt < KT
                      ? load_a8(p.A + m * p.lda, kt * 128 + j * 32 + t * 8, p.K, vec_a)
                      : make_uint4(0u, 0u, 0u, 0u);
    }
  };

#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(first + s * step, s);
  uint32_t meta[CT][MREGS];
  uint4 a[NT][4];
  load_meta(first, meta);
  load_a(first, a);

  float acc[CT][NT][4] = {};
  int s = 0;
  for (int kt = first; kt < KT; kt += step) {
    issue(kt + (STAGES - 1) * step, s == 0 ? STAGES - 1 : s - 1);
    cp_async_wait<STAGES - 1>();
    uint32_t mine[CT][MREGS];
    uint4 x[NT][4];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int r = 0; r < MREGS; ++r) mine[c][r] = meta[c][r];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = a[i][j];
    load_meta(kt + step, meta);
    if (NT == 1) load_a(kt + step, a);
    const uint8_t* st = ring + s * CT * kW4TileBytes;
    if (++s == STAGES) s = 0;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (c > 0 && nt0 + c >= NTILES) break;
      const uint4 h0 = *reinterpret_cast<const uint4*>(st + c * kW4TileBytes);
      const uint4 h1 = *reinterpret_cast<const uint4*>(st + c * kW4TileBytes + 512);
      const uint32_t w0[4] = {h0.x, h0.y, h0.z, h0.w};
      const uint32_t w1[4] = {h1.x, h1.y, h1.z, h1.w};
#pragma unroll
      for (int grp = 0; grp < GPT; ++grp) {
        const uint32_t g0 = __shfl_sync(0xFFFFFFFFu, mine[c][grp / 2], (grp % 2) * 16 + g);
        const uint32_t g1 = __shfl_sync(0xFFFFFFFFu, mine[c][grp / 2], (grp % 2) * 16 + 8 + g);
        const uint32_t z0 = __byte_perm(g0, 0, 0x1010), z1 = __byte_perm(g1, 0, 0x1010);
        float part[NT][4] = {};
#pragma unroll
        for (int j = grp * (4 / GPT); j < (grp + 1) * (4 / GPT); ++j) {
          uint32_t v0[4], v1[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v0[i] = sub_bf16x2(decode_pair(w0[j], i), z0);
            v1[i] = sub_bf16x2(decode_pair(w1[j], i), z1);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mma_bf16(part[i], v0[0], v1[0], v0[1], v1[1], x[i][j].x, x[i][j].y);
            mma_bf16(part[i], v0[2], v1[2], v0[3], v1[3], x[i][j].z, x[i][j].w);
          }
        }
        const float s0 = bf16_hi(g0), s1 = bf16_hi(g1);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          acc[c][i][0] = fmaf(s0, part[i][0], acc[c][i][0]);
          acc[c][i][1] = fmaf(s0, part[i][1], acc[c][i][1]);
          acc[c][i][2] = fmaf(s1, part[i][2], acc[c][i][2]);
          acc[c][i][3] = fmaf(s1, part[i][3], acc[c][i][3]);
        }
      }
    }
    if (NT > 1) load_a(kt + step, a);
  }
  cp_async_wait<0>();
  __syncthreads();  // every copy of the block has landed: the ring becomes the exchange
  float(*red)[CT * 16][RED] = reinterpret_cast<float(*)[CT * 16][RED]>(smem);
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      red[warp][c * 16 + g][i * 8 + 2 * t] = acc[c][i][0];
      red[warp][c * 16 + g][i * 8 + 2 * t + 1] = acc[c][i][1];
      red[warp][c * 16 + 8 + g][i * 8 + 2 * t] = acc[c][i][2];
      red[warp][c * 16 + 8 + g][i * 8 + 2 * t + 1] = acc[c][i][3];
    }
  __syncthreads();
  constexpr int OUT = CT * 16 * 8 * NT;
  if (blocks > 1) {
    // this block's sums, in its first warp's place, then all blocks' by rank
    for (int i = threadIdx.x; i < OUT; i += kThreads) {
      const int col = i % (CT * 16), row = i / (CT * 16);
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[w][col][row];
      red[0][col][row] = v;
    }
    cluster_sync();
  }
  for (int i = threadIdx.x + rank * kThreads; i < OUT; i += kThreads * blocks) {
    const int col = i % (CT * 16), row = i / (CT * 16);
    const int n = nt0 * 16 + col, m = m0 + row;
    if (n >= p.N || m >= p.M) continue;
    float v = 0.0f;
    if (blocks > 1) {
      const uint32_t at = smem_u32(&red[0][col][row]);
      for (int r = 0; r < blocks; ++r) v += ld_cluster_f32(map_to_rank(at, r));
    } else {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[w][col][row];
    }
    const float bias = p.epi.bias != nullptr ? p.epi.bias[n] : 0.0f;
    if (p.c_bf16) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.C) + m * p.ldc + n;
      *o = __float2bfloat16_rn(
          epi_apply(p.epi, v, p.epi.beta != 0.0f ? __bfloat162float(*o) : 0.0f, bias));
    } else {
      float* o = static_cast<float*>(p.C) + m * p.ldc + n;
      *o = epi_apply(p.epi, v, p.epi.beta != 0.0f ? *o : 0.0f, bias);
    }
  }
  if (blocks > 1) cluster_sync();  // no block leaves while others read its sums
}

// Position of code (k, n) in the packed matrix: word index and shift.
__device__ __forceinline__ int64_t packed_word(int k, int n, int KT, int* shift) {
  const int kk = k & 127, nn = n & 15;
  *shift = nibble_shift(kk & 7);
  return (static_cast<int64_t>(n >> 4) * KT + (k >> 7)) * 256 +
         (((nn >> 3) * 8 + (nn & 7)) * 4 + ((kk >> 3) & 3)) * 4 + (kk >> 5);
}

// One thread per packed word (eight rows of a column), column fastest among
// threads so that the reads of the codes are contiguous.
__global__ void w4_pack_kernel(int K, int N, const uint8_t* __restrict__ codes, int64_t ld,
                               uint32_t* __restrict__ packed) {
  grid_dependency_wait();
  grid_dependents_go();
  const int KT = (K + 127) / 128;
  const int np = (N + 15) / 16 * 16;
  const int64_t total = static_cast<int64_t>(KT) * 16 * np;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int n = static_cast<int>(i % np), k0 = static_cast<int>(i / np) * 8;
    uint32_t w = 0;
    for (int e = 0; e < 8; ++e)
      if (n < N && k0 + e < K)
        w |= static_cast<uint32_t>(codes[(k0 + e) * ld + n] & 15u) << nibble_shift(e);
    int shift;
    packed[packed_word(k0, n, KT, &shift)] = w;
  }
}

// One thread per (group, column): the group's range gives its scale (and zero
// point), then its codes.  Symmetric: s = max|w| / 7, codes 1..15 around 8.
// With zero points: s = (hi - lo) / 15 over the range widened to hold 0,
// z = round(-lo / s).  The scale is rounded to BF16 first and the codes are
// taken for the rounded scale.  A group with a value that is not finite gets a
// NaN scale.  Groups divide the 128-row tiles, so no word is shared by groups.
template <typename T>
__global__ void w4_quantize_kernel(int K, int N, int group, const T* __restrict__ B, int64_t ldb,
                                   uint32_t* __restrict__ packed,
                                   __nv_bfloat16* __restrict__ scales, int64_t ld_scales,
                                   uint8_t* __restrict__ zeros, int64_t ld_zeros) {
  grid_dependency_wait();
  grid_dependents_go();
  const int KT = (K + 127) / 128;
  const int np = (N + 15) / 16 * 16;
  const int groups = KT * 128 / group;  // the padding rows' words are written too
  const int64_t total = static_cast<int64_t>(groups) * np;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int n = static_cast<int>(i % np), grp = static_cast<int>(i / np);
    const int k0 = grp * group, k1 = min(k0 + group, K);
    float lo = 0.0f, hi = 0.0f;
    bool finite = true;
    if (n < N)
      for (int k = k0; k < k1; ++k) {
        const float v = to_f32(B[k * ldb + n]);
        finite &= fabsf(v) <= 3.402823466e38f;
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
      }
    float s = zeros ? hi * (1.0f / 15.0f) - lo * (1.0f / 15.0f) : fmaxf(-lo, hi) * (1.0f / 7.0f);
    s = __bfloat162float(__float2bfloat16_rn(s));
    float z = 8.0f;
    if (zeros) z = s > 0.0f ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 8.0f;
    for (int k = k0; k < k0 + group; k += 8) {
      uint32_t w = 0;
      for (int e = 0; e < 8; ++e) {
        float q = z;
        if (n < N && k + e < K && s > 0.0f && finite)
          q = fminf(fmaxf(rintf(to_f32(B[(k + e) * ldb + n]) / s) + z, 0.0f), 15.0f);
        w |= static_cast<uint32_t>(q) << nibble_shift(e);
      }
      int shift;
      packed[packed_word(k, n, KT, &shift)] = w;
    }
    if (n < N && k0 < K) {
      scales[grp * ld_scales + n] =
          __float2bfloat16_rn(finite ? s : __int_as_float(0x7FC00000));
      if (zeros) zeros[grp * ld_zeros + n] = static_cast<uint8_t>(z);
    }
  }
}

// W as BF16, rounded once from the exact FP32 product (q - z) * s (4 signed
// bits by 8: at most 12 significant bits, so exact in FP32).
__global__ void w4_unpack_kernel(int K, int N, int group, const uint32_t* __restrict__ packed,
                                 const __nv_bfloat16* __restrict__ scales, int64_t ld_scales,
                                 const uint8_t* __restrict__ zeros, int64_t ld_zeros,
                                 __nv_bfloat16* __restrict__ B, int64_t ldb) {
  grid_dependency_wait();
  grid_dependents_go();
  const int KT = (K + 127) / 128;
  const int k8 = (K + 7) / 8;
  const int64_t total = static_cast<int64_t>(k8) * N;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int n = static_cast<int>(i % N), k0 = static_cast<int>(i / N) * 8;
    int shift;
    const uint32_t w = packed[packed_word(k0, n, KT, &shift)];
    const int grp = k0 / group;
    const float s = __bfloat162float(scales[grp * ld_scales + n]);
    const float z = zeros ? static_cast<float>(zeros[grp * ld_zeros + n]) : 8.0f;
    for (int e = 0; e < 8 && k0 + e < K; ++e)
      B[(k0 + e) * ldb + n] = __float2bfloat16_rn(
          (static_cast<float>((w >> nibble_shift(e)) & 15u) - z) * s);
  }
}

int blocks_for(int64_t total, int threads) {
  const int64_t b = (total + threads - 1) / threads;
  return static_cast<int>(b < 8192 ? (b > 0 ? b : 1) : 8192);
}

template <int CT, int NT, int GPT>
cudaError_t launch_tile(const W4Args& a, bool vec_a, int blocks, cudaStream_t stream) {
  constexpr int STAGES = CT == 4 ? 3 : 4;
  constexpr size_t kRing = static_cast<size_t>(kWarps) * STAGES * CT * kW4TileBytes;
  constexpr size_t kExchange = sizeof(float) * kWarps * CT * 16 * (8 * NT + 1);
  constexpr size_t kSmem = kRing > kExchange ? kRing : kExchange;
  const auto kernel = w4_kernel<CT, NT, GPT, STAGES>;
  if (kSmem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
  }
  const int ntiles = (a.N + kW4TileN - 1) / kW4TileN;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = static_cast<unsigned>(blocks);
  cfg.gridDim = dim3(static_cast<unsigned>((ntiles + CT - 1) / CT),
                     static_cast<unsigned>((a.M + 8 * NT - 1) / (8 * NT)),
                     static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, vec_a ? 1 : 0);
}

template <int CT, int NT>
cudaError_t launch_groups(const W4Args& a, bool vec_a, int blocks, cudaStream_t stream) {
  if (a.group == 128) return launch_tile<CT, NT, 1>(a, vec_a, blocks, stream);
  if (a.group == 64) return launch_tile<CT, NT, 2>(a, vec_a, blocks, stream);
  return launch_tile<CT, NT, 4>(a, vec_a, blocks, stream);
}

template <int NT>
cudaError_t launch_columns(int ct, const W4Args& a, bool vec_a, int blocks, cudaStream_t stream) {
  if (ct == 4) return launch_groups<4, NT>(a, vec_a, blocks, stream);
  if (ct == 2) return launch_groups<2, NT>(a, vec_a, blocks, stream);
  return launch_groups<1, NT>(a, vec_a, blocks, stream);
}

}  // namespace

cudaError_t launch_w4(const W4Args& a, const LayerDevice& dev, cudaStream_t stream) {
  const bool vec_a = (reinterpret_cast<uintptr_t>(a.A) & 15u) == 0 && (a.lda % 8 == 0 || a.M == 1);
  const int ntiles = (a.N + kW4TileN - 1) / kW4TileN, kts = (a.K + kW4TileK - 1) / kW4TileK;
  // A is read once per CT tiles of columns: wide where that would be more than
  // the weights (M of 3 and up), as long as every SM still gets a block.
  int ct = a.M > 4 ? 4 : a.M > 2 ? 2 : 1;
  while (ct > 1 && ntiles < ct * dev.sms) ct /= 2;
  // Few columns: K is shared by the blocks of a cluster too, at least two
  // steps to a warp.
  int blocks = 1;
  while (blocks < 8 && (ntiles + ct - 1) / ct * blocks * 2 <= 2 * dev.sms &&
         kts >= 4 * kWarps * blocks)
    blocks *= 2;
  const cudaError_t e = a.M <= 8 ? launch_columns<1>(ct, a, vec_a, blocks, stream)
                                 : launch_columns<2>(ct, a, vec_a, blocks, stream);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_w4_pack(int K, int N, const uint8_t* codes, int64_t ld, uint8_t* packed,
                           cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>((K + 127) / 128) * 16 * ((N + 15) / 16 * 16);
  const cudaError_t e = launch_pdl(w4_pack_kernel, dim3(blocks_for(total, 256)), dim3(256), 0,
                                   stream, K, N, codes, ld, reinterpret_cast<uint32_t*>(packed));
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_w4_quantize(int K, int N, int group, const void* B, int64_t ldb, bool b_bf16,
                               uint8_t* packed, __nv_bfloat16* scales, int64_t ld_scales,
                               uint8_t* zeros, int64_t ld_zeros, cudaStream_t stream) {
  const int64_t total =
      static_cast<int64_t>((K + 127) / 128) * (128 / group) * ((N + 15) / 16 * 16);
  const dim3 grid(blocks_for(total, 128)), block(128);
  uint32_t* out = reinterpret_cast<uint32_t*>(packed);
  const cudaError_t e =
      b_bf16 ? launch_pdl(w4_quantize_kernel<__nv_bfloat16>, grid, block, 0, stream, K, N, group,
                          static_cast<const __nv_bfloat16*>(B), ldb, out, scales, ld_scales, zeros,
                          ld_zeros)
             : launch_pdl(w4_quantize_kernel<float>, grid, block, 0, stream, K, N, group,
                          static_cast<const float*>(B), ldb, out, scales, ld_scales, zeros,
                          ld_zeros);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_w4_unpack(int K, int N, int group, const uint8_t* packed,
                             const __nv_bfloat16* scales, int64_t ld_scales, const uint8_t* zeros,
                             int64_t ld_zeros, __nv_bfloat16* B, int64_t ldb,
                             cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>((K + 7) / 8) * N;
  const cudaError_t e = launch_pdl(w4_unpack_kernel, dim3(blocks_for(total, 256)), dim3(256), 0,
                                   stream, K, N, group, reinterpret_cast<const uint32_t*>(packed),
                                   scales, ld_scales, zeros, ld_zeros, B, ldb);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace g07
