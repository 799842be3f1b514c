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
  if (vec && k + 8 <= K) return *reinterpret_cast<const uint4*>(row + k);
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

// One block: CT tiles of 16 columns by up to 8 * NT rows of A.  Its warps take
// the 128-row tiles of K in turn and add their sums in warp order.
template <int CT, int NT>
__global__ void __launch_bounds__(kThreads) w4_kernel(W4Args p, int vec_a) {
  __shared__ float red[kWarps][CT * 16][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int KT = (p.K + kW4TileK - 1) / kW4TileK;
  const int NTILES = (p.N + kW4TileN - 1) / kW4TileN;
  const int nt0 = blockIdx.x * CT;
  const int m0 = blockIdx.y * 8 * NT;
  const int G = (p.K + p.group - 1) / p.group;
  const int per = p.group / 32;  // 32-row blocks of a group: 1, 2 or 4
  grid_dependency_wait();
  grid_dependents_go();

  float acc[CT][NT][4] = {};
  for (int kt = warp; kt < KT; kt += kWarps) {
    uint4 a[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int m = m0 + i * 8 + g;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[i][j] = m < p.M ? load_a8(p.A + m * p.lda, kt * 128 + j * 32 + t * 8, p.K, vec_a)
                          : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (nt0 + c >= NTILES) break;
      const uint4* tile = reinterpret_cast<const uint4*>(
          p.packed + (static_cast<int64_t>(nt0 + c) * KT + kt) * kW4TileBytes);
      const uint4 h0 = tile[lane], h1 = tile[32 + lane];
      const uint32_t w0[4] = {h0.x, h0.y, h0.z, h0.w};
      const uint32_t w1[4] = {h1.x, h1.y, h1.z, h1.w};
      const int n_lo = min((nt0 + c) * 16 + g, p.N - 1), n_hi = min((nt0 + c) * 16 + 8 + g, p.N - 1);
      float part[NT][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int grp = min((kt * 128 + j * 32) / p.group, G - 1);
        uint32_t z0 = 8, z1 = 8;
        if (p.zeros != nullptr) {
          z0 = p.zeros[grp * p.ld_zeros + n_lo];
          z1 = p.zeros[grp * p.ld_zeros + n_hi];
        }
        z0 = (z0 | (z0 << 16)) | 0x43004300u;  // 128 + z, twice
        z1 = (z1 | (z1 << 16)) | 0x43004300u;
        uint32_t v0[4], v1[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v0[i] = sub_bf16x2(decode_pair(w0[j], i), z0);
          v1[i] = sub_bf16x2(decode_pair(w1[j], i), z1);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          mma_bf16(part[i], v0[0], v1[0], v0[1], v1[1], a[i][j].x, a[i][j].y);
          mma_bf16(part[i], v0[2], v1[2], v0[3], v1[3], a[i][j].z, a[i][j].w);
        }
        if ((j + 1) % per == 0) {
          const float s0 = __bfloat162float(p.scales[grp * p.ld_scales + n_lo]);
          const float s1 = __bfloat162float(p.scales[grp * p.ld_scales + n_hi]);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            acc[c][i][0] = fmaf(s0, part[i][0], acc[c][i][0]);
            acc[c][i][1] = fmaf(s0, part[i][1], acc[c][i][1]);
            acc[c][i][2] = fmaf(s1, part[i][2], acc[c][i][2]);
            acc[c][i][3] = fmaf(s1, part[i][3], acc[c][i][3]);
            part[i][0] = part[i][1] = part[i][2] = part[i][3] = 0.0f;
          }
        }
      }
    }
  }
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
  for (int i = threadIdx.x; i < CT * 16 * 8 * NT; i += kThreads) {
    const int col = i % (CT * 16), row = i / (CT * 16);
    const int n = nt0 * 16 + col, m = m0 + row;
    if (n >= p.N || m >= p.M) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][col][row];
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

template <int CT, int NT>
cudaError_t launch_tile(const W4Args& a, bool vec_a, cudaStream_t stream) {
  const int64_t ntiles = (a.N + kW4TileN - 1) / kW4TileN;
  const dim3 grid(static_cast<unsigned>((ntiles + CT - 1) / CT),
                  static_cast<unsigned>((a.M + 8 * NT - 1) / (8 * NT)));
  return launch_pdl(w4_kernel<CT, NT>, grid, dim3(kThreads), 0, stream, a, vec_a ? 1 : 0);
}

}  // namespace

cudaError_t launch_w4(const W4Args& a, const LayerDevice& dev, cudaStream_t stream) {
  (void)dev;
  const bool vec_a = (reinterpret_cast<uintptr_t>(a.A) & 15u) == 0 && (a.lda % 8 == 0 || a.M == 1);
  const cudaError_t e = a.M <= 8 ? launch_tile<1, 1>(a, vec_a, stream)
                                 : launch_tile<1, 2>(a, vec_a, stream);
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
