// w4.cu -- C = act(alpha * A * W + beta * C + bias) for a few rows of A and a
// matrix W of 4-bit codes:
//   W[k][n] = (q[k][n] - z[g][n]) * s[g][n],  g = k / group,
// q and z whole numbers 0..15 (z = 8 without zero points), s BF16.  Also the
// kernels that bring codes into the packed order, quantise a matrix, and write
// W back as BF16.
//
// The product reads K * N / 2 bytes of codes once and does 2 M K N operations
// on them, so at M <= 16 memory should bound it.  Each weight is turned into the
// exact BF16 whole number q - z and multiplied on the tensor cores
// (mma.sync m16n8k16: 16 columns of W by 8 rows of A, FP32 sums), and the
// scale is applied to a group's FP32 sum, so nothing is rounded to fewer bits
// than 32 between the codes and the result.  mma.sync, not tcgen05: an operand
// decoded in registers would have to be stored to tensor memory or shared
// memory first, and at 16 rows the products are a small part of the time.
//
// Decoding takes 11 operations for 8 weights (3 shifts, 4 logic, 4 subtractions).
// At sixteen rows no unit is full (16 x 16384 x 8192, groups of 64, counters: 1.9
// of 4 instructions a cycle, integer pipe 35 %, tensor pipe 27 %): 16 warps an SM,
// which 128 registers a thread allow, do not cover the latencies of decoding and
// products.  With groups of 32 and two tiles a warp the ring and its scales take
// 118 KB a block at more than eight rows (116 KB at four rows, K over the warps),
// so one block and 8 warps an SM.  Measured (M x K x N, inputs beyond L2): 1 x 8192
// x 32768, groups of 128, 33 us, 4.2 TB/s (62 % of the measured copy rate); 16 x
// 8192 x 32768 46 us, 3.0 TB/s, with zero points and groups of 64 52 us, 2.8 TB/s,
// of 32 71 us, 2.2 TB/s; 4 x 8192 x 32768 with groups of 32 50 us, 3.2 TB/s; 1 x
// 4096 x 4096 6.1 us, mostly launch and latency.  Tried without gain: shifts as
// high products (16 x 8192 x 32768: 46 -> 56 us), rings of three and five stages
// (52 and 68 us against 52 with groups of 64).
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
// 0x4300 | q are exactly 128 + q.  (Whole numbers made into floating point under a
// fixed exponent are a published way of decoding few-bit weights: Kim et al., "Who
// Says Elephants Can't Run", 2022.)
// One three-input logic operation for both (written as & and | it became two).
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, int i) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;"  // (a & b) | c
      : "=r"(d)
      : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(0x43004300u));
  return d;
}
// Exact: both operands are whole numbers of at most 8 bits.
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The same with a sum that starts here.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------- one warp's share of W
//
// Per step a warp takes CT packed tiles (16 columns each) of one 128-row block
// of K with their GPT = 128 / group groups.  Both come through a ring in shared
// memory by asynchronous copies: a lane copies the 16-byte pieces of the tiles
// that it decodes itself, and pieces of the groups' scales and zero points,
// whose rows start anywhere: the 16-byte granules that hold a tile's 16 scales
// (3 at most) and 16 zero points (2) are copied and read from an offset.
constexpr int kMetaBytes = 80;    // a group's granules: 48 of scales, 32 of zero points
constexpr int kMetaPieces = 5;

template <int CT, int GPT>
struct WarpWeights {
  static constexpr int kStageBytes = CT * (kW4TileBytes + GPT * kMetaBytes);
  static constexpr int kMetaJobs = (CT * GPT * kMetaPieces + 31) / 32;

  const int lane, tiles, KT, G;
  const bool zeros;
  const uint8_t* src;     // this lane's piece of tile (nt0, 0)
  int64_t tile_stride;    // from a tile to the next 16 columns
  // What a step costs besides its weights is kept small by working out here
  // what does not change from step to step.  Jobs: the granules that this lane
  // copies (job i * 32 + lane).
  uintptr_t row0[kMetaJobs];      // the row of the job's group in step 0
  int64_t step_bytes[kMetaJobs];  // from there to its row in the next step
  int job_steps[kMetaJobs];       // steps in which that group lies in the matrix
  int job_to[kMetaJobs];          // offset in the stage
  int job_skip[kMetaJobs];        // bytes of granules between the row's first and the job's
  int job_len[kMetaJobs];         // bytes wanted from the row (-16: no job)
  // Low address bits of the arrays' first rows: where in its granules a row
  // starts (tiles are 32 and 16 bytes apart, so all of them start alike).
  uint32_t scale_low, zero_low, scale_row, zero_row;

  __device__ __forceinline__ WarpWeights(const W4Args& p, int nt0)
      : lane(threadIdx.x & 31), tiles((p.N + kW4TileN - 1) / kW4TileN - nt0),
        KT((p.K + kW4TileK - 1) / kW4TileK), G((p.K + p.group - 1) / p.group),
        zeros(p.zeros != nullptr),
        src(p.packed + static_cast<int64_t>(nt0) * KT * kW4TileBytes + lane * 16),
        tile_stride(static_cast<int64_t>(KT) * kW4TileBytes) {
    const uintptr_t scale0 = reinterpret_cast<uintptr_t>(p.scales + nt0 * kW4TileN);
    const uintptr_t zero0 = reinterpret_cast<uintptr_t>(p.zeros + nt0 * kW4TileN);
#pragma unroll
    for (int i = 0; i < kMetaJobs; ++i) {
      const int job = i * 32 + lane, cg = job / kMetaPieces, piece = job % kMetaPieces;
      const int c = cg / GPT;
      const bool scale = piece < 3;
      const int cols = min(kW4TileN, p.N - (nt0 + c) * kW4TileN);
      const bool live = cg < CT * GPT && c < tiles && (scale || zeros);
      const int64_t row_bytes = scale ? p.ld_scales * 2 : p.ld_zeros;
      row0[i] = (scale ? scale0 + c * 32 : zero0 + c * 16) + cg % GPT * row_bytes;
      step_bytes[i] = GPT * row_bytes;
      job_steps[i] = (G - cg % GPT + GPT - 1) / GPT;
      job_to[i] = CT * kW4TileBytes + cg * kMetaBytes + piece * 16;
      job_skip[i] = (scale ? piece : piece - 3) * 16;
      job_len[i] = !live ? -16 : scale ? cols * 2 : cols;
    }
    scale_row = static_cast<uint32_t>(p.ld_scales * 2);
    zero_row = static_cast<uint32_t>(p.ld_zeros);
    scale_low = static_cast<uint32_t>(scale0);
    zero_low = static_cast<uint32_t>(zero0);
  }

  // Zeroes the group words of this warp's stages: nothing is copied to those of
  // columns past the matrix, and they are read (for sums that are never written).
  __device__ __forceinline__ void clear(uint8_t* ring, int stages, int stage_bytes) const {
    for (int s = 0; s < stages; ++s)
      for (int i = lane; i < CT * GPT * kMetaBytes / 16; i += 32)
        *reinterpret_cast<uint4*>(ring + s * stage_bytes + CT * kW4TileBytes + i * 16) =
            make_uint4(0u, 0u, 0u, 0u);
    __syncwarp();
  }

  // Starts the copies of step kt into a stage; the caller commits.  A group past
  // the matrix gets the scale 0: A and its products are 0 past K, but 0 times what
  // the stage held before need not be.  (The row of an earlier step that started
  // elsewhere in its granules has the scales of other columns, or the gap between
  // two rows, in the same place, and its own column's may be infinite.)
  __device__ __forceinline__ void copy(uint8_t* stage, int kt) const {
    const uint8_t* from = src + static_cast<int64_t>(kt) * kW4TileBytes;
    uint8_t* to = stage + lane * 16;
#pragma unroll
    for (int c = 0; c < CT; ++c)
      if (c < tiles) {
        cp_async_16(to + c * kW4TileBytes, from + c * tile_stride);
        cp_async_16(to + c * kW4TileBytes + 512, from + c * tile_stride + 512);
      }
#pragma unroll
    for (int i = 0; i < kMetaJobs; ++i) {
      const uintptr_t at = row0[i] + kt * step_bytes[i];
      const int skip = job_skip[i] - static_cast<int>(at & 15u);
      if (skip < job_len[i]) {
        const bool there = GPT == 1 || kt < job_steps[i];  // (one group a step: all are)
        cp_async_16(stage + job_to[i], there ? reinterpret_cast<const void*>(at + skip) : from,
                    there ? 16u : 0u);
      }
    }
  }

  // Adds the step's products to acc: x holds this lane's pieces of A (row 8 i +
  // lane / 4, 8 values of each 32-row block).
  template <int NT>
  __device__ __forceinline__ void multiply(const uint8_t* stage, int kt, const uint4 (&x)[NT][4],
                                           float (&acc)[CT][NT][4]) const {
    // Tiles past the matrix are decoded too, from whatever the stage holds: their
    // sums are never written, and without a branch the tiles' work interleaves.
    const uint8_t* words = stage + CT * kW4TileBytes + (lane >> 2) * 2;
#pragma unroll
    for (int grp = 0; grp < GPT; ++grp) {
      const uint32_t row = kt * GPT + grp;
      const uint32_t s_off = (scale_low + row * scale_row) & 15u;
      const uint32_t z_off = 48 + ((zero_low + row * zero_row) & 15u);
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        // scales and zero points of columns lane / 4 and 8 + lane / 4
        const uint8_t* m = words + (c * GPT + grp) * kMetaBytes;
        const uint16_t* sc = reinterpret_cast<const uint16_t*>(m + s_off);
        const float s0 = __uint_as_float(sc[0] * 65536u), s1 = __uint_as_float(sc[8] * 65536u);
        uint32_t z0 = 0x43084308u, z1 = 0x43084308u;  // 128 + z, twice
        if (zeros) {
          const uint8_t* zp = m + z_off - (lane >> 2);
          z0 = zp[0] * 0x00010001u + 0x43004300u;
          z1 = zp[8] * 0x00010001u + 0x43004300u;
        }
        const uint8_t* tile = stage + c * kW4TileBytes + lane * 16;
        float part[NT][4];
#pragma unroll
        for (int jj = 0; jj < 4 / GPT; ++jj) {
          const int j = grp * (4 / GPT) + jj;
          const uint32_t w0 = word(tile, j), w1 = word(tile + 512, j);
          uint32_t v0[4], v1[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v0[i] = sub_bf16x2(decode_pair(w0, i), z0);
            v1[i] = sub_bf16x2(decode_pair(w1, i), z1);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (jj == 0)
              mma_bf16_first(part[i], v0[0], v1[0], v0[1], v1[1], x[i][j].x, x[i][j].y);
            else
              mma_bf16(part[i], v0[0], v1[0], v0[1], v1[1], x[i][j].x, x[i][j].y);
            mma_bf16(part[i], v0[2], v1[2], v0[3], v1[3], x[i][j].z, x[i][j].w);
          }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          acc[c][i][0] = fmaf(s0, part[i][0], acc[c][i][0]);
          acc[c][i][1] = fmaf(s0, part[i][1], acc[c][i][1]);
          acc[c][i][2] = fmaf(s1, part[i][2], acc[c][i][2]);
          acc[c][i][3] = fmaf(s1, part[i][3], acc[c][i][3]);
        }
      }
    }
  }

  // Word j of this lane's 16-byte piece (the four of a piece are one load).
  static __device__ __forceinline__ uint32_t word(const uint8_t* piece, int j) {
    const uint4 v = *reinterpret_cast<const uint4*>(piece);
    return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
  }
};

// Elements k .. k + 7 of a row of A into 16 bytes of shared memory, zeros past
// K; a row off the 16-byte grid goes element by element.
__device__ __forceinline__ void copy_a8(uint8_t* to, const __nv_bfloat16* row, int k, int K,
                                        bool vec) {
  if (vec) {
    const int n = K - k;
    cp_async_16(to, n > 0 ? row + k : row, n >= 8 ? 16u : n > 0 ? 2u * n : 0u);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo =
        k + 2 * i < K ? *reinterpret_cast<const uint16_t*>(row + k + 2 * i) : 0u;
    const uint32_t hi =
        k + 2 * i + 1 < K ? *reinterpret_cast<const uint16_t*>(row + k + 2 * i + 1) : 0u;
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void write_c(const W4Args& p, int m, int n, float v) {
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

// The sums at red[0], one per output of the block (OUT of them at `at(i)`), added
// over the cluster's blocks by rank, each block writing its share.
template <typename At, typename Put>
__device__ __forceinline__ void finish(int outs, int rank, int blocks, At at, Put put) {
  if (blocks > 1) cluster_sync();
  for (int i = threadIdx.x + rank * kThreads; i < outs; i += kThreads * blocks) {
    const float* here = at(i);
    float v = *here;
    if (blocks > 1) {
      v = 0.0f;
      for (int r = 0; r < blocks; ++r) v += ld_cluster_f32(map_to_rank(smem_u32(here), r));
    }
    put(i, v);
  }
  if (blocks > 1) cluster_sync();  // no block leaves while others read its sums
}

// ------------------------------------------- few rows: K goes over the warps
//
// Up to kFewRows rows of A; a cluster takes CT tiles of columns, the 128-row blocks
// of K go round over the warps of its blocks.  A's pieces come through the ring
// like the weights.  The warps' sums are added in warp order.
constexpr int kFewRows = 4;

template <int CT, int GPT, int STAGES>
__global__ void __launch_bounds__(kThreads, 2) w4_rows_kernel(W4Args p, int vec_a) {
  extern __shared__ __align__(16) uint8_t smem[];
  using Weights = WarpWeights<CT, GPT>;
  constexpr int RED = 9;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int blocks = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);
  const int nt0 = blockIdx.x * CT, rows = p.M;
  const int first = rank * kWarps + warp, step = blocks * kWarps;
  const int stage_bytes = Weights::kStageBytes + rows * 256;
  uint8_t* ring = smem + warp * STAGES * stage_bytes;
  const bool mine = g < rows;
  const Weights w(p, nt0);
  w.clear(ring, STAGES, stage_bytes);
  const __nv_bfloat16* a_row = p.A + (mine ? g : 0) * p.lda;
  const int whole = p.K / kW4TileK;  // blocks of K that end inside the row
  grid_dependency_wait();
  grid_dependents_go();

  auto issue = [&](int kt, int s) {
    if (kt < w.KT) {
      uint8_t* stage = ring + s * stage_bytes;
      w.copy(stage, kt);
      if (mine) {
        uint8_t* to = stage + Weights::kStageBytes + g * 256 + t * 16;
        const int k = kt * 128 + t * 8;
        if (vec_a && kt < whole) {
#pragma unroll
          for (int j = 0; j < 4; ++j) cp_async_16(to + j * 64, a_row + k + j * 32);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) copy_a8(to + j * 64, a_row, k + j * 32, p.K, vec_a);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(first + s * step, s);
  float acc[CT][1][4] = {};
  int s = 0;
  for (int kt = first; kt < w.KT; kt += step) {
    __syncwarp();  // every lane has read the stage that is filled next
    issue(kt + (STAGES - 1) * step, s == 0 ? STAGES - 1 : s - 1);
    cp_async_wait<STAGES - 1>();
    __syncwarp();  // the group words were copied by other lanes
    const uint8_t* stage = ring + s * stage_bytes;
    if (++s == STAGES) s = 0;
    uint4 x[1][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[0][j] = mine ? *reinterpret_cast<const uint4*>(stage + Weights::kStageBytes + g * 256 +
                                                       j * 64 + t * 16)
                     : make_uint4(0u, 0u, 0u, 0u);
    w.multiply(stage, kt, x, acc);
  }
  cp_async_wait<0>();
  __syncthreads();  // every copy of the block has landed: the ring becomes the exchange
  float(*red)[CT * 16][RED] = reinterpret_cast<float(*)[CT * 16][RED]>(smem);
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    red[warp][c * 16 + g][2 * t] = acc[c][0][0];
    red[warp][c * 16 + g][2 * t + 1] = acc[c][0][1];
    red[warp][c * 16 + 8 + g][2 * t] = acc[c][0][2];
    red[warp][c * 16 + 8 + g][2 * t + 1] = acc[c][0][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < CT * 16 * rows; i += kThreads) {
    const int col = i % (CT * 16), row = i / (CT * 16);
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += red[k][col][row];
    red[0][col][row] = v;
  }
  // (a thread's share below is what it has just added when there is one block)
  finish(CT * 16 * rows, rank, blocks,
         [&](int i) { return &red[0][i % (CT * 16)][i / (CT * 16)]; },
         [&](int i, float v) {
           const int n = nt0 * 16 + i % (CT * 16);
           if (n < p.N) write_c(p, i / (CT * 16), n, v);
         });
}

// -------------------------------------- more rows: columns go over the warps
//
// Up to 8 * NT rows of A; each warp takes CT tiles of columns of its own and
// all of the block's share of K (K is cut over a cluster's blocks when there are
// few columns).  A is staged for the whole block, kPhase steps at a time in two
// buffers, so it is read once per 128 CT columns.
constexpr int kPhase = 4;
constexpr int kPhaseRow = kPhase * 256 + 64;  // bytes of a staged row: 64 off a multiple of 128,
                                              // so 8 lanes of two rows read all banks once

template <int CT, int NT, int GPT, int STAGES>
__global__ void __launch_bounds__(kThreads, 2) w4_columns_kernel(W4Args p, int vec_a) {
  extern __shared__ __align__(16) uint8_t smem[];
  using Weights = WarpWeights<CT, GPT>;
  static_assert(STAGES <= kPhase + 1, "a phase of A lands before its first step");
  constexpr int ROWS = 8 * NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int blocks = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);
  const int nt0 = (blockIdx.x * kWarps + warp) * CT, m0 = blockIdx.y * ROWS;
  const int rows = min(ROWS, p.M - m0);
  const Weights w(p, nt0);
  const int k0 = static_cast<int>(static_cast<int64_t>(w.KT) * rank / blocks);
  const int k1 = static_cast<int>(static_cast<int64_t>(w.KT) * (rank + 1) / blocks);
  uint8_t* staged = smem;  // [2][ROWS][kPhaseRow]
  uint8_t* ring = smem + 2 * ROWS * kPhaseRow + warp * STAGES * Weights::kStageBytes;
  w.clear(ring, STAGES, Weights::kStageBytes);
  // rows that A does not have stay zero in both buffers
  for (int i = threadIdx.x; i < 2 * (ROWS - rows) * (kPhaseRow / 16); i += kThreads) {
    const int per = (ROWS - rows) * (kPhaseRow / 16);
    const int b = i / per, at = i % per;
    *reinterpret_cast<uint4*>(staged + (b * ROWS + rows) * kPhaseRow + at * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  grid_dependency_wait();
  grid_dependents_go();

  auto stage_a = [&](int kt, int b) {  // steps kt .. kt + kPhase - 1
    if (kt >= k1) return;
    for (int i = threadIdx.x; i < rows * kPhase * 16; i += kThreads) {
      const int row = i / (kPhase * 16), piece = i % (kPhase * 16);
      copy_a8(staged + (b * ROWS + row) * kPhaseRow + piece * 16, p.A + (m0 + row) * p.lda,
              kt * 128 + piece * 8, p.K, vec_a);
    }
  };
  auto issue = [&](int kt, int s) {
    if (kt < k1) w.copy(ring + s * Weights::kStageBytes, kt);
    cp_async_commit();
  };
  stage_a(k0, 0);  // in the first group
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(k0 + s, s);
  float acc[CT][NT][4] = {};
  int s = 0;
  for (int kt = k0; kt < k1; ++kt) {
    const int i = kt - k0;
    if (i % kPhase == 0) {
      // This phase of A was copied kPhase steps ago (or first of all): its
      // group is complete once at most STAGES - 2 later ones are not.
      cp_async_wait<STAGES - 2>();
      __syncthreads();  // all of it has landed, and the other buffer has been read
      stage_a(kt + kPhase, (i / kPhase + 1) & 1);
    } else {
      __syncwarp();  // every lane has read the stage that is filled next
    }
    issue(kt + STAGES - 1, s == 0 ? STAGES - 1 : s - 1);
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const uint8_t* a = staged + (i / kPhase & 1) * ROWS * kPhaseRow + g * kPhaseRow +
                       (i % kPhase) * 256 + t * 16;
    uint4 x[NT][4];
#pragma unroll
    for (int r = 0; r < NT; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[r][j] = *reinterpret_cast<const uint4*>(a + r * 8 * kPhaseRow + j * 64);
    w.multiply(ring + s * Weights::kStageBytes, kt, x, acc);
    if (++s == STAGES) s = 0;
  }
  cp_async_wait<0>();
  __syncthreads();
  // through shared memory for whole rows of C: [row][columns of the block + 4]
  constexpr int COLS = kWarps * CT * 16;
  float(*red)[COLS + 4] = reinterpret_cast<float(*)[COLS + 4]>(smem);
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const int col = (warp * CT + c) * 16 + g, row = r * 8 + 2 * t;
      red[row][col] = acc[c][r][0];
      red[row + 1][col] = acc[c][r][1];
      red[row][col + 8] = acc[c][r][2];
      red[row + 1][col + 8] = acc[c][r][3];
    }
  __syncthreads();
  finish(COLS * rows, rank, blocks, [&](int i) { return &red[i / COLS][i % COLS]; },
         [&](int i, float v) {
           const int n = blockIdx.x * COLS + i % COLS;
           if (n < p.N) write_c(p, m0 + i / COLS, n, v);
         });
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

cudaError_t launch_cluster(void (*kernel)(W4Args, int), const W4Args& a, bool vec_a, int gx,
                           int gy, int blocks, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = static_cast<unsigned>(blocks);
  cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy),
                     static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, vec_a ? 1 : 0);
}

size_t larger(size_t a, size_t b) { return a > b ? a : b; }

template <int CT, int GPT>
cudaError_t launch_rows(const W4Args& a, bool vec_a, int gx, int blocks, cudaStream_t stream) {
  constexpr int STAGES = 4;
  static std::atomic<uint64_t> allowed{0};
  auto smem = [](int rows) {
    return larger(
        static_cast<size_t>(kWarps) * STAGES * (WarpWeights<CT, GPT>::kStageBytes + rows * 256),
        sizeof(float) * kWarps * CT * 16 * 9);
  };
  const auto kernel = w4_rows_kernel<CT, GPT, STAGES>;
  const cudaError_t e = allow_shared(kernel, smem(kFewRows), &allowed);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, a, vec_a, gx, 1, blocks, smem(a.M), stream);
}

template <int CT, int NT, int GPT>
cudaError_t launch_columns(const W4Args& a, bool vec_a, int gx, int blocks, cudaStream_t stream) {
  constexpr int STAGES = CT == 4 ? 2 : 4;
  static std::atomic<uint64_t> allowed{0};
  const size_t smem =
      larger(static_cast<size_t>(2) * 8 * NT * kPhaseRow +
                 static_cast<size_t>(kWarps) * STAGES * WarpWeights<CT, GPT>::kStageBytes,
             sizeof(float) * 8 * NT * (kWarps * CT * 16 + 4));
  const auto kernel = w4_columns_kernel<CT, NT, GPT, STAGES>;
  const cudaError_t e = allow_shared(kernel, smem, &allowed);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, a, vec_a, gx, (a.M + 8 * NT - 1) / (8 * NT), blocks, smem, stream);
}

template <int GPT>
cudaError_t launch_groups(const W4Args& a, const LayerDevice& dev, cudaStream_t stream) {
  const bool vec_a = (reinterpret_cast<uintptr_t>(a.A) & 15u) == 0 && (a.lda % 8 == 0 || a.M == 1);
  const int ntiles = (a.N + kW4TileN - 1) / kW4TileN, kts = (a.K + kW4TileK - 1) / kW4TileK;
  int blocks = 1;
  if (a.M <= kFewRows) {
    const bool two = ntiles >= 4 * dev.sms;
    const int gx = two ? (ntiles + 1) / 2 : ntiles;
    // few columns: at least two steps to a warp of each block
    while (blocks < 8 && gx * blocks * 2 <= 2 * dev.sms && kts >= 4 * kWarps * blocks) blocks *= 2;
    return two ? launch_rows<2, GPT>(a, vec_a, gx, blocks, stream)
               : launch_rows<1, GPT>(a, vec_a, gx, blocks, stream);
  }
  // As wide as still gives every SM a block when K is cut in eight.  (Sixteen
  // rows at four tiles do not fit 128 registers: with one group a step 8 bytes
  // spill, with two 128, which took 57 us at 16 x 8192 x 32768 against 52 at two
  // tiles; with four 76.)
  const int widest = a.M <= 8 || GPT == 1 ? 4 : 2;
  int ct = ntiles >= 4 * dev.sms ? 4 : ntiles >= 2 * dev.sms ? 2 : 1;
  if (ct > widest) ct = widest;
  const int gx = (ntiles + kWarps * ct - 1) / (kWarps * ct);
  while (blocks < 8 && gx * blocks * 2 <= 2 * dev.sms && kts >= 4 * blocks) blocks *= 2;
  if (a.M <= 8) {
    if (ct == 4) return launch_columns<4, 1, GPT>(a, vec_a, gx, blocks, stream);
    if (ct == 2) return launch_columns<2, 1, GPT>(a, vec_a, gx, blocks, stream);
    return launch_columns<1, 1, GPT>(a, vec_a, gx, blocks, stream);
  }
  if constexpr (GPT == 1)
    if (ct == 4) return launch_columns<4, 2, GPT>(a, vec_a, gx, blocks, stream);
  if (ct == 2) return launch_columns<2, 2, GPT>(a, vec_a, gx, blocks, stream);
  return launch_columns<1, 2, GPT>(a, vec_a, gx, blocks, stream);
}

}  // namespace

cudaError_t launch_w4(const W4Args& a, const LayerDevice& dev, cudaStream_t stream) {
  const cudaError_t e = a.group == 128  ? launch_groups<1>(a, dev, stream)
                        : a.group == 64 ? launch_groups<2>(a, dev, stream)
                                        : launch_groups<4>(a, dev, stream);
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
