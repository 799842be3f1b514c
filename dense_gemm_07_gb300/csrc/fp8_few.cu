// fp8_few.cu -- products of 8-bit floating-point matrices with a scale for each
// block of 128 values, on 128-column tiles of C:
//   C[m][n] = act(alpha * sum_kb sa[kb][m] * sb * P[m][n][kb] + beta * C + bias[n]),
//   P = sum over the 128 k of block kb of a[m][k] * b[n][k].
// The tensor core forms P (products of 8-bit codes are exact, at most 128 of them
// are added in tensor memory), and every P is scaled and added in registers in
// FP32: one multiply-add for each element of C and block of 128 k.
//
// The rows of B (columns of C) are the MMA's 128 lanes and the rows of A its 16 to
// 128 columns, as many as the tile has in steps of 16: a few rows cost a narrow MMA.
// The scales of A's rows change along a thread's sums and are read from shared memory;
// so a thread takes its part of P in the form in which it holds every fourth pair of
// columns of four lanes (tcgen05.ld 16x256b) and needs a quarter of them.  The tile's K
// is shared by the 1 to 8 CTAs of a cluster; their partial sums meet in distributed
// shared memory and are added in rank order.
//
// Roles, 384 threads: warp 0 copies both operands by TMA (a ring of 128-byte
// rows), warp 1 issues the MMAs, warp 2 sends the scales of up to 8 blocks of K ahead
// (one block ahead, a load took longer than a block: 4096 x 4096 x 11008 with scales of
// B's rows 455 us, 8 ahead 306), warps 4-11 add (two groups of four take turns at 32
// columns) and write C.  Two CTAs share an SM, so that one's start and end overlap the
// other's copies.  Every wait is bounded.
//
// Reading the weights bounds a few rows: 32 rows of 8 experts, 4096 x 4096 each, 134
// MB, 26 us, 77 % of the measured copy rate; 1 x 4096 x 4096 6.8 us, of which the
// kernel's start, one pass and the exchange are most.
#include <atomic>

#include "experts.h"
#include "fp8.cuh"
#include "kernels.h"
#include "sm103_ptx.cuh"

namespace g07 {
namespace {

constexpr int TILE_N = 128;
constexpr int BK = kFp8Block;
constexpr int B_BYTES = TILE_N * BK;
constexpr int THREADS = 384;
constexpr int SUM_WARPS = 8;
constexpr int MAX_STAGES = 8;
constexpr int MAX_SPLIT = 8;  // CTAs of a cluster
constexpr int SLOTS = 8;  // blocks of K whose scales are staged
// Words from one row of A's sums to the next: what a warp stores at once (8 lanes of 4
// columns) falls into 32 banks.
constexpr int PART_ROW = TILE_N + 4;
// Shared memory of a CTA when two share an SM (228 KB, 1 KB of it reserved for each).
constexpr int kSmemBytes = 228 * 1024 / 2 - 1024;

// Registers a thread of the wide kernel's roles (setmaxnreg): together what the
// block is launched with, 384 x 80.
constexpr int kRegsOther = 32, kRegsSum = 104;
constexpr int kRegsBlock = 128 * kRegsOther + 256 * kRegsSum;
static_assert(kRegsBlock <= THREADS * 80, "register split");

template <int COLS, bool SQUARE>
struct alignas(16) Control {
  static constexpr int ACCS = COLS <= 32 ? 4 : 2;
  float scale[SLOTS][COLS];  // of A's rows
  float scale_b[SLOTS][SQUARE ? 4 : TILE_N];  // of the block of B, or of its rows
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t acc_full[ACCS];
  uint64_t acc_empty[ACCS];
  uint64_t scale_full[SLOTS];
  uint64_t scale_empty[SLOTS];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  Fp8Rows rows;  // the tile's expert and rows
};

struct FewArgs {
  Fp8GemmArgs g;
  int cols, stages, split, n_tiles;
  unsigned int* status;
};

__device__ __forceinline__ void give_up(volatile int* abort, unsigned int* status) {
  *abort = 1;
  atomicOr(status, 1u);
}

// Numbers of the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ float4 part4_of(uint32_t at, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(map_to_rank(at, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ float part_of(uint32_t at, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_rank(at, rank)) : "memory");
  return v;
}

// The tile's part of C from the partial sums, a warp a row of A.  WIDE: a lane takes four
// adjacent columns; else every 32nd, so that a warp's stores are adjacent.
struct OutRows {
  const Fp8GemmArgs& g;
  const float* part;
  const Fp8Rows& rows;
  int n0, split, warp;

  template <bool WIDE, typename T>
  __device__ __forceinline__ void store(T* C) const {
    const int lane = threadIdx.x & 31;
    const float* bias =
        g.epi.bias ? g.epi.bias + static_cast<int64_t>(rows.expert) * g.N + n0 : nullptr;
    int col[4];
    float b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      col[i] = WIDE ? 4 * lane + i : lane + 32 * i;
      b[i] = bias && n0 + col[i] < g.N ? __ldg(bias + col[i]) : 0.0f;
    }
    C += rows.first * g.ldc + n0;
    for (int c = warp; c < rows.count; c += SUM_WARPS * split) {
      const float* mine = part + c * PART_ROW;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (split == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mine[col[i]];
      } else {
        // four parts of a sum are on their way together, and are added in rank order
#pragma unroll 1
        for (int r0 = 0; r0 < split; r0 += 4) {
          float u[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (r0 + r >= split) {
#pragma unroll
              for (int i = 0; i < 4; ++i) u[r][i] = 0.0f;
            } else if (WIDE) {
              const float4 q = part4_of(smem_u32(mine + 4 * lane), r0 + r);
              u[r][0] = q.x; u[r][1] = q.y; u[r][2] = q.z; u[r][3] = q.w;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) u[r][i] = part_of(smem_u32(mine + col[i]), r0 + r);
            }
          }
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += u[r][i];
        }
      }
      T* o = C + c * g.ldc;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = WIDE || n0 + col[i] < g.N;
        v[i] = epi_apply(g.epi, v[i], g.epi.beta != 0.0f && in ? to_f32(o[col[i]]) : 0.0f, b[i]);
      }
      if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + col[i] < g.N) o[col[i]] = from_f32<T>(v[i]);
      } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint2*>(o + 4 * lane) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      } else {
        *reinterpret_cast<float4*>(o + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
  }
};

// SQUARE: a block of B's scales is 128 x 128, so that sa * sb is staged; else every
// row of B has its own and a thread multiplies by its row's.
template <int COLS, bool SQUARE>
__global__ void __launch_bounds__(THREADS, 2)
fp8_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ FewArgs p) {
  using Ctl = Control<COLS, SQUARE>;
  constexpr int ACCS = Ctl::ACCS;
  // 32-column chunks of a group of four sum warps, and halves of their 32 lanes: a
  // group takes every other chunk, or where there is one chunk every other half.
  constexpr int CHUNKS = COLS > 32 ? COLS / 64 : 1, HALVES = COLS > 32 ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int stage_bytes = B_BYTES + p.cols * BK;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + p.stages * stage_bytes);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile = static_cast<int>(blockIdx.x) / p.split;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int a = 0; a < ACCS; ++a) {
      mbar_init(&ctl->acc_full[a], 1);
      mbar_init(&ctl->acc_empty[a], SUM_WARPS);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&ctl->scale_full[s], 32);
      mbar_init(&ctl->scale_empty[s], SUM_WARPS);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_barrier_init();
    if (p.g.K > 0) {
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmB);
    }
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, ACCS * COLS);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_dependents_go();
  if (warp == 2) {
    const int unit = tile / p.n_tiles;
    Fp8Rows r;
    if (p.g.E > 0) {
      r = fp8_expert_rows(p.g.offsets, p.g.E, p.g.M, p.cols, unit);
    } else {
      r.expert = 0;
      r.first = unit * p.cols;
      r.count = p.g.M - r.first < p.cols ? p.g.M - r.first : p.cols;
    }
    if (lane == 0) ctl->rows = r;
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  const uint64_t limit = wait_limit_ns(p.status);
  const Fp8Rows rows = ctl->rows;
  const int n0 = tile % p.n_tiles * TILE_N;
  const int kbs = (p.g.K + BK - 1) / BK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(kbs) * rank / p.split);
  const int kb1 = rows.count > 0 ? static_cast<int>(static_cast<int64_t>(kbs) * (rank + 1) / p.split)
                                 : kb0;
  const int ncols = (rows.count + 15) & ~15;

  const int group = (warp >> 2) & 1;         // of the sum warps: takes chunks group, group + 2, ...
  // The sums leave through the ring, once every MMA that read it has completed:
  // 128 columns of C a row of A, PART_ROW apart.
  float* part = reinterpret_cast<float*>(smem);

  if (warp < 4) {
    if constexpr (COLS > 32) regs_dec<kRegsOther>();
    if (warp == 0 && lane == 0) {
      // ----------------------------------------------------------- copies
      // test fault: the first stage is never copied
      const bool skip = p.status[1] == 1u;
      const int brow = rows.expert * p.g.N + n0;
      int stage = 0;
      uint32_t phase = 0;
      int last[MAX_STAGES];
      for (int s = 0; s < MAX_STAGES; ++s) last[s] = -1;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_soon(&ctl->empty[stage], phase ^ 1u, abort, limit)) {
          give_up(abort, p.status);
          break;
        }
        if (!(skip && kb == kb0)) {
          uint8_t* b = smem + stage * stage_bytes;
          mbar_arrive_expect_tx(&ctl->full[stage], stage_bytes);
          tma_load_2d(b, &tmB, &ctl->full[stage], kb * BK, brow);
          tma_load_2d(b + B_BYTES, &tmA, &ctl->full[stage], kb * BK, rows.first);
#pragma unroll
          for (int s = 0; s < MAX_STAGES; ++s)
            if (s == stage) last[s] = static_cast<int>(phase);
        }
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // copies in flight land before the CTA may exit
      volatile int never = 0;
#pragma unroll
      for (int s = 0; s < MAX_STAGES; ++s)
        if (last[s] >= 0 &&
            !wait_soon(&ctl->full[s], static_cast<uint32_t>(last[s]), &never, limit))
          give_up(abort, p.status);
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------- MMAs
      const uint32_t idesc = idesc_e4m3_f32(TILE_N, ncols);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool issued = false;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_soon(&ctl->acc_empty[acc], acc_phase ^ 1u, abort, limit) ||
            !wait_soon(&ctl->full[stage], phase, abort, limit)) {
          give_up(abort, p.status);
          break;
        }
        tc_fence_after_sync();
        const uint32_t b = smem_u32(smem + stage * stage_bytes);
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          mma_e4m3_ss(tmem + acc * COLS, sdesc_sw128(b + kk * 32, 16, 1024),
                      sdesc_sw128(b + B_BYTES + kk * 32, 16, 1024), idesc, kk != 0 ? 1u : 0u);
        issued = true;
        mma_commit(&ctl->empty[stage]);
        mma_commit(&ctl->acc_full[acc]);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++acc == ACCS) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (issued) {
        mma_commit(&ctl->drain);
        volatile int never = 0;
        if (!wait_soon(&ctl->drain, 0u, &never, limit)) give_up(abort, p.status);
      }
    } else if (warp == 2) {
      // ----------------------------------------------------------- scales
      const float* sa = p.g.sa + rows.first;
      const float* sb = p.g.sb;
      if (SQUARE)
        sb += (static_cast<int64_t>(rows.expert) * p.n_tiles + n0 / TILE_N) * p.g.ld_sb;
      int slot = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu,
                        wait_soon(&ctl->scale_empty[slot], phase ^ 1u, abort, limit))) {
          if (lane == 0) give_up(abort, p.status);
          break;
        }
#pragma unroll
        for (int i = 0; i < COLS / 32; ++i) {
          const bool in = i * 32 + lane < rows.count;
          copy_scale(&ctl->scale[slot][i * 32 + lane],
                     in ? sa + kb * p.g.ld_sa + i * 32 + lane : p.g.sa, in);
        }
        if (SQUARE) {
          if (lane == 0) copy_scale(&ctl->scale_b[slot][0], sb + kb, true);
        } else {
#pragma unroll
          for (int i = 0; i < TILE_N / 32; ++i) {
            const bool in = n0 + i * 32 + lane < p.g.N;
            copy_scale(&ctl->scale_b[slot][SQUARE ? 0 : i * 32 + lane],
                       in ? sb + kb * p.g.ld_sb + n0 + i * 32 + lane : p.g.sb, in);
          }
        }
        arrive_when_copied(&ctl->scale_full[slot]);
        if (++slot == SLOTS) {
          slot = 0;
          phase ^= 1u;
        }
      }
      cp_async_wait_all();  // nothing is on its way when the ring is used again
    }
  } else {
    // --------------------------------------------------------------- sums
    if constexpr (COLS > 32) regs_inc<kRegsSum>();
    const int quad = warp & 3, pos = lane >> 2, at2 = 2 * (lane & 3);
    const int h0 = COLS > 32 ? 0 : group, c0 = COLS > 32 ? group * 32 : 0;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32 + 16 * h0) << 16) + c0;
    const int at = quad * 32 + 16 * h0 + pos;  // lane: at + 16 h + 8 q
    // [chunk][16 h][8 q][columns 8 i + at2 and the next]
    uint64_t sum[CHUNKS][HALVES][2][4];
#pragma unroll
    for (int j = 0; j < CHUNKS * HALVES * 8; ++j)
      sum[j / (HALVES * 8)][j / 8 % HALVES][j / 4 % 2][j % 4] = 0;
    int acc = 0, slot = 0;
    uint32_t acc_phase = 0, phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      const bool ok = wait_soon(&ctl->scale_full[slot], phase, abort, limit) &&
                      wait_soon(&ctl->acc_full[acc], acc_phase, abort, limit);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        if (lane == 0) give_up(abort, p.status);
        break;
      }
      tc_fence_after_sync();
      uint64_t mine[HALVES * 2];  // of B's rows (or of their block)
#pragma unroll
      for (int q = 0; q < HALVES * 2; ++q) {
        const float v = ctl->scale_b[slot][SQUARE ? 0 : at + 8 * q];
        mine[q] = pack2(v, v);
      }
#pragma unroll
      for (int j = 0; j < CHUNKS; ++j) {
        if (j * 64 + c0 < ncols) {
          uint64_t f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[i] = *reinterpret_cast<const uint64_t*>(&ctl->scale[slot][c0 + j * 64 + at2 + 8 * i]);
          if (SQUARE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], mine[0]);
          }
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            uint32_t r[16];
            tmem_ld_16x256b_x4(taddr + (static_cast<uint32_t>(16 * h) << 16) + acc * COLS + j * 64, r);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                fma2_loaded(sum[j][h][q][i], r[4 * i + 2 * q], r[4 * i + 2 * q + 1],
                            SQUARE ? f[i] : mul2(f[i], mine[2 * h + q]));
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->acc_empty[acc]);
        mbar_arrive(&ctl->scale_empty[slot]);
      }
      if (++acc == ACCS) {
        acc = 0;
        acc_phase ^= 1u;
      }
      if (++slot == SLOTS) {
        slot = 0;
        phase ^= 1u;
      }
    }
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = c0 + j * 64 + 8 * (i / 2) + at2 + (i & 1);
            if (c < rows.count)
              part[c * PART_ROW + at + 16 * h + 8 * q] = half_of(sum[j][h][q][i / 2], i & 1);
          }
  }

  // ------------------------------------------------------------------ output
  if (p.split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp >= 4 && n0 < p.g.N) {
    const bool bf16 = p.g.c_bf16 != 0;
    const bool whole = n0 + TILE_N <= p.g.N && ((reinterpret_cast<uintptr_t>(p.g.C) |
                                                 (p.g.ldc * (bf16 ? 2 : 4))) & (bf16 ? 7u : 15u)) == 0;
    const OutRows out = {p.g, part, rows, n0, p.split, rank * SUM_WARPS + warp - 4};
    if (bf16) {
      if (whole)
        out.store<true>(static_cast<__nv_bfloat16*>(p.g.C));
      else
        out.store<false>(static_cast<__nv_bfloat16*>(p.g.C));
    } else {
      if (whole)
        out.store<true>(static_cast<float*>(p.g.C));
      else
        out.store<false>(static_cast<float*>(p.g.C));
    }
  }
  if (p.split > 1) cluster_sync();  // the others have read this CTA's sums
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, ACCS * COLS);
  }
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const FewArgs);
Kernel kernel_of(int cols, bool square) {
  if (cols <= 32) return square ? fp8_few_kernel<32, true> : fp8_few_kernel<32, false>;
  return square ? fp8_few_kernel<128, true> : fp8_few_kernel<128, false>;
}
std::atomic<uint64_t> g_allowed[4], g_registers[2];

// The shared-memory limit and the wide kernel's registers.
cudaError_t prepare(Kernel kernel, bool wide, bool square) {
  const cudaError_t e =
      allow_shared(kernel, kSmemBytes, &g_allowed[(wide ? 2 : 0) + (square ? 1 : 0)]);
  if (e != cudaSuccess || !wide) return e;
  return check_registers(kernel, kRegsBlock, THREADS, &g_registers[square ? 1 : 0]);
}

}  // namespace

cudaError_t fp8_few_plan(const Fp8GemmArgs& a, const LayerDevice& dev, Fp8FewPlan* plan) {
  const int64_t n_tiles = (a.N + TILE_N - 1) / TILE_N;
  const int64_t kbs = (static_cast<int64_t>(a.K) + BK - 1) / BK;
  int64_t rows = a.M, units;
  if (a.E > 0) rows = 2 * ((a.M + static_cast<int64_t>(a.E) - 1) / a.E);
  const int64_t cols = rows > 112 ? 128 : (rows + 15) / 16 * 16;
  if (a.E > 0) {  // at most floor(M / cols) full units and one ragged one an expert
    units = a.M / cols + (a.E < a.M ? a.E : a.M);
  } else {
    units = (a.M + cols - 1) / cols;
  }
  plan->cols = static_cast<int>(cols);
  plan->tiles = units * n_tiles;
  // K is shared until there is a block for each SM, and on to two where that leaves a
  // block 6 blocks of K at least (4 with few columns, whose exchange is small).  Measured,
  // in us one after another (1, 2, 4, 8 ways): 128 x 4096 x 4096 22.5, 16.0, 11.7, 13.7;
  // 200 x 2000 x 500 (K = 500) 9.6, 9.5, 8.1, -; 1000 x 1000 x 3001 22.0, 16.1, 14.7, 24.3;
  // 700 x 3000 x 2000 17.0, 16.9, 23.4, 47; 1 x 4096 x 4096 14.6, 9.9, 7.3, 6.8.
  const int64_t least = cols <= 32 ? 4 : 6;
  int split = 1;
  for (int twice = 2; twice <= MAX_SPLIT && twice <= kbs; twice *= 2) {
    const int64_t blocks = plan->tiles * twice;
    if (blocks > dev.sms && (blocks > 2 * dev.sms || kbs / twice < least)) break;
    split = twice;
  }
  plan->split = split;
  const int control = static_cast<int>(
      cols <= 32 ? (a.b_square ? sizeof(Control<32, true>) : sizeof(Control<32, false>))
                 : (a.b_square ? sizeof(Control<128, true>) : sizeof(Control<128, false>)));
  int stages = (kSmemBytes - 1024 - control) / (B_BYTES + plan->cols * BK);
  plan->stages = stages < MAX_STAGES ? stages : MAX_STAGES;
  return plan->tiles * split <= 0x7FFFFFFF ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_fp8_few(const CUtensorMap& tmA, const CUtensorMap& tmB, const Fp8GemmArgs& a,
                           const Fp8FewPlan& plan, unsigned int* status, cudaStream_t stream) {
  const Kernel kernel = kernel_of(plan.cols, a.b_square);
  cudaError_t e = prepare(kernel, plan.cols > 32, a.b_square);
  if (e != cudaSuccess) return e;
  const FewArgs p = {a, plan.cols, plan.stages, plan.split, (a.N + TILE_N - 1) / TILE_N, status};
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = plan.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg.gridDim = dim3(static_cast<unsigned>(plan.tiles * plan.split));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, tmA, tmB, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace g07
