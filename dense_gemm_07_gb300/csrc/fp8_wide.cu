// fp8_wide.cu -- products of 8-bit floating-point matrices (the formula is in
// fp8_few.cu) of many rows, on tiles of 128 rows by 256 columns of C, B with square
// scales.
//
// A persistent block an SM walks over tiles.  The rows of A are the MMA's lanes, so that
// a thread has one row's scale, times its 128 columns' block's of B, for all the sums it
// adds: one multiply-add for each of them and block of 128 k, no scales to read.  Two
// accumulators of 256 columns take turns: while the sum warps read one (tcgen05.ld
// 32x32b: the forms that spread columns over lanes read tensor memory at half the rate),
// the MMAs fill the other.
//
// Roles, 384 threads: warp 0 copies both operands by TMA (3 stages of 48 KB), warp 1
// issues the MMAs, warp 2 works out the experts' rows, warps 4-11 add 128 columns of 32
// rows each, and write them.
//
// What bounds it is the turn of an accumulator, MMAs, signal, reading, signal, which the
// two hide only in part: four MMAs of 128 x 256 x 32 take 641 clocks back to back (of
// 128 x 128 x 32 404; timed apart, by a program that is not kept), a block of K about 1040
// (1024 x 4864 x 8192 less 1024 x 4864 x 4096, one tile an SM: 534 ns at 2.0 GHz).  4096 x
// 4096 x 11008: 195 us, 1.89 PFLOP/s, 49 % of twice the measured BF16 rate; 226 with bias and GELU, whose
// exponentials and quotients keep the sum warps from the next tile; 16384 rows of 64
// experts, 4096 x 2048, 197 us.  The last of ten waves has 8 tiles of 152.
//
// Tried: MMAs of 128 columns from two threads, each half with its own signals, 230 us;
// 16 sum warps 418 to 460; the tiles on pairs of SMs (cta_group::2, 256 x 256), whose
// signals cross SMs at every block of K, 390 to 400; scalar multiply-adds 238; the scales
// through shared memory 252; output 16 columns at a time 220 (and 10000 clocks a tile
// with that code written out eight times, which the instruction cache does not hold).
#include <atomic>

#include "experts.h"
#include "fp8.cuh"
#include "kernels.h"
#include "normal_tail.cuh"
#include "sm103_ptx.cuh"
#include "tile_order.cuh"

namespace g07 {
namespace {

constexpr int TILE_M = kFp8WideRows;  // rows of C: the MMA's lanes
constexpr int TILE_N = 256;           // columns of C, in two halves
constexpr int HALF = 128;
constexpr int BK = kFp8Block;
constexpr int STAGES = 3;
constexpr int A_BYTES = TILE_M * BK;
constexpr int B_BYTES = TILE_N * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int THREADS = 384;
constexpr int SUM_WARPS = 8;
constexpr int GROUP = 12;
// A sum warp's 32 rows of 64 numbers on their way out, 68 words from one row to the
// next: rows stay on 16 bytes, and what 8 lanes store at once falls into 32 banks.
constexpr int STAGED_COLS = 64;
constexpr int STAGED_ROW = STAGED_COLS + 4;
constexpr int STAGED_FLOATS = 32 * STAGED_ROW;
constexpr int STAGED_AT = STAGES * STAGE_BYTES;
constexpr int CONTROL_AT = STAGED_AT + SUM_WARPS * STAGED_FLOATS * 4;
// Registers a thread of the roles (setmaxnreg): together at most the 384 x 168 that
// the block is launched with.
constexpr int kRegsOther = 88, kRegsSum = 208;
constexpr int kRegsBlock = 128 * kRegsOther + 256 * kRegsSum;
static_assert(kRegsBlock <= THREADS * 168, "register split");

struct alignas(16) Control {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int tiles;
  int start[kRouteMaxExperts + 1];   // experts: first row of each
  int before[kRouteMaxExperts + 1];  // experts: units of rows before each
};
constexpr size_t kSmemBytes = 1024 + CONTROL_AT + sizeof(Control);  // 1024: to align the ring
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a block");

struct WideArgs {
  Fp8GemmArgs g;
  int n_tiles, units;  // dense: units of rows
  unsigned int* status;
};

struct Tile {
  int expert, first, count, n0;
};

__device__ __forceinline__ Tile tile_at(const WideArgs& p, const Control* ctl, int t) {
  Tile r;
  int left;
  if (p.g.E == 0) {
    const TileCoord c = tile_order(t, p.units, p.n_tiles, GROUP);
    r.expert = 0;
    r.first = c.m * TILE_M;
    r.n0 = c.n * TILE_N;
    left = p.g.M - r.first;
  } else {
    // the last expert with before[e] * n_tiles <= t: it has units.  Its units share the
    // columns of B and follow each other.
    int lo = 0, hi = p.g.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (ctl->before[mid] * p.n_tiles <= t)
        lo = mid;
      else
        hi = mid;
    }
    const int units = ctl->before[lo + 1] - ctl->before[lo];
    const int in = t - ctl->before[lo] * p.n_tiles;
    r.expert = lo;
    r.first = ctl->start[lo] + in % units * TILE_M;
    r.n0 = in / units * TILE_N;
    left = ctl->start[lo + 1] - r.first;
  }
  r.count = left < TILE_M ? left : TILE_M;
  return r;
}

__device__ __forceinline__ void give_up(volatile int* abort, unsigned int* status) {
  *abort = 1;
  atomicOr(status, 1u);
}

struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// act(alpha * v + beta * old + bias) of N consecutive columns.
template <int N>
__device__ __forceinline__ void finish(const EpiParams& e, const float (&bias)[N],
                                       const float (&old)[N], float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] *= e.alpha;
    if (e.beta != 0.0f) v[i] = fmaf(e.beta, old[i], v[i]);
    v[i] += bias[i];
    if (e.act == 1) v[i] = fmaxf(v[i], 0.0f);
    if (e.act == 2) {
      float ignored;
      const float tail = 0.5f * normal_tail2(v[i], &ignored);
      v[i] *= v[i] > 0.0f ? 1.0f - tail : tail;
    }
  }
}

// 64 columns of C from n on, of the `rows` rows from `first` on, from a warp's staged
// sums: eight lanes a row, so that a row's part leaves as whole 128-byte lines.
template <typename T>
__device__ __forceinline__ void store_rows(const Fp8GemmArgs& g, T* C, const float* stage,
                                           int expert, int first, int rows, int n) {
  const int lane = threadIdx.x & 31;
  C += first * g.ldc + n;
  const float* bias = g.epi.bias ? g.epi.bias + static_cast<int64_t>(expert) * g.N + n : nullptr;
  if (n + STAGED_COLS <= g.N &&
      ((reinterpret_cast<uintptr_t>(g.C) | (g.ldc * sizeof(T))) & 15u) == 0) {
    const int c = (lane & 7) * 8;
    float b[8], old[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = bias ? __ldg(bias + c + i) : 0.0f;
#pragma unroll 2
    for (int r = lane >> 3; r < rows; r += 4) {
      float v[8];
      load_vec<8>(stage + r * STAGED_ROW + c, v);
      T* o = C + r * g.ldc + c;
      if (g.epi.beta != 0.0f) load_vec<8>(o, old);
      finish(g.epi, b, old, v);
      store_vec<8>(o, v);
    }
  } else {  // a lane a column
    for (int c = lane; c < STAGED_COLS && n + c < g.N; c += 32) {
      const float b[1] = {bias ? __ldg(bias + c) : 0.0f};
#pragma unroll 4
      for (int r = 0; r < rows; ++r) {
        float v[1] = {stage[r * STAGED_ROW + c]}, old[1];
        T* o = C + r * g.ldc + c;
        if (g.epi.beta != 0.0f) old[0] = to_f32(*o);
        finish(g.epi, b, old, v);
        *o = from_f32<T>(v[0]);
      }
    }
  }
}

__global__ void __launch_bounds__(THREADS, 1)
fp8_wide_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ WideArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Control* ctl = reinterpret_cast<Control*>(smem + CONTROL_AT);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int step = gridDim.x;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&ctl->acc_full[a], 1);
      mbar_init(&ctl->acc_empty[a], SUM_WARPS);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, 2 * TILE_N);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_dependents_go();
  if (warp == 2) {
    int units = p.units;
    if (p.g.E > 0)
      units = fp8_expert_table(p.g.offsets, p.g.E, p.g.M, TILE_M, ctl->start, ctl->before);
    if (lane == 0) ctl->tiles = units * p.n_tiles;
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  const int tiles = ctl->tiles;
  const uint64_t limit = wait_limit_ns(p.status);
  const int kbs = (p.g.K + BK - 1) / BK;

  if (warp < 4) {
    regs_dec<kRegsOther>();
    if (warp == 0 && lane == 0) {
      // ----------------------------------------------------------- copies
      // test faults: the first stage is never copied (2: by the first block alone)
      const unsigned int fault = p.status[1];
      const bool skip = fault == 1 || (fault == 2 && blockIdx.x == 0);
      Ring ring;
      int last[STAGES];
#pragma unroll
      for (int s = 0; s < STAGES; ++s) last[s] = -1;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += step) {
        const Tile w = tile_at(p, ctl, t);
        const int brow = w.expert * p.g.N + w.n0;
        for (int kb = 0; kb < kbs; ++kb) {
          ok = wait_soon(&ctl->empty[ring.at], ring.phase ^ 1u, abort, limit);
          if (!ok) break;
          if (!(skip && t == static_cast<int>(blockIdx.x) && kb == 0)) {
            uint8_t* a = smem + ring.at * STAGE_BYTES;
            mbar_arrive_expect_tx(&ctl->full[ring.at], STAGE_BYTES);
            tma_load_2d(a, &tmA, &ctl->full[ring.at], kb * BK, w.first);
            tma_load_2d(a + A_BYTES, &tmB, &ctl->full[ring.at], kb * BK, brow);
#pragma unroll
            for (int s = 0; s < STAGES; ++s)
              if (s == ring.at) last[s] = static_cast<int>(ring.phase);
          }
          ring.next(STAGES);
        }
      }
      if (!ok) give_up(abort, p.status);
      // copies in flight land before the block may exit
      volatile int never = 0;
#pragma unroll
      for (int s = 0; s < STAGES; ++s)
        if (last[s] >= 0 &&
            !wait_soon(&ctl->full[s], static_cast<uint32_t>(last[s]), &never, limit))
          give_up(abort, p.status);
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------- MMAs
      const uint64_t desc_a = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t desc_b = sdesc_sw128(smem_u32(smem) + A_BYTES, 16, 1024);
      Ring ring, acc;
      bool ok = true, issued = false;
      for (int t = blockIdx.x; ok && t < tiles; t += step) {
        const Tile w = tile_at(p, ctl, t);
        const int cols = p.g.N - w.n0 < TILE_N ? (p.g.N - w.n0 + 15) & ~15 : TILE_N;
        const uint32_t idesc = idesc_e4m3_f32(TILE_M, cols);
        for (int kb = 0; kb < kbs; ++kb) {
          ok = wait_soon(&ctl->full[ring.at], ring.phase, abort, limit) &&
               wait_soon(&ctl->acc_empty[acc.at], acc.phase ^ 1u, abort, limit);
          if (!ok) break;
          tc_fence_after_sync();
          const uint64_t at = static_cast<uint64_t>(ring.at * (STAGE_BYTES >> 4));
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma_e4m3_ss(tmem + acc.at * TILE_N, desc_a + at + 2 * kk, desc_b + at + 2 * kk, idesc,
                        kk != 0 ? 1u : 0u);
          issued = true;
          mma_commit(&ctl->acc_full[acc.at]);
          mma_commit(&ctl->empty[ring.at]);
          ring.next(STAGES);
          acc.next(2);
        }
      }
      if (!ok) give_up(abort, p.status);
      if (issued) {
        mma_commit(&ctl->drain);
        volatile int never = 0;
        if (!wait_soon(&ctl->drain, 0u, &never, limit)) give_up(abort, p.status);
      }
    }
  } else {
    // --------------------------------------------------------------- sums
    regs_inc<kRegsSum>();
    const int half = (warp >> 2) - 1;  // its 128 columns of the tile
    const int quad = warp & 3;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * HALF;
    float* stage = reinterpret_cast<float*>(smem + STAGED_AT) + (warp - 4) * STAGED_FLOATS;
    Ring acc;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += step) {
      const Tile w = tile_at(p, ctl, t);
      const int n0 = w.n0 + half * HALF;
      const int rows = w.count - quad * 32 < 32 ? w.count - quad * 32 : 32;  // of this warp's
      const bool live = n0 < p.g.N;
      uint64_t sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      // A thread has a row of A: its scale times the block's of B.
      const int blocks = (p.g.N + 127) / 128;
      const float* sb =
          p.g.sb + (static_cast<int64_t>(w.expert) * blocks + (live ? n0 / 128 : 0)) * p.g.ld_sb;
      const float* sa = p.g.sa + w.first + quad * 32 + lane;
      const bool mine = lane < rows;
      float fa[3], fb[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        fa[i] = mine && i < kbs ? __ldg(sa + i * p.g.ld_sa) : 0.0f;
        fb[i] = i < kbs ? __ldg(sb + i) : 0.0f;
      }
      for (int kb = 0; kb < kbs; ++kb) {
        const float scale = fa[0] * fb[0];
#pragma unroll
        for (int i = 0; i + 1 < 3; ++i) {
          fa[i] = fa[i + 1];
          fb[i] = fb[i + 1];
        }
        if (kb + 3 < kbs) {
          if (mine) fa[2] = __ldg(sa + (kb + 3) * p.g.ld_sa);
          fb[2] = __ldg(sb + kb + 3);
        }
        const bool got = wait_soon(&ctl->acc_full[acc.at], acc.phase, abort, limit);
        ok = __all_sync(0xFFFFFFFFu, got);
        if (!ok) break;
        tc_fence_after_sync();
        const uint64_t f = pack2(scale, scale);
        const uint32_t from = taddr + acc.at * TILE_N;
        uint32_t r[2][32];  // 32 columns are added while the next are on their way
        tmem_ld_32x32b_x32(from, r[0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tmem_ld_wait();
          if (j < 3) tmem_ld_32x32b_x32(from + (j + 1) * 32, r[(j + 1) & 1]);
          if (j == 3) {  // everything has been read
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&ctl->acc_empty[acc.at]);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            fma2_loaded(sum[j * 16 + i], r[j & 1][2 * i], r[j & 1][2 * i + 1], f);
        }
        acc.next(2);
      }
      if (!ok) break;
      if (live && rows > 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (n0 + j * STAGED_COLS < p.g.N) {
            __syncwarp();  // the last ones have been read
#pragma unroll
            for (int i = 0; i < 16; ++i)
              *reinterpret_cast<float4*>(stage + lane * STAGED_ROW + 4 * i) = make_float4(
                  half_of(sum[j * 32 + 2 * i], 0), half_of(sum[j * 32 + 2 * i], 1),
                  half_of(sum[j * 32 + 2 * i + 1], 0), half_of(sum[j * 32 + 2 * i + 1], 1));
            __syncwarp();
            if (p.g.c_bf16)
              store_rows(p.g, static_cast<__nv_bfloat16*>(p.g.C), stage, w.expert,
                         w.first + quad * 32, rows, n0 + j * STAGED_COLS);
            else
              store_rows(p.g, static_cast<float*>(p.g.C), stage, w.expert, w.first + quad * 32,
                         rows, n0 + j * STAGED_COLS);
          }
        }
      }
    }
    if (!ok && lane == 0) give_up(abort, p.status);
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 2 * TILE_N);
  }
}

std::atomic<uint64_t> g_allowed, g_registers;

}  // namespace

// The most units of 128 rows there are (experts: only the device knows their rows).
int units_of(const Fp8GemmArgs& a) {
  return a.E == 0 ? (a.M + TILE_M - 1) / TILE_M : a.M / TILE_M + (a.E < a.M ? a.E : a.M);
}

// Many rows, for which a thread of fp8_wide has one scale of A for 128 columns, where
// one of fp8_few reads the scales of its columns, and enough tiles, of which fp8_wide does
// not share K: measured, in us one after another (few, wide), M x N x K.
// By tiles: 256 x 4096 x 4096 15, 21 (32); 384 x 4096 x 4096 22.0, 22.0 (48); 512 x 4096 x
// 4096 22.2, 22.1 (64); 700 x 3000 x 2000 16.7, 13.9 (72); 300 x 8192 x 4096 30.6, 22.3
// (96); 2048^3 18.8, 14.1; 4096 x 11008 x 4096 260, 191.  By rows, where the tiles are
// enough: 1 x 16384 x 4096 16.1, 21.8; 16 x 32000 x 4096 26.6, 36.0; 32 x 128256 x 4096
// 92.5, 100.6; 64 x 16384 x 4096 18.1, 22.4; 64 x 32000 x 4096 28.0, 28.7; 65 x 32000 x
// 4096 29.0, 28.6; 128 x 16384 x 4096 22.8, 22.9; 128 x 32000 x 4096 33.0, 29.7; 129 x
// 16384 x 4096 31.2, 23.2.  Experts, by their average number of rows: 48 rows of 8, 4096 x
// 4096, 29.2, 30.0 and of 64, 4096 x 2048, 111.7, 100.4; 64 rows of 8, 4096 x 4096, 31.8,
// 30.1 and of 64, 4096 x 2048, 119, 109; 128 rows of 16, 2048 x 4096, 53, 47; 2048 rows of
// 8, 2048 x 4096, 197, 142; by tiles: 64 rows of 1, 4096 x 4096, 9.6, 21.0 (16); 1000 rows
// of 1, 1024 x 2048, 12.6, 13.7 (32); 256 rows of 8, 512 x 4096, 21.5, 21.8 (48); 128 rows
// of 8, 1024 x 1024, 10.5, 10.1 (64).  Where B's rows have scales of their own, both have
// to be read per column, and fp8_few's narrower tiles are faster (4096 x 11008 x 4096: 306,
// 318 with an L2 flush).
bool fp8_takes_wide(const Fp8GemmArgs& a, const LayerDevice& dev) {
  if (a.K == 0 || !a.b_square) return false;
  const int64_t tiles = static_cast<int64_t>(units_of(a)) *
                        ((static_cast<int64_t>(a.N) + TILE_N - 1) / TILE_N);
  const bool rows = a.E > 0 ? a.M / a.E >= TILE_M / 2 : a.M > TILE_M / 2;
  return rows && 5 * tiles >= 2 * dev.sms;
}

cudaError_t launch_fp8_wide(const CUtensorMap& tmA, const CUtensorMap& tmB, const Fp8GemmArgs& a,
                            const LayerDevice& dev, cudaStream_t stream) {
  cudaError_t e = allow_shared(fp8_wide_kernel, kSmemBytes, &g_allowed);
  // The roles' register shares are drawn from what the block is launched with.
  if (e == cudaSuccess) e = check_registers(fp8_wide_kernel, kRegsBlock, THREADS, &g_registers);
  if (e != cudaSuccess) return e;
  const WideArgs p = {a, (a.N + TILE_N - 1) / TILE_N, units_of(a), dev.status};
  const int64_t tiles = static_cast<int64_t>(p.units) * p.n_tiles;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles < dev.sms ? tiles : dev.sms));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fp8_wide_kernel, tmA, tmB, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace g07
