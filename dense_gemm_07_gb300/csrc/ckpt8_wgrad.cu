// ckpt8_wgrad.cu -- dW = X^T dY + beta dW with X (T x K) kept in 8 bits
// (ckpt8.cu) and dY (T x N) BF16, on pairs of SMs.
//
// 2 T K N operations on T K + 2 T N + 4 K N bytes: the tensor cores bound it
// (4096 x 4096 x 11008: 190 us at their measured rate, 51 us of traffic).  The
// kept values are exact BF16 numbers, so the products are exact; what has to be
// looked after is the sum.  The tensor core adds to its FP32 accumulator
// rounding toward zero, an error of one sign that grows with the length of the
// sum (measured on normal data, relative: 4.7e-7 over 512 rows, 2.1e-6 over
// 4096, 9.1e-6 over 16384, against 2e-7 to 1.5e-6 for FP32 FMAs).  So a sum in
// tensor memory covers 512 rows at most, and those sums are added in registers,
// rounded to nearest.
//
// One cluster of two CTAs computes 256 x 256 tiles of dW (tcgen05.mma
// cta_group::2, M = 256, N = 256, K = 16, accumulators of 256 columns, two of
// them taking turns).  Both operands are staged per 128 rows of X and dY in a
// ring of 3 stages; CTA r owns rows 128 r .. of the tile (columns of X) and
// stages 128 columns of dY.  Roles, 640 threads per CTA:
//   warp 0       copies dY boxes by TMA (64 columns x 128 rows, N-major);
//   warp 1       issues the MMAs (even CTA);
//   warps 2, 3   of the odd CTA tell the even one that a stage of X is decoded,
//                taking turns.  (A release across the pair takes longer than a
//                stage and waits for the loads its thread has in flight: done
//                by the decoding warps it emptied their read-ahead at every
//                stage, 732 us at 4096 x 4096 x 11008; done by one warp, 520.)
//   warps 4-11   load X as kept (16 rows of one column are 16 bytes, so a
//                thread owns a row of X^T and reads its 64 values of a stage as
//                four 16-byte loads, one stage ahead), turn them into BF16 and
//                store them K-major in the swizzle the MMA reads.  Nothing is
//                written back to memory in 16 bits, and 8 bits of X are read
//                per 256 columns of dW;
//   warps 12-19  add each finished accumulator to 128 sums a thread, and write
//                the tile.
// 8 bits to BF16, per two values: a byte permutation sets the bytes under the
// exponent of 128, two masks split the sign bit off (128 + low 7 bits, and 128
// or 256), a subtraction gives the whole number exactly and a multiplication by
// the power of two its value.
//
// Measured: 4096 x 4096 x 11008 273 to 277 us, 1.34 PFLOP/s, 69 % of the measured
// BF16 rate, where gemm_bf16_f32acc on X in 16 bits, without these sums, takes
// 206 (with beta, which reads dW, 345 us); 3001 x 1000 x 3000 28 to 31 us.  The 96
// registers a thread that the block is launched with spill 148 bytes.  In parts:
// without the copies of dY and the loads of X, and sums of 1024 rows, 214 us;
// without decoding as well 185.  Adding in registers costs 6.  Tried without
// gain: dY in 6 slices (293 us), sums of 1024 rows (270, left alone for their
// larger error), other register splits (274 to 381).
//
// Work sharing (stream_k.cuh): whole tiles round-robin over the resident pairs;
// the tiles of a partial last wave, with those of the last whole one, are cut
// into equal runs of stages, one per pair, where that saves more than it costs.
// A tile cut into segments is finished by the warp that arrives last on its
// counter: the others have left their sums in a workspace before they count, so
// it waits for nothing, and it adds all of them in row order.  (A pair whose
// bounded wait ran out counts its segments without summing them: the counters are
// at zero after every launch, and a later call finds no trace of it.)
#include <atomic>
#include <cstring>

#include "kernels.h"
#include "layer.h"
#include "sm103_ptx.cuh"
#include "tile_order.cuh"

namespace g07 {
namespace {

constexpr int TILE = 256;
constexpr int CTA_M = 128;                       // rows of the tile per CTA
constexpr int CTA_N = 128;                       // columns of dY staged per CTA
constexpr int BK = kCkptStageRows;               // rows of X and dY per stage
constexpr int STAGES = 3;
constexpr int A_PART_BYTES = CTA_M * 64 * 2;     // 16 KB: 64 rows of X, K-major lines of 128 bytes
constexpr int A_BYTES = CTA_M * BK * 2;          // 32 KB
constexpr int B_BOX_BYTES = BK * 64 * 2;         // 16 KB
constexpr int B_BYTES = BK * CTA_N * 2;          // 32 KB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int CHUNK = 4;                         // stages per sum in tensor memory
constexpr int TMEM_COLS = 2 * TILE;
constexpr int THREADS = 640;
constexpr int DECODE_WARPS = 8;
constexpr int EPI_WARPS = 8;
constexpr int BOX_BYTES = 32 * 32 * 4;
constexpr int EPI_BYTES = EPI_WARPS * BOX_BYTES;
constexpr int GROUP = 8;
// Stages (0.5 us) that a split of the last wave's tiles has to save.
constexpr int kSplitStages = 24;
// Registers per thread of the roles (setmaxnreg): together at most the 640 x
// 96 that the block is launched with.
constexpr int kRegsCopy = 32, kRegsDecode = 56, kRegsSum = 168;
constexpr int kRegsBlock = 128 * kRegsCopy + 256 * kRegsDecode + 256 * kRegsSum;
static_assert(kRegsBlock <= THREADS * 96, "register split");

struct alignas(8) Control {
  uint64_t full[STAGES];  // even CTA: dY bytes and decoded X of both CTAs
  uint64_t decoded[STAGES];  // odd CTA: its decoding warps
  uint64_t empty[STAGES];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];  // even CTA: 8 warps of both CTAs
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

struct WgradArgs {
  int T, K, N;
  const uint8_t* q;
  const uint8_t* scales;
  float* dW;
  int64_t ldw;
  float beta;
  float* partial;          // segments' sums: [pair][slot][rank][warp][column][lane]
  unsigned int* counters;  // [stream-K tile][rank][warp], zero between launches
  unsigned int* status;
};

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// As mbar_wait, acquiring what the other CTA of the pair released.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             uint64_t limit_ns) {
  const uint32_t a = smem_u32(bar);
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(a), "r"(parity)
        : "memory");
    if (done) return true;
    if ((i & 15u) == 15u) {
      if (*abort) return false;
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > limit_ns) return false;
    }
  }
}

__device__ __forceinline__ void give_up(volatile int* abort, uint32_t peer_abort,
                                        unsigned int* status) {
  *abort = 1;
  st_cluster_u32(peer_abort, 1u);
  atomicOr(status, 1u);
}

struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// The stages of a pair's units, one after another; the tile's place is worked
// out once a unit (its divisions cost as much as a stage's decoding).
struct StageWalk {
  WorkIter it;
  WorkUnit w;
  TileCoord tc;
  int kb;
  bool any;
  __device__ __forceinline__ void init(const PairSchedule& s, int pair, int pairs) {
    it.init(s, pair);
    next(s, pairs);
  }
  // True when a new unit begins.
  __device__ __forceinline__ bool advance(const PairSchedule& s, int pairs) {
    if (++kb < w.k1) return false;
    next(s, pairs);
    return true;
  }
  __device__ __forceinline__ void next(const PairSchedule& s, int pairs) {
    any = it.next(s, pairs, w);
    if (!any) return;
    kb = w.k0;
    tc = tile_order(w.tile, s.tiles_m, s.tiles_n, GROUP);
  }
};

__device__ __forceinline__ uint32_t step_pair(uint32_t code) {
  const uint32_t h = code == 255u ? 0x7FC0u : code << 7;
  return h | (h << 16);
}

__device__ __forceinline__ uint32_t value_pair(uint32_t p, uint32_t step) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(p & 0xFF7FFF7Fu), "r"(p & 0xFF80FF80u));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(d) : "r"(step));
  return d;
}
// Four values (bytes) as two BF16 pairs.
__device__ __forceinline__ uint2 values(uint32_t w, uint32_t step) {
  return make_uint2(value_pair(__byte_perm(w, 0x43434343u, 0x4140), step),
                    value_pair(__byte_perm(w, 0x43434343u, 0x4342), step));
}

__global__ void __launch_bounds__(THREADS, 1)
ckpt8_wgrad_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmW,
                   const PairSchedule sched, WgradArgs p, int tma_w) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* boxes = smem + STAGES * STAGE_BYTES;
  Control* ctl = reinterpret_cast<Control*>(boxes + EPI_BYTES);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctl->full[s], 1 + DECODE_WARPS + 1);  // dY's copier; X; the odd CTA's X
      mbar_init(&ctl->decoded[s], DECODE_WARPS);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&ctl->acc_full[a], 1);
      mbar_init(&ctl->acc_empty[a], 2 * EPI_WARPS);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmY);
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctl->tmem_base, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before anyone signals them
  tc_fence_after_sync();
  grid_dependency_wait();
  grid_dependents_go();
  const uint32_t tmem = ctl->tmem_base;
  const uint64_t limit = wait_limit_ns(p.status);
  const uint32_t peer_abort = map_to_rank(smem_u32(&ctl->abort), rank ^ 1u);

  if (warp < 4) {
    regs_dec<kRegsCopy>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------- copies of dY
      // test faults: the first stage is never copied (2: by the first pair alone)
      const unsigned int fault = p.status[1];
      const bool skip = fault == 1 || (fault == 2 && pair == 0);
      Ring ring;
      int last[STAGES];
      for (int s = 0; s < STAGES; ++s) last[s] = -1;
      WorkIter it;
      it.init(sched, pair);
      WorkUnit w;
      bool ok = true;
      for (bool first = true; ok && it.next(sched, pairs, w);) {
        const TileCoord tc = tile_order(w.tile, sched.tiles_m, sched.tiles_n, GROUP);
        const int col = tc.n * TILE + static_cast<int>(rank) * CTA_N;
        for (int kb = w.k0; kb < w.k1; ++kb, first = false) {
          ok = mbar_wait(&ctl->empty[ring.stage], ring.phase ^ 1u, abort, limit);
          if (!ok) break;
          if (!(skip && first)) {
            if (rank == 0) {
              mbar_arrive_expect_tx(&ctl->full[ring.stage], 2u * B_BYTES);
              last[ring.stage] = static_cast<int>(ring.phase);
            }
            const uint32_t full0 = map_to_rank(smem_u32(&ctl->full[ring.stage]), 0);
            uint8_t* b = smem + ring.stage * STAGE_BYTES + A_BYTES;
            tma_load_2d_pair(b, &tmY, full0, col, kb * BK);
            tma_load_2d_pair(b + B_BOX_BYTES, &tmY, full0, col + 64, kb * BK);
          }
          ring.advance();
        }
      }
      if (!ok) give_up(abort, peer_abort, p.status);
      // copies in flight land before the pair may exit.  A phase also counts
      // the decoding warps, which may have given up: its bytes are then waited
      // for only as long as the limit allows.
      volatile int never = 0;
      for (int s = 0; s < STAGES; ++s)
        if (last[s] >= 0 &&
            !mbar_wait(&ctl->full[s], static_cast<uint32_t>(last[s]), &never, limit))
          give_up(abort, peer_abort, p.status);
    } else if (warp >= 2 && rank == 1 && lane == 0) {
      // ------------------------------------------------- decoded X, to the even CTA
      const uint32_t full0 = map_to_rank(smem_u32(&ctl->full[0]), 0);
      Ring ring;
      WorkIter it;
      it.init(sched, pair);
      WorkUnit w;
      bool ok = true;
      int turn = warp - 2;
      while (ok && it.next(sched, pairs, w))
        for (int kb = w.k0; kb < w.k1; ++kb, turn ^= 1) {
          if (turn == 0) {
            ok = mbar_wait(&ctl->decoded[ring.stage], ring.phase, abort, limit);
            if (!ok) break;
            mbar_arrive_cluster(full0 + ring.stage * 8);
          }
          ring.advance();
        }
      if (!ok) give_up(abort, peer_abort, p.status);
    } else if (warp == 1 && rank == 0 && lane == 0) {
      // -------------------------------------------------------------- MMAs
      constexpr uint32_t IDESC = idesc_bf16_f32(TILE, TILE, false, true);
      Ring ring;
      WorkIter it;
      it.init(sched, pair);
      WorkUnit w;
      bool ok = true, issued = false;
      int acc = 0;
      uint32_t acc_phase = 0;
      while (ok && it.next(sched, pairs, w)) {
        for (int k = w.k0; ok && k < w.k1; k += CHUNK) {
          const int k1 = k + CHUNK < w.k1 ? k + CHUNK : w.k1;
          ok = wait_cluster(&ctl->acc_empty[acc], acc_phase ^ 1u, abort, limit);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t d = tmem + acc * TILE;
          for (int kb = k; kb < k1; ++kb) {
            ok = wait_cluster(&ctl->full[ring.stage], ring.phase, abort, limit);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t a_addr = smem_u32(smem + ring.stage * STAGE_BYTES);
            const uint32_t b_addr = a_addr + A_BYTES;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_f16_ss_pair(d, sdesc_sw128(a_addr + kk / 4 * A_PART_BYTES + kk % 4 * 32, 16, 1024),
                              sdesc_sw128(b_addr + kk * 2048, B_BOX_BYTES, 1024), IDESC,
                              kb != k || kk != 0 ? 1u : 0u);
            issued = true;
            mma_commit_pair(&ctl->empty[ring.stage], 0x3);
            ring.advance();
          }
          if (!ok) break;
          mma_commit_pair(&ctl->acc_full[acc], 0x3);
          acc_phase ^= static_cast<uint32_t>(acc);
          acc ^= 1;
        }
      }
      if (!ok) give_up(abort, peer_abort, p.status);
      if (issued) {
        mma_commit_pair(&ctl->drain, 0x1);
        volatile int never = 0;
        if (!mbar_wait(&ctl->drain, 0u, &never, limit)) give_up(abort, peer_abort, p.status);
      }
    }
  } else if (warp < 4 + DECODE_WARPS) {
    // ------------------------------------------------- X: 8 bits to BF16
    regs_dec<kRegsDecode>();
    const int m = static_cast<int>(threadIdx.x) & 127;  // row of this CTA's part of the tile
    const int part = (warp - 4) / 4;                     // which 64 of a stage's rows of X
    const int blocks = (p.T + kCkptRun - 1) / kCkptRun * 2;  // 16-row pieces kept
    Ring ring;
    StageWalk sw;
    sw.init(sched, pair, pairs);
    bool ok = true;
    // Where this thread's row of X^T is kept: the stage's first 16-row piece
    // and its first scale.
    const uint4* src = nullptr;
    const uint8_t* codes = nullptr;
    int left = 0;  // 16-row pieces from there on; 0: the row is outside dW
    auto place = [&]() {
      left = 0;
      if (!sw.any) return;
      const int row = sw.tc.m * TILE + static_cast<int>(rank) * CTA_M + m;
      if (row >= p.K) return;
      const int64_t first = sw.kb * 8 + part * 4;
      src = reinterpret_cast<const uint4*>(p.q) + row + first * p.K;
      codes = p.scales + row + first / 2 * p.K;
      left = blocks - static_cast<int>(first);
    };
    auto next = [&]() {
      src += 8 * static_cast<int64_t>(p.K);
      codes += 4 * static_cast<int64_t>(p.K);
      left -= 8;
      if (sw.advance(sched, pairs)) place();
    };
    uint4 v[4];        // 16 values each
    uint32_t code[2];  // a run's scale byte each
    auto piece = [&](int i) {
      v[i] = i < left ? __ldg(src + static_cast<int64_t>(i) * p.K) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto scale = [&](int i) {
      code[i] = 2 * i < left ? __ldg(codes + static_cast<int64_t>(i) * p.K) : 1u;
    };
    place();
#pragma unroll
    for (int i = 0; i < 4; ++i) piece(i);
#pragma unroll
    for (int i = 0; i < 2; ++i) scale(i);
    uint64_t* done = rank == 0 ? ctl->full : ctl->decoded;
    while (sw.any) {
      ok = __all_sync(0xFFFFFFFFu,
                      mbar_wait(&ctl->empty[ring.stage], ring.phase ^ 1u, abort, limit));
      if (!ok) break;
      next();
      uint8_t* a = smem + ring.stage * STAGE_BYTES + part * A_PART_BYTES + m * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // 16 values to two 16-byte pieces; the next stage's take their place
        const uint32_t st = step_pair(code[i / 2]);
        const uint2 x = values(v[i].x, st), y = values(v[i].y, st);
        const uint2 z = values(v[i].z, st), w = values(v[i].w, st);
        piece(i);
        if (i % 2 == 1) scale(i / 2);
        *reinterpret_cast<uint4*>(a + (((2 * i) ^ (m & 7)) << 4)) = make_uint4(x.x, x.y, y.x, y.y);
        *reinterpret_cast<uint4*>(a + (((2 * i + 1) ^ (m & 7)) << 4)) =
            make_uint4(z.x, z.y, w.x, w.y);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(done + ring.stage);
      ring.advance();
    }
    if (!ok && lane == 0) give_up(abort, peer_abort, p.status);
  } else {
    // ------------------------------------------------------ sums and output
    regs_inc<kRegsSum>();
    const int ew = warp - 4 - DECODE_WARPS;  // 0..7
    const int quad = warp & 3;               // the tensor-memory lanes of this warp
    const int half = ew >> 2;                // its 128 columns of the tile
    uint8_t* box = boxes + ew * BOX_BYTES;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) +
                           static_cast<uint32_t>(half * 128);
    const uint32_t empty0 = map_to_rank(smem_u32(&ctl->acc_empty[0]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    WorkIter it;
    it.init(sched, pair);
    WorkUnit w;
    bool ok = true;
    auto counter = [&]() {  // of the unit's tile
      return p.counters + (static_cast<int64_t>(w.tile - sched.dp_tiles) * 2 + rank) * EPI_WARPS + ew;
    };
    while (ok && it.next(sched, pairs, w)) {
      float sum[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) sum[i] = 0.0f;
      for (int kb = w.k0; kb < w.k1; kb += CHUNK) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->acc_full[acc], acc_phase, abort, limit));
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(taddr + acc * TILE + c * 32, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[c * 32 + i] += __uint_as_float(r[i]);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(empty0 + acc * 8);
        acc_phase ^= static_cast<uint32_t>(acc);
        acc ^= 1;
      }
      if (!ok) break;
      const TileCoord tc = tile_order(w.tile, sched.tiles_m, sched.tiles_n, GROUP);
      const int row0 = tc.m * TILE + static_cast<int>(rank) * CTA_M + quad * 32;
      const int col0 = tc.n * TILE + half * 128;
      if (w.k0 != 0 || w.k1 != sched.num_kb) {
        // A segment.  Every segment but the last to arrive leaves its sums and
        // then counts; the last one adds all of them in row order.
        const SkTile st = sk_tile(sched, w.tile);
        auto slot = [&](int q) {
          return p.partial +
                 ((static_cast<int64_t>(q) * 2 + sk_slot(sched, q, w.tile)) * 2 + rank) *
                     (EPI_WARPS * 128 * 32) +
                 ew * (128 * 32) + lane;
        };
        float* mine = slot(pair);
#pragma unroll
        for (int i = 0; i < 128; ++i) mine[i * 32] = sum[i];
        __threadfence();
        __syncwarp();
        unsigned int before = 0;
        if (lane == 0) {
          before = atomicAdd(counter(), 1u);
          if (before + 1 == static_cast<unsigned int>(st.nseg)) *counter() = 0u;  // for the next launch
        }
        before = __shfl_sync(0xFFFFFFFFu, before, 0);
        __threadfence();
        if (before + 1 != static_cast<unsigned int>(st.nseg)) continue;
        // (of two segments only the other's: a + b == b + a)
        for (int s = 0; s < st.nseg; ++s) {
          const float* other = slot(st.q_first + s);
          if (st.nseg == 2) {
            if (st.q_first + s == pair) continue;
#pragma unroll
            for (int i = 0; i < 128; ++i) sum[i] += __ldcg(other + i * 32);
          } else if (s == 0) {
#pragma unroll
            for (int i = 0; i < 128; ++i) sum[i] = __ldcg(other + i * 32);
          } else {
#pragma unroll
            for (int i = 0; i < 128; ++i) sum[i] += __ldcg(other + i * 32);
          }
        }
      }
      const int rows = p.K - row0 < 32 ? p.K - row0 : 32;
      if (rows <= 0) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n0 = col0 + c * 32;
        if (n0 < p.N) {
          if (tma_w) {
            if (lane == 0) bulk_wait_read<0>();  // the box's last store has read it
            __syncwarp();
            if (p.beta != 0.0f && lane < rows) {
              const float* old = p.dW + static_cast<int64_t>(row0 + lane) * p.ldw + n0;
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                if (n0 + j < p.N) {  // N is a multiple of 4 on this path
                  const float4 o = *reinterpret_cast<const float4*>(old + j);
                  sum[c * 32 + j] = fmaf(p.beta, o.x, sum[c * 32 + j]);
                  sum[c * 32 + j + 1] = fmaf(p.beta, o.y, sum[c * 32 + j + 1]);
                  sum[c * 32 + j + 2] = fmaf(p.beta, o.z, sum[c * 32 + j + 2]);
                  sum[c * 32 + j + 3] = fmaf(p.beta, o.w, sum[c * 32 + j + 3]);
                }
            }
          } else {
            __syncwarp();  // the box's last rows have been read
          }
          uint8_t* mine = box + lane * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(mine + ((j ^ (lane & 7)) << 4)) =
                make_float4(sum[c * 32 + 4 * j], sum[c * 32 + 4 * j + 1], sum[c * 32 + 4 * j + 2],
                            sum[c * 32 + 4 * j + 3]);
          if (tma_w) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmW, box, n0, row0);
              bulk_commit();
            }
          } else {
            __syncwarp();
            if (n0 + lane < p.N) {
              float* out = p.dW + static_cast<int64_t>(row0) * p.ldw + n0 + lane;
#pragma unroll 4
              for (int r = 0; r < rows; ++r) {
                const float v = *reinterpret_cast<const float*>(
                    box + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                float* o = out + static_cast<int64_t>(r) * p.ldw;
                *o = p.beta != 0.0f ? fmaf(p.beta, *o, v) : v;
              }
            }
          }
        }
      }
    }
    if (!ok && lane == 0) {
      give_up(abort, peer_abort, p.status);
      // The segments left are not summed, but they count all the same, so that
      // the counters are at zero after this launch too.
      do {
        if (w.k0 == 0 && w.k1 == sched.num_kb) continue;
        if (atomicAdd(counter(), 1u) + 1 == static_cast<unsigned int>(sk_tile(sched, w.tile).nseg))
          *counter() = 0u;
      } while (it.next(sched, pairs, w));
    }
    if (lane == 0) bulk_wait_all();  // every store has completed before the CTA exits
  }

  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

constexpr size_t kSmemBytes = 1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + EPI_BYTES +
                              sizeof(Control);

void config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int pairs, cudaStream_t stream) {
  *cfg = cudaLaunchConfig_t{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg->gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg->blockDim = dim3(THREADS);
  cfg->dynamicSmemBytes = kSmemBytes;
  cfg->stream = stream;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

// Per device: resident pairs + 1 once the shared-memory attribute is set.
std::atomic<int> g_pairs_plus1[64];

}  // namespace

int ckpt8_wgrad_pairs() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int known = g_pairs_plus1[dev].load(std::memory_order_acquire);
  if (known > 0) return known - 1;
  // The role's register shares are drawn from what the block is launched with.
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, ckpt8_wgrad_kernel) != cudaSuccess ||
      fa.numRegs * THREADS < kRegsBlock)
    return 0;
  if (cudaFuncSetAttribute(ckpt8_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemBytes)) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  config(&cfg, attr, 1, nullptr);
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, ckpt8_wgrad_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  g_pairs_plus1[dev].store(n + 1, std::memory_order_release);
  return n;
}

PairSchedule ckpt8_wgrad_schedule(int64_t T, int64_t K, int64_t N, int max_pairs) {
  PairSchedule s;
  s.tiles_m = static_cast<int>((K + TILE - 1) / TILE);
  s.tiles_n = static_cast<int>((N + TILE - 1) / TILE);
  s.num_kb = static_cast<int>((T + BK - 1) / BK);
  const int64_t tiles = static_cast<int64_t>(s.tiles_m) * s.tiles_n;
  const int64_t rest = tiles % max_pairs;
  int64_t sk = 0;
  // What the split saves of the last wave, in stages, against the exchange of
  // the segments' sums (kSplitStages).
  if (rest > 0 && (max_pairs - rest) * s.num_kb > kSplitStages * max_pairs) {
    // the partial last wave, with the last whole one if there is one
    sk = tiles > max_pairs ? rest + max_pairs : rest;
    // runs of at least half a tile: at most kSkMaxSeg segments a tile
    int64_t p = 2 * sk < max_pairs ? 2 * sk : max_pairs;
    s.sk_pairs = static_cast<int>(p);
  }
  s.sk_tiles = static_cast<int>(sk);
  s.dp_tiles = static_cast<int>(tiles - sk);
  s.num_full = s.dp_tiles;
  const int64_t most = s.dp_tiles > s.sk_pairs ? s.dp_tiles : s.sk_pairs;
  s.pairs = static_cast<int>(most < max_pairs ? most : max_pairs);
  return s;
}

int64_t ckpt8_wgrad_partial_bytes(const PairSchedule& s) {
  return static_cast<int64_t>(s.sk_pairs) * 2 * 2 * EPI_WARPS * 128 * 32 * 4;
}
int64_t ckpt8_wgrad_counters(const PairSchedule& s) {
  return static_cast<int64_t>(s.sk_tiles) * 2 * EPI_WARPS;
}

cudaError_t launch_ckpt8_wgrad(const CUtensorMap& tmY, const CUtensorMap* tmW,
                               const PairSchedule& s, int T, int K, int N, const uint8_t* q,
                               const uint8_t* scales, float* dW, int64_t ldw, float beta,
                               float* partial, unsigned int* counters, unsigned int* status,
                               cudaStream_t stream) {
  if (s.pairs <= 0) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  config(&cfg, attr, s.pairs, stream);
  CUtensorMap none;
  std::memset(&none, 0, sizeof(none));
  const WgradArgs a = {T, K, N, q, scales, dW, ldw, beta, partial, counters, status};
  const cudaError_t e = cudaLaunchKernelEx(&cfg, ckpt8_wgrad_kernel, tmY, tmW ? *tmW : none, s, a,
                                           tmW ? 1 : 0);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace g07
