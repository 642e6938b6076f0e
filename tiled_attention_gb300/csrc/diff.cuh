// diff.cuh — differential attention forward for sm_103a: dense and document masks, and chunks of
// new tokens over a paged KV cache.
//
// A head has two maps of D/2 channels side by side in q and k and one value row of D channels:
//   A_m = softmax(scale q_m k_m^T + mask),  y = A_1 v - lam A_2 v,
//   O = out_scale * y * w / sqrt(mean y^2 + eps)        (without w: O = out_scale * y)
//
// Both maps run over the same keys, so one pass over K and V serves them: a work unit is one
// 128-row query tile of one (batch or segment, query head), and what the ordinary kernel's two
// query tiles are there, the two maps are here. K_j and V_j are loaded once for both, and the
// difference and the norm are taken in registers at the end, so that neither A_1 v nor A_2 v ever
// leaves the SM. Each map keeps its own running max and sum (the sums differ, so the accumulators
// cannot be joined before the end).
//
// Roles (384 threads, or 256):
//   warp 0      finds the CTA's units (below) and loads by TMA: the unit's Q tile, then K_j and V_j
//               of a tile into one stage of a ring
//   warps 1, 2  MMA issuers of map 0 and 1: S_m = Q_m K_m^T (SS; map m is k-steps [m D/32,
//               (m + 1) D/32) of the tile's swizzled rows) and O_m += P_m V (P from TMEM); warp 1
//               owns TMEM. One issuer for both maps kept the tensor core waiting (causal 2 x 8192
//               1158 us against 1105).
//   warp 3      paged, pages under 64 tokens: the V pages
//   warps 4-7   softmax of map 0, warps 8-11 of map 1; a thread owns one query row. At the end
//               warps q of both take columns [0, D/2) and [D/2, D) of both accumulators: x = O_0 /
//               l_0 - lam O_1 / l_1, the row's sum of squares is exchanged through shared
//               memory, and the scaled row goes out by TMA. (Or four warps take both maps in turn,
//               and a thread has all of its row.)
// TMEM columns: S of map m, buffer b of kSBufs at (kSBufs m + b) BN (P takes the place of its S),
// then O_0 and O_1, D each.
//
// Key tiles are of 64 keys with two S buffers a map (one tile of 128 and one buffer: causal 2 x 8192
// 1253 us against 1105); 96 where d = 64 leaves the columns. At d = 64 and with many units two CTAs
// share an SM, with one S buffer a map each: the softmax is what bounds it there, and more of it is
// in flight (a window of 1000 over 3 x 5003 150 us with one CTA and 131 with two, chunks of 64 heads
// over 16K contexts 1030 and 863). Over pages eight softmax warps a CTA hide one another's waits, with
// 32 columns of scores in registers at a time (all 64 spilled: the window 183 us with eight warps,
// which take 141 without spills). Else four warps, which take both maps in turn (window 131, 200
// prompts of 17 tokens 48 against 55; over pages they take 897 against 862).
//
// A warp goes by its own 32 rows: a tile that all of them see all of takes the short loop, one that
// none sees gets P = 0 (by the unit's 128 rows: window 146 us against 142).
//
// Units: the grid has a block a unit, the longest first (two-sided documents go in the order of causal
// ones: the first units of a long one, as long as its last, begin at the end); a resident CTA takes
// over a block that has not begun by cancelling its launch (cluster launch control), so that uneven
// units (chunks of many lengths) spread as CTAs get done: 16 chunks 2926 to 2636 us against a fixed
// walk, five small ones 78 to 57. Finding units costs warp 0 alone; the other warps read them from
// shared memory.
//
// What bounds it: a tile of 64 keys takes the tensor core 854 cycles for both maps at D = 128 (S
// with N = 64 runs below the full rate; 768 would be the operations'), the exponentials 512 and the
// loop 1068. P is rounded to bf16 (2^-8 of a weight at most), which is most of the output's error:
// 2.6e-3 of |O| in 2-norm, where the output's own rounding is 1.7e-3. The rounding's rest as a second
// bf16 term in the other half of S's columns leaves 1.7e-3 and costs a quarter to a third: causal 2 x
// 8192 1080 to 1387 us, 16 chunks 2356 to 3035, window of 1000 131 to 165, chunks of 64 heads over 16K
// 864 to 1175. So one term; sums are those of the unrounded weights, in fp32.
//
// Measured (heads 32 over 8, D = 128): causal 2 x 8192 1077 us in bursts of three at 2.07 GHz = 1.53
// PFLOP/s of the pairs under the mask, and 1171 on end, where the power limit holds the clock at 1.90
// GHz; 16 chunks of up to 2048 tokens over up to 16K 2.33 ms, and 2.56 at 1.83 GHz. D = 64, 3 x 5003,
// window of 1000 131 to 134 us at 2.07 GHz either way.
#pragma once

#include <cuda_bf16.h>

#include "norm.cuh"
#include "prefill.cuh"
#include "ptx.cuh"
#include "sched.h"
#include "share.cuh"

namespace ta {

struct DiffParams {
  PrefillParams base;    // o, lse [planes, 2, N], lengths, table, sizes; scale of the maps' scores
  const float* lam;      // [Hq]
  const float* weight;   // [D] or null
  float eps, out_scale;
  int mask;              // of the dense and document kinds
  int head_shift;        // log2 of the heads that may share a tile: a power of two that divides group
};

// A tile's sum of a row's weights above which its reference max is raised: 2^24, so that weights
// times values stay finite for values up to 2^80.
constexpr float kDiffRaise = 16777216.f;

constexpr int imin_c(int a, int b) { return a < b ? a : b; }

// CTAS: of an SM.
template <int D, int PACK, int CTAS>
struct DiffCfg {
  static_assert(CTAS == 1 || D == 64, "TMEM holds two CTAs' accumulators of 64 columns");
  static constexpr int BM = 128;
  static constexpr int BN = D == 64 && PACK != kMaskPagedPrefill && CTAS == 1 ? 96 : 64;
  static constexpr int kCtas = CTAS;
  static constexpr int kSBufs = 3 - kCtas;           // S buffers a map
  static constexpr int kMapsPerWarp = CTAS == 2 && PACK != kMaskPagedPrefill ? 2 : 1;
  static constexpr int kSoftmaxWarps = 8 / kMapsPerWarp;
  static constexpr int kThreads = 128 + 32 * kSoftmaxWarps;
  static constexpr int kPanels = D / 64;
  static constexpr int kQPanelBytes = BM * 128;      // 64 columns of a Q tile
  static constexpr int kQBytes = BM * D * 2;
  static constexpr int kPanelBytes = BN * 128;       // 64 columns of a K or V tile
  static constexpr int kTileBytes = BN * D * 2;
  static constexpr int kStageBytes = 2 * kTileBytes; // K, then V
  static constexpr int kQBufs = 2;                   // this unit's and the next one's
  static constexpr int kCtrlBytes = 2048;
  static constexpr int kStages =
      imin_c((233472 / kCtas - 2048 - kCtrlBytes - kQBufs * kQBytes) / kStageBytes, 8);
  static constexpr int kSmemBytes = 1024 + kQBufs * kQBytes + kStages * kStageBytes + kCtrlBytes;
  static constexpr int kTmemCols = 512 / kCtas;
  static constexpr int kOCol = 2 * kSBufs * BN;
  static constexpr int kSteps = D / 32;              // 16-channel k-steps of one map
  static constexpr int kHalf = D / 2;                // columns of O a softmax warp writes
  static constexpr int kRegsLaunch = 65536 / kCtas / kThreads / 8 * 8;
  static constexpr uint32_t kRegsControl = CTAS == 1 ? 88 : 48;
  static constexpr uint32_t kRegsSoftmax = CTAS == 2 && kMapsPerWarp == 1 ? 96 : 208;
  static_assert(128 * kRegsControl + 32 * kSoftmaxWarps * kRegsSoftmax <= kThreads * kRegsLaunch,
                "register split");
  static_assert((kSmemBytes + 1024) * kCtas <= 233472, "shared memory");
  static_assert(kOCol + 2 * D <= kTmemCols, "TMEM columns");
  static constexpr uint32_t kIdescS = idesc_bf16(BM, BN, false, false);
  static constexpr uint32_t kIdescO = idesc_bf16(BM, D, false, true);
};

// A work unit as the producer hands it to the other warps, with its key tiles. Where at most 64 rows
// of a segment are left, the tile takes those of several heads of one kv head, a power of two (at
// least 8) of rows each; the other heads' units are not there (dense masks) or have no work (32 chunks
// of up to 16 tokens over 500-4000, 64 heads over 4, d = 64: 278 to 97 us; 32 over 8, d = 128: 192 to
// 101; 64 dense prompts of 40 tokens 43 to 30).
struct DiffTask {
  Unit un;
  KvRange rng;
  int rows_log2;  // of one head's rows in the tile
};

struct DiffCtrl {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t s_ready[2][2], p_ready[2][2];  // of map m, buffer b
  uint64_t o_done, drain[2];
  uint64_t both[4];          // warps q of the two softmax warpgroups
  uint64_t task_full[2], task_empty[2], asked[2];
  alignas(16) uint4 answer[2];  // of the requests for another unit
  DiffTask task[2];
  uint32_t tmem_base;
  int abort_flag;
  float coef[2][128];        // 1 / l of map 0's rows, lam / l of map 1's
  alignas(16) float weight[128];  // out_scale * w
};

// One lane's commit to a barrier by its shared-memory address: `lead` is set in the lane that
// issues the MMAs.
__device__ __forceinline__ void commit_at(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(
          bar),
      "r"(lead)
      : "memory");
}

// N SS MMAs of one accumulator from the lane where `lead` is set: k-steps of 16 columns, 32 bytes
// apart in both operands; the first overwrites D.
template <int N>
__device__ __forceinline__ void mma_ss_steps(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t lead) {
  static_assert(N == 2 || N == 4, "k-steps");
  if constexpr (N == 4)
    asm volatile(
        "{\n .reg .pred e, t, f;\n .reg .b64 a1, b1, a2, b2, a3, b3;\n"
        " setp.ne.b32 t, 1, 0;\n setp.ne.b32 f, 0, 0;\n"
        " add.s64 a1, %1, 2;\n add.s64 b1, %2, 2;\n add.s64 a2, %1, 4;\n add.s64 b2, %2, 4;\n"
        " add.s64 a3, %1, 6;\n add.s64 b3, %2, 6;\n"
        " setp.ne.b32 e, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred e, t, f;\n .reg .b64 a1, b1;\n"
        " setp.ne.b32 t, 1, 0;\n setp.ne.b32 f, 0, 0;\n"
        " add.s64 a1, %1, 2;\n add.s64 b1, %2, 2;\n"
        " setp.ne.b32 e, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(lead)
        : "memory");
}

// N TS MMAs of one accumulator from the lane where `lead` is set: A from TMEM, 8 columns a 16-key
// step, B an MN-major operand whose steps are 2048 bytes apart; the first accumulates iff acc0.
template <int N>
__device__ __forceinline__ void mma_ts_steps(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                             uint32_t acc0, uint32_t lead) {
  static_assert(N == 4 || N == 6, "k-steps");
  asm volatile(
      "{\n .reg .pred e, t, p;\n .reg .b64 b1, b2, b3;\n .reg .b32 a1, a2, a3;\n"
      " setp.ne.b32 t, 1, 0;\n setp.ne.b32 p, %4, 0;\n"
      " add.s32 a1, %1, 8;\n add.s32 a2, %1, 16;\n add.s32 a3, %1, 24;\n"
      " add.s64 b1, %2, 128;\n add.s64 b2, %2, 256;\n add.s64 b3, %2, 384;\n"
      " setp.ne.b32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc0), "r"(lead)
      : "memory");
  if constexpr (N == 6)
    asm volatile(
        "{\n .reg .pred e, t;\n .reg .b64 b1;\n .reg .b32 a1;\n setp.ne.b32 t, 1, 0;\n"
        " add.s32 a1, %1, 8;\n add.s64 b1, %2, 128;\n"
        " setp.ne.b32 e, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n}" ::"r"(d),
        "r"(a + 32), "l"(b + 512), "r"(idesc), "r"(lead)
        : "memory");
}

// Asks for the launch of a block that has not begun to be cancelled and handed to this CTA; the
// answer (16 bytes) lands in `to` and on `bar`. One thread. Not to be asked again after a refusal.
__device__ __forceinline__ void ask_unit(uint4* to, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(smem_u32(to)),
      "r"(smem_u32(bar))
      : "memory");
}
// The cancelled block's index, -1 where none was left.
__device__ __forceinline__ int unit_answer(const uint4* from) {
  int x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 h;\n .reg .b32 y;\n ld.shared.b128 h, [%1];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n mov.b32 %0, -1;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n}"
      : "=r"(x)
      : "r"(smem_u32(from))
      : "memory");
  return x;
}

// log2 of one head's rows in a tile that begins with `left` rows of a segment left.
TA_HD int tile_rows_log2(int left, int head_shift) {
  int log2 = 7 - head_shift;
  if (log2 < 3) log2 = 3;
  while (log2 < 7 && (1 << log2) < left) ++log2;
  return log2;
}

// Work unit u in launch order: 128-row tiles from the last one down, then batch and head; packed
// kinds take the two halves of prefill.cuh's 256-row units, the later (longer) one first. q_row0
// may lie past the segment (an odd number of tiles): that unit has no key tiles.
template <int PACK>
__device__ __forceinline__ Unit diff_unit(int u, const DiffParams& dp, UnitCursor& cur) {
  const PrefillParams& p = dp.base;
  if constexpr (PACK != kMaskNone) {
    Unit r = decode_unit<PACK>(u >> 1, p, cur);
    if (r.valid && !(u & 1)) r.q_row0 += 128;
    return r;
  } else {
    Unit r{0, 0, 0, 0, 0, 0, 0};
    const int per_level = p.B * p.Hq;
    // The last tiles, several heads of which may be one unit.
    const int top = tiles_for_rows(p.N) - 1;
    const int s = 7 - tile_rows_log2(p.N - 128 * top, dp.head_shift);
    const int over = u - (per_level >> s);
    const int level = over < 0 ? top : top - 1 - over / per_level;
    if (level < 0) return r;
    const int bh = over < 0 ? u << s : over % per_level;
    r.valid = 1;
    r.bh = bh;
    r.kvh = (bh / p.Hq) * p.Hkv + (bh % p.Hq) / p.group;
    r.q_row0 = level * 128;
    r.k_end = p.N;
    return r;
  }
}

template <int D, int PACK, int CTAS>
__global__ void __launch_bounds__((DiffCfg<D, PACK, CTAS>::kThreads), CTAS)
    diff_prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_q8,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_o, const DiffParams dp) {
  using C = DiffCfg<D, PACK, CTAS>;
  constexpr int BM = C::BM, BN = C::BN, STAGES = C::kStages, QB = C::kQBufs;
  constexpr int SB = C::kSBufs, MW = C::kMapsPerWarp;
  constexpr bool kPaged = PACK == kMaskPagedPrefill;
  constexpr unsigned kFull = 0xffffffffu;
  const PrefillParams& p = dp.base;
  const int mask = kPaged ? static_cast<int>(kMaskPagedPrefill) : dp.mask;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* q_s = smem;
  uint8_t* kv_s = smem + QB * C::kQBytes;
  DiffCtrl* ctl = reinterpret_cast<DiffCtrl*>(kv_s + STAGES * C::kStageBytes);
  static_assert(sizeof(DiffCtrl) <= C::kCtrlBytes, "control block");

  const int warp = static_cast<int>(threadIdx.x >> 5);
  const int lane = static_cast<int>(lane_id());
  if (warp == 0) {
    if (lane == 0) {
      ctl->abort_flag = 0;
      for (int q = 0; q < QB; ++q) {
        mbar_init(&ctl->q_full[q], 1);
        mbar_init(&ctl->q_empty[q], C::kSoftmaxWarps);  // one arrival per softmax warp
      }
      for (int s = 0; s < STAGES; ++s) {
        mbar_init(&ctl->kv_full[s], kPaged ? 2 : 1);  // an arrival for K, one for V
        mbar_init(&ctl->kv_empty[s], 2);  // one release per issuing warp
      }
      for (int m = 0; m < 2; ++m) {
        for (int x = 0; x < 2; ++x) {
          mbar_init(&ctl->s_ready[m][x], 1);
          mbar_init(&ctl->p_ready[m][x], 4);  // one arrival per warp
        }
        mbar_init(&ctl->drain[m], 1);
      }
      mbar_init(&ctl->o_done, 2);
      for (int q = 0; q < 4; ++q) mbar_init(&ctl->both[q], 2);
      const int readers = 2 + C::kSoftmaxWarps + (kPaged && p.page_shift < 6 ? 1 : 0);
      for (int s = 0; s < 2; ++s) {
        mbar_init(&ctl->task_full[s], 1);
        mbar_init(&ctl->task_empty[s], readers);  // the issuers, softmax warps and V's producer
        mbar_init(&ctl->asked[s], 1);
      }
      fence_mbar_init();
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
      prefetch_tensormap(&tm_o);
    }
  } else if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, C::kTmemCols);
    tmem_relinquish();
  } else if (warp >= 4) {
    const int c = static_cast<int>(threadIdx.x) - 128;
    if (c < D) ctl->weight[c] = dp.weight ? __ldg(dp.weight + c) * dp.out_scale : dp.out_scale;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = ctl->tmem_base;
  const WaitCtl wc{p.timeout_ns, p.status, &ctl->abort_flag};
  const WaitCtl wc_drain{p.timeout_ns, p.status, nullptr};
  // Unit n of this CTA, from the producer; false at the end.
  auto read_task = [&](int n, DiffTask& task) {
    if (!wait_at(smem_u32(&ctl->task_full[n & 1]), (n >> 1) & 1, wc)) return false;
    task = ctl->task[n & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->task_empty[n & 1]);
    return task.un.valid != 0;
  };

  if (warp < 4) {
    regs_decrease<C::kRegsControl>();
    const bool split_v = kPaged && p.page_shift < 6;
    if (warp == 0 || (split_v && warp == 3)) {
      // -------------------------------------------------------------- TMA producer
      // Warp 0 finds the CTA's units: the first by its block index, another by cancelling the
      // launch of the next block that waits (the grid has a block a unit, longest units first), so
      // that CTAs take units as they get done with theirs. It asks one unit ahead.
      int e = 0;   // K/V stages
      int qn = 0;  // Q loads issued
      int asked = 0, answered = 0;
      bool ok = true;
      UnitCursor cur{0, 0, 0, 0};
      int u = static_cast<int>(blockIdx.x);
      DiffTask task;
      for (int n = 0; ok;) {
        if (warp == 0) {
          if (lane == 0) ask_unit(&ctl->answer[asked & 1], &ctl->asked[asked & 1]);
          ++asked;
          task.un = diff_unit<PACK>(u, dp, cur);  // warp-collective
          task.rows_log2 = tile_rows_log2(task.un.k_end - task.un.q_row0, dp.head_shift);
          if (task.un.bh & ((128 >> task.rows_log2) - 1)) task.un.valid = 0;
          task.rng = kv_tile_range(mask, p.window, task.un.q_row0, BM, task.un.k_end, task.un.k_org,
                                   task.un.k_end, BN);
          const bool work = task.un.valid && task.rng.hi > task.rng.lo;
          if (work) {
            ok = wait_at(smem_u32(&ctl->task_empty[n & 1]), ((n >> 1) & 1) ^ 1, wc);
            if (!ok) break;
            if (lane == 0) {
              ctl->task[n & 1] = task;
              mbar_arrive(&ctl->task_full[n & 1]);
            }
            __syncwarp();
          } else {
            task.rng.hi = task.rng.lo = 0;
          }
          if (work) ++n;
        } else {
          if (!read_task(n, task)) break;
          ++n;
        }
        const Unit& un = task.un;
        const KvRange rng = task.rng;
        const int npos = rng.hi - rng.lo;
        if (npos > 0) {
          if (warp == 0) {
            const int qb = qn % QB;
            ok = wait_at(smem_u32(&ctl->q_empty[qb]), ((qn / QB) & 1) ^ 1, wc);
            if (!ok) break;
            ++qn;
            if (lane == 0) mbar_arrive_expect_tx(&ctl->q_full[qb], C::kQBytes);
            __syncwarp();
            uint8_t* dst = q_s + qb * C::kQBytes;
            if (task.rows_log2 == 7) {
              if (lane < C::kPanels)
                tma_load_3d(dst + lane * C::kQPanelBytes, &tm_q, &ctl->q_full[qb], lane * 64,
                            un.q_row0, un.bh);
            } else if (lane < 16) {  // rows of several heads, eight at a time
              const int at = 8 * lane;
              for (int c = 0; c < C::kPanels; ++c)
                tma_load_3d(dst + c * C::kQPanelBytes + at * 128, &tm_q8, &ctl->q_full[qb], c * 64,
                            un.q_row0 + (at & ((1 << task.rows_log2) - 1)),
                            un.bh + (at >> task.rows_log2));
            }
          }
          for (int x = 0; !kPaged && x < npos; ++x, ++e) {
            const int st = e % STAGES;
            ok = wait_at(smem_u32(&ctl->kv_empty[st]), ((e / STAGES) & 1) ^ 1, wc);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&ctl->kv_full[st], C::kStageBytes);
            __syncwarp();
            if (lane < 2 * C::kPanels)  // panels of K, then of V
              tma_load_3d(kv_s + st * C::kStageBytes + lane * C::kPanelBytes,
                          lane < C::kPanels ? &tm_k : &tm_v, &ctl->kv_full[st],
                          lane % C::kPanels * 64, un.k_org + (rng.lo + x) * BN, un.kvh);
          }
          if constexpr (kPaged) {
            // A lane issues a box of a page of the key tile (one half of a page of 128);
            // pages past the context or outside the pool come from the zero-filled plane past it.
            const int lp = p.page_shift;
            const int run = imin(BN, 1 << lp), nb = BN / run, sb = lane & (nb - 1);
            const int lk = un.k_end - un.k_org;
            const int* trow = p.table + static_cast<size_t>(un.seq) * p.max_pages;
            PageEntries pages(trow, rng.lo * BN, run, lp, lk);
            // With pages under 64 tokens warp 0 brings K and warp 3 V, else warp 0 both.
            const int first = warp == 3 ? 1 : 0, last = split_v && warp == 0 ? 0 : 1;
            for (int x = 0; x < npos && ok; ++x, ++e) {
              const int st = e % STAGES;
              ok = wait_at(smem_u32(&ctl->kv_empty[st]), ((e / STAGES) & 1) ^ 1, wc);
              if (!ok) break;
              if (lane == 0)
                for (int y = first; y <= last; ++y)
                  mbar_arrive_expect_tx(&ctl->kv_full[st], C::kTileBytes);
              __syncwarp();
              const int raw = pages.at(x * nb, sb);
              int pl = p.num_pages * p.Hkv;
              if (raw >= 0 && raw < p.num_pages)
                pl = raw * p.Hkv + un.kvh;
              else if (lane < nb && (rng.lo + x) * BN + sb * run < lk)
                report_status(p.status, -5);
              const int kind = first * C::kPanels + lane / nb;  // panels of K, then of V
              if (kind < (last + 1) * C::kPanels) {
                const int row0 = nb > 1 ? 0 : ((rng.lo + x) * BN) & ((1 << lp) - 1);
                tma_load_3d(kv_s + st * C::kStageBytes + kind * C::kPanelBytes + sb * run * 128,
                            kind < C::kPanels ? &tm_k : &tm_v, &ctl->kv_full[st],
                            kind % C::kPanels * 64, row0, pl);
              }
            }
          }
        }
        if (warp == 0 && ok) {
          ok = wait_at(smem_u32(&ctl->asked[answered & 1]), (answered >> 1) & 1, wc);
          if (!ok) break;
          const int before = u;
          u = unit_answer(&ctl->answer[answered & 1]);
          // Every lane's read of the answer comes before the request that has its place next.
          fence_proxy_async_smem();
          __syncwarp();
          ++answered;
          if (u < before) cur = UnitCursor{0, 0, 0, 0};  // the cursor only goes up
          if (u < 0) {  // no unit left: tell the others
            ok = wait_at(smem_u32(&ctl->task_empty[n & 1]), ((n >> 1) & 1) ^ 1, wc);
            if (ok && lane == 0) {
              ctl->task[n & 1].un.valid = 0;
              mbar_arrive(&ctl->task_full[n & 1]);
            }
            break;
          }
        }
      }
      if (lane == 0) {
        // Let copies and answers still in flight land before the CTA can exit (no-op on the normal
        // path).
        for (; answered < asked; ++answered)
          mbar_wait(&ctl->asked[answered & 1], (answered >> 1) & 1, wc_drain);
        for (int x = imax(0, e - STAGES); x < e; ++x)
          mbar_wait(&ctl->kv_full[x % STAGES], (x / STAGES) & 1, wc_drain);
        for (int x = imax(0, qn - QB); x < qn; ++x)
          mbar_wait(&ctl->q_full[x % QB], (x / QB) & 1, wc_drain);
      }
    } else if (warp == 1 || warp == 2) {
      // -------------------------------------------------------------- MMA issuers
      // Warp 1 issues map 0's MMAs, warp 2 map 1's. S of the first SB positions go first; step x is
      // P V of position x, then S of x + SB into the buffer that P V has just read (MMAs of one
      // thread run in order). With two buffers the map's next S is there when its softmax is done
      // with this one. Every ring entry takes one release from each issuer.
      const int m = warp - 1;
      uint32_t lead;
      asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}"
                   : "=r"(lead));
      const uint32_t full0 = smem_u32(ctl->kv_full), empty0 = smem_u32(ctl->kv_empty);
      const uint32_t s_bar = smem_u32(ctl->s_ready[m]), p_bar = smem_u32(ctl->p_ready[m]);
      // Operands of map m in stage 0 and the Q tiles: a map's k-steps are 32 bytes apart inside a
      // 128-byte swizzle row, four steps a panel.
      constexpr int kPer = 4 / C::kSteps;  // maps of a panel
      const uint64_t k_desc0 =
          sw128_desc(smem_u32(kv_s), 16, 1024) +
          ((m / kPer * C::kPanelBytes + m % kPer * C::kSteps * 32) >> 4);
      const uint64_t v_desc0 = sw128_desc(smem_u32(kv_s) + C::kTileBytes, C::kPanelBytes, 1024);
      const uint64_t q_desc0 =
          sw128_desc(smem_u32(q_s), 16, 1024) +
          ((m / kPer * C::kQPanelBytes + m % kPer * C::kSteps * 32) >> 4);
      const uint32_t d_s = tmem + C::kSBufs * m * BN, d_o = tmem + C::kOCol + m * D;
      // Stage of the next S and of the next P V, the parity of the former's, and of Q's and P's.
      int st_s = 0, st_v = 0, qn = 0;
      uint32_t ph_s = 0, ph_p = 0;
      uint32_t buf = 0;  // S buffer of the next P
      bool ok = true;
      DiffTask task;
      for (int n = 0; ok && read_task(n, task); ++n) {
        const int npos = task.rng.hi - task.rng.lo;
        const uint64_t q_desc = q_desc0 + (qn % QB) * (C::kQBytes >> 4);
        auto issue_s = [&](uint32_t b) {
          mma_ss_steps<C::kSteps>(d_s + b * BN, q_desc, k_desc0 + st_s * (C::kStageBytes >> 4),
                                  C::kIdescS, lead);
          commit_at(s_bar + 8 * b, lead);
          if (++st_s == STAGES) st_s = 0, ph_s ^= 1;
        };
        ok = wait_at(smem_u32(&ctl->q_full[qn % QB]), (qn / QB) & 1, wc);
        for (int x = 0; x < SB && x < npos && ok; ++x) {
          ok = wait_at(full0 + 8 * st_s, ph_s, wc);
          if (!ok) break;
          tc_fence_after();
          issue_s(buf ^ x);
        }
        if (!ok) break;
        for (int x = 0; x < npos; ++x) {
          // P and the next K together: looking at a barrier takes 80 cycles, and the tensor core
          // may run dry meanwhile.
          const bool more = x + SB < npos;
          const bool rp = try_wait_at(p_bar + 8 * buf, ph_p);
          const bool rk = !more || try_wait_at(full0 + 8 * st_s, ph_s);
          if (!__all_sync(kFull, rp && rk)) {
            ok = wait_at(p_bar + 8 * buf, ph_p, wc) &&
                 (!more || wait_at(full0 + 8 * st_s, ph_s, wc));
            if (!ok) break;
          }
          tc_fence_after();
          // The unit's first P V overwrites O_m: both warps of every row published this P after
          // they had read O of the unit before.
          mma_ts_steps<BN / 16>(d_o, d_s + buf * BN, v_desc0 + st_v * (C::kStageBytes >> 4),
                                C::kIdescO, x > 0, lead);
          if (more) issue_s(buf);
          commit_at(empty0 + 8 * st_v, lead);  // K and V of the stage are done with
          if (++st_v == STAGES) st_v = 0;
          ph_p ^= buf | (SB == 1);
          buf ^= SB - 1;
        }
        commit_at(smem_u32(&ctl->o_done), lead);
        ++qn;
      }
      // Every MMA this warp issued has completed before TMEM can be released.
      commit_at(smem_u32(&ctl->drain[m]), lead);
      mbar_wait(&ctl->drain[m], 0, wc_drain);
    }
  } else {
    regs_increase<C::kRegsSoftmax>();
    // ---------------------------------------------------------------- softmax warpgroups
    // A warp takes one map, or both in turn, so that one map's products run under the other's
    // exponentials.
    int m = MW == 2 ? 0 : (warp - 4) >> 2;  // map
    const int quarter = warp & 3;           // TMEM lanes [32*quarter, 32*quarter + 32)
    const int r = quarter * 32 + lane;      // row inside the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_bar0 = smem_u32(ctl->s_ready);
    const float c = p.scale_log2;
    int sc = 0;          // S tiles of a map consumed
    int un_done = 0;     // units with work finished
    int e = 0;           // stage of the unit's first key tile
    int pending_q = -1;  // Q buffer whose O store may still be reading it
    auto release_pending = [&]() {
      if (pending_q >= 0) {
        if (lane == 0) {
          bulk_wait_group_read0();
          mbar_arrive(&ctl->q_empty[pending_q]);
        }
        __syncwarp();
        pending_q = -1;
      }
    };
    bool ok = true;
    DiffTask task;
    for (int n = 0; ok && read_task(n, task); ++n) {
      const Unit un = task.un;
      const KvRange rng = task.rng;
      // This thread's row: of head bh, which several of may lie in the tile.
      const int rl = task.rows_log2;
      const int k_org = un.k_org, k_end = un.k_end, bh = un.bh + (r >> rl);
      const int row = un.q_row0 + (r & ((1 << rl) - 1));
      const int key0 = k_org + rng.lo * BN;  // keys below are counted from it
      // A row past the segment goes as the last one.
      const int see_lo = vis_lo(mask, p.window, k_org, imin(row, k_end - 1)) - key0;
      const int see_hi = vis_hi(mask, p.window, k_end, imin(row, k_end - 1)) - key0;
      // This warp's rows: all of them see all of a tile that begins in [full_lo, full_hi], and the
      // tiles before j_full begin by full_hi; none sees any of one outside [some_lo, some_hi].
      const int last = imin(31, (1 << rl) - 1);  // lane 0 has the first row, this one the last
      const int full_lo = __shfl_sync(kFull, see_lo, last);
      const int full_hi = __shfl_sync(kFull, see_hi, 0) - (BN - 1);
      const int some_lo = __shfl_sync(kFull, see_lo, 0) - (BN - 1);
      const int some_hi = __shfl_sync(kFull, see_hi, last);
      const int j_full = full_hi < 0 ? rng.lo : imin(rng.hi, rng.lo + full_hi / BN + 1);
      const float lam = MW == 2 || m ? __ldg(dp.lam + bh % p.Hq) : 1.f;
      // Reference max in log2 units and sum of the map in hand, and of the other one.
      float m_run = -INFINITY, m_other = -INFINITY;
      float l_run = 0.f, l_other = 0.f;
      constexpr int kParts = BN / 32;
      // Parts of a row's scores held in registers: all, but one where those are few.
      constexpr int kHeld = C::kRegsSoftmax < 128 ? 1 : kParts;
      const float2 cc2 = make_float2(c, c);
      int j = rng.lo;
      // P of tile j is in TMEM: on to the next tile.
      auto publish = [&]() {
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_ready[m][sc % SB]);
        if (MW == 1 || m == 1) {
          ++sc;
          ++j;
          release_pending();
        }
        if constexpr (MW == 2) {
          const float mo = m_other, lo = l_other;
          m_other = m_run, l_other = l_run, m_run = mo, l_run = lo;
          m ^= 1;
        }
      };
      bool fresh = true;  // some row has no key yet (of either map)
      for (bool find = true; j < rng.hi; find = fresh) {
        // Tiles that every row sees. Weights 2^(c s - m_run) against the reference max that the row
        // has so far: weights are floating-point, so that a score far above it costs no accuracy,
        // only range, and a sum above 2^24 tells of one. A row's first tile, such a one (S is still
        // in TMEM) and boundary tiles take the longer way below. (One loop for both compiled to a
        // slower one: causal 2 x 8192 1241 us, 1069 this way.)
        if (!find && (j - rng.lo) * BN >= full_lo) {
#pragma unroll 1
          while (j < j_full) {
            ok = wait_at(s_bar0 + 16 * m + 8 * (sc % SB), (sc / SB) & 1, wc);
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_col = lane_base + (SB * m + sc % SB) * BN;
            uint32_t s[kHeld][32], pk[kParts][16];
            if constexpr (kHeld > 1) {
#pragma unroll
              for (int y = 0; y < kParts; ++y) tmem_ld_x32(s_col + 32 * y, s[y]);
#pragma unroll
              for (int y = 0; y < kParts; ++y) tmem_wait_ld_x32(s[y]);
            }
            float2 sa = make_float2(0.f, 0.f), sb = sa;
            const float2 mm = make_float2(-m_run, -m_run);  // of a row yet without keys: +inf
#pragma unroll
            for (int y = 0; y < kParts; ++y) {
              if constexpr (kHeld == 1) {
                tmem_ld_x32(s_col + 32 * y, s[0]);
                tmem_wait_ld_x32(s[0]);
              }
              exp2_pack_32(reinterpret_cast<const float*>(s[y % kHeld]), cc2, mm, sa, sb, pk[y]);
            }
            sa = __fadd2_rn(sa, sb);
            const float sum = sa.x + sa.y;
            find = __any_sync(kFull, !(sum <= kDiffRaise));
            if (find) break;
            l_run += sum;
#pragma unroll
            for (int y = 0; y < kParts; ++y) tmem_st_x16(s_col + 16 * y, pk[y]);
            publish();
          }
          if (!ok || j >= rng.hi) break;
        }
        ok = wait_at(s_bar0 + 16 * m + 8 * (sc % SB), (sc / SB) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_col = lane_base + (SB * m + sc % SB) * BN;
        const int at = (j - rng.lo) * BN;
        const bool edge = at < full_lo || at > full_hi;
        if (at < some_lo || at > some_hi) {
          const uint32_t none[16] = {};
#pragma unroll
          for (int y = 0; y < kParts; ++y) tmem_st_x16(s_col + 16 * y, none);
        } else {
          uint32_t s[kHeld][32], pk[kParts][16];
          float2 sa, sb;
          auto masked = [&](int y) {
            tmem_wait_ld_x32(s[y % kHeld]);
            if (edge) {
              const uint32_t bits = vis_bits32(see_lo - at - 32 * y, see_hi - at - 32 * y);
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (!(bits & (1u << x))) s[y % kHeld][x] = 0xff800000u;  // -inf
            }
          };
          auto load = [&](int y) {
            tmem_ld_x32(s_col + 32 * y, s[0]);
            masked(y);
          };
          if constexpr (kHeld > 1) {
#pragma unroll
            for (int y = 0; y < kParts; ++y) tmem_ld_x32(s_col + 32 * y, s[y]);
#pragma unroll
            for (int y = 0; y < kParts; ++y) masked(y);
          }
#pragma unroll 1
          for (;;) {
            if (find) {
              float mx[kParts];
#pragma unroll
              for (int y = 0; y < kParts; ++y) {
                if constexpr (kHeld == 1) load(y);
                const uint32_t(&sy)[32] = s[y % kHeld];
                mx[y] = -INFINITY;
#pragma unroll
                for (int t = 0; t < 32; t += 2)
                  mx[y] = fmax3(mx[y], __uint_as_float(sy[t]), __uint_as_float(sy[t + 1]));
              }
              const float top = fmax3(mx[0], mx[1], mx[kParts - 1]) * c;
              // Move the reference only when it grows by more than 8 (a factor of 256).
              float alpha = 1.f;
              if (top > m_run + 8.f) {
                // (A row without keys so far has O = 0.)
                alpha = m_run == -INFINITY ? 1.f : fast_exp2(m_run - top);
                m_run = top;
              }
              l_run *= alpha;
              if (j > rng.lo && __any_sync(kFull, alpha < 1.f)) {
                // This tile's S was issued before the P V of the one before, which ends with its
                // stage's release.
                const int ep = e + j - 1 - rng.lo;
                ok = wait_at(smem_u32(&ctl->kv_empty[ep % STAGES]), (ep / STAGES) & 1, wc);
                if (!ok) break;
                tc_fence_after();
                const uint32_t o_col = lane_base + C::kOCol + m * D;
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 16) {
                  uint32_t ov[16];
                  tmem_ld_x16(o_col + cc, ov);
                  tmem_wait_ld_x16(ov);
#pragma unroll
                  for (int t = 0; t < 16; ++t)
                    ov[t] = __float_as_uint(__uint_as_float(ov[t]) * alpha);
                  tmem_st_x16(o_col + cc, ov);
                }
              }
            }
            const float msub = find && m_run == -INFINITY ? 0.f : m_run;
            sa = sb = make_float2(0.f, 0.f);
#pragma unroll
            for (int y = 0; y < kParts; ++y) {
              if constexpr (kHeld == 1) load(y);
              exp2_pack_32(reinterpret_cast<const float*>(s[y % kHeld]), cc2,
                           make_float2(-msub, -msub), sa, sb, pk[y]);
            }
            sa = __fadd2_rn(sa, sb);
            if (find) break;
            find = __any_sync(kFull, !(sa.x + sa.y <= kDiffRaise));
            if (!find) break;
          }
          if (!ok) break;
          fresh = fresh && __any_sync(kFull, m_run == -INFINITY || (MW == 2 && m_other == -INFINITY));
          l_run += sa.x + sa.y;
#pragma unroll
          for (int y = 0; y < kParts; ++y) tmem_st_x16(s_col + 16 * y, pk[y]);
        }
        if constexpr (kPaged) {
          // The context ends inside a page of this tile: its slots past the end may hold
          // anything, and a NaN there would survive p = 0. Both warpgroups clear their V rows
          // (the first P V may be either's).
          const int left = k_end - k_org - j * BN;  // tokens of the context from the tile's first
          const int clear = imin(BN, (left + p.page_size - 1) & -p.page_size);
          if (left < clear && (MW == 1 || m == 0)) {
            const int ev = e + j - rng.lo;  // V came with the K that S was made of
            ok = __all_sync(kFull,
                            mbar_wait(&ctl->kv_full[ev % STAGES], (ev / STAGES) & 1, wc));
            if (!ok) break;
            const uint32_t v0 = smem_u32(kv_s + (ev % STAGES) * C::kStageBytes + C::kTileBytes);
            for (int i = left * 8 + r; i < clear * 8; i += 128)
#pragma unroll
              for (int cp = 0; cp < C::kPanels; ++cp)
                st_shared_v4(v0 + cp * C::kPanelBytes + i * 16, 0, 0, 0, 0);
            fence_proxy_async_smem();
          }
        }
        publish();
      }
      if (!ok) break;
      // -------------------------------------------------------------- epilogue
      const bool live = row < k_end;
      float f0, f1;  // of O_0 and O_1
      if constexpr (MW == 2) {
        f0 = l_run != 0.f ? __frcp_rn(l_run) : 0.f;
        f1 = l_other != 0.f ? -lam * __frcp_rn(l_other) : 0.f;
      } else {
        ctl->coef[m][r] = l_run != 0.f ? lam * __frcp_rn(l_run) : 0.f;  // for both warps of the row
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->both[quarter]);
      }
      if (live) {
        float* to = p.lse + (static_cast<size_t>(bh) * 2 + m) * p.N + row;
        *to = l_run != 0.f ? (m_run + log2f(l_run)) * 0.69314718055994530942f : -INFINITY;
        if (MW == 2)
          to[p.N] =
              l_other != 0.f ? (m_other + log2f(l_other)) * 0.69314718055994530942f : -INFINITY;
      }
      ok = (MW == 2 || wait_at(smem_u32(&ctl->both[quarter]), 0, wc)) &&
           wait_at(smem_u32(&ctl->o_done), un_done & 1, wc);
      if (!ok) break;
      tc_fence_after();
      if constexpr (MW == 1) f0 = ctl->coef[0][r], f1 = -ctl->coef[1][r];
      // This warp's columns of the row: one half of the head's or both.
      constexpr int kCols = C::kHalf * MW, kX = kCols / 32;
      const int half0 = MW == 2 ? 0 : m;
      const uint32_t o0 = lane_base + C::kOCol + half0 * C::kHalf;
      float x[kCols];
      float2 ss2 = make_float2(0.f, 0.f), ss3 = ss2;
      uint32_t xa[kX][32], xb[kX][32];
#pragma unroll
      for (int y = 0; y < kX; ++y) {
        tmem_ld_x32(o0 + y * 32, xa[y]);
        tmem_ld_x32(o0 + D + y * 32, xb[y]);
      }
#pragma unroll
      for (int y = 0; y < kX; ++y) {
        tmem_wait_ld_x32(xa[y]);
        tmem_wait_ld_x32(xb[y]);
      }
#pragma unroll
      for (int y = 0; y < kX; ++y)
#pragma unroll
        for (int t = 0; t < 32; t += 2) {
          const float2 d2 = __ffma2_rn(
              make_float2(__uint_as_float(xa[y][t]), __uint_as_float(xa[y][t + 1])),
              make_float2(f0, f0),
              __fmul2_rn(make_float2(__uint_as_float(xb[y][t]), __uint_as_float(xb[y][t + 1])),
                         make_float2(f1, f1)));
          x[y * 32 + t] = d2.x;
          x[y * 32 + t + 1] = d2.y;
          if (t & 2)
            ss3 = __ffma2_rn(d2, d2, ss3);
          else
            ss2 = __ffma2_rn(d2, d2, ss2);
        }
      ss2 = __fadd2_rn(ss2, ss3);
      // The row's place in the staging area: this Q buffer, whose last MMA is done. Columns of half
      // a head: rows of D bytes, 16-byte chunks swizzled as TMA expects them.
      uint8_t* stage = q_s + (un_done % QB) * C::kQBytes;
      auto chunk_at = [&](int half, int ch) {
        const int sw = D == 128 ? (r & 7) : ((r >> 1) & 3);
        return stage + half * (128 * D) + r * D + ((ch ^ sw) << 4);
      };
      float ss = ss2.x + ss2.y;
      // Half a row's squares go to the warp with the other half where its chunk `ch` will be, which it
      // writes only after it has read them. Two halves in a fixed order, so that both warps scale by
      // the same number.
      auto whole_row = [&](int ch, uint32_t phase) {
        *reinterpret_cast<float*>(chunk_at(1 - m, ch)) = ss;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->both[quarter]);
        if (!wait_at(smem_u32(&ctl->both[quarter]), phase, wc)) return false;
        const float other = *reinterpret_cast<const float*>(chunk_at(m, ch));
        ss = m ? other + ss : ss + other;
        return true;
      };
      if constexpr (MW == 1) {
        ok = whole_row(0, 1);
        if (!ok) break;
      } else {
        tc_fence_before();
        __syncwarp();
      }
      const float by = dp.weight ? norm_scale(ss, dp.eps) : 1.f;
      if (__any_sync(kFull, by != 1.f)) {  // in both warps of these rows
        const float as_it_is = ss;
        ss = 0.f;
#pragma unroll
        for (int t = 0; t < kCols; ++t) {
          x[t] *= by;
          ss = fmaf(x[t], x[t], ss);
        }
        if constexpr (MW == 1) {
          ok = whole_row(1, 0);
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->both[quarter]);  // the next unit begins at phase 0
          ok = wait_at(smem_u32(&ctl->both[quarter]), 1, wc);
          if (!ok) break;
        }
        if (by == 1.f) ss = as_it_is;
      }
      const float rs = dp.weight ? norm_factor<D>(ss, by, dp.eps) : 1.f;
      const int warp_row0 = un.q_row0 + quarter * 32;
      const bool staged = rl == 7 && (PACK == kMaskNone || warp_row0 + 31 < k_end);
      uint8_t* orow = static_cast<uint8_t*>(p.o) +
                      (static_cast<size_t>(bh) * p.N + static_cast<size_t>(row)) * D * 2;
      const float2 rs2 = make_float2(rs, rs);
#pragma unroll
      for (int hh = 0; hh < MW; ++hh)
#pragma unroll
        for (int ch = 0; ch < C::kHalf / 8; ++ch) {
          uint32_t w[4];
          const int half = half0 + hh;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int at = ch * 8 + 4 * t;
            const float* xt = x + hh * C::kHalf + at;
            const float4 wt = *reinterpret_cast<const float4*>(&ctl->weight[half * C::kHalf + at]);
            const float2 y0 = __fmul2_rn(__fmul2_rn(make_float2(xt[0], xt[1]), rs2),
                                         make_float2(wt.x, wt.y));
            const float2 y1 = __fmul2_rn(__fmul2_rn(make_float2(xt[2], xt[3]), rs2),
                                         make_float2(wt.z, wt.w));
            w[2 * t] = pack_bf16x2(y0.x, y0.y);
            w[2 * t + 1] = pack_bf16x2(y1.x, y1.y);
          }
          if (staged)
            st_shared_v4(smem_u32(chunk_at(half, ch)), w[0], w[1], w[2], w[3]);
          else if (live)
            st_global_v4(orow + half * D + ch * 16, w[0], w[1], w[2], w[3]);
        }
      // What every lane read and wrote of the buffer comes before TMA's reads of it here and before its
      // next Q there, whether this warp's rows go out by TMA or not.
      fence_proxy_async_smem();
      __syncwarp();
      if (staged && warp_row0 < k_end && lane == 0) {
        for (int half = half0; half < half0 + MW; ++half)
          tma_store_3d(&tm_o, stage + half * (128 * D) + quarter * 32 * D, half * C::kHalf, warp_row0,
                       un.bh);
        bulk_commit_group();
      }
      // The buffer goes back to the producer once the store has read it, after this warp's next
      // key tile: it takes the Q of the unit after the next.
      pending_q = un_done % QB;
      ++un_done;
      e += rng.hi - rng.lo;
    }
    release_pending();  // the last unit's store, before shared memory goes away
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace ta
