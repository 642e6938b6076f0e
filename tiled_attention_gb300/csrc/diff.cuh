// diff.cuh — differential attention forward for sm_103a: dense and document masks, and chunks of
// new tokens over a paged KV cache.
//
// A head has two maps of D/2 channels side by side in q and k and one value row of D channels:
//   A_m = softmax(scale q_m k_m^T + mask),  y = A_1 v - lam A_2 v,
//   O = out_scale * y * w / sqrt(mean y^2 + eps)        (without w: O = out_scale * y)
//
// Both maps run over the same keys, so one pass over K and V serves them: a work unit is one
// 128-row query tile of one (batch or segment, query head), and what the ordinary kernel's two
// query tiles are there, the two maps are here. K_j and V_j are loaded once for both; the two
// softmaxes alternate on the tensor core, S of one map under the other's exponentials; the
// difference and the norm are taken in registers at the end, so that neither A_1 v nor A_2 v ever
// leaves the SM. Each map keeps its own running max and sum (the sums differ, so the accumulators
// cannot be joined before the end).
//
// Roles (384 threads), as in prefill.cuh:
//   warp 0      TMA producer: the unit's Q tile, then K_j, V_j into a ring
//   warp 1      MMA issuer: S_m = Q_m K_m^T (SS; map m is k-steps [m D/32, (m + 1) D/32) of the
//               tile's swizzled rows) and O_m += P_m V_j (P from TMEM); owns TMEM
//   warp 3      paged, pages under 64 tokens: the V entries
//   warps 4-7   softmax of map 0, warps 8-11 of map 1; a thread owns one query row. At the end
//               warps q of both take columns [0, D/2) and [D/2, D) of both accumulators: x = O_0 /
//               l_0 - lam O_1 / l_1, the row's sum of squares is exchanged through shared
//               memory, and the scaled row goes out by TMA.
// TMEM columns: S_0/P_0 [0, 128), S_1/P_1 [128, 256), O_0 and O_1 from 256 on, D each.
//
// Per key tile of 128 the tensor core needs 2 x (D/64) x 128 cycles for S and 2 x (D/128) x 512 for
// P V at D = 128 (1536 in all), the exponentials 1024 (32 a cycle and SM), and shared memory moves
// 192 KB (1536 cycles at 128 bytes).
#pragma once

#include <cuda_bf16.h>

#include "prefill.cuh"
#include "ptx.cuh"
#include "sched.h"

namespace ta {

struct DiffParams {
  PrefillParams base;    // o, lse [planes, 2, N], lengths, table, sizes; scale of the maps' scores
  const float* lam;      // [Hq]
  const float* weight;   // [D] or null
  float eps, out_scale;
  int mask;              // of the dense and document kinds
};

template <int D>
struct DiffCfg {
  static constexpr int BM = 128, BN = 128;
  static constexpr int kThreads = 384;
  static constexpr int kPanels = D / 64;
  static constexpr int kChunkBytes = 128 * 128;      // 64 columns of 128 rows
  static constexpr int kTileBytes = 128 * D * 2;     // Q, K or V
  static constexpr int kQBufs = 2;                   // this unit's and the next one's
  static constexpr int kStages = D == 128 ? 5 : 12;
  static constexpr int kCtrlBytes = 2048;
  static constexpr int kSmemBytes = 1024 + (kQBufs + kStages) * kTileBytes + kCtrlBytes;
  static constexpr int kTmemCols = 512;
  static constexpr int kOCol = 256;
  static constexpr int kSteps = D / 32;              // 16-channel k-steps of one map
  static constexpr int kHalf = D / 2;                // columns of O a softmax warp writes
  static constexpr uint32_t kRegsControl = 88, kRegsSoftmax = 208;
  static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= 384 * 168, "register split");
  static_assert(kSmemBytes <= 232448, "shared memory");
  static constexpr uint32_t kIdescS = idesc_bf16(BM, BN, false, false);
  static constexpr uint32_t kIdescO = idesc_bf16(BM, D, false, true);
};

struct DiffCtrl {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[12], kv_empty[12];
  uint64_t s_ready[2], p_ready[2], o_done, drain;
  uint64_t both[4];          // warps q of the two softmax warpgroups
  uint32_t tmem_base;
  int abort_flag;
  float coef[2][128];        // 1 / l of map 0's rows, lam / l of map 1's
  float weight[128];         // out_scale * w
};

// Work unit u in launch order: 128-row tiles from the last one down, then batch and head; packed
// kinds take the two halves of prefill.cuh's 256-row units, the later (longer) one first. q_row0
// may lie past the segment (an odd number of tiles): that unit has no key tiles.
template <int PACK>
__device__ __forceinline__ Unit diff_unit(int u, const PrefillParams& p, UnitCursor& cur) {
  if constexpr (PACK != kMaskNone) {
    Unit r = decode_unit<PACK>(u >> 1, p, cur);
    if (r.valid && !(u & 1)) r.q_row0 += 128;
    return r;
  } else {
    Unit r{0, 0, 0, 0, 0, 0, 0};
    const int per_level = p.B * p.Hq;
    const int level = tiles_for_rows(p.N) - 1 - u / per_level;
    if (level < 0) return r;
    const int bh = u % per_level;
    r.valid = 1;
    r.bh = bh;
    r.kvh = (bh / p.Hq) * p.Hkv + (bh % p.Hq) / p.group;
    r.q_row0 = level * 128;
    r.k_end = p.N;
    return r;
  }
}

template <int D, int PACK>
__global__ void __launch_bounds__(384, 1)
    diff_prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_o, const DiffParams dp) {
  using C = DiffCfg<D>;
  constexpr int BM = C::BM, BN = C::BN, STAGES = C::kStages, QB = C::kQBufs;
  constexpr bool kPaged = PACK == kMaskPagedPrefill;
  constexpr unsigned kFull = 0xffffffffu;
  const PrefillParams& p = dp.base;
  const int mask = kPaged ? static_cast<int>(kMaskPagedPrefill) : dp.mask;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* q_s = smem;
  uint8_t* kv_s = smem + QB * C::kTileBytes;
  DiffCtrl* ctl = reinterpret_cast<DiffCtrl*>(kv_s + STAGES * C::kTileBytes);
  static_assert(sizeof(DiffCtrl) <= C::kCtrlBytes, "control block");

  const int warp = static_cast<int>(threadIdx.x >> 5);
  const int lane = static_cast<int>(lane_id());
  if (warp == 0) {
    if (lane == 0) {
      ctl->abort_flag = 0;
      for (int q = 0; q < QB; ++q) {
        mbar_init(&ctl->q_full[q], 1);
        mbar_init(&ctl->q_empty[q], 8);  // one arrival per softmax warp
      }
      for (int s = 0; s < STAGES; ++s) {
        mbar_init(&ctl->kv_full[s], 1);
        mbar_init(&ctl->kv_empty[s], 1);
      }
      for (int m = 0; m < 2; ++m) {
        mbar_init(&ctl->s_ready[m], 1);
        mbar_init(&ctl->p_ready[m], 128);
      }
      mbar_init(&ctl->o_done, 1);
      mbar_init(&ctl->drain, 1);
      for (int q = 0; q < 4; ++q) mbar_init(&ctl->both[q], 2);
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
  const int G = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
  auto unit_of = [&](int k) { return k * G + ((k & 1) ? G - 1 - b : b); };
  auto range_of = [&](const Unit& un) {
    return kv_tile_range(mask, p.window, un.q_row0, BM, un.k_end, un.k_org, un.k_end, BN);
  };
  UnitCursor cur{0, 0, 0, 0};  // this role's place in the packed unit list

  if (warp < 4) {
    regs_decrease<C::kRegsControl>();
    const bool split_v = kPaged && p.page_shift < 6;
    if (warp == 0 || (split_v && warp == 3)) {
      // -------------------------------------------------------------- TMA producer
      int e = 0;   // K/V ring entries
      int qn = 0;  // Q loads issued
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int u = unit_of(k);
        if (u >= p.num_units) break;
        const Unit un = diff_unit<PACK>(u, p, cur);  // warp-collective
        if (!un.valid) break;
        const KvRange rng = range_of(un);
        const int npos = rng.hi - rng.lo;
        if (npos <= 0) continue;
        if (lane == 0) {
          if (warp == 0) {
            const int qb = qn % QB;
            ok = mbar_wait(&ctl->q_empty[qb], ((qn / QB) & 1) ^ 1, wc);
            if (ok) {
              ++qn;
              mbar_arrive_expect_tx(&ctl->q_full[qb], C::kTileBytes);
              for (int c = 0; c < C::kPanels; ++c)
                tma_load_3d(q_s + qb * C::kTileBytes + c * C::kChunkBytes, &tm_q,
                            &ctl->q_full[qb], c * 64, un.q_row0, un.bh);
            }
          }
          // Ring entry: K (even x) or V of the key tile at position x / 2.
          for (int x = 0; !kPaged && x < 2 * npos && ok; ++x, ++e) {
            const int st = e % STAGES;
            ok = mbar_wait(&ctl->kv_empty[st], ((e / STAGES) & 1) ^ 1, wc);
            if (!ok) break;
            mbar_arrive_expect_tx(&ctl->kv_full[st], C::kTileBytes);
            for (int c = 0; c < C::kPanels; ++c)
              tma_load_3d(kv_s + st * C::kTileBytes + c * C::kChunkBytes, (x & 1) ? &tm_v : &tm_k,
                          &ctl->kv_full[st], c * 64, un.k_org + (rng.lo + x / 2) * BN, un.kvh);
          }
        }
        ok = __shfl_sync(kFull, ok, 0);
        if constexpr (kPaged) {
          // Lane sb owns page sb of every key tile, as in prefill.cuh: it reads the page's entry a
          // tile ahead and issues its boxes; pages past the context or outside the pool come
          // from the zero-filled plane past it.
          const int lp = p.page_shift;
          const int nb = BN >> lp;
          const int lk = un.k_end - un.k_org;
          const int* trow = p.table + static_cast<size_t>(un.seq) * p.max_pages;
          auto plane_of = [&](int j) {
            const int tok = j * BN + (lane << lp);
            int pl = p.num_pages * p.Hkv;
            if (lane < nb && tok < lk) {
              const int raw = __ldg(trow + (tok >> lp));
              if (raw < 0 || raw >= p.num_pages)
                report_status(p.status, -5);
              else
                pl = raw * p.Hkv + un.kvh;
            }
            return pl;
          };
          int pl_next = plane_of(rng.lo), pl = 0;
          for (int x = 0; x < 2 * npos && ok; ++x, ++e) {
            if (split_v && (x & 1) != (warp == 3 ? 1 : 0)) continue;  // the other warp's entry
            const int st = e % STAGES;
            if (lane == 0) ok = mbar_wait(&ctl->kv_empty[st], ((e / STAGES) & 1) ^ 1, wc);
            ok = __shfl_sync(kFull, ok, 0);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&ctl->kv_full[st], C::kTileBytes);
            __syncwarp();
            if (split_v || !(x & 1)) pl = pl_next;  // the first entry of its tile this warp issues
            if (lane < nb) {
              for (int c = 0; c < C::kPanels; ++c)
                tma_load_3d(kv_s + st * C::kTileBytes + c * C::kChunkBytes + (lane << lp) * 128,
                            (x & 1) ? &tm_v : &tm_k, &ctl->kv_full[st], c * 64, 0, pl);
            }
            if ((split_v || !(x & 1)) && x / 2 + 1 < npos) pl_next = plane_of(rng.lo + x / 2 + 1);
          }
        }
      }
      if (lane == 0) {
        // Let copies still in flight land before the CTA can exit (no-op on the normal path).
        for (int x = imax(0, e - STAGES); x < e; ++x)
          if (!split_v || (x & 1) == (warp == 3 ? 1 : 0))
            mbar_wait(&ctl->kv_full[x % STAGES], (x / STAGES) & 1, wc_drain);
        for (int x = imax(0, qn - QB); x < qn; ++x)
          mbar_wait(&ctl->q_full[x % QB], (x / QB) & 1, wc_drain);
      }
    } else if (warp == 1) {
      // -------------------------------------------------------------- MMA issuer
      int e = 0;   // ring entry of the unit's first K
      int qn = 0;  // Q tiles used
      int pn = 0;  // P tiles consumed, of each map
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int u = unit_of(k);
        if (u >= p.num_units) break;
        const Unit un = diff_unit<PACK>(u, p, cur);  // warp-collective
        if (!un.valid) break;
        const KvRange rng = range_of(un);
        const int npos = rng.hi - rng.lo;
        if (npos <= 0) continue;
        const uint64_t q_desc = sw128_desc(smem_u32(q_s + (qn % QB) * C::kTileBytes), 16, 1024);
        // Step x: P V of the key tile at position x - 1, then S of the one at x, map by map.
        for (int x = 0; x <= npos && ok; ++x) {
          const bool have_v = x > 0, have_k = x < npos;
          const int ev = e + 2 * x - 1, ek = e + 2 * x;
          {
            const bool rv = !have_v || mbar_try_wait(&ctl->kv_full[ev % STAGES], (ev / STAGES) & 1);
            const bool rk = !have_k || mbar_try_wait(&ctl->kv_full[ek % STAGES], (ek / STAGES) & 1);
            if (!__all_sync(kFull, rv && rk)) {
              if (have_v)
                ok = __all_sync(kFull,
                                mbar_wait(&ctl->kv_full[ev % STAGES], (ev / STAGES) & 1, wc));
              if (have_k && ok)
                ok = __all_sync(kFull,
                                mbar_wait(&ctl->kv_full[ek % STAGES], (ek / STAGES) & 1, wc));
            }
            if (ok && x == 0)
              ok = __all_sync(kFull, mbar_wait(&ctl->q_full[qn % QB], (qn / QB) & 1, wc));
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t v_desc =
              sw128_desc(smem_u32(kv_s + (ev % STAGES) * C::kTileBytes), C::kChunkBytes, 1024);
          const uint64_t k_desc =
              sw128_desc(smem_u32(kv_s + (ek % STAGES) * C::kTileBytes), 16, 1024);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (have_v) {
              const int ph = (pn + x - 1) & 1;
              if (!__all_sync(kFull, mbar_try_wait(&ctl->p_ready[m], ph)))
                ok = __all_sync(kFull, mbar_wait(&ctl->p_ready[m], ph, wc));
              if (!ok) break;
              tc_fence_after();
              // The unit's first P V overwrites O_m: both warps of every row published this P
              // after they had read O of the unit before.
              mma_ts_chain8(tmem + C::kOCol + m * D, tmem + m * 128, v_desc, C::kIdescO, x > 1);
              if (m == 1) {
                mma_commit(&ctl->kv_empty[ev % STAGES]);
                if (!have_k) mma_commit(&ctl->o_done);
              }
            }
            if (have_k) {
#pragma unroll
              for (int s = 0; s < C::kSteps; ++s) {
                // 32 bytes a step inside a 128-byte swizzle row, four steps a panel.
                const int at = m * C::kSteps + s;
                const uint32_t off16 = ((at >> 2) * C::kChunkBytes + (at & 3) * 32) >> 4;
                mma_ss(tmem + m * 128, q_desc + off16, k_desc + off16, C::kIdescS, s > 0);
              }
              mma_commit(&ctl->s_ready[m]);
              if (m == 1) mma_commit(&ctl->kv_empty[ek % STAGES]);
            }
          }
        }
        e += 2 * npos;
        pn += npos;
        ++qn;
      }
      // Every MMA this warp issued has completed before TMEM can be released.
      mma_commit(&ctl->drain);
      mbar_wait(&ctl->drain, 0, wc_drain);
    }
  } else {
    regs_increase<C::kRegsSoftmax>();
    // ---------------------------------------------------------------- softmax warpgroups
    const int m = (warp - 4) >> 2;          // map
    const int quarter = warp & 3;           // TMEM lanes [32*quarter, 32*quarter + 32)
    const int r = quarter * 32 + lane;      // row inside the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_col = lane_base + m * 128;
    const float c = p.scale_log2;
    int sc = 0;          // S tiles consumed
    int un_done = 0;     // units with work finished
    int e = 0;           // ring entry of the unit's first K
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
    for (int k = 0; ok; ++k) {
      const int u = unit_of(k);
      if (u >= p.num_units) break;
      const Unit un = diff_unit<PACK>(u, p, cur);  // warp-collective
      if (!un.valid) break;
      const KvRange rng = range_of(un);
      if (rng.hi <= rng.lo) continue;
      const int k_org = un.k_org, k_end = un.k_end, bh = un.bh;
      const int row = un.q_row0 + r;
      // Keys that every row of the tile sees, and those that this row sees, from the range's first
      // key on.
      const int key0 = k_org + rng.lo * BN;
      const int full_lo = vis_lo(mask, p.window, k_org, imin(un.q_row0 + BM, k_end) - 1) - key0;
      const int full_hi = vis_hi(mask, p.window, k_end, un.q_row0) - key0 - (BN - 1);
      const int see_lo = vis_lo(mask, p.window, k_org, row) - key0;
      const int see_hi = vis_hi(mask, p.window, k_end, row) - key0;
      float m_run = -INFINITY;  // running max in log2 units (may trail the true max by < 8)
      float l_run = 0.f;
      for (int j = rng.lo; j < rng.hi && ok; ++j) {
        ok = __all_sync(kFull, mbar_wait(&ctl->s_ready[m], (sc++) & 1, wc));
        if (!ok) break;
        tc_fence_after();
        uint32_t s0[32], s1[32], s2[32], s3[32];
        tmem_ld_x32(s_col + 0, s0);
        tmem_ld_x32(s_col + 32, s1);
        tmem_ld_x32(s_col + 64, s2);
        tmem_ld_x32(s_col + 96, s3);
        tmem_wait_ld_x32(s0);
        tmem_wait_ld_x32(s1);
        tmem_wait_ld_x32(s2);
        tmem_wait_ld_x32(s3);
        float* f0 = reinterpret_cast<float*>(s0);
        float* f1 = reinterpret_cast<float*>(s1);
        float* f2 = reinterpret_cast<float*>(s2);
        float* f3 = reinterpret_cast<float*>(s3);
        const int at = (j - rng.lo) * BN;
        if (at < full_lo || at > full_hi) {
          const int lo_k = see_lo - at, hi_k = see_hi - at;
          const uint32_t b0 = vis_bits32(lo_k, hi_k), b1 = vis_bits32(lo_k - 32, hi_k - 32);
          const uint32_t b2 = vis_bits32(lo_k - 64, hi_k - 64);
          const uint32_t b3 = vis_bits32(lo_k - 96, hi_k - 96);
#pragma unroll
          for (int t = 0; t < 32; ++t) {
            if (!(b0 & (1u << t))) f0[t] = -INFINITY;
            if (!(b1 & (1u << t))) f1[t] = -INFINITY;
            if (!(b2 & (1u << t))) f2[t] = -INFINITY;
            if (!(b3 & (1u << t))) f3[t] = -INFINITY;
          }
        }
        // Row max: four independent chains of 3-input max over the 128 scores.
        float mx0 = fmax3(f0[0], f0[1], f0[2]), mx1 = fmax3(f1[0], f1[1], f1[2]);
        float mx2 = fmax3(f2[0], f2[1], f2[2]), mx3 = fmax3(f3[0], f3[1], f3[2]);
#pragma unroll
        for (int t = 3; t < 31; t += 2) {
          mx0 = fmax3(mx0, f0[t], f0[t + 1]);
          mx1 = fmax3(mx1, f1[t], f1[t + 1]);
          mx2 = fmax3(mx2, f2[t], f2[t + 1]);
          mx3 = fmax3(mx3, f3[t], f3[t + 1]);
        }
        mx0 = fmax3(mx0, f0[31], f1[31]);
        mx2 = fmax3(mx2, f2[31], f3[31]);
        const float m_tile = fmax3(fmaxf(mx0, mx1), mx2, mx3) * c;
        float alpha = 1.f;
        // Move the reference max only when it grows by more than 8 (a factor 256).
        if (m_tile > m_run + 8.f) {
          alpha = fast_exp2(m_run - m_tile);  // 0 when m_run is -inf
          m_run = m_tile;
        }
        if (j > rng.lo && __any_sync(kFull, alpha < 1.f)) {
          const uint32_t o_col = lane_base + C::kOCol + m * D;
#pragma unroll
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t ov[16];
            tmem_ld_x16(o_col + cc * 16, ov);
            tmem_wait_ld_x16(ov);
#pragma unroll
            for (int t = 0; t < 16; ++t)
              ov[t] = __float_as_uint(__uint_as_float(ov[t]) * alpha);
            tmem_st_x16(o_col + cc * 16, ov);
          }
        }
        const float msub = (m_run == -INFINITY) ? 0.f : m_run;
        const float2 cc2 = make_float2(c, c);
        const float2 mm = make_float2(-msub, -msub);
        float2 sa = make_float2(0.f, 0.f), sb = make_float2(0.f, 0.f);
        uint32_t pk[16];
        exp2_pack_32(f0, cc2, mm, sa, sb, pk);
        tmem_st_x16(s_col + 0, pk);
        exp2_pack_32(f1, cc2, mm, sa, sb, pk);
        tmem_st_x16(s_col + 16, pk);
        exp2_pack_32(f2, cc2, mm, sa, sb, pk);
        tmem_st_x16(s_col + 32, pk);
        exp2_pack_32(f3, cc2, mm, sa, sb, pk);
        tmem_st_x16(s_col + 48, pk);
        l_run = l_run * alpha + ((sa.x + sa.y) + (sb.x + sb.y));
        if constexpr (kPaged) {
          // The context ends inside a page of this tile: its slots past the end may hold
          // anything, and a NaN there would survive p = 0. Both warpgroups clear their V rows
          // (the first P V may be either's).
          const int left = k_end - k_org - j * BN;  // tokens of the context from the tile's first
          const int clear = imin(BN, (left + p.page_size - 1) & -p.page_size);
          if (left < clear) {
            const int ev = e + 2 * (j - rng.lo) + 1;
            ok = __all_sync(kFull,
                            mbar_wait(&ctl->kv_full[ev % STAGES], (ev / STAGES) & 1, wc));
            if (!ok) break;
            const uint32_t v0 = smem_u32(kv_s + (ev % STAGES) * C::kTileBytes);
            for (int i = left * 8 + r; i < clear * 8; i += 128)
#pragma unroll
              for (int cp = 0; cp < C::kPanels; ++cp)
                st_shared_v4(v0 + cp * C::kChunkBytes + i * 16, 0, 0, 0, 0);
            fence_proxy_async_smem();
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&ctl->p_ready[m]);
        release_pending();
      }
      if (!ok) break;
      // -------------------------------------------------------------- epilogue
      // This row's factor of O_m, for both warps of the row.
      ctl->coef[m][r] = l_run != 0.f ? (m ? __ldg(dp.lam + bh % p.Hq) : 1.f) / l_run : 0.f;
      const bool live = row < k_end;
      if (live)
        p.lse[(static_cast<size_t>(bh) * 2 + m) * p.N + row] =
            l_run != 0.f ? (m_run + log2f(l_run)) * 0.69314718055994530942f : -INFINITY;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->both[quarter]);
      ok = __all_sync(kFull, mbar_wait(&ctl->both[quarter], 0, wc) &&
                                 mbar_wait(&ctl->o_done, un_done & 1, wc));
      if (!ok) break;
      tc_fence_after();
      const float f0 = ctl->coef[0][r], f1 = -ctl->coef[1][r];
      float x[C::kHalf];
      float2 ss2 = make_float2(0.f, 0.f);
      const uint32_t o0 = lane_base + C::kOCol + m * C::kHalf;
#pragma unroll
      for (int cc = 0; cc < C::kHalf / 32; ++cc) {
        uint32_t va[32], vb[32];
        tmem_ld_x32(o0 + cc * 32, va);
        tmem_ld_x32(o0 + D + cc * 32, vb);
        tmem_wait_ld_x32(va);
        tmem_wait_ld_x32(vb);
#pragma unroll
        for (int t = 0; t < 32; t += 2) {
          const float2 y = __ffma2_rn(
              make_float2(__uint_as_float(va[t]), __uint_as_float(va[t + 1])),
              make_float2(f0, f0),
              __fmul2_rn(make_float2(__uint_as_float(vb[t]), __uint_as_float(vb[t + 1])),
                         make_float2(f1, f1)));
          x[cc * 32 + t] = y.x;
          x[cc * 32 + t + 1] = y.y;
          ss2 = __ffma2_rn(y, y, ss2);
        }
      }
      // The row's place in the staging area: this Q buffer, whose last MMA is done. Columns of
      // warpgroup m: rows of D bytes, 16-byte chunks swizzled as TMA expects them.
      uint8_t* stage = q_s + (un_done % QB) * C::kTileBytes;
      auto chunk_at = [&](int half, int ch) {
        const int sw = D == 128 ? (r & 7) : ((r >> 1) & 3);
        return stage + half * (128 * D) + r * D + ((ch ^ sw) << 4);
      };
      // Half a row's squares, put where the partner's first chunk will be, which it writes only
      // after it has read them.
      *reinterpret_cast<float*>(chunk_at(1 - m, 0)) = ss2.x + ss2.y;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->both[quarter]);
      ok = __all_sync(kFull, mbar_wait(&ctl->both[quarter], 1, wc));
      if (!ok) break;
      // Two halves in a fixed order, so that both warps scale by the same number.
      const float mine = ss2.x + ss2.y, other = *reinterpret_cast<const float*>(chunk_at(m, 0));
      const float ss = m ? other + mine : mine + other;
      // A row without keys stays zero whatever eps is.
      const float rs = dp.weight && l_run != 0.f ? rsqrtf(ss * (1.f / D) + dp.eps) : 1.f;
      const int warp_row0 = un.q_row0 + quarter * 32;
      const bool staged = PACK == kMaskNone || warp_row0 + 31 < k_end;
      uint8_t* orow = static_cast<uint8_t*>(p.o) +
                      (static_cast<size_t>(bh) * p.N + static_cast<size_t>(row)) * D * 2 + m * D;
#pragma unroll
      for (int ch = 0; ch < C::kHalf / 8; ++ch) {
        uint32_t w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float2 wt =
              *reinterpret_cast<const float2*>(&ctl->weight[m * C::kHalf + ch * 8 + 2 * t]);
          w[t] = pack_bf16x2(x[ch * 8 + 2 * t] * rs * wt.x, x[ch * 8 + 2 * t + 1] * rs * wt.y);
        }
        if (staged)
          st_shared_v4(smem_u32(chunk_at(m, ch)), w[0], w[1], w[2], w[3]);
        else if (live)
          st_global_v4(orow + ch * 16, w[0], w[1], w[2], w[3]);
      }
      if (staged && warp_row0 < k_end) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&tm_o, stage + m * (128 * D) + quarter * 32 * D, m * C::kHalf, warp_row0,
                       bh);
          bulk_commit_group();
        }
      }
      // The buffer goes back to the producer once the store has read it, after this warp's next
      // key tile: it takes the Q of the unit after the next.
      pending_q = un_done % QB;
      ++un_done;
      e += 2 * (rng.hi - rng.lo);
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
