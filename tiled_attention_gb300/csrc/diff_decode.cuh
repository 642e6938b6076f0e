// diff_decode.cuh — differential attention's paged decode: one query token a sequence, the
// difference of two softmax maps over one set of values (diff.cuh has the formulas).
//
// K and V are read once for both maps, and both maps' products cost as many MMAs as one map of
// ordinary attention with up to 16 heads a kv head: rows r < 8 of an m16n8k16 tile are head r's
// first map, rows r + 8 its second. K holds the maps' channels side by side, so the queries enter
// block-diagonally, (q_1, 0) in rows r and (0, q_2) in rows r + 8: the k-steps over the first D / 2
// channels leave S_1 in rows r, those over the others S_2 in rows r + 8, and P of both maps is one A
// fragment for V. Decode reads 512 bytes a token and kv head at D = 128 and is bound by HBM.
//
// Work: contexts are cut into 64-token blocks and shared out evenly over two CTAs an SM
// (share.cuh), each of which walks its range of (sequence, kv head, block), one or more segments of
// one (sequence, kv head). A producer warp brings 64-token stages into a ring by TMA, page by page
// through the block table, and runs ahead over the segments' ends. Each of four consumer warps owns
// a 16-token slice of every stage with its own running max, sum and O; at a segment's end the four
// are merged in the slot of its last stage. A segment that is its whole context writes O and LSE
// itself, normed; the others (a CTA's first and last at most) leave O, max and sum of both maps in
// the workspace, two slots a CTA, and a second kernel, under programmatic dependent launch, joins
// them in the workers' order: results do not depend on timing.
//
// So with up to 8 heads a kv head; with 9 to 16 a warp takes one map, whose tile has a row a head,
// over twice the tokens.
//
// Measured (32 heads over 8, D = 128): 32 sequences of 1K to 16K tokens 166 us, 0.98 of the copy
// rate; one sequence of 16K 20.0 us, of which the bytes are 9.9 and the rest is the launch, the
// ring's fill and the join. With 16 heads a kv head (D = 64, pages of 16, 48 sequences) 69.8 us,
// where the bytes take 56.4. A copy that only streams takes 161 and 71 us (the latter with less even
// shares): what is left is that some SMs get their bytes later than others, 135 to 160 us in the
// batch.
#pragma once

#include <type_traits>

#include "decode.cuh"
#include "norm.cuh"
#include "ptx.cuh"
#include "sched.h"
#include "share.cuh"

namespace ta {

struct DiffDecodeParams {
  const uint32_t* q;     // bf16 [B, Hq, 1, D]
  const int* cu;         // [B+1] cumulative context lengths
  const int* table;      // [B, max_pages]
  uint16_t* o;           // bf16 [B, Hq, 1, D]
  float* lse;            // [B, Hq, 2]
  const float* lam;      // [Hq]
  const float* weight;   // [D] or null
  float* part_o;         // [2 * slots, 2 maps, group, D]
  float* part_ml;        // [2 * slots, 2 maps, group, 2]
  int B, Hq, Hkv, max_pages, num_pages, group, page_shift, max_len;
  int slots;             // CTAs of the decode kernel
  int join_heads;        // query heads a CTA of the joining kernel takes
  int join_workers;      // it goes by workers, not by contexts
  float scale_log2, eps, out_scale;
  int* status;
  unsigned long long timeout_ns;
};

constexpr int kDiffDecodeCtas = 2;  // per SM
constexpr float kDiffDecodeRaise = 16777216.f;  // 2^24

// Beginning a context costs a CTA's pipeline about as much at both head dims, and a block of d = 64
// half the bytes. 48 sequences of up to 16K tokens, 16 heads a kv head, d = 64: 76.0 us with 2, 72.6
// with 4, 70.4 with 8, 71.6 with 16; at d = 128 one sequence of 16K 20.1 with 2, 20.4 with 3 to 6,
// batches within 1 %.
template <int D>
using DiffShare = Share<DiffDecodeParams, 64, D == 64 ? 8 : 2, 32, 1>;

template <int D>
struct DiffDecodeCfg {
  static constexpr int kTok = 64;  // tokens per ring stage; consumer warp w owns 16 w .. 16 w + 15
  static constexpr int kWarps = 4;
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kThreads = kConsumers + 32;
  static constexpr int kPanels = D / 64;
  static constexpr int kPanelBytes = kTok * 128;
  static constexpr int kHalfBytes = kTok * D * 2;            // K or V of a stage
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kStages = (96 * 1024) / kStageBytes;  // 3 (D = 128), 6 (D = 64)
  static constexpr int kSteps = D / 16;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kMiscBytes = 768;
  static constexpr int kSmemBytes = 1024 + kRingBytes + kMiscBytes;
  static_assert(kWarps * 16 * D * 4 <= kStageBytes, "a tile's rows are merged in one slot");
  static_assert(kDiffDecodeCtas * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs an SM");
};

struct DiffDecodeCtrl {
  uint64_t full[8], empty[8];
  int abort_flag;
};

// A worker's walk over its range of blocks, segment by segment.
template <class S, class P>
struct SegmentWalk {
  int u, end, b, seq_u;           // next unit, the range's end, sequence and its first unit
  int g, L, nb, blk0, nblk;       // the segment: kv head, context, its blocks, first and count
  __device__ __forceinline__ SegmentWalk(const S& share, const P& p, int worker) {
    u = share.start(worker);
    end = share.start(worker + 1);
    share.find(p, u, b, seq_u);
    seq_u *= p.Hkv;
  }
  __device__ __forceinline__ bool next(const P& p) {  // false: the range holds no more blocks
    if (u >= end) return false;
    L = context_length(p, b, false);
    nb = S::blocks(L);
    int w = S::units(nb);
    while (u >= seq_u + w * p.Hkv) {  // on to the next sequence that has blocks
      seq_u += w * p.Hkv;
      L = context_length(p, ++b, false);
      nb = S::blocks(L);
      w = S::units(nb);
    }
    g = (u - seq_u) / w;
    int pos = u - seq_u - g * w;
    if (pos < S::kStart) {
      u += S::kStart - pos;
      pos = S::kStart;
      if (u >= end) return false;
    }
    blk0 = pos - S::kStart;
    nblk = imin(nb - blk0, end - u);
    u += nblk;
    return true;
  }
};

// Four columns of one head's row from both maps' sums: the difference, its norm over the D / 4
// lanes that hold the row side by side, and the store.
template <int D>
__device__ __forceinline__ void diff_finish(const DiffDecodeParams& p, size_t row, float lam,
                                            float4 w, int quad, float4 a0, float4 a1, float2 ml0,
                                            float2 ml1, unsigned lanes) {
  // A map without a score above -inf (an empty context has none in either) adds nothing.
  const float f0 = ml0.y != 0.f ? 1.f / ml0.y : 0.f, f1 = ml1.y != 0.f ? lam / ml1.y : 0.f;
  float4 y = make_float4(a0.x * f0 - a1.x * f1, a0.y * f0 - a1.y * f1, a0.z * f0 - a1.z * f1,
                         a0.w * f0 - a1.w * f1);
  float rs = p.out_scale;
  if (p.weight) {
    auto squares = [&] {  // the same bits in all of the row's lanes
      float ss = (y.x * y.x + y.y * y.y) + (y.z * y.z + y.w * y.w);
#pragma unroll
      for (int off = D / 8; off; off >>= 1) ss += __shfl_xor_sync(lanes, ss, off);
      return ss;
    };
    float ss = squares();
    const float by = norm_scale(ss, p.eps);
    if (by != 1.f) {
      y = make_float4(y.x * by, y.y * by, y.z * by, y.w * by);
      ss = squares();
    }
    rs *= norm_factor<D>(ss, by, p.eps);
  }
  *reinterpret_cast<uint2*>(p.o + row * D + 4 * quad) =
      make_uint2(pack_bf16x2(y.x * rs * w.x, y.y * rs * w.y),
                 pack_bf16x2(y.z * rs * w.z, y.w * rs * w.w));
  auto lse = [](float2 ml) {
    return ml.y != 0.f ? (ml.x + log2f(ml.y)) * 0.69314718055994530942f : -INFINITY;
  };
  if (quad == 0) *reinterpret_cast<float2*>(p.lse + 2 * row) = make_float2(lse(ml0), lse(ml1));
}
// Four norm weights (ones without a norm).
__device__ __forceinline__ float4 diff_weight(const DiffDecodeParams& p, int quad) {
  return p.weight ? __ldg(reinterpret_cast<const float4*>(p.weight) + quad)
                  : make_float4(1.f, 1.f, 1.f, 1.f);
}

// NT: 1 for up to 8 heads a kv head, 2 for up to 16.
template <int D, int NT>
__global__ void __launch_bounds__(160, kDiffDecodeCtas)
    diff_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const DiffDecodeParams p) {
  using C = DiffDecodeCfg<D>;
  constexpr int S = C::kStages;
  const int G = p.group;  // 1 <= G <= 8 NT
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5;
  const int lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  DiffDecodeCtrl* ctl = reinterpret_cast<DiffDecodeCtrl*>(ring + C::kRingBytes);
  float* red_m = reinterpret_cast<float*>(ring + C::kRingBytes + 256);  // [warps][16]
  float* red_l = red_m + C::kWarps * 16;
  static_assert(256 + 2 * C::kWarps * 16 * 4 <= C::kMiscBytes, "misc area");

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == C::kConsumers) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], C::kWarps);
    }
    ctl->abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  const int worker = static_cast<int>(blockIdx.x);
  const DiffShare<D> share(p, 0, worker == 0 && warp == 0);
  __syncthreads();
  if (worker >= share.n) return;
  SegmentWalk<DiffShare<D>, DiffDecodeParams> seg(share, p, worker);
  const WaitCtl wc{p.timeout_ns, p.status, &ctl->abort_flag};
  const WaitCtl wc_drain{p.timeout_ns, p.status, nullptr};

  if (warp == C::kWarps) {
    // ---------------------------------------------------------------- TMA producer
    // A stage is one box a panel of a page of 64 tokens or of half a page of 128, or whole pages of
    // 16 or 32, a lane a box. A page past
    // the context, or whose entry lies outside the pool (never addressed; the status word
    // reports it), comes from the plane past the pool, which TMA fills with zeros.
    const int lp = p.page_shift;
    const int run = imin(C::kTok, 1 << lp), nbox = C::kTok / run, sb = lane & (nbox - 1);
    int e = 0;  // stages issued
    bool ok = true;
    while (ok && seg.next(p)) {
      const int* row = p.table + static_cast<size_t>(seg.b) * p.max_pages;
      PageEntries pages(row, seg.blk0 * C::kTok, run, lp, seg.L);
      for (int i = 0; i < seg.nblk; ++i, ++e) {
        const int st = e % S;
        ok = wait_at(smem_u32(&ctl->empty[st]), ((e / S) & 1) ^ 1, wc);
        if (!ok) break;
        const int raw = pages.at(i * nbox, sb);
        int pl = p.num_pages * p.Hkv;
        if (raw >= 0 && raw < p.num_pages)
          pl = raw * p.Hkv + seg.g;
        else if (lane < nbox && (seg.blk0 + i) * C::kTok + sb * run < seg.L)
          report_status(p.status, -5);
        const int row0 = ((seg.blk0 + i) * C::kTok) & ((1 << lp) - 1);  // second half of a page
        if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], C::kStageBytes);
        __syncwarp();
        const int kind = lane / nbox;  // panels of K, then of V
        if (kind < 2 * C::kPanels)
          tma_load_3d(ring + st * C::kStageBytes + kind * C::kPanelBytes + sb * run * 128,
                      kind < C::kPanels ? &tm_k : &tm_v, &ctl->full[st], kind % C::kPanels * 64, row0,
                      pl);
      }
    }
    if (lane == 0)
      for (int x = imax(0, e - S); x < e; ++x)
        mbar_wait(&ctl->full[x % S], (x / S) & 1, wc_drain);
    return;  // the producer takes no part in the consumer barriers below
  }

  // ------------------------------------------------------------------ consumers
  // A lane holds rows r and r + 8 of its warp's tile. NT = 1: head r's maps 0 and 1, over a slice of
  // 16 tokens of every stage. NT = 2: heads r and r + 8 of map warp & 1, over 32 tokens. (With both
  // maps' tiles in every warp D = 128 needs more registers than two CTAs leave: 100 sequences of up
  // to 8K, 12 heads on one kv head 81 us against 51; with both maps in one tile, as for NT = 1, 100.)
  constexpr int kTiles = NT;                         // 16-token tiles of a slice
  constexpr int kQSteps = C::kSteps / NT;            // k-steps of a warp's S
  constexpr int kMerge = C::kWarps / NT;             // warps that hold the same rows
  const int r = lane >> 2;
  const int q = lane & 3;
  const float c = p.scale_log2;
  const int map = NT == 2 ? warp & 1 : 0;
  const int tok_w = (NT == 2 ? warp >> 1 : warp) * 16 * kTiles;
  // ldmatrix row addresses: lane -> (matrix, row).
  const int mrow = lane & 7, msel = lane >> 3;
  const int k_token = tok_w + 8 * (msel >> 1) + mrow;  // K: matrices (n-tile, k half)
  const int k_half = (msel & 1) * 8 + map * (D / 2);
  const int v_token = tok_w + 8 * (msel & 1) + mrow;   // V: matrices (n-tile, token half)
  const int v_sub = (msel >> 1) * 8;
  int e = 0;
  bool ok = true;
  for (bool first = true; seg.next(p); first = false) {
    const size_t head0 = (static_cast<size_t>(seg.b) * p.Hkv + seg.g) * G;
    // Q as the A operand, rows r and r + 8 and both halves of a k-step. NT = 1: k-step kk lies in
    // map 2 kk / kSteps, whose rows alone are not zero. (Asking for the next segment's before this
    // one's rows are joined gained nothing.)
    uint32_t qa[kQSteps][NT][2];
#pragma unroll
    for (int kk = 0; kk < kQSteps; ++kk)
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        const int head = 8 * h + r;
        const uint32_t* from = p.q + (head0 + head) * (D / 2) + map * (D / 4) + kk * 8 + q;
        qa[kk][h][0] = head < G ? __ldg(from) : 0u;
        qa[kk][h][1] = head < G ? __ldg(from + 4) : 0u;
      }
    float o[D / 8][4];
    float mx[2], l[2];  // of rows r and r + 8: reference max in log2 units, sum
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    mx[0] = mx[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    int last_st = 0;
    for (int i = 0; i < seg.nblk; ++i, ++e) {
      const int st = e % S;
      last_st = st;
      ok = wait_at(smem_u32(&ctl->full[st]), (e / S) & 1, wc);
      if (ok) {
        const uint32_t kp = smem_u32(ring + st * C::kStageBytes);
        const uint32_t vp = kp + C::kHalfBytes;
        const int left = seg.L - (seg.blk0 + i) * C::kTok - tok_w;  // tokens from this slice on
        float s[kTiles][2][4];
        // Scores; apart (NT = 1): each map's rows from its own k-steps alone.
        auto scores = [&](auto apart) {
          constexpr bool kApart = decltype(apart)::value;
          float rows[2][2];
#pragma unroll
          for (int tt = 0; tt < kTiles; ++tt)
#pragma unroll
            for (int x = 0; x < 8; ++x) s[tt][x >> 2][x & 3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < kQSteps; ++kk) {
            const bool lo = kk < kQSteps / 2;  // NT = 1: map 0's
            const uint32_t a[4] = {NT == 2 || lo ? qa[kk][0][0] : 0u,
                                   NT == 2 ? qa[kk][NT - 1][0] : lo ? 0u : qa[kk][0][0],
                                   NT == 2 || lo ? qa[kk][0][1] : 0u,
                                   NT == 2 ? qa[kk][NT - 1][1] : lo ? 0u : qa[kk][0][1]};
            if (kApart && kk == kQSteps / 2)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                rows[y][0] = s[0][y][0], rows[y][1] = s[0][y][1];
                s[0][y][2] = s[0][y][3] = 0.f;
              }
#pragma unroll
            for (int tt = 0; tt < kTiles; ++tt) {
              uint32_t kb[4];
              ldmatrix_x4(kb, kp + page_chunk(k_token + 16 * tt, kk * 16 + k_half));
              mma_bf16_16816(s[tt][0], a, kb[0], kb[1]);
              mma_bf16_16816(s[tt][1], a, kb[2], kb[3]);
            }
          }
          if constexpr (kApart)
#pragma unroll
            for (int y = 0; y < 2; ++y) s[0][y][0] = rows[y][0], s[0][y][1] = rows[y][1];
          // Slots past the context may hold anything.
          if (left < 16 * kTiles)
#pragma unroll
            for (int tt = 0; tt < kTiles; ++tt)
#pragma unroll
              for (int x = 0; x < 8; ++x)
                if (16 * tt + 8 * (x >> 2) + 2 * q + (x & 1) >= left)
                  s[tt][x >> 2][x & 3] = -INFINITY;
        };
        scores(std::false_type{});
        if (left < 16 * kTiles) {
          // Values past the context are cleared: a NaN would survive a weight of zero.
          for (int x = lane; x < 16 * kTiles * (D / 8); x += 32) {
            const int tok = x / (D / 8);
            if (tok >= left)
              st_shared_v4(vp + page_chunk(tok_w + tok, (x % (D / 8)) * 8), 0, 0, 0, 0);
          }
          __syncwarp();
        }
        // Weights 2^(c s - mx) against the reference max of the row so far; one of a sum above 2^24
        // (a score far above it), and a row's first, has the max found. Element x of n-tile y: row
        // r + 8 (x >> 1), token 8 y + 2 q + (x & 1) of the tile.
        float w[kTiles][2][4], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int tt = 0; tt < kTiles; ++tt) {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            w[tt][x >> 2][x & 3] = fast_exp2(fmaf(s[tt][x >> 2][x & 3], c, -mx[(x & 3) >> 1]));
#pragma unroll
          for (int h = 0; h < 2; ++h)
            sum[h] += (w[tt][0][2 * h] + w[tt][0][2 * h + 1]) +
                      (w[tt][1][2 * h] + w[tt][1][2 * h + 1]);
        }
        if (__any_sync(0xffffffffu, !(sum[0] + sum[1] <= kDiffDecodeRaise))) {
          if constexpr (NT == 1) {
            // An infinite key channel of one map is NaN times the other one's zeros. (Both maps apart
            // from the start spill at D = 128: 512 short contexts 102.5 to 107 us.)
            bool nan = false;
#pragma unroll
            for (int x = 0; x < 8; ++x) nan |= isnan(s[0][x >> 2][x & 3]);
            if (__any_sync(0xffffffffu, nan)) scores(std::true_type{});
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float top = -INFINITY;
#pragma unroll
            for (int tt = 0; tt < kTiles; ++tt)
              top = fmaxf(top, fmaxf(fmaxf(s[tt][0][2 * h], s[tt][0][2 * h + 1]),
                                     fmaxf(s[tt][1][2 * h], s[tt][1][2 * h + 1])) * c);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // Move the reference only when it grows by more than 8 (a factor of 256).
            if (top > mx[h] + 8.f) {
              const float al = fast_exp2(mx[h] - top);  // 0 when the reference is -inf
              mx[h] = top;
              l[h] *= al;
#pragma unroll
              for (int i = 0; i < D / 8; ++i) o[i][2 * h] *= al, o[i][2 * h + 1] *= al;
            }
            const float sub = mx[h] == -INFINITY ? 0.f : mx[h];
            sum[h] = 0.f;
#pragma unroll
            for (int tt = 0; tt < kTiles; ++tt) {
#pragma unroll
              for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int x = 2 * h; x < 2 * h + 2; ++x)
                  w[tt][y][x] = fast_exp2(fmaf(s[tt][y][x], c, -sub));
              sum[h] += (w[tt][0][2 * h] + w[tt][0][2 * h + 1]) +
                        (w[tt][1][2 * h] + w[tt][1][2 * h + 1]);
            }
          }
        }
        l[0] += sum[0];
        l[1] += sum[1];
        // The accumulators of the two n-tiles are, as bf16 pairs, the A fragment of P; what their
        // rounding leaves goes in as a second term, so that weights are good to 2^-16. One term
        // would leave 1.9e-3 of |O| (2-norm) beside the output's own 1.7e-3, and the products have
        // time while the bytes come: 32 sequences 166.2 us against 163.8 with one term, 48 of 16
        // heads a kv head 69.8 against 70.8, 512 short ones 101.8 against 100.2.
#pragma unroll
        for (int tt = 0; tt < kTiles; ++tt) {
          uint32_t pa[4], pb[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const float w0 = w[tt][f >> 1][2 * (f & 1)], w1 = w[tt][f >> 1][2 * (f & 1) + 1];
            pa[f] = pack_bf16x2(w0, w1);
            pb[f] = pack_bf16x2(w0 - __uint_as_float(pa[f] << 16),
                                w1 - __uint_as_float(pa[f] & 0xffff0000u));
          }
#pragma unroll
          for (int pair = 0; pair < D / 16; ++pair) {
            uint32_t vb[4];
            ldmatrix_x4_trans(vb, vp + page_chunk(v_token + 16 * tt, pair * 16 + v_sub));
            mma_bf16_16816(o[2 * pair], pa, vb[0], vb[1]);
            mma_bf16_16816(o[2 * pair + 1], pa, vb[2], vb[3]);
            mma_bf16_16816(o[2 * pair], pb, vb[0], vb[1]);
            mma_bf16_16816(o[2 * pair + 1], pb, vb[2], vb[3]);
          }
        }
      }
      __syncwarp();
      // The segment's last slot is kept for the merge.
      if (lane == 0 && i + 1 < seg.nblk) mbar_arrive(&ctl->empty[st]);
    }
    // ---------------------------------------------------------------- the segment's rows
    // Row 8 h + r of a warp's tile is map h of head r (NT = 1) or the warp's map of head 8 h + r;
    // warps w, w + NT, ... hold the same rows.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (q == 0) {
        red_m[warp * 16 + 8 * h + r] = mx[h];
        red_l[warp * 16 + 8 * h + r] = l[h];
      }
    }
    named_barrier_sync(1, C::kConsumers);  // and every consumer is past its last read of the slot
    // Each warp's rows, rescaled to the common max: [warp][16][D] fp32, columns rotated by eight a
    // row against bank conflicts.
    float* buf = reinterpret_cast<float*>(ring + last_st * C::kStageBytes);
    const bool whole = seg.nblk == seg.nb;
    const size_t slot = 2 * static_cast<size_t>(worker) + (first ? 0 : 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 8 * h + r;
      float M = -INFINITY;
#pragma unroll
      for (int x = 0; x < kMerge; ++x) M = fmaxf(M, red_m[((warp & (NT - 1)) + x * NT) * 16 + row]);
      const float f = l[h] != 0.f ? fast_exp2(mx[h] - M) : 0.f;
      if ((NT == 2 ? row : r) < G) {
        float* to = buf + (warp * 16 + row) * D;
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
          *reinterpret_cast<float2*>(to + ((8 * t + 2 * q + 8 * r) & (D - 1))) =
              make_float2(o[t][2 * h] * f, o[t][2 * h + 1] * f);
      }
    }
    named_barrier_sync(1, C::kConsumers);
    constexpr int kQuads = D / 4;
    for (int idx = tid; idx < G * kQuads; idx += C::kConsumers) {
      const int hg = idx / kQuads, quad = idx % kQuads;
      const int col = (4 * quad + 8 * (hg & 7)) & (D - 1);
      float4 a[2];
      float2 ml[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int w0 = NT == 2 ? m : 0, row = NT == 2 ? hg : 8 * m + hg;
        const float* from = buf + (w0 * 16 + row) * D + col;
        float4 w[kMerge];
#pragma unroll
        for (int x = 0; x < kMerge; ++x)
          w[x] = *reinterpret_cast<const float4*>(from + x * NT * 16 * D);
        a[m] = make_float4(w[0].x + w[1].x, w[0].y + w[1].y, w[0].z + w[1].z, w[0].w + w[1].w);
        if constexpr (kMerge == 4)
          a[m] = make_float4(a[m].x + (w[2].x + w[3].x), a[m].y + (w[2].y + w[3].y),
                             a[m].z + (w[2].z + w[3].z), a[m].w + (w[2].w + w[3].w));
        float M = -INFINITY, Ls = 0.f;
#pragma unroll
        for (int x = 0; x < kMerge; ++x) M = fmaxf(M, red_m[(w0 + x * NT) * 16 + row]);
#pragma unroll
        for (int x = 0; x < kMerge; ++x) {
          const float lw = red_l[(w0 + x * NT) * 16 + row];
          if (lw != 0.f) Ls += lw * fast_exp2(red_m[(w0 + x * NT) * 16 + row] - M);
        }
        ml[m] = make_float2(M, Ls);
      }
      if (whole) {
        const unsigned lanes = kQuads == 32 ? 0xffffffffu : 0xffffu << (lane & 16);
        diff_finish<D>(p, head0 + hg, __ldg(p.lam + seg.g * G + hg), diff_weight(p, quad), quad,
                       a[0], a[1], ml[0], ml[1], lanes);
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const size_t at = (slot * 2 + m) * G + hg;
          *reinterpret_cast<float4*>(p.part_o + at * D + 4 * quad) = a[m];
          if (quad == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = ml[m];
        }
      }
    }
    fence_proxy_async_smem();  // the merge's plain accesses, before the slot's next copy
    named_barrier_sync(1, C::kConsumers);
    if (lane == 0) mbar_arrive(&ctl->empty[last_st]);
  }
}

// Joins the parts of contexts that several workers share, and writes the rows of empty ones:
//   M = max_c m_c,  L = sum_c l_c 2^(m_c - M),  A = sum_c O_c 2^(m_c - M)  of each map.
// A CTA takes join_heads heads of a (kv head, sequence); where there are more of those than workers
// it goes by a worker instead, and joins the context that this worker's share is the first to cut
// (512 sequences of 20 to 400 tokens, 8 kv heads: 130 us in all by contexts, whose 4096 CTAs mostly
// find a whole one, and 101; 256 of 1K 189 and 179). A warp takes one head, and set s of the
// `sets` warps of a head the parts s, s + sets, ... (at D = 64 a half warp the even ones of those
// and the other the odd); lanes hold the parts' m and l, of all parts in every warp, so that the
// sets' sums of O are added as they are, in order. 32 parts at most (64 at D = 64) take one round
// trip to L2. Eight parts a warp at once (64 a round) need 186 registers, with which a CTA does not
// fit beside one that still decodes: one sequence of 16K tokens 19.7 us against 20.2, but 16 heads
// a kv head 81 against 76.6. 16 warps a CTA: 19.8 and 77.9.
constexpr int kDiffJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(kDiffJoinWarps * 32, 2)
    diff_join_kernel(const DiffDecodeParams p) {
  constexpr int kQuads = D / 4, kHalves = 32 / kQuads, kBatch = 4;
  __shared__ float4 so[2][kDiffJoinWarps][32];
  const int G = p.group, H = p.join_heads;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int idx = static_cast<int>(blockIdx.x);  // the (sequence, kv head), or the worker
  const bool workers = p.join_workers != 0;
  // Without keys this kernel runs alone, and reports what is wrong with the lengths.
  const bool report = p.max_len == 0 && idx == 0 && blockIdx.y == 0 && tid < 32;
  int b = workers ? 0 : idx / p.Hkv, g = idx % p.Hkv;
  const DiffShare<D> share(p, b, report);
  // The context's first unit, its blocks and units.
  int u0 = 0, nb = 0, w = 0;
  const bool cut = !workers || (idx > 0 && idx < share.n);
  if (workers && cut) {
    int ahead;
    share.find(p, share.start(idx), b, ahead);
    nb = share.blocks(context_length(p, b, false));
    w = share.units(nb);
    g = (share.start(idx) - ahead * p.Hkv) / w;
    u0 = ahead * p.Hkv + g * w;
  } else if (cut) {
    nb = share.blocks(context_length(p, b, false));
    w = share.units(nb);
    u0 = share.before * p.Hkv + g * w;
  }
  const int h0 = g * G + static_cast<int>(blockIdx.y) * H, hg = static_cast<int>(blockIdx.y) * H;
  const size_t head0 = static_cast<size_t>(b) * p.Hq + h0;
  // Rows of empty contexts. (Every CTA waits, those without work too: this kernel must not end
  // before the first one.)
  auto clear = [&](size_t row, int rows) {
    for (int i = tid; i < rows * kQuads; i += kDiffJoinWarps * 32)
      reinterpret_cast<uint2*>(p.o + row * D)[i] = make_uint2(0, 0);
    for (int i = tid; i < 2 * rows; i += kDiffJoinWarps * 32) p.lse[2 * row + i] = -INFINITY;
  };
  if (workers && blockIdx.y == 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int s = idx; s < p.B; s += static_cast<int>(gridDim.x))
      if (context_length(p, s, false) == 0) clear(static_cast<size_t>(s) * p.Hq, p.Hq);
  }
  if (nb == 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!workers) clear(head0, H);
    return;
  }
  // The workers of the context's first and last block; the first part is its worker's first segment
  // only if that has no block of a context before.
  const int c0 = share.worker_of(u0 + share.kStart);
  const int parts = share.worker_of(u0 + w - 1) - c0 + 1;
  const int slot0 = 2 * c0 + (share.start(c0) >= u0 ? 0 : 1);
  const int sets = imax(1, kDiffJoinWarps / H);
  const int set = sets > 1 ? warp / H : 0;
  const int quad = lane % kQuads, half = lane / kQuads;
  const float4 weight = diff_weight(p, quad);
  float lam = __ldg(p.lam + h0 + imin(sets > 1 ? warp % H : warp, H - 1));
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // One worker held the whole context, or another CTA joins it.
  if (parts == 1 || (workers && c0 + 1 != idx)) return;
  const int take = sets * kHalves;                 // parts that are taken side by side
  const int round = imin(kBatch * take, 64);       // parts of a round
  for (int hh = sets > 1 ? warp % H : warp; hh < H || sets > 1; hh += kDiffJoinWarps) {
    float4 a[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f};
    const bool here = set < sets;
    for (int x0 = 0; here && x0 < parts; x0 += round) {
      const int n = imin(round, parts - x0);
      auto at = [&](int x, int m) {
        return (static_cast<size_t>(x ? 2 * (c0 + x) : slot0) * 2 + m) * G + hg + hh;
      };
      float2 ml[2][2];
      float4 po[2][kBatch];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          ml[m][i] = lane + 32 * i < n ? __ldcg(reinterpret_cast<const float2*>(p.part_ml) +
                                                at(x0 + lane + 32 * i, m))
                                       : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int t = 0; t < kBatch; ++t)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int x = t * take + set * kHalves + half;
          po[m][t] =
              x < n ? __ldcg(reinterpret_cast<const float4*>(p.part_o + at(x0 + x, m) * D) + quad)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float top = fmaxf(ml[m][0].x, ml[m][1].x);
#pragma unroll
        for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float Mn = fmaxf(M[m], top);
        const float f = L[m] != 0.f ? exp2f(M[m] - Mn) : 0.f;
        M[m] = Mn;
        // A part whose sum is not 0 had scores; NaN among them alone leaves its max at -inf.
        const float w0 = ml[m][0].y != 0.f ? exp2f(ml[m][0].x - Mn) : 0.f;
        const float w1 = ml[m][1].y != 0.f ? exp2f(ml[m][1].x - Mn) : 0.f;
        float sum = ml[m][0].y * w0 + ml[m][1].y * w1;
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        L[m] = L[m] * f + sum;
        a[m].x *= f, a[m].y *= f, a[m].z *= f, a[m].w *= f;
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
          const int x = t * take + set * kHalves + half;
          const float v0 = __shfl_sync(0xffffffffu, w0, x & 31);
          const float v1 = __shfl_sync(0xffffffffu, w1, x & 31);
          const float wt = x < n ? (x < 32 ? v0 : v1) : 0.f;
          a[m].x += po[m][t].x * wt, a[m].y += po[m][t].y * wt;
          a[m].z += po[m][t].z * wt, a[m].w += po[m][t].w * wt;
        }
      }
    }
    if (kHalves == 2) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        a[m].x += __shfl_xor_sync(0xffffffffu, a[m].x, 16);
        a[m].y += __shfl_xor_sync(0xffffffffu, a[m].y, 16);
        a[m].z += __shfl_xor_sync(0xffffffffu, a[m].z, 16);
        a[m].w += __shfl_xor_sync(0xffffffffu, a[m].w, 16);
      }
    }
    if (sets > 1) {
      so[0][warp][lane] = a[0], so[1][warp][lane] = a[1];
      __syncthreads();
      if (set == 0)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          for (int i = 1; i < sets; ++i) {
            const float4 x = so[m][warp + i * H][lane];
            a[m].x += x.x, a[m].y += x.y, a[m].z += x.z, a[m].w += x.w;
          }
    }
    if (set == 0 && half == 0) {
      const unsigned lanes = kQuads == 32 ? 0xffffffffu : 0xffffu;
      diff_finish<D>(p, head0 + hh, lam, weight, quad, a[0], a[1], make_float2(M[0], L[0]),
                     make_float2(M[1], L[1]), lanes);
    }
    if (sets > 1) break;
    lam = __ldg(p.lam + h0 + imin(hh + kDiffJoinWarps, H - 1));
  }
}

}  // namespace ta
