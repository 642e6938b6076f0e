// decode_fp4.cuh — paged decode (one query token per sequence) over a 4-bit KV cache
// (fp4.cuh), with split-KV partials and a fused log-sum-exp-weighted combine.
//
//   O = softmax(scale K q) V,  LSE = ln sum_j exp(scale k_j . q),
//   k_j, v_j = code * block scale * tensor scale
//
// The key scale joins the softmax scale and the value scale the last division, so the
// kernel works on code * block scale, which is exact in f16. A token and kv head are 144
// bytes at d = 128 (K and V) against 512 in bf16, so per byte read there is 3.6 times the
// arithmetic of the bf16 decode: the instructions per token decide whether HBM stays the
// bound. The layout of the products follows from that:
//   * S^T = K Q^T and O^T = V^T P^T: tokens (then channels) are the 16 rows of an m16n8k16
//     MMA and the group's query heads its 8 columns. Up to 8 heads cost one MMA where heads as
//     rows would cost two, and K and V, the operands that are dequantized, are A fragments,
//     whose 4-bit codes each lane loads from shared memory in the order it needs them.
//   * The channels of a k-step (for S) and the rows of an m-tile (for O) may be any
//     permutation, as long as Q and the output use the same. Lane (r, q) = (lane / 4, lane % 4)
//     takes channels [D/4 q, D/4 (q + 1)) of token rows r and r + 8 in one 16-byte load, and
//     channels [D/8 r, D/8 (r + 1)) of the four tokens 2q, 2q + 1, 2q + 8, 2q + 9 of V: whole
//     scale blocks (at d = 64 half a block for V), so scales are fetched once per lane.
//   * Q in f16: bf16 values times a power of two per head (its largest magnitude lands in
//     [1, 2)), which f16 holds exactly down to 2^-14 of the largest; the power goes back into
//     the head's scale. P in f16: 2^(s - m + 7), at most 2^15, where m trails the running
//     max by less than 8; f16 keeps 11 bits of it where bf16 would keep 8.
//
// Work: the contexts are cut into blocks (of 128 tokens; of a stage where SOLO), numbered over
// sequence, kv head and position, with a few units more at each context's start for the cost of
// beginning it, and shared out evenly over the workers in that order: every worker has the same work whatever the
// lengths are, and finds its range from cu_seqlens alone. A worker is a CTA where contexts are
// few, so that they fall into few parts, and a single warp where they are many (SOLO), which
// then begins and ends contexts without waiting for three others. A range is one or more
// segments, each of one (sequence, kv head). A segment that is the whole context writes O and
// LSE itself; the others (a worker's first and last at most) leave the unnormalised O, the
// reference max and the sum in the workspace, two slots a worker, and a second kernel joins them
// in the workers' order, so results do not depend on timing:
//   M = max_c m_c,  L = sum_c l_c 2^(m_c - M),  O = sum_c O_c 2^(m_c - M) / L,
//   LSE = (M + log2 L) ln 2.
// The second kernel starts under programmatic dependent launch: with CTAs as workers it takes a
// context a CTA and finds the parts from cu_seqlens while the first still runs; with warps a
// worker a CTA, and each warp leaves word of the context that it begins and others end (going
// by contexts there, 1000 sequences x 8 kv heads took 31 us longer). No counters, so no memset.
//
// CTA: four warps; warp w takes stages w, w + 4, ... of a segment (64 tokens, 128 at d = 64), or
// all stages of its own segments, through a ring of its own in shared memory: it brings the next
// stage in with bulk copies while it works on one, so no warp waits for another before a
// segment's end.
//
// Measured (GB300, device time): 32 sequences of 1K-16K tokens, 8 kv heads of 4 query heads,
// d = 128, 313 MB: 62 us, 5.1 TB/s, 75 % of the copy rate; 48 sequences of 1-32K, 4 kv heads of
// 16, d = 64, pages of 16, 216 MB: 73 us (pages of 64: 67; 8 heads a kv head: 60 and 53); one
// sequence of 16K: 13 us. Bound by issue: 224 instructions of a warp per 16 tokens at d = 128, of
// which 64 convert and 64 scale at half rate; computing alone takes 54 us on the first, streaming
// alone 53, ~10 of each start-up and joining. At d = 64 with two head tiles 217 instructions.
#pragma once

#include "fp4.cuh"
#include "ptx.cuh"
#include "sched.h"

namespace ta {

struct DecodeFp4Params {
  const uint4* q;        // bf16 [B, Hq, 1, D]
  const uint8_t* k;      // 4-bit pools
  const uint8_t* v;
  const int* cu;         // [B+1] cumulative context lengths
  const int* table;      // [B, max_pages]
  uint16_t* o;           // bf16 [B, Hq, 1, D]
  float* lse;            // [B, Hq]
  float* part_o;         // [2 * workers, group, D]: two rows a worker; room for four workers a CTA
  float* part_ml;        // [2 * workers, group, 2]
  int4* joins;           // [workers], SOLO: the context that a worker begins and others end:
                         // its number, first part's slot, parts (0: none)
  int B, Hq, Hkv, max_pages, num_pages, group, page_shift, max_len;
  int slots;             // CTAs of the decode kernel
  int join_heads;        // query heads a CTA of the joining kernel takes
  float scale_log2;      // softmax scale * K tensor scale * log2 e
  float v_scale;
  int* status;
  unsigned long long timeout_ns;
};

// Units of work that beginning a context costs a CTA, in 128-token blocks. Measured: a CTA that
// begins one context more ends about 2.5 us later, and a block takes it 1.35 us (d = 128) or
// 0.9 us. With 0, 1, 2, 3 and 4 units 32 sequences of 1K-16K take 68.3, 65.7, 63.7, 63.2 and
// 63.8 us; with 0, 2, 3, 4 and 6 units 48 sequences of up to 32K at d = 64 take 81, 75.0, 74.5,
// 73.6 and 74.6 us.
template <int D>
struct DecodeFp4Start {
  static constexpr int kUnits = D == 128 ? 3 : 4;
};

template <int D, int NT>  // NT: 8-head column tiles (1 or 2)
struct DecodeFp4Cfg {
  static constexpr int kTok = 32;     // tokens per slice: two 16-row tiles
  static constexpr int kStage = 64 * 128 / D;  // tokens per ring stage
  static constexpr int kWarps = 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kCtas = D == 128 && NT == 2 ? 2 : 3;  // per SM
  static constexpr int kCode = D / 2, kScale = D / 16;
  // A stage in shared memory: K, then V, each as blocks of min(page, stage) tokens laid out like
  // the pool's: codes, then scales.
  static constexpr int kOffV = kStage * (kCode + kScale);
  static constexpr int kStageBytes = 2 * kOffV;      // 9216
  static constexpr int kStages = 2;                  // of one warp's ring
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kSteps = D / 16;              // k-steps of S^T, m-tiles of O^T
  static constexpr int kMiscBytes = 256 + 2 * kWarps * 16 * 4;
  static constexpr int kSmemBytes = kWarps * kRingBytes + kMiscBytes + 128;
  static_assert(kHeads * D * 4 <= kStageBytes, "a warp's O rows reuse one slot");
  static_assert(kWarps * kStages <= 8, "barriers");
};

struct DecodeFp4Ctrl {
  uint64_t full[8];  // [warps][stages]
  int abort_flag;
  int idle[4];       // ring slot each warp's rows are merged in
};

// D(16x8, fp32) += A(16x16, f16, row-major) * B(16x8, f16, column-major).
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a zero accumulator.
__device__ __forceinline__ void mma_f16_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1,
                                                   uint32_t a2, uint32_t a3, uint32_t b0,
                                                   uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// a * (b.lo, b.lo) or (b.hi, b.hi).
template <bool HI>
__device__ __forceinline__ uint32_t hmul2_dup(uint32_t a, uint32_t b) {
  const __half2 x = *reinterpret_cast<const __half2*>(&a);
  const __half2 y = *reinterpret_cast<const __half2*>(&b);
  const __half2 z = __hmul2(x, HI ? __high2half2(y) : __low2half2(y));
  return *reinterpret_cast<const uint32_t*>(&z);
}

// Slice h of stage `sl` (blocks of `run` tokens): S^T, the softmax step and O^T of 32 tokens, of
// which the first `left` belong to the context. EDGE: some do not; the others run without a
// mask.
template <int D, int NT, bool EDGE>
__device__ __forceinline__ void fp4_slice(const uint8_t* sl, int h, int run, int left, int r, int q,
                                          const uint32_t (&qb)[NT][D / 16][2],
                                          const float (&sc)[NT][2], float (&o)[NT][D / 16][4],
                                          float (&mref)[NT][2], float (&l)[NT][2]) {
  using C = DecodeFp4Cfg<D, NT>;
  constexpr int kWords = D / 64;  // 32-bit words of V codes per lane and token; K: 2 kWords
  // Codes and scales of the two 16-token tiles (K; V lies kOffV further): tile token tb is token
  // tb - first of the block that starts with token `first`.
  const uint8_t *codes[2], *scales[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int tb = 32 * h + 16 * u, first = tb & -run;
    codes[u] = sl + tb * C::kCode + first * C::kScale;
    scales[u] = sl + tb * C::kScale + (first + run) * C::kCode;
  }
  // ---- S^T = K Q^T, tiles of 16 tokens
  float s[2][NT][4];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t kw[2][2 * kWords], sf[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = r + 8 * x;
      if constexpr (D == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(codes[u] + row * C::kCode + 16 * q);
        kw[x][0] = v.x, kw[x][1] = v.y, kw[x][2] = v.z, kw[x][3] = v.w;
        sf[x] = e4m3x2_to_f16(
            *reinterpret_cast<const uint16_t*>(scales[u] + row * C::kScale + 2 * q));
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(codes[u] + row * C::kCode + 8 * q);
        kw[x][0] = v.x, kw[x][1] = v.y;
        sf[x] = e4m3x2_to_f16(scales[u][row * C::kScale + q]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * kWords; ++i) {
      uint32_t a[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        e2m1x8_to_f16(kw[x][i], a[x]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          a[x][e] = i < 2 ? hmul2_dup<false>(a[x][e], sf[x]) : hmul2_dup<true>(a[x][e], sf[x]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (i == 0)
          mma_f16_16816_zero(s[u][nt], a[0][0], a[1][0], a[0][1], a[1][1], qb[nt][0][0],
                             qb[nt][0][1]);
        else
          mma_f16_16816(s[u][nt], a[0][0], a[1][0], a[0][1], a[1][1], qb[nt][2 * i][0],
                        qb[nt][2 * i][1]);
        mma_f16_16816(s[u][nt], a[0][2], a[1][2], a[0][3], a[1][3], qb[nt][2 * i + 1][0],
                      qb[nt][2 * i + 1][1]);
      }
    }
  }
  // V's codes and scale pairs of both tiles, asked for before the softmax step, whose branch the
  // loads would not pass (32 sequences: 63.0 us without, 60.8 with).
  constexpr int kPer = D == 128 ? 1 : 2;  // lanes r of one scale block
  uint32_t w[2][4][kWords], two[2][2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint8_t* at = codes[u] + C::kOffV + (2 * q + (x & 1) + 8 * (x >> 1)) * C::kCode;
      if constexpr (D == 128) {
        const uint2 v = *reinterpret_cast<const uint2*>(at + 8 * r);
        w[u][x][0] = v.x, w[u][x][1] = v.y;
      } else {
        w[u][x][0] = *reinterpret_cast<const uint32_t*>(at + 4 * r);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint8_t* at = scales[u] + C::kOffV + (2 * q + 8 * x) * C::kScale + r / kPer;
      two[u][x] = __byte_perm(at[0], at[C::kScale], 0x5540);
    }
  }
  // ---- softmax: columns are heads 2q, 2q + 1, rows tokens r and r + 8 of each tile
  bool live[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) live[x] = !EDGE || r + 8 * x < left;
  // Weights 2^(x - mref) and their sums. A weight above 2^15 (a score past the reference max by
  // more than 8) shows in the sums, which are needed anyway; a sum may also pass it without one,
  // and the slow path then finds nothing to move, or moves early.
  float e[2][NT][4], sum[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[u][nt][i] = fast_exp2(fmaf(s[u][nt][i], sc[nt][i & 1], -mref[nt][i & 1]));
        if (EDGE && !live[2 * u + (i >> 1)]) e[u][nt][i] = 0.f;
      }
#pragma unroll
    for (int c = 0; c < 2; ++c)
      sum[nt][c] = (e[0][nt][c] + e[0][nt][c + 2]) + (e[1][nt][c] + e[1][nt][c + 2]);
  }
  float all = sum[0][0] + sum[0][1];
  if (NT == 2) all += sum[NT - 1][0] + sum[NT - 1][1];
  if (__any_sync(0xffffffffu, !(all <= 32768.f))) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = -INFINITY;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (live[x]) mx = fmaxf(mx, s[x >> 1][nt][c + 2 * (x & 1)] * sc[nt][c]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = mx - 7.f;
        if (mn > mref[nt][c]) {
          const float f = fast_exp2(mref[nt][c] - mn);
          mref[nt][c] = mn;
          l[nt][c] *= f;
#pragma unroll
          for (int i = 0; i < C::kSteps; ++i) o[nt][i][c] *= f, o[nt][i][c + 2] *= f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int u = x >> 1, i = c + 2 * (x & 1);
            e[u][nt][i] = live[x] ? fast_exp2(fmaf(s[u][nt][i], sc[nt][c], -mn)) : 0.f;
          }
          sum[nt][c] = (e[0][nt][c] + e[0][nt][c + 2]) + (e[1][nt][c] + e[1][nt][c + 2]);
        }
      }
  }
  uint32_t pb[2][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    l[nt][0] += sum[nt][0];
    l[nt][1] += sum[nt][1];
    // The weights' fragment, transposed, is the B operand of O^T: k = tokens.
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        pb[u][nt][i] = movmatrix_trans(pack_f16x2(e[u][nt][2 * i], e[u][nt][2 * i + 1]));
  }
  // ---- O^T += V^T P^T
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t sv[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (EDGE) {
        // Slots past the context may hold anything; a NaN scale would survive p = 0.
        const int tok = 16 * u + 2 * q + 8 * x;
        if (tok >= left) two[u][x] &= 0xFF00u;
        if (tok + 1 >= left) two[u][x] &= 0x00FFu;
      }
      sv[x] = e4m3x2_to_f16(two[u][x]);
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      // Token pairs side by side: byte j holds channel 2j (lo) or 2j + 1 (hi) of both.
      constexpr uint32_t kLow = 0x0F0F0F0Fu;
      uint32_t lo[2][4], hi[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t w0 = w[u][2 * x][i], w1 = w[u][2 * x + 1][i];
        e2m1x8_to_f16((w0 & kLow) | ((w1 << 4) & ~kLow), lo[x]);
        e2m1x8_to_f16(((w0 >> 4) & kLow) | (w1 & ~kLow), hi[x]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[x][e] = hmul2(lo[x][e], sv[x]);
          hi[x][e] = hmul2(hi[x][e], sv[x]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16_16816(o[nt][4 * i + e], lo[0][e], hi[0][e], lo[1][e], hi[1][e], pb[u][nt][0],
                        pb[u][nt][1]);
    }
  }
}

// Context length of sequence b; 0 (and a report, if asked) where cu_seqlens is malformed.
__device__ __forceinline__ int fp4_length(const DecodeFp4Params& p, int b, bool report) {
  const int L = __ldg(p.cu + b + 1) - __ldg(p.cu + b);
  if (L >= 0 && L <= p.max_len) return L;
  if (report) report_status(p.status, -7);
  return 0;
}

// How the blocks are shared out. Every warp of both kernels works it out by itself, from
// cu_seqlens alone: a context counts its blocks and kStart units before them for what beginning
// it costs, and worker i of n takes an even share of the units, the first r workers q + 1, the
// others q. A share that ends among a context's kStart units holds none of it. Cutting small
// batches into equal parts of whole rounds of the four warps instead, a CTA a part, so that no
// CTA begins two contexts, gained 0.6 us on one sequence of 16K tokens (13.7 us) and lost 0.5 to
// 1 us on one of 700, one of 4K and four of 1K to 16K. Warps as workers, with blocks of a stage:
// with 1, 2 and 3 units 1000 sequences of 20-400 tokens x 8 kv heads take 78.7, 79.3 and 80.2 us,
// 512 of 200-1000 81.0, 82.1 and 84.4 (blocks of 128 tokens at d = 128 and one unit: 81.9, 83.4).
template <int D, bool SOLO>
struct Fp4Share {
  static constexpr int kStart = SOLO ? 1 : DecodeFp4Start<D>::kUnits;
  static constexpr int kTok = SOLO ? DecodeFp4Cfg<D, 1>::kStage : 128;  // tokens of a block
  // Parts of a context that join well: with CTAs as workers the joining kernel reads 32 in one
  // round. Warps: one sequence of 16K tokens among 63 empty ones takes 26 us, in 128 parts 28.
  static constexpr int kParts = SOLO ? 64 : 32;
  int total;    // units of one kv head, all sequences
  int before;   // those of the sequences before `upto`
  int n, q, r;
  int w0;       // units of sequence `lane`

  __device__ __forceinline__ static int blocks(int L) { return (L + kTok - 1) / kTok; }
  __device__ __forceinline__ static int units(int nb) { return nb > 0 ? nb + kStart : 0; }

  __device__ __forceinline__ Fp4Share(const DecodeFp4Params& p, int upto, bool report) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    w0 = lane < p.B ? units(blocks(fp4_length(p, lane, report))) : 0;
    int all = w0, ahead = lane < upto ? w0 : 0;
    for (int b0 = lane + 32; b0 < p.B; b0 += 128) {
#pragma unroll
      for (int b = b0; b < b0 + 128; b += 32) {  // four loads at a time
        const int w = b < p.B ? units(blocks(fp4_length(p, b, report))) : 0;
        all += w;
        if (b < upto) ahead += w;
      }
    }
    total = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, ahead);
    const int U = total * p.Hkv;
    // As many workers as the GPU holds, but over kParts a context only at four units or more each.
    // Contexts are counted by the lanes that have any, up to 32 x kv heads (enough for every
    // worker), and a padded batch's empty ones are none: with B counted instead, one sequence of
    // 16K tokens x 8 kv heads took 18 us among 55 empty ones and 54 among 63, now 15.6 and 26.
    const int live = __popc(__ballot_sync(0xffffffffu, all > 0)) * p.Hkv;
    n = imin((SOLO ? DecodeFp4Cfg<D, 1>::kWarps : 1) * p.slots, imin(U, imax(live * kParts, U / 4)));
    q = n ? U / n : 0;
    r = U - q * n;
  }
  // First unit of worker i, and the worker that takes unit u.
  __device__ __forceinline__ int start(int i) const { return i * q + imin(i, r); }
  __device__ __forceinline__ int worker_of(int u) const {
    const int large = r * (q + 1);
    return u < large ? u / (q + 1) : r + (u - large) / q;
  }
  // The sequence whose heads hold unit u, and the units (of one kv head) before it.
  __device__ __forceinline__ void find(const DecodeFp4Params& p, int u, int& seq,
                                       int& ahead) const {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    int run = 0;
    for (int b0 = 0; b0 < p.B;) {
      const int b = b0 + lane;
      const int w = b0 == 0 ? w0 : b < p.B ? units(blocks(fp4_length(p, b, false))) : 0;
      int sum = w;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += x;
      }
      sum += run;
      const unsigned past = __ballot_sync(0xffffffffu, u < sum * p.Hkv);
      if (past) {
        const int l = __ffs(past) - 1;
        seq = b0 + l;
        ahead = __shfl_sync(0xffffffffu, sum - w, l);
        return;
      }
      run = __shfl_sync(0xffffffffu, sum, 31);
      for (b0 += 32; b0 < p.B; b0 += 128) {  // past four times 32 sequences at once
        int four = 0;
#pragma unroll
        for (int c = b0 + lane; c < b0 + lane + 128; c += 32)
          four += units(c < p.B ? blocks(fp4_length(p, c, false)) : 0);
        four = run + __reduce_add_sync(0xffffffffu, four);
        if (u < four * p.Hkv) break;
        run = four;
      }
    }
    seq = p.B - 1;  // not reached: u lies below the total
    ahead = run;
  }
};

template <int D, int NT, bool SOLO>
__global__ void __launch_bounds__(128, DecodeFp4Cfg<D, NT>::kCtas)
    decode_fp4_kernel(const DecodeFp4Params p) {
  using C = DecodeFp4Cfg<D, NT>;
  constexpr int S = C::kStages;
  static_assert(S == 2, "two slots a ring");
  const int G = p.group;  // 1 <= G <= 8 NT
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5;
  const int lane = tid & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint8_t* ring = base + warp * C::kRingBytes;
  uint8_t* misc = base + C::kWarps * C::kRingBytes;
  DecodeFp4Ctrl* ctl = reinterpret_cast<DecodeFp4Ctrl*>(misc);
  float* red_m = reinterpret_cast<float*>(misc + 256);   // [warps][16 heads]
  float* red_l = red_m + C::kWarps * 16;
  uint64_t* full = ctl->full + warp * S;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 32);
    if (warp == 0) ctl->abort_flag = 0;
    fence_mbar_init();
  }
  const int cta = static_cast<int>(blockIdx.x);
  const Fp4Share<D, SOLO> share(p, 0, cta == 0 && warp == 0);
  const int worker = SOLO ? C::kWarps * cta + warp : cta;
  if (SOLO && lane == 0) p.joins[worker] = make_int4(0, 0, 0, 0);  // so far
  __syncthreads();  // barriers and flag
  if (worker >= share.n) return;
  int u = share.start(worker);
  const int end = share.start(worker + 1);
  int b, seq_u;
  share.find(p, u, b, seq_u);
  seq_u *= p.Hkv;  // first unit of sequence b
  const WaitCtl wc{p.timeout_ns, p.status, &ctl->abort_flag};
  const WaitCtl wc_drain{p.timeout_ns, p.status, nullptr};

  // Copies of one stage: lane 4 sub + part brings K (part 0) or V (part 2) of the stage's tokens
  // in its page `sub` (up to eight pages of 16 tokens), a whole (page, head) block in one
  // copy; where a page is longer than a stage, parts 0 and 2 bring its codes and parts 1 and 3
  // its scales. Every lane arrives on the stage's barrier with the bytes it asked for. Stages
  // lie at the same place of their pages, but for `flip` below. Pages past the context are not
  // copied. A page whose entry lies outside the pool is never addressed: the status word reports it
  // and it reads as zeros. A stage's table entries are read one stage ahead of its copies.
  const int lp = p.page_shift;
  const int sub = lane >> 2, part = lane & 3;
  const int run = imin(C::kStage, 1 << lp);  // tokens of the stage in one page
  const bool whole_pages = (1 << lp) == run;
  const bool copies = sub * run < C::kStage && !(whole_pages && (part & 1));
  constexpr int kHop = (SOLO ? 1 : C::kWarps) * C::kStage;  // tokens from stage to stage
  const int tok_w = SOLO ? 0 : warp * C::kStage;  // the warp's first token in a segment
  const int tok0 = tok_w + sub * run;             // this lane's first token in the warp's stage 0
  const uint32_t bytes = static_cast<uint32_t>(run) *
                         (whole_pages ? C::kCode + C::kScale : (part & 1) ? C::kScale : C::kCode);
  // Shared-memory addresses of this lane's copy and of its barrier, for the next stage; the
  // other slot's follow by adding, then subtracting, the distance.
  uint32_t dst = smem_u32(ring) + ((part & 2) ? C::kOffV : 0) +
                 ((part & 1) ? run * C::kCode : 0) + sub * run * (C::kCode + C::kScale);
  uint32_t bar = smem_u32(full);
  int step = 1;
  const int in_page = tok0 & ((1 << lp) - 1);
  const uint8_t* const src0 =
      ((part & 2) ? p.v : p.k) +
      ((part & 1) ? (C::kCode << lp) + in_page * C::kScale : in_page * C::kCode);
  // A page of 128 tokens at d = 128 holds two stages; a warp that takes all goes to and fro
  // between the halves.
  const uint32_t flip = SOLO && (C::kStage << 1) == (1 << lp)
                            ? static_cast<uint32_t>(run * ((part & 1) ? C::kScale : C::kCode))
                            : 0;
  uint32_t half = 0;
  const uint32_t blk_bytes = static_cast<uint32_t>(C::kCode + C::kScale) << lp;
  const uint32_t page_bytes = static_cast<uint32_t>(p.Hkv) * blk_bytes;  // the host checks it

  const int r = lane >> 2, q = lane & 3;
  int st_out = 0;              // ring slot of the next stage
  uint32_t parity = 0;         // of slot st_out
  bool aborted = false;

  // The segment that starts at block u, and its first stage on the way.
  int g, n, t0, t1, next;
  bool whole;         // the segment is its whole context
  int begins;         // the context's last unit, if others end it; else -1
  const int* row;
  const uint8_t* src_g;
  // Table entry of this lane's page of stage i: -2 nothing to copy, -1 outside the pool.
  auto entry = [&](int i) {
    const int tok = t0 + tok0 + i * kHop;
    if (!copies || i >= n || tok >= t1) return -2;
    const int e = __ldg(row + (tok >> lp));
    return static_cast<unsigned>(e) < static_cast<unsigned>(p.num_pages) ? e : -1;
  };
  auto issue = [&](int phys) {
    if (phys >= 0) {
      asm volatile(
          "mbarrier.arrive.expect_tx.shared::cta.b64 _, [%3], %2;\n"
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
          "[%3];" ::"r"(dst),
          "l"(src_g + half + static_cast<uint64_t>(static_cast<uint32_t>(phys)) * page_bytes),
          "r"(bytes), "r"(bar)
          : "memory");
    } else {
      if (phys == -1) {
        report_status(p.status, -5);
        for (uint32_t x = 0; x < bytes; x += 16) st_shared_v4(dst + x, 0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
    }
    half ^= flip;
    dst += step * C::kStageBytes;
    bar += step * 8;
    step = -step;
  };
  auto open = [&]() {  // false: the range holds no more blocks
    if (u >= end) return false;
    int L = fp4_length(p, b, false), nb = share.blocks(L), w = share.units(nb);
    while (u >= seq_u + w * p.Hkv) {  // the sequence is done: on to the next that has blocks
      seq_u += w * p.Hkv;
      L = fp4_length(p, ++b, false);
      nb = share.blocks(L);
      w = share.units(nb);
    }
    g = (u - seq_u) / w;
    int pos = u - seq_u - g * w;
    if (pos < share.kStart) {
      u += share.kStart - pos;
      pos = share.kStart;
      if (u >= end) return false;
    }
    const int blk0 = pos - share.kStart;
    const int nblk = imin(nb - blk0, end - u);
    u += nblk;
    whole = nblk == nb;
    begins = blk0 || whole ? -1 : seq_u + (g + 1) * w - 1;
    // Stages of the segment's tokens [t0, t1): this warp takes stage warp, warp + 4, ...
    t0 = blk0 * share.kTok;
    t1 = imin(t0 + nblk * share.kTok, L);
    n = aborted ? 0 : (t1 - t0 - tok_w + kHop - 1) / kHop;
    half = t0 & C::kStage ? flip : 0;  // flip is 0 where the page holds one stage
    row = p.table + static_cast<size_t>(b) * p.max_pages;
    src_g = src0 + static_cast<size_t>(g) * blk_bytes;
    if (n > 0) {
      issue(entry(0));
      next = entry(1);
    }
    return true;
  };
  bool more = open();
  for (bool first = true; more; first = false) {
    const int ctx = b * p.Hkv + g;
    const size_t head0 = static_cast<size_t>(ctx) * G;
    // Q as the B operand: column (head) r, k-step kk = channels D/4 q + 4 kk + {0, 1 | 2, 3}.
    uint32_t qb[NT][C::kSteps][2];
    float sc[NT][2];  // scale of heads 8 nt + 2 q, + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint4 w[D / 32];
      const int h = 8 * nt + r;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        w[i] =
            h < G ? __ldg(p.q + (head0 + h) * (D / 8) + q * (D / 32) + i) : make_uint4(0, 0, 0, 0);
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[e] << 16)),
                                   fabsf(__uint_as_float(x[e] & 0xFFFF0000u))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int e2 = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
      e2 = amax == 0.f ? 0 : imax(-126, imin(126, e2));
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);  // 2^-e2
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          qb[nt][2 * i + (e >> 1)][e & 1] = pack_f16x2(__uint_as_float(x[e] << 16) * down,
                                                       __uint_as_float(x[e] & 0xFFFF0000u) * down);
      }
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23) * p.scale_log2;
      sc[nt][0] = __shfl_sync(0xffffffffu, up, 8 * q);
      sc[nt][1] = __shfl_sync(0xffffffffu, up, 8 * q + 4);
    }
    float o[NT][C::kSteps][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < C::kSteps; ++i)
        o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    // p = 2^(x - mref): mref is the running max less 7, and the max trails by less than 8.
    float mref[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      mref[nt][0] = mref[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;

    int left = t1 - t0 - tok_w;  // tokens from the stage's first on
    const bool was_whole = whole;
    const int begun = begins;
    int stages = aborted ? 0 : n;
    for (int i = 0;; ++i, left -= kHop) {
      // Into the slot of stage i - 1, which the whole warp has left: the next stage, or the next
      // segment's first one.
      if (i + 1 < stages) {
        issue(next);
        next = entry(i + 2);
      } else if (i == imax(stages - 1, 0)) {
        more = open();
      }
      if (i >= stages) break;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[st_out], parity, wc))) {
        // Let the copies in flight land (with a limit) before their slots are used again; there
        // are no more after that. The rest of the range is walked without stages.
        aborted = true;
        mbar_wait(&full[st_out], parity, wc_drain);
        if (i + 1 < stages || (more && n > 0))
          mbar_wait(&full[st_out ^ 1], parity ^ static_cast<uint32_t>(st_out), wc_drain);
        if (i + 1 >= stages) break;  // the next segment is open already
        stages = 0;
        i = -1;
        continue;
      }
      const uint8_t* sl = ring + st_out * C::kStageBytes;
      if (left >= C::kStage) {
#pragma unroll 1
        for (int h = 0; h < C::kStage / C::kTok; ++h)
          fp4_slice<D, NT, false>(sl, h, run, C::kTok, r, q, qb, sc, o, mref, l);
      } else {
#pragma unroll 1
        for (int h = 0; h * C::kTok < left; ++h)
          fp4_slice<D, NT, true>(sl, h, run, left - h * C::kTok, r, q, qb, sc, o, mref, l);
      }
      if (++st_out == S) st_out = 0, parity ^= 1;
      __syncwarp();
    }
    // ---------------------------------------------------------------- the segment's rows
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
    const size_t slot = 2 * static_cast<size_t>(worker) + (first ? 0 : 1);
    if constexpr (SOLO) {
      if (begun >= 0 && lane == 0)
        p.joins[worker] = make_int4(ctx, static_cast<int>(slot),
                                    share.worker_of(begun) - worker + 1, 0);
      // Lane (r, q): heads 2q, 2q + 1, channels D/8 r ..; m-tile i holds channels 2i and 2i + 1.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int h = 8 * nt + 2 * q + c;
          if (h >= G) continue;
          const float Ls = l[nt][c];
          if (was_whole) {
            const float inv = Ls != 0.f ? p.v_scale / Ls : 0.f;
            uint16_t* to = p.o + (head0 + h) * D + r * (D / 8);
#pragma unroll
            for (int i = 0; i < C::kSteps; i += 4)
              *reinterpret_cast<uint4*>(to + 2 * i) =
                  make_uint4(pack_bf16x2(o[nt][i][c] * inv, o[nt][i][c + 2] * inv),
                             pack_bf16x2(o[nt][i + 1][c] * inv, o[nt][i + 1][c + 2] * inv),
                             pack_bf16x2(o[nt][i + 2][c] * inv, o[nt][i + 2][c + 2] * inv),
                             pack_bf16x2(o[nt][i + 3][c] * inv, o[nt][i + 3][c + 2] * inv));
            if (r == 0)
              p.lse[head0 + h] =
                  Ls != 0.f ? (mref[nt][c] + log2f(Ls)) * 0.69314718055994530942f : -INFINITY;
          } else {
            float* to = p.part_o + (slot * G + h) * D + r * (D / 8);
#pragma unroll
            for (int i = 0; i < C::kSteps; i += 2)
              *reinterpret_cast<float4*>(to + 2 * i) = make_float4(
                  o[nt][i][c], o[nt][i][c + 2], o[nt][i + 1][c], o[nt][i + 1][c + 2]);
            if (r == 0)
              *reinterpret_cast<float2*>(p.part_ml + 2 * (slot * G + h)) =
                  make_float2(mref[nt][c], Ls);
          }
        }
    } else {
      // The slot of the stage just used; the next segment's first stage is on its way into the
      // other one, and its latency hides behind the merge.
      float* const mine =
          reinterpret_cast<float*>(ring + (st_out ^ 1) * C::kStageBytes);
      // [head][D] fp32 in each warp's idle slot. Lane (r, q): heads 2q, 2q + 1, channels D/8 r ..;
      // m-tile i holds channels 2i and 2i + 1 of them.
      if (lane == 0) ctl->idle[warp] = st_out ^ 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int h = 8 * nt + 2 * q + c;
          if (r == 0) {
            red_m[warp * 16 + h] = mref[nt][c];
            red_l[warp * 16 + h] = l[nt][c];
          }
          if (h < G) {
            float* to = mine + h * D + r * (D / 8);
#pragma unroll
            for (int i = 0; i < C::kSteps; i += 2)
              *reinterpret_cast<float4*>(to + 2 * i) = make_float4(
                  o[nt][i][c], o[nt][i][c + 2], o[nt][i + 1][c], o[nt][i + 1][c + 2]);
          }
        }
      __syncthreads();
      constexpr int kQuads = D / 4;  // four-column groups of one head's row
      for (int idx = tid; idx < G * kQuads; idx += C::kThreads) {
        const int hh = idx / kQuads, d0 = (idx % kQuads) * 4;
        float M = red_m[hh];
#pragma unroll
        for (int w = 1; w < C::kWarps; ++w) M = fmaxf(M, red_m[w * 16 + hh]);
        float Ls = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
          const float lw = red_l[w * 16 + hh];
          if (lw != 0.f) {  // the warp had tokens; a NaN among their scores is a sum of NaN
            const float f = fast_exp2(red_m[w * 16 + hh] - M);
            const float4 x = *reinterpret_cast<const float4*>(
                base + w * C::kRingBytes + ctl->idle[w] * C::kStageBytes + (hh * D + d0) * 4);
            Ls += lw * f;
            a.x += x.x * f, a.y += x.y * f, a.z += x.z * f, a.w += x.w * f;
          }
        }
        if (was_whole) {
          const size_t orow = head0 + hh;
          const float inv = Ls != 0.f ? p.v_scale / Ls : 0.f;
          *reinterpret_cast<uint2*>(p.o + orow * D + d0) =
              make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
          if (d0 == 0)
            p.lse[orow] = Ls != 0.f ? (M + log2f(Ls)) * 0.69314718055994530942f : -INFINITY;
        } else {
          *reinterpret_cast<float4*>(p.part_o + (slot * G + hh) * D + d0) = a;
          if (d0 == 0)
            *reinterpret_cast<float2*>(p.part_ml + 2 * (slot * G + hh)) = make_float2(M, Ls);
        }
      }
      fence_proxy_async_smem();  // the merge's plain writes, before the next segment's copies
      __syncthreads();
    }
  }
}

// Joins the parts of contexts that several workers share, and writes the rows of empty ones. One
// CTA per (kv head, sequence), per query head, or per worker (SOLO); a thread takes four columns of
// one head, and where that leaves threads over, set s of them takes the parts s, s + sets, ...;
// the sets' sums are added in order.
constexpr int kCombineThreads = 256;  // at most

template <int D, bool SOLO>
__global__ void __launch_bounds__(kCombineThreads) combine_fp4_kernel(const DecodeFp4Params p) {
  constexpr int kQuads = D / 4, kBatch = 4;
  __shared__ float2 sml[kCombineThreads];
  __shared__ float4 so[kCombineThreads];
  const int G = p.group, H = SOLO ? G : p.join_heads;
  const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
  size_t head0;  // first query head's row
  int hg, slot0, c0, parts;  // its place in the group; first part's slot and worker; parts
  auto empty = [&](size_t row, int heads) {  // O = 0, LSE = -inf
    for (int i = tid; i < heads * kQuads; i += threads)
      reinterpret_cast<uint2*>(p.o + row * D)[i] = make_uint2(0, 0);
    for (int i = tid; i < heads; i += threads) p.lse[row + i] = -INFINITY;
  };
  // Every CTA waits, those without work too: this kernel must not end before the first one.
  if constexpr (SOLO) {
    for (int b = static_cast<int>(blockIdx.x); b < p.B; b += static_cast<int>(gridDim.x))
      if (fp4_length(p, b, false) == 0) empty(static_cast<size_t>(b) * p.Hq, p.Hq);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 join = __ldcg(p.joins + blockIdx.x);
    if (join.z == 0) return;
    head0 = static_cast<size_t>(join.x) * G, hg = 0, slot0 = join.y, parts = join.z;
    c0 = slot0 >> 1;
  } else {
    const int h0 = static_cast<int>(blockIdx.x) * H, b = static_cast<int>(blockIdx.y);
    const int g = h0 / G;  // kv head
    hg = h0 % G;
    const Fp4Share<D, SOLO> share(p, b, false);
    const int nb = share.blocks(fp4_length(p, b, false));
    head0 = static_cast<size_t>(b) * p.Hq + h0;
    if (nb == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      empty(head0, H);
      return;
    }
    // The context's first unit, and those of its first and last block.
    const int w = share.units(nb), u0 = share.before * p.Hkv + g * w;
    c0 = share.worker_of(u0 + share.kStart);
    parts = share.worker_of(u0 + w - 1) - c0 + 1;
    // The first part is its worker's first segment only if that has no block of the context
    // before.
    slot0 = 2 * c0 + (share.start(c0) >= u0 ? 0 : 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (parts == 1) return;  // one worker held the whole context
  }
  const int items = H * kQuads;
  const int sets = imax(1, imin(threads / items, parts));
  const int set = items < threads ? tid / items : 0;
  for (int it0 = 0; it0 < items; it0 += threads) {
    const int item = it0 + (items < threads ? tid % items : tid);
    const bool here = item < items && set < sets;
    const int hh = item / kQuads, quad = item % kQuads;
    float M = -INFINITY, Ls = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = here ? set : parts; x0 < parts; x0 += sets * kBatch) {
      float2 ml[kBatch];
      float4 ov[kBatch];
#pragma unroll
      for (int t = 0; t < kBatch; ++t) {
        const int x = imin(x0 + t * sets, parts - 1);
        const size_t at = static_cast<size_t>(x ? 2 * (c0 + x) : slot0) * G + hg + hh;
        ml[t] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + 2 * at));
        ov[t] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + 4 * quad));
      }
      float Mn = M;
#pragma unroll
      for (int t = 0; t < kBatch; ++t) Mn = fmaxf(Mn, ml[t].x);
      const float f = M == -INFINITY ? 0.f : exp2f(M - Mn);
      M = Mn;
      Ls *= f;
      a.x *= f, a.y *= f, a.z *= f, a.w *= f;
#pragma unroll
      for (int t = 0; t < kBatch; ++t)
        if (x0 + t * sets < parts) {
          const float wt = exp2f(ml[t].x - M);
          Ls += ml[t].y * wt;
          a.x += ov[t].x * wt, a.y += ov[t].y * wt, a.z += ov[t].z * wt, a.w += ov[t].w * wt;
        }
    }
    if (sets > 1) {
      so[tid] = a;
      sml[tid] = make_float2(M, Ls);
      __syncthreads();
      if (set == 0) {
        for (int i = 1; i < sets; ++i) M = fmaxf(M, sml[tid + i * items].x);
        Ls = 0.f;
        a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < sets; ++i) {
          const float2 ml = sml[tid + i * items];
          if (ml.y == 0.f) continue;  // more sets than parts
          const float f = exp2f(ml.x - M);
          const float4 x = so[tid + i * items];
          Ls += ml.y * f;
          a.x += x.x * f, a.y += x.y * f, a.z += x.z * f, a.w += x.w * f;
        }
      }
    }
    if (here && set == 0) {
      const float inv = p.v_scale / Ls;
      const size_t orow = head0 + hh;
      *reinterpret_cast<uint2*>(p.o + orow * D + 4 * quad) =
          make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
      if (quad == 0) p.lse[orow] = (M + log2f(Ls)) * 0.69314718055994530942f;
    }
  }
}

}  // namespace ta
