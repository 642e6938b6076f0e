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
// CTA: one split (a run of 128-token stages) of one (sequence, kv head); four consumer warps,
// 32 tokens of a stage each, and a producer warp that brings every page of a stage in with one
// bulk copy for K and one for V. The split, merge and ticket scheme is the bf16 decode's.
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
  float* part_o;         // [B*Hkv, max_splits, G, D]
  float* part_ml;        // [B*Hkv, max_splits, G, 2]
  int* counters;         // [B*Hkv], zero before the launch
  int Hq, Hkv, max_pages, num_pages, max_splits, chunk_stages, group, page_shift, max_len;
  float scale_log2;      // softmax scale * K tensor scale * log2 e
  float v_scale;
  int* status;
  unsigned long long timeout_ns;
};

template <int D, int NT>  // NT: 8-head column tiles (1 or 2)
struct DecodeFp4Cfg {
  static constexpr int kTok = 128;  // tokens per ring stage
  static constexpr int kWarps = 4;
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kThreads = kConsumers + 32;
  static constexpr int kCode = D / 2, kScale = D / 16, kRow = kCode + kScale;
  static constexpr int kHalf = kTok * kRow;        // K (or V) of a stage
  static constexpr int kStageBytes = 2 * kHalf;
  static constexpr int kStages = 4 * 128 / D;      // 4 x 18 KB (D = 128), 8 x 9 KB (D = 64)
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kSteps = D / 16;            // k-steps of S^T, m-tiles of O^T
  static constexpr int kMiscBytes = 256 + 2 * kWarps * 16 * 4;
  static constexpr int kSmemBytes = kRingBytes + kMiscBytes + 128;
  static_assert(kWarps * kHeads * D * 4 <= kRingBytes, "the warps' O rows reuse the ring");
};

struct DecodeFp4Ctrl {
  uint64_t full[8];
  uint64_t empty[8];
  int abort_flag;
  int is_last;
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

__device__ __forceinline__ uint32_t dup_lo(uint32_t a) { return __byte_perm(a, a, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t a) { return __byte_perm(a, a, 0x3232); }

template <int D, int NT>
__global__ void __launch_bounds__(160, NT == 1 ? 3 : 2)
    decode_fp4_kernel(const DecodeFp4Params p) {
  using C = DecodeFp4Cfg<D, NT>;
  constexpr int S = C::kStages;
  constexpr int kWords = D / 64;  // 32-bit words of V codes per lane and token; K: 2 kWords
  const int G = p.group;          // 1 <= G <= 8 NT
  const int split = static_cast<int>(blockIdx.x);
  const int g = static_cast<int>(blockIdx.y);
  const int b = static_cast<int>(blockIdx.z);
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const size_t head0 = static_cast<size_t>(b) * p.Hq + static_cast<size_t>(g) * G;

  int L = p.cu[b + 1] - p.cu[b];
  if (L < 0 || L > p.max_len) {
    if (split == 0 && tid == 0) report_status(p.status, -7);
    L = 0;
  }
  const int nstages = (L + C::kTok - 1) / C::kTok;
  const int nsplit = (nstages + p.chunk_stages - 1) / p.chunk_stages;
  if (L == 0) {
    // Empty context: O = 0, LSE = -inf.
    if (split == 0) {
      for (int idx = tid; idx < G * D; idx += C::kThreads) p.o[head0 * D + idx] = 0;
      if (tid < G) p.lse[head0 + tid] = -INFINITY;
    }
    return;
  }
  if (split >= nsplit) return;
  const int st0 = split * p.chunk_stages;
  const int n = imin(nstages - st0, p.chunk_stages);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint8_t* misc = ring + C::kRingBytes;
  DecodeFp4Ctrl* ctl = reinterpret_cast<DecodeFp4Ctrl*>(misc);
  float* red_m = reinterpret_cast<float*>(misc + 256);   // [warps][16 heads]
  float* red_l = red_m + C::kWarps * 16;

  if (tid == C::kConsumers) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], C::kWarps);
    }
    ctl->abort_flag = 0;
    ctl->is_last = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtl wc{p.timeout_ns, p.status, &ctl->abort_flag};
  const WaitCtl wc_drain{p.timeout_ns, p.status, nullptr};
  const int lp = p.page_shift;

  if (warp == C::kWarps) {
    // ---------------------------------------------------------------- producer
    // Lane 2i + kv < 2 * (128 >> lp) brings K (kv = 0) or V of page i of every stage: whole
    // (page, head) blocks, one copy each. It reads its table entry one stage ahead. Pages
    // past the context are not copied (no consumer reads them). A page whose entry lies
    // outside the pool is never addressed: the status word reports it and it reads as zeros.
    const int* row = p.table + static_cast<size_t>(b) * p.max_pages;
    const int pages = C::kTok >> lp;
    const uint32_t bytes = static_cast<uint32_t>(C::kRow) << lp;
    const uint8_t* pool = (lane & 1) ? p.v : p.k;
    const int sub = lane >> 1;
    int issued = 0;
    auto entry = [&](int k) {  // -2: nothing to copy, -1: bad entry
      const int tok = (st0 + k) * C::kTok + (sub << lp);
      if (sub >= pages || tok >= L) return -2;
      const int e = __ldg(row + (tok >> lp));
      return e < 0 || e >= p.num_pages ? -1 : e;
    };
    int next = entry(0);
    for (int k = 0; k < n; ++k) {
      const int st = k % S;
      bool okw = true;
      if (lane == 0) okw = mbar_wait(&ctl->empty[st], ((k / S) & 1) ^ 1, wc);
      if (!__shfl_sync(0xffffffffu, okw, 0)) break;
      ++issued;
      const int phys = next;
      uint8_t* dst = ring + st * C::kStageBytes + (lane & 1) * C::kHalf + sub * bytes;
      const uint32_t good = __ballot_sync(0xffffffffu, phys >= 0);
      if (phys == -1) {
        report_status(p.status, -5);
        for (uint32_t i = 0; i < bytes; i += 16)
          *reinterpret_cast<uint4*>(dst + i) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], __popc(good) * bytes);
      __syncwarp();
      if (phys >= 0)
        bulk_load(dst, pool + (static_cast<size_t>(phys) * p.Hkv + g) * bytes, bytes,
                  &ctl->full[st]);
      if (k + 1 < n) next = entry(k + 1);
    }
    if (lane == 0) {
      for (int k = imax(0, issued - S); k < issued; ++k)
        mbar_wait(&ctl->full[k % S], (k / S) & 1, wc_drain);
    }
    return;  // the producer takes no part in the consumer barriers below
  }

  // ------------------------------------------------------------------ consumers
  const int r = lane >> 2, q = lane & 3;
  // Q as the B operand: column (head) r, k-step kk = channels D/4 q + 4 kk + {0, 1 | 2, 3}.
  uint32_t qb[NT][C::kSteps][2];
  float sc[NT][2];  // scale of heads 8 nt + 2 q, + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint4 w[D / 32];
    const int h = 8 * nt + r;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      w[i] = h < G ? __ldg(p.q + (head0 + h) * (D / 8) + q * (D / 32) + i) : make_uint4(0, 0, 0, 0);
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
  const uint32_t pmask = (1u << lp) - 1;
  bool ok = true;

  for (int k = 0; k < n; ++k) {
    const int st = k % S;
    ok = __all_sync(0xffffffffu, mbar_wait(&ctl->full[st], (k / S) & 1, wc));
    if (ok) {
      const uint8_t* stage = ring + st * C::kStageBytes;
      const int left = L - (st0 + k) * C::kTok;  // tokens of the context from this stage on
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int tb = warp * 32 + half * 16;
        if (tb < left) {  // the same for the whole warp
          const uint8_t* kblk = stage + (tb >> lp) * (C::kRow << lp);
          const int in = tb & pmask;  // the tile's first token in its page
          const uint8_t* kc = kblk + in * C::kCode;
          const uint8_t* ks = kblk + (C::kCode << lp) + in * C::kScale;
          const uint8_t* vc = kc + C::kHalf;
          const uint8_t* vs = ks + C::kHalf;
          const bool edge = tb + 16 > left;
          // ---- S^T = K Q^T
          float s[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
          {
            uint32_t w[2][2 * kWords], sf[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int row = r + 8 * x;
              if constexpr (D == 128) {
                const uint4 u = *reinterpret_cast<const uint4*>(kc + row * C::kCode + 16 * q);
                w[x][0] = u.x, w[x][1] = u.y, w[x][2] = u.z, w[x][3] = u.w;
                sf[x] = e4m3x2_to_f16(
                    *reinterpret_cast<const uint16_t*>(ks + row * C::kScale + 2 * q));
              } else {
                const uint2 u = *reinterpret_cast<const uint2*>(kc + row * C::kCode + 8 * q);
                w[x][0] = u.x, w[x][1] = u.y;
                sf[x] = e4m3x2_to_f16(ks[row * C::kScale + q]);
              }
            }
#pragma unroll
            for (int i = 0; i < 2 * kWords; ++i) {
              uint32_t a[2][4];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t ss = i < 2 ? dup_lo(sf[x]) : dup_hi(sf[x]);
                e2m1x8_to_f16(w[x][i], a[x]);
#pragma unroll
                for (int e = 0; e < 4; ++e) a[x][e] = hmul2(a[x][e], ss);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16_16816(s[nt], a[0][0], a[1][0], a[0][1], a[1][1], qb[nt][2 * i][0],
                              qb[nt][2 * i][1]);
                mma_f16_16816(s[nt], a[0][2], a[1][2], a[0][3], a[1][3], qb[nt][2 * i + 1][0],
                              qb[nt][2 * i + 1][1]);
              }
            }
          }
          // ---- softmax: columns are heads 2q, 2q + 1, rows tokens r and r + 8
          const bool live0 = !edge || tb + r < left, live1 = !edge || tb + r + 8 < left;
          float y[NT][4];
          bool over = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[nt][e] = fmaf(s[nt][e], sc[nt][e & 1], -mref[nt][e & 1]);
              if (!((e & 2) ? live1 : live0)) y[nt][e] = -INFINITY;
              over |= y[nt][e] > 15.f;
            }
          if (__any_sync(0xffffffffu, over)) {
            // Some score passed the reference max by more than 8: move that head's.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float x0 = live0 ? s[nt][c] * sc[nt][c] : -INFINITY;
                float x1 = live1 ? s[nt][c + 2] * sc[nt][c] : -INFINITY;
                float mx = fmaxf(x0, x1);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                if (mx > mref[nt][c] + 15.f) {
                  const float mn = mx - 7.f;
                  const float f = fast_exp2(mref[nt][c] - mn);
                  mref[nt][c] = mn;
                  l[nt][c] *= f;
#pragma unroll
                  for (int i = 0; i < C::kSteps; ++i) o[nt][i][c] *= f, o[nt][i][c + 2] *= f;
                  y[nt][c] = live0 ? fmaf(s[nt][c], sc[nt][c], -mn) : -INFINITY;
                  y[nt][c + 2] = live1 ? fmaf(s[nt][c + 2], sc[nt][c], -mn) : -INFINITY;
                }
              }
          }
          uint32_t pb[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = fast_exp2(y[nt][i]);
            l[nt][0] += e[0] + e[2];
            l[nt][1] += e[1] + e[3];
            // The scores' fragment, transposed, is the B operand of O^T: k = tokens.
            pb[nt][0] = movmatrix_trans(pack_f16x2(e[0], e[1]));
            pb[nt][1] = movmatrix_trans(pack_f16x2(e[2], e[3]));
          }
          // ---- O^T += V^T P^T
          {
            uint32_t w[4][kWords], sv[2];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int tok = 2 * q + (x & 1) + 8 * (x >> 1);
              if constexpr (D == 128) {
                const uint2 u = *reinterpret_cast<const uint2*>(vc + tok * C::kCode + 8 * r);
                w[x][0] = u.x, w[x][1] = u.y;
              } else {
                w[x][0] = *reinterpret_cast<const uint32_t*>(vc + tok * C::kCode + 4 * r);
              }
            }
            constexpr int kPer = D == 128 ? 1 : 2;  // lanes r of one scale block
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int tok = 2 * q + 8 * x;
              const uint8_t* at = vs + tok * C::kScale + r / kPer;
              uint32_t two = at[0] | (static_cast<uint32_t>(at[C::kScale]) << 8);
              if (edge) {
                // Slots past the context may hold anything; a NaN scale would survive p = 0.
                if (tb + tok >= left) two &= 0xFF00u;
                if (tb + tok + 1 >= left) two &= 0x00FFu;
              }
              sv[x] = e4m3x2_to_f16(two);
            }
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
              // Token pairs side by side: byte j holds channel 2j (lo) or 2j + 1 (hi) of both.
              constexpr uint32_t kLow = 0x0F0F0F0Fu;
              uint32_t lo[2][4], hi[2][4];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t w0 = w[2 * x][i], w1 = w[2 * x + 1][i];
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
                  mma_f16_16816(o[nt][4 * i + e], lo[0][e], hi[0][e], lo[1][e], hi[1][e],
                                pb[nt][0], pb[nt][1]);
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->empty[st]);
  }

  // ------------------------------------------------------------------ merge the four warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
  named_barrier_sync(1, C::kConsumers);  // every consumer is past its last ring read
  // [warp][head][D] fp32 in the idle ring. Lane (r, q): heads 2q, 2q + 1, channels D/8 r ..;
  // m-tile i holds channels 2i and 2i + 1 of them.
  float* buf = reinterpret_cast<float*>(ring);
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
        float* to = buf + (warp * C::kHeads + h) * D + r * (D / 8);
#pragma unroll
        for (int i = 0; i < C::kSteps; i += 2)
          *reinterpret_cast<float4*>(to + 2 * i) = make_float4(
              o[nt][i][c], o[nt][i][c + 2], o[nt][i + 1][c], o[nt][i + 1][c + 2]);
      }
    }
  named_barrier_sync(1, C::kConsumers);

  const size_t bg = static_cast<size_t>(b) * p.Hkv + g;
  const bool single = nsplit == 1;
  constexpr int kQuads = D / 4;  // four-column groups of one head's row
  for (int idx = tid; idx < G * kQuads; idx += C::kConsumers) {
    const int hh = idx / kQuads, d0 = (idx % kQuads) * 4;
    float M = red_m[hh];
#pragma unroll
    for (int w = 1; w < C::kWarps; ++w) M = fmaxf(M, red_m[w * 16 + hh]);
    float Ls = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      const float mw = red_m[w * 16 + hh];
      if (mw != -INFINITY) {
        const float f = fast_exp2(mw - M);
        const float4 x = *reinterpret_cast<const float4*>(buf + (w * C::kHeads + hh) * D + d0);
        Ls += red_l[w * 16 + hh] * f;
        a.x += x.x * f, a.y += x.y * f, a.z += x.z * f, a.w += x.w * f;
      }
    }
    const size_t orow = head0 + hh;
    if (single) {
      const float inv = Ls > 0.f ? p.v_scale / Ls : 0.f;
      *reinterpret_cast<uint2*>(p.o + orow * D + d0) =
          make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
      if (d0 == 0)
        p.lse[orow] = Ls > 0.f ? (M + log2f(Ls)) * 0.69314718055994530942f : -INFINITY;
    } else {
      const size_t base = (bg * p.max_splits + split) * G + hh;
      *reinterpret_cast<float4*>(p.part_o + base * D + d0) = a;
      if (d0 == 0) {
        p.part_ml[2 * base] = M;
        p.part_ml[2 * base + 1] = Ls;
      }
    }
  }
  if (single) return;

  // Ticket: the split that draws the last one merges all splits in split order, so the result
  // does not depend on which CTA finishes last.
  named_barrier_sync(1, C::kConsumers);
  if (tid == 0) {
    __threadfence();
    const int ticket = atomicAdd(&p.counters[bg], 1);
    __threadfence();
    ctl->is_last = ticket == nsplit - 1;
  }
  named_barrier_sync(1, C::kConsumers);
  if (!ctl->is_last) return;
  __threadfence();
  constexpr int kBatch = 8;
  const size_t base_bg = bg * p.max_splits * G;
  for (int idx = tid; idx < G * kQuads; idx += C::kConsumers) {
    const int hh = idx / kQuads, d0 = (idx % kQuads) * 4;
    const float* ml = p.part_ml + 2 * (base_bg + hh);
    const float* po = p.part_o + (base_bg + hh) * D + d0;
    // The running max over batches of splits, with the sums rescaled when it grows.
    float M = -INFINITY, Ls = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < nsplit; c0 += kBatch) {
      float2 mlv[kBatch];
      float4 ov[kBatch];
#pragma unroll
      for (int t = 0; t < kBatch; ++t) {
        const size_t c = static_cast<size_t>(imin(c0 + t, nsplit - 1));
        mlv[t] = __ldcg(reinterpret_cast<const float2*>(ml + 2 * c * G));
        ov[t] = __ldcg(reinterpret_cast<const float4*>(po + c * G * D));
      }
      float Mn = M;
#pragma unroll
      for (int t = 0; t < kBatch; ++t) Mn = fmaxf(Mn, mlv[t].x);
      const float f = M == -INFINITY ? 0.f : exp2f(M - Mn);
      M = Mn;
      Ls *= f;
      a.x *= f, a.y *= f, a.z *= f, a.w *= f;
#pragma unroll
      for (int t = 0; t < kBatch; ++t)
        if (c0 + t < nsplit) {
          const float wt = exp2f(mlv[t].x - M);
          Ls += mlv[t].y * wt;
          a.x += ov[t].x * wt, a.y += ov[t].y * wt, a.z += ov[t].z * wt, a.w += ov[t].w * wt;
        }
    }
    const size_t orow = head0 + hh;
    const float inv = p.v_scale / Ls;
    *reinterpret_cast<uint2*>(p.o + orow * D + d0) =
        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    if (d0 == 0) p.lse[orow] = (M + log2f(Ls)) * 0.69314718055994530942f;
  }
}

}  // namespace ta
