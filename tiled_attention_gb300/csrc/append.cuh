// append.cuh — per-head norm and rotation of queries and keys, and the append of new tokens'
// keys and values to a paged cache, in bf16 or in 4 bits. Every (token, head) row of the
// projection is read once and written once where its reader wants it.
//
// Mathematics of one row x of D channels, all in fp32:
//   norm      y_c = x_c * rsqrt(mean_c x_c^2 + eps) * w_c                   (optional)
//   rotation  pairs (i, i + R/2), or (2i, 2i + 1), i < R/2, by the position's angle i:
//             a' = a cos - b sin,  b' = b cos + a sin                       (optional)
//             for keys that go to 4 bits each product and sum is rounded on its own (no FMA):
//             the codes then depend on the inputs alone, not on how a compiler contracts
//   bf16 out  round to nearest even, once
//   4-bit out xs = y * RN(1 / tensor scale); s = E4M3(max over 16 channels |xs| / 6);
//             code = E2M1(xs / s), the division rounded as IEEE does; 0 where s is 0
//
// A row is D/16 lanes wide (8 at D = 128), 16 channels a lane in two 16-byte chunks: the two
// halves of a half-split rotation meet in one lane, and the row's sums are shuffles. A warp
// takes rows of one token, so the position, its cosines and the page are found once for them.
// The kernel only moves bytes: each lane issues the loads of up to kBatch row groups before
// it uses any.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "fp4.cuh"
#include "ptx.cuh"
#include "sched.h"

namespace ta {

enum CacheKind { kCacheNone = 0, kCacheBf16 = 1, kCacheFp4 = 2 };

struct RowParams {
  const uint8_t* in[3];      // q, k, v: bf16 rows
  long long stride[3];       // bytes from token to token
  uint8_t* out[2];           // q, k in head-major layout [total / N, H, N, D] (k: no cache)
  uint8_t* pool[2];          // K, V page pools
  const float* weight[2];    // norm weights [D] of q and k, or null
  const float* cos_sin;      // [max_pos, rot]: rot/2 cosines, rot/2 sines
  const int* positions;      // no cache: position of every token, or null for t % N
  const int* cu;             // cache: [B + 1] starts of the sequences' new tokens
  const int* lens;           // cache: [B] context lengths, new tokens included
  const int* table;          // cache: [B, max_pages]
  float inv_scale[2];        // 4-bit pools: RN(1 / tensor scale) of K and V
  float eps;
  int heads[3];              // rows of a token: Hq, Hkv, Hkv (0: absent)
  int groups[3];             // row groups of a token: heads over rows per warp, rounded up
  int total, N, B, max_pos, rot, interleaved, max_pages, page_shift, num_pages;
  int groups_per_task;       // row groups a warp takes of its token; the grid's y picks which
  int* status;
};

// Two CTAs of eight warps an SM and four row groups in flight a warp, measured on 16384 tokens of
// 32 + 8 heads (norm and rotation) and on 17754 tokens of 32 + 8 + 8 appended to 16-token
// pages: 60.0 and 80.6 us; three CTAs with two groups 58.4 and 74.5, but spilling; 128 threads,
// five CTAs, four groups 57.5 and 76.7, spilling; three CTAs of 128 with six groups 67 and 94.
// With the rows prefetched (below) the first takes 55.5 and 75.0.
constexpr int kRowThreads = 256;

// Sequence of token t: b with cu[b] <= t < cu[b + 1], by the whole warp; -1 where t lies
// behind the last sequence, -2 where cu gives no such b. Single tokens of every sequence
// (cu[t] = t) are found at once; else each step narrows the range 32-fold.
__device__ __forceinline__ int find_sequence(const int* __restrict__ cu, int B, int t, int lane) {
  if (t >= __ldg(cu + B)) return -1;
  if (t < B && __ldg(cu + t) == t && __ldg(cu + t + 1) == t + 1) return t;
  int lo = 0, n = B;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, lane * step < n && __ldg(cu + i) <= t);
    if (!(le & 1u)) return -2;
    const int j = 31 - __clz(le);
    const int lo2 = lo + j * step;
    n = imin(step, lo + n - lo2);
    lo = lo2;
  }
  return __ldg(cu + lo) <= t && t < __ldg(cu + lo + 1) ? lo : -2;
}

// x / s as IEEE division rounds it, for every element of four pairs and one s >= 2^-9 with
// rc = RN(1/s): q = RN(x rc) is within an ulp, its remainder is exact in one FMA, and one more
// FMA rounds correctly (Markstein's correction, as in the FP8 quantizer). A zero quotient keeps
// the sign of x.
__device__ __forceinline__ void divide8(float2 (&x)[4], float s, float rc) {
  const float2 rc2 = make_float2(rc, rc), ns2 = make_float2(-s, -s);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 q0 = __fmul2_rn(x[e], rc2);
    const float2 q1 = __ffma2_rn(__ffma2_rn(q0, ns2, x[e]), rc2, q0);
    x[e] = make_float2(copysignf(q1.x, x[e].x), copysignf(q1.y, x[e].y));
  }
}

__device__ __forceinline__ float2 clamp2(float2 x, float m) {
  return make_float2(fminf(fmaxf(x.x, -m), m), fminf(fmaxf(x.y, -m), m));
}

template <int D, int CACHE>
__global__ void __launch_bounds__(kRowThreads, 2) rows_kernel(const RowParams p) {
  constexpr int R = D / 16;          // lanes per row
  constexpr int kRows = 32 / R;      // rows per warp
  constexpr int kBatch = 4;             // row groups in flight
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int l = lane % R, rr = lane / R;

  // Block (0, 0) looks the lengths over, so that a fault in a sequence without tokens is
  // reported too; each warp checks its own token's sequence before it writes.
  if (CACHE != kCacheNone && blockIdx.x == 0 && blockIdx.y == 0) {
    bool bad = threadIdx.x == 0 && (p.cu[0] != 0 || p.cu[p.B] > p.total);
    for (int b = static_cast<int>(threadIdx.x); b < p.B; b += kRowThreads) {
      const long long n = static_cast<long long>(p.cu[b + 1]) - p.cu[b];
      bad |= n < 0 || p.lens[b] < n ||
             p.lens[b] > (static_cast<long long>(p.max_pages) << p.page_shift);
    }
    if (bad) report_status(p.status, -7);
  }

  const long long tl =
      static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (tl >= p.total) return;
  const int t = static_cast<int>(tl);

  // A warp that takes all rows of its token asks for them now, lane by kind, so that they come
  // into L2 while it looks up the position, its page and its angles (four dependent loads).
  // Split tokens do not: one step of 32 sequences takes 3.3 us without, 3.6 with.
  if (gridDim.y == 1 && lane < (CACHE == kCacheNone ? 2 : 3) && p.heads[lane] > 0)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.in[lane] +
                                                                   t * p.stride[lane]),
                 "r"(p.heads[lane] * 2 * D));

  int pos, phys = -1;
  if constexpr (CACHE == kCacheNone) {
    pos = p.positions ? __ldg(p.positions + t) : t % p.N;
  } else {
    const int b = find_sequence(p.cu, p.B, t, lane);
    if (b == -1) return;  // rows behind the last sequence
    int start = 0, n = 0, len = 0;
    bool ok = b >= 0;
    if (ok) {
      start = __ldg(p.cu + b);
      n = __ldg(p.cu + b + 1) - start;
      len = __ldg(p.lens + b);
      ok = start >= 0 && n <= p.total - start && len >= n &&
           len <= (static_cast<long long>(p.max_pages) << p.page_shift);
    }
    if (!ok) {
      if (lane == 0) report_status(p.status, -7);
      return;
    }
    pos = len - n + (t - start);
    phys = __ldg(p.table + static_cast<size_t>(b) * p.max_pages + (pos >> p.page_shift));
    if (phys < 0 || phys >= p.num_pages) {
      if (lane == 0) report_status(p.status, -5);
      phys = -1;
    }
  }
  if (p.rot && (pos < 0 || pos >= p.max_pos)) {
    if (lane == 0) report_status(p.status, -5);
    return;
  }

  // This lane's chunks (8 channels each) and angles. Half-split: lane l < hl holds chunk l and
  // its partner l + hl; the lanes past the rotated channels hold two neighbours. Otherwise
  // chunks l and l + R.
  const bool split = p.rot && !p.interleaved;
  const int hl = split ? p.rot / 16 : R;
  const bool paired = l < hl;
  const int ca = paired ? l : 2 * hl + 2 * (l - hl);
  const int cb = paired ? l + hl : ca + 1;
  const bool turn_a = p.rot && 8 * ca < p.rot, turn_b = p.rot && 8 * cb < p.rot;
  // Angles: half-split, of the eight pairs (a, b); interleaved, of the four pairs of a, then of
  // b. Channels that do not turn get no angle and are left alone below.
  float2 cs[4], sn[4], ns[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = make_float2(1.f, 1.f), sn[i] = make_float2(0.f, 0.f);
  if (p.rot) {
    const float* row = p.cos_sin + static_cast<size_t>(pos) * p.rot;
    const float* srow = row + p.rot / 2;
    auto four = [](const float* from, float2* to) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(from));
      to[0] = make_float2(v.x, v.y), to[1] = make_float2(v.z, v.w);
    };
    if (split) {
      if (paired) {
        four(row + 8 * l, cs), four(row + 8 * l + 4, cs + 2);
        four(srow + 8 * l, sn), four(srow + 8 * l + 4, sn + 2);
      }
    } else {
      if (turn_a) four(row + 4 * ca, cs), four(srow + 4 * ca, sn);
      if (turn_b) four(row + 4 * cb, cs + 2), four(srow + 4 * cb, sn + 2);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) ns[i] = make_float2(-sn[i].x, -sn[i].y);

  // Rows of one kind (0 q, 1 k, 2 v): groups [g0, g1) of kRows heads.
  auto rows = [&](auto kind_c, int g0, int g1) {
    constexpr int kind = decltype(kind_c)::value;
    const int heads = p.heads[kind];
    const uint8_t* src = p.in[kind] + t * p.stride[kind];
    const float* w = kind < 2 ? p.weight[kind] : nullptr;
    float2 wa[4], wb[4];
    if (kind < 2 && w) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(w + 8 * ca) + e);
        const float4 y = __ldg(reinterpret_cast<const float4*>(w + 8 * cb) + e);
        wa[2 * e] = make_float2(x.x, x.y), wa[2 * e + 1] = make_float2(x.z, x.w);
        wb[2 * e] = make_float2(y.x, y.y), wb[2 * e + 1] = make_float2(y.z, y.w);
      }
    }
    uint8_t* dst = nullptr;   // of head 0; null: this token has no page
    size_t dst_step = 0;      // from head to head
    const int slot = pos & ((1 << p.page_shift) - 1);
    if (CACHE == kCacheNone || kind == 0) {
      const unsigned blk = static_cast<unsigned>(t) / static_cast<unsigned>(p.N);
      const unsigned row = static_cast<unsigned>(t) - blk * static_cast<unsigned>(p.N);
      dst_step = static_cast<size_t>(p.N) * (2 * D);
      dst = p.out[kind == 0 ? 0 : 1] + static_cast<size_t>(blk) * heads * dst_step +
            static_cast<size_t>(row) * (2 * D);
    } else if (phys >= 0) {
      const size_t tok = CACHE == kCacheFp4 ? fp4_row_bytes(D) : 2 * D;
      dst_step = tok << p.page_shift;
      dst = p.pool[kind - 1] + static_cast<size_t>(phys) * heads * dst_step;
      if (CACHE == kCacheBf16) dst += static_cast<size_t>(slot) * (2 * D);
    }
    for (int gb = g0; gb < g1; gb += kBatch) {
      uint4 va[kBatch], vb[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int head = (gb + i) * kRows + rr;
        va[i] = vb[i] = make_uint4(0, 0, 0, 0);
        if (gb + i < g1 && head < heads) {
          const uint4* from =
              reinterpret_cast<const uint4*>(src + static_cast<size_t>(head) * (2 * D));
          va[i] = __ldg(from + ca);
          vb[i] = __ldg(from + cb);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (gb + i >= g1) break;  // the same for the whole warp
        const int head = (gb + i) * kRows + rr;
        const bool live = head < heads && dst != nullptr;
        uint8_t* to = dst + static_cast<size_t>(head) * dst_step;
        if constexpr (kind == 2 && CACHE == kCacheBf16) {
          if (live) {
            reinterpret_cast<uint4*>(to)[ca] = va[i];
            reinterpret_cast<uint4*>(to)[cb] = vb[i];
          }
          continue;
        }
        float2 a[4], b[4];
        {
          const uint32_t xa[4] = {va[i].x, va[i].y, va[i].z, va[i].w};
          const uint32_t xb[4] = {vb[i].x, vb[i].y, vb[i].z, vb[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = make_float2(__uint_as_float(xa[e] << 16), __uint_as_float(xa[e] & 0xFFFF0000u));
            b[e] = make_float2(__uint_as_float(xb[e] << 16), __uint_as_float(xb[e] & 0xFFFF0000u));
          }
        }
        if (kind < 2 && w) {
          float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s2 = __ffma2_rn(a[e], a[e], s2);
            s2 = __ffma2_rn(b[e], b[e], s2);
          }
          float ss = s2.x + s2.y;
#pragma unroll
          for (int off = R / 2; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          const float rs = rsqrtf(ss * (1.f / D) + p.eps);
          const float2 rs2 = make_float2(rs, rs);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = __fmul2_rn(__fmul2_rn(a[e], rs2), wa[e]);
            b[e] = __fmul2_rn(__fmul2_rn(b[e], rs2), wb[e]);
          }
        }
        if (kind < 2 && p.rot) {
          if (split) {
            if (paired) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 x = a[e], y = b[e];
                if constexpr (CACHE == kCacheFp4 && kind == 1) {
                  // Scalar: packed products and sums get contracted, whatever their rounding.
                  a[e] = make_float2(__fsub_rn(__fmul_rn(x.x, cs[e].x), __fmul_rn(y.x, sn[e].x)),
                                     __fsub_rn(__fmul_rn(x.y, cs[e].y), __fmul_rn(y.y, sn[e].y)));
                  b[e] = make_float2(__fadd_rn(__fmul_rn(y.x, cs[e].x), __fmul_rn(x.x, sn[e].x)),
                                     __fadd_rn(__fmul_rn(y.y, cs[e].y), __fmul_rn(x.y, sn[e].y)));
                } else {
                  a[e] = __ffma2_rn(x, cs[e], __fmul2_rn(y, ns[e]));
                  b[e] = __ffma2_rn(y, cs[e], __fmul2_rn(x, sn[e]));
                }
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              auto turn = [](float2& v, float c, float s) {
                v = make_float2(__fsub_rn(__fmul_rn(v.x, c), __fmul_rn(v.y, s)),
                                __fadd_rn(__fmul_rn(v.y, c), __fmul_rn(v.x, s)));
              };
              const int h = e >> 1;
              if (turn_a) turn(a[e], e & 1 ? cs[h].y : cs[h].x, e & 1 ? sn[h].y : sn[h].x);
              if (turn_b)
                turn(b[e], e & 1 ? cs[2 + h].y : cs[2 + h].x, e & 1 ? sn[2 + h].y : sn[2 + h].x);
            }
          }
        }
        if constexpr (CACHE == kCacheFp4 && kind >= 1) {
          // 16-channel blocks: this lane's chunk a with the partner lane's (chunk a ^ 1), and
          // b with its; past the rotated channels of a half-split, a with b.
          const float2 inv = make_float2(p.inv_scale[kind - 1], p.inv_scale[kind - 1]);
          float ma = 0.f, mb = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = __fmul2_rn(a[e], inv);
            b[e] = __fmul2_rn(b[e], inv);
            ma = fmax_nan(ma, fmax_nan(fabsf(a[e].x), fabsf(a[e].y)));
            mb = fmax_nan(mb, fmax_nan(fabsf(b[e].x), fabsf(b[e].y)));
          }
          const float oa = __shfl_xor_sync(0xffffffffu, ma, 1);
          const float ob = __shfl_xor_sync(0xffffffffu, mb, 1);
          if (paired) {
            ma = fmax_nan(ma, oa), mb = fmax_nan(mb, ob);
          } else {
            ma = mb = fmax_nan(ma, mb);
          }
          // From kFp4Large on scale and codes saturate (448 * 6 < kFp4Large); infinities would
          // not go through the divisions below. A NaN stays, gives its block the scale NaN and,
          // as that is not > 0, zero codes.
          if (ma >= kFp4Large) {
            ma = kFp4Large;
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = clamp2(a[e], kFp4Large);
          }
          if (mb >= kFp4Large) {
            mb = kFp4Large;
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = clamp2(b[e], kFp4Large);
          }
          // max / 6, correctly rounded as in divide8, then to E4M3.
          constexpr float kSixth = 1.f / 6.f;
          const float qa = ma * kSixth, qm = mb * kSixth;
          const float da = fmaf(fmaf(qa, -6.f, ma), kSixth, qa);
          const float db = fmaf(fmaf(qm, -6.f, mb), kSixth, qm);
          const uint32_t sf = f32x2_to_e4m3(da, db);
          const uint32_t sh = e4m3x2_to_f16(sf);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&sh));
          // A zero scale: zeros, not quotients.
          divide8(a, f.x, f.x > 0.f ? __frcp_rn(f.x) : 0.f);
          divide8(b, f.y, f.y > 0.f ? __frcp_rn(f.y) : 0.f);
          if (live) {
            uint32_t* codes = reinterpret_cast<uint32_t*>(to + slot * fp4_code_bytes(D));
            uint8_t* scales = to + (fp4_code_bytes(D) << p.page_shift) + slot * fp4_scale_bytes(D);
            codes[ca] = f.x > 0.f ? f32x8_to_e2m1(a) : 0u;
            codes[cb] = f.y > 0.f ? f32x8_to_e2m1(b) : 0u;
            if (!(ca & 1)) scales[ca >> 1] = static_cast<uint8_t>(sf);
            if (!(cb & 1)) scales[cb >> 1] = static_cast<uint8_t>(sf >> 8);
          }
        } else if (live) {
          reinterpret_cast<uint4*>(to)[ca] =
              make_uint4(pack_bf16x2(a[0].x, a[0].y), pack_bf16x2(a[1].x, a[1].y),
                         pack_bf16x2(a[2].x, a[2].y), pack_bf16x2(a[3].x, a[3].y));
          reinterpret_cast<uint4*>(to)[cb] =
              make_uint4(pack_bf16x2(b[0].x, b[0].y), pack_bf16x2(b[1].x, b[1].y),
                         pack_bf16x2(b[2].x, b[2].y), pack_bf16x2(b[3].x, b[3].y));
        }
      }
    }
  };
  // This warp's share of the token's row groups: [g0, g1) of q's, then k's, then v's.
  const int g0 = static_cast<int>(blockIdx.y) * p.groups_per_task;
  const int g1 = g0 + p.groups_per_task;
  const int nq = p.groups[0], nk = p.groups[1], nv = p.groups[2];
  if (g0 < nq) rows(std::integral_constant<int, 0>{}, g0, imin(g1, nq));
  if (g1 > nq && g0 < nq + nk)
    rows(std::integral_constant<int, 1>{}, imax(g0 - nq, 0), imin(g1 - nq, nk));
  if (CACHE != kCacheNone && g1 > nq + nk && g0 < nq + nk + nv)
    rows(std::integral_constant<int, 2>{}, imax(g0 - nq - nk, 0), imin(g1 - nq - nk, nv));
}

// 4-bit pages -> bf16 pages: page p of sequence b, as the table lists it, goes to dst page
// b * max_pages + p. A thread turns 4 bytes of codes into 16 bytes and has kUnpackBatch such
// loads in flight; a CTA takes 256 * kUnpackBatch of a page, so that a few pages of many heads
// still fill the GPU. Slots past the sequence's length get zeros (a reader multiplies them by
// zero, so they have to be finite), pages past it are left alone.
constexpr int kUnpackBatch = 8;

struct UnpackParams {
  const uint8_t* pool;
  uint4* dst;
  const int* table;
  const int* lens;
  float scale;
  int max_pages, Hkv, page_shift, num_pages;
  int* status;
};

template <int D>
__global__ void __launch_bounds__(256) unpack_fp4_kernel(const UnpackParams p) {
  const int pg = static_cast<int>(blockIdx.x), b = static_cast<int>(blockIdx.y);
  const int P = 1 << p.page_shift;
  const int len = __ldg(p.lens + b);
  const int phys = __ldg(p.table + static_cast<size_t>(b) * p.max_pages + pg);
  if (len < 0 || len > (static_cast<long long>(p.max_pages) << p.page_shift)) {
    if (pg == 0 && blockIdx.z == 0 && threadIdx.x == 0) report_status(p.status, -7);
    return;
  }
  const int here = imin(len - (pg << p.page_shift), P);  // valid tokens of this page
  if (here <= 0) return;
  if (phys < 0 || phys >= p.num_pages) {
    if (blockIdx.z == 0 && threadIdx.x == 0) report_status(p.status, -5);
    return;
  }
  constexpr int kChunks = D / 8;             // 8-channel chunks of a row
  constexpr int kRowsPer = 256 / kChunks;    // rows the CTA's threads cover at once
  const int c = static_cast<int>(threadIdx.x) % kChunks;
  const int row0 = static_cast<int>(blockIdx.z) * (kRowsPer * kUnpackBatch) +
                   static_cast<int>(threadIdx.x) / kChunks;
  const int rows = p.Hkv << p.page_shift;    // (head, token) rows of the page
  const size_t blk = static_cast<size_t>(P * fp4_row_bytes(D));
  const uint8_t* src = p.pool + static_cast<size_t>(phys) * p.Hkv * blk;
  uint4* dst = p.dst + (static_cast<size_t>(b) * p.max_pages + pg) * rows * kChunks + c;
  uint32_t w[kUnpackBatch];
  uint8_t sf[kUnpackBatch];
#pragma unroll
  for (int i = 0; i < kUnpackBatch; ++i) {
    const int row = row0 + i * kRowsPer, tok = row & (P - 1);
    w[i] = 0, sf[i] = 0;
    if (row < rows && tok < here) {
      const uint8_t* q = src + static_cast<size_t>(row >> p.page_shift) * blk;
      w[i] = __ldg(reinterpret_cast<const uint32_t*>(q) + tok * kChunks + c);
      sf[i] = __ldg(q + (fp4_code_bytes(D) << p.page_shift) + tok * (kChunks / 2) + c / 2);
    }
  }
  const float2 scale = make_float2(p.scale, p.scale);
#pragma unroll
  for (int i = 0; i < kUnpackBatch; ++i) {
    const int row = row0 + i * kRowsPer;
    if (row >= rows) break;
    uint32_t v[4], o[4];
    e2m1x8_to_f16(w[i], v);
    const __half2 s = __half2half2(__ushort_as_half(e4m3x2_to_f16(sf[i]) & 0xFFFFu));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // code * scale is exact in f16; one product in fp32, one rounding to bf16.
      const float2 f =
          __fmul2_rn(__half22float2(__hmul2(*reinterpret_cast<const __half2*>(&v[e]), s)), scale);
      o[e] = pack_bf16x2(f.x, f.y);
    }
    dst[static_cast<size_t>(row) * kChunks] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace ta
