// append.cuh — per-head norm and rotation of queries and keys, and the append of new tokens'
// keys and values to a paged cache, in bf16 or in 4 bits. Every (token, head) row of the
// projection is read once and written once where its reader wants it.
//
// Mathematics of one row x of D channels, all in fp32:
//   norm      y_c = x_c * rsqrt(mean_c x_c^2 + eps) * w_c                   (optional)
//   rotation  pairs (i, i + R/2), or (2i, 2i + 1), i < R/2, by the position's angle i:
//             a' = a cos - b sin,  b' = b cos + a sin                       (optional)
//             each product and each sum rounded on its own (no FMA): the 4-bit codes then
//             depend on the inputs alone, not on how a compiler contracts
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
  int tasks_per_token, groups_per_task;
  int* status;
};

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

template <int D, int CACHE>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowParams p) {
  constexpr int R = D / 16;          // lanes per row
  constexpr int kRows = 32 / R;      // rows per warp
  constexpr int kBatch = 4;          // row groups in flight
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int l = lane % R, rr = lane / R;
  const long long task =
      static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);

  // Block 0 looks the lengths over, so that a fault in a sequence without tokens is reported
  // too; each warp checks its own token's sequence before it writes.
  if (CACHE != kCacheNone && blockIdx.x == 0) {
    bool bad = threadIdx.x == 0 && (p.cu[0] != 0 || p.cu[p.B] > p.total);
    for (int b = static_cast<int>(threadIdx.x); b < p.B; b += kRowThreads) {
      const long long n = static_cast<long long>(p.cu[b + 1]) - p.cu[b];
      bad |= n < 0 || p.lens[b] < n ||
             p.lens[b] > (static_cast<long long>(p.max_pages) << p.page_shift);
    }
    if (bad) report_status(p.status, -7);
  }

  const int t = static_cast<int>(task / p.tasks_per_token);
  if (t >= p.total) return;
  const int part = static_cast<int>(task % p.tasks_per_token);

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
      ok = start >= 0 && len >= n && len <= (static_cast<long long>(p.max_pages) << p.page_shift);
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
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (p.rot) {
    const float* row = p.cos_sin + static_cast<size_t>(pos) * p.rot;
    const float* srow = row + p.rot / 2;
    auto four = [](const float* from, float* to) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(from));
      to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
    };
    if (split) {
      if (paired) {
        four(row + 8 * l, cs), four(row + 8 * l + 4, cs + 4);
        four(srow + 8 * l, sn), four(srow + 8 * l + 4, sn + 4);
      }
    } else {
      if (turn_a) four(row + 4 * ca, cs), four(srow + 4 * ca, sn);
      if (turn_b) four(row + 4 * cb, cs + 4), four(srow + 4 * cb, sn + 4);
    }
  }

  const int all = p.groups[0] + p.groups[1] + p.groups[2];
  const int g0 = part * p.groups_per_task;
  const int g1 = imin(g0 + p.groups_per_task, all);
  // (kind, head) of row group g on this lane; head < 0: no row.
  auto row_of = [&](int g, int& kind, int& head) {
    kind = g < p.groups[0] ? 0 : g < p.groups[0] + p.groups[1] ? 1 : 2;
    const int first = kind == 0 ? 0 : kind == 1 ? p.groups[0] : p.groups[0] + p.groups[1];
    head = (g - first) * kRows + rr;
    if (g >= g1 || head >= p.heads[kind]) head = -1;
  };
  for (int gb = g0; gb < g1; gb += kBatch) {
    uint4 va[kBatch], vb[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      int kind, head;
      row_of(gb + i, kind, head);
      va[i] = vb[i] = make_uint4(0, 0, 0, 0);
      if (head >= 0) {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.in[kind] + t * p.stride[kind] + static_cast<size_t>(head) * (2 * D));
        va[i] = __ldg(src + ca);
        vb[i] = __ldg(src + cb);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (gb + i >= g1) break;  // the same for the whole warp
      int kind, head;
      row_of(gb + i, kind, head);
      float a[8], b[8];
      {
        const uint32_t wa[4] = {va[i].x, va[i].y, va[i].z, va[i].w};
        const uint32_t wb[4] = {vb[i].x, vb[i].y, vb[i].z, vb[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[2 * e] = __uint_as_float(wa[e] << 16);
          a[2 * e + 1] = __uint_as_float(wa[e] & 0xFFFF0000u);
          b[2 * e] = __uint_as_float(wb[e] << 16);
          b[2 * e + 1] = __uint_as_float(wb[e] & 0xFFFF0000u);
        }
      }
      const float* w = kind < 2 ? p.weight[kind] : nullptr;
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
#pragma unroll
        for (int off = R / 2; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float rs = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(w + 8 * ca + e));
          const float4 y = __ldg(reinterpret_cast<const float4*>(w + 8 * cb + e));
          a[e] *= rs * x.x, a[e + 1] *= rs * x.y, a[e + 2] *= rs * x.z, a[e + 3] *= rs * x.w;
          b[e] *= rs * y.x, b[e + 1] *= rs * y.y, b[e + 2] *= rs * y.z, b[e + 3] *= rs * y.w;
        }
      }
      if (kind < 2 && p.rot) {
        if (split) {
          if (paired) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = a[e], y = b[e];
              a[e] = __fsub_rn(__fmul_rn(x, cs[e]), __fmul_rn(y, sn[e]));
              b[e] = __fadd_rn(__fmul_rn(y, cs[e]), __fmul_rn(x, sn[e]));
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (turn_a) {
              const float x = a[2 * e], y = a[2 * e + 1];
              a[2 * e] = __fsub_rn(__fmul_rn(x, cs[e]), __fmul_rn(y, sn[e]));
              a[2 * e + 1] = __fadd_rn(__fmul_rn(y, cs[e]), __fmul_rn(x, sn[e]));
            }
            if (turn_b) {
              const float x = b[2 * e], y = b[2 * e + 1];
              b[2 * e] = __fsub_rn(__fmul_rn(x, cs[4 + e]), __fmul_rn(y, sn[4 + e]));
              b[2 * e + 1] = __fadd_rn(__fmul_rn(y, cs[4 + e]), __fmul_rn(x, sn[4 + e]));
            }
          }
        }
      }
      if (CACHE == kCacheFp4 && kind >= 1) {
        // 16-channel blocks: this lane's chunk a with the partner lane's (chunk a ^ 1), and b
        // with its; past the rotated channels of a half-split, a with b.
        const float inv = p.inv_scale[kind - 1];
        float ma = 0.f, mb = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] *= inv, b[e] *= inv;
          ma = fmaxf(ma, fabsf(a[e]));
          mb = fmaxf(mb, fabsf(b[e]));
        }
        const float oa = __shfl_xor_sync(0xffffffffu, ma, 1);
        const float ob = __shfl_xor_sync(0xffffffffu, mb, 1);
        if (paired) {
          ma = fmaxf(ma, oa), mb = fmaxf(mb, ob);
        } else {
          ma = mb = fmaxf(ma, mb);
        }
        const uint32_t sa = f32_to_e4m3(__fdiv_rn(ma, 6.f)), sb = f32_to_e4m3(__fdiv_rn(mb, 6.f));
        const float fa = e4m3_to_f32(sa), fb = e4m3_to_f32(sb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] = fa > 0.f ? __fdiv_rn(a[e], fa) : 0.f;
          b[e] = fb > 0.f ? __fdiv_rn(b[e], fb) : 0.f;
        }
        if (phys >= 0 && head >= 0) {
          const int P = 1 << p.page_shift, slot = pos & (P - 1);
          uint8_t* blk = p.pool[kind - 1] +
                         (static_cast<size_t>(phys) * p.heads[1] + head) *
                             static_cast<size_t>(P * fp4_row_bytes(D));
          uint32_t* codes = reinterpret_cast<uint32_t*>(blk + slot * fp4_code_bytes(D));
          uint8_t* scales = blk + P * fp4_code_bytes(D) + slot * fp4_scale_bytes(D);
          codes[ca] = f32x8_to_e2m1(a);
          codes[cb] = f32x8_to_e2m1(b);
          if (!(ca & 1)) scales[ca >> 1] = static_cast<uint8_t>(sa);
          if (!(cb & 1)) scales[cb >> 1] = static_cast<uint8_t>(sb);
        }
      } else if (head >= 0) {
        uint4* dst = nullptr;
        if (CACHE == kCacheBf16 && kind >= 1) {
          const int slot = pos & ((1 << p.page_shift) - 1);
          if (phys >= 0)
            dst = reinterpret_cast<uint4*>(
                p.pool[kind - 1] +
                (((static_cast<size_t>(phys) * p.heads[1] + head) << p.page_shift) + slot) *
                    (2 * D));
        } else {
          const int blk = t / p.N, row = t % p.N;
          dst = reinterpret_cast<uint4*>(
              p.out[kind] +
              ((static_cast<size_t>(blk) * p.heads[kind] + head) * p.N + row) * (2 * D));
        }
        if (dst) {
          dst[ca] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                               pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
          dst[cb] = make_uint4(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]),
                               pack_bf16x2(b[4], b[5]), pack_bf16x2(b[6], b[7]));
        }
      }
    }
  }
}

// 4-bit pages -> bf16 pages: page p of sequence b, as the table lists it, goes to dst page
// b * max_pages + p. One CTA per page; a thread turns 4 bytes of codes into 16 bytes. Slots
// past the sequence's length get zeros (a reader multiplies them by zero, so they have to be
// finite), pages past it are left alone.
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
  const int len = p.lens[b];
  if (len < 0 || len > (static_cast<long long>(p.max_pages) << p.page_shift)) {
    if (pg == 0 && threadIdx.x == 0) report_status(p.status, -7);
    return;
  }
  const int here = imin(len - (pg << p.page_shift), P);  // valid tokens of this page
  if (here <= 0) return;
  const int phys = p.table[static_cast<size_t>(b) * p.max_pages + pg];
  if (phys < 0 || phys >= p.num_pages) {
    if (threadIdx.x == 0) report_status(p.status, -5);
    return;
  }
  constexpr int kChunks = D / 8;  // 8-channel chunks of a row
  const size_t blk = static_cast<size_t>(P * fp4_row_bytes(D));
  const uint8_t* src = p.pool + static_cast<size_t>(phys) * p.Hkv * blk;
  uint4* dst = p.dst + (static_cast<size_t>(b) * p.max_pages + pg) * p.Hkv *
                           (static_cast<size_t>(P) * kChunks);
  const int n = p.Hkv * P * kChunks;
  for (int i = static_cast<int>(threadIdx.x); i < n; i += blockDim.x) {
    const int c = i % kChunks, row = i / kChunks, tok = row & (P - 1), h = row >> p.page_shift;
    uint4 out = make_uint4(0, 0, 0, 0);
    if (tok < here) {
      const uint8_t* q = src + h * blk;
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q) + tok * kChunks + c);
      const float s = e4m3_to_f32(__ldg(q + P * fp4_code_bytes(D) + tok * (kChunks / 2) + c / 2));
      uint32_t v[4], o[4];
      e2m1x8_to_f16(w, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[e]));
        o[e] = pack_bf16x2(f.x * s * p.scale, f.y * s * p.scale);
      }
      out = make_uint4(o[0], o[1], o[2], o[3]);
    }
    dst[i] = out;
  }
}

}  // namespace ta
