// share.cuh — how the split decodes share a batch's contexts out over their workers.
#pragma once

#include "ptx.cuh"
#include "sched.h"

namespace ta {

// P: a kernel's parameters, with cu ([B + 1] cumulative context lengths), B, Hkv, max_len, slots
// (CTAs of the decode kernel) and status.

// Context length of sequence b; 0 (and a report, if asked) where cu_seqlens is malformed.
template <class P>
__device__ __forceinline__ int context_length(const P& p, int b, bool report) {
  const int L = __ldg(p.cu + b + 1) - __ldg(p.cu + b);
  if (L >= 0 && L <= p.max_len) return L;
  if (report) report_status(p.status, -7);
  return 0;
}

// The block-table entries of a TMA producer's boxes of `run` tokens (a page, or part of one) from
// token `first` of a context on. A lane holds one entry of 32 boxes, and the next 32 are asked for
// when these come into use: an entry read a tile ahead is waited for on the spot, since it is
// checked there, which held a warp up for an L2 latency a tile (decode of 32 sequences of up to 8K,
// 16 kv heads, d = 64, 16-token pages 88.7 to 83.6 us; chunks of 2K tokens over 16K contexts 2583 to
// 2488).
struct PageEntries {
  const int* row;  // of the block table
  int first, run, page_shift, length;
  int now, next;
  __device__ __forceinline__ PageEntries(const int* row_, int first_, int run_, int page_shift_,
                                         int length_)
      : row(row_), first(first_), run(run_), page_shift(page_shift_), length(length_), now(0) {
    next = load(0);
  }
  __device__ __forceinline__ int load(int box) const {
    const int tok = first + (box + static_cast<int>(lane_id())) * run;
    return tok < length ? __ldg(row + (tok >> page_shift)) : -1;
  }
  // Entry of box `box` + i (-1 past the context), i below the boxes a tile has, a power of two.
  // Warp-collective, for multiples of those in order from 0 on.
  __device__ __forceinline__ int at(int box, int i) {
    if ((box & 31) == 0) {
      now = next;
      next = load(box + 32);
    }
    return __shfl_sync(0xffffffffu, now, (box + i) & 31);
  }
};

// Contexts are cut into blocks of TOK tokens, numbered over sequence, kv head and position. Every
// warp of a decode kernel and of the kernel that joins its parts works the shares out by itself,
// from cu_seqlens alone: a context counts its blocks and START units before them for what beginning
// it costs, and worker i of n takes an even share of the units, the first r workers q + 1, the
// others q. A share that ends among a context's START units holds none of it. PER_SLOT: workers of
// a CTA. PARTS: parts of a context that join well.
template <class P, int TOK, int START, int PARTS, int PER_SLOT>
struct Share {
  static constexpr int kTok = TOK;      // tokens of a block
  static constexpr int kStart = START;  // units that beginning a context costs
  int total;    // units of one kv head, all sequences
  int before;   // those of the sequences before `upto`
  int n, q, r;
  int w0;       // units of sequence `lane`

  __device__ __forceinline__ static int blocks(int L) { return (L + kTok - 1) / kTok; }
  __device__ __forceinline__ static int units(int nb) { return nb > 0 ? nb + kStart : 0; }

  __device__ __forceinline__ Share(const P& p, int upto, bool report) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    w0 = lane < p.B ? units(blocks(context_length(p, lane, report))) : 0;
    int all = w0, ahead = lane < upto ? w0 : 0;
    for (int b0 = lane + 32; b0 < p.B; b0 += 128) {
#pragma unroll
      for (int b = b0; b < b0 + 128; b += 32) {  // four loads at a time
        const int w = b < p.B ? units(blocks(context_length(p, b, report))) : 0;
        all += w;
        if (b < upto) ahead += w;
      }
    }
    total = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, ahead);
    const int U = total * p.Hkv;
    // As many workers as the GPU holds, but over PARTS a context only at four units or more each.
    // Contexts are counted by the lanes that have any, up to 32 x kv heads (enough for every
    // worker), and a padded batch's empty ones are none.
    const int live = __popc(__ballot_sync(0xffffffffu, all > 0)) * p.Hkv;
    n = imin(PER_SLOT * p.slots, imin(U, imax(live * PARTS, U / 4)));
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
  __device__ __forceinline__ void find(const P& p, int u, int& seq,
                                       int& ahead) const {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    int run = 0;
    for (int b0 = 0; b0 < p.B;) {
      const int b = b0 + lane;
      const int w = b0 == 0 ? w0 : b < p.B ? units(blocks(context_length(p, b, false))) : 0;
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
          four += units(c < p.B ? blocks(context_length(p, c, false)) : 0);
        four = run + __reduce_add_sync(0xffffffffu, four);
        if (u < four * p.Hkv) break;
        run = four;
      }
    }
    seq = p.B - 1;  // not reached: u lies below the total
    ahead = run;
  }
};

}  // namespace ta
