// diff.cu — differential attention's prefill instantiations (head dim 64 / 128; dense, document and
// paged) and their entry points.
#include "diff.cuh"

#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "api.h"
#include "diff.h"
#include "launch.h"

namespace ta {
namespace {

// Q by tiles of 128 rows and by boxes of 8 (where heads may share a tile), K and V, and O by boxes of
// 32 rows of half a head.
struct DiffMaps {
  CUtensorMap q, q8, k, v, o;
};

template <int D, int PACK, int CTAS>
cudaError_t launch_one(const DiffMaps& t, const DiffParams& p, int grid, cudaStream_t stream) {
  static unsigned long long done = 0;
  auto kern = diff_prefill_kernel<D, PACK, CTAS>;
  using C = DiffCfg<D, PACK, CTAS>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::kThreads, C::kSmemBytes, stream>>>(t.q, t.q8, t.k, t.v, t.o, p);
  return cudaGetLastError();
}

template <int D, int CTAS>
cudaError_t launch(int mask, const DiffMaps& t, const DiffParams& p, int grid,
                   cudaStream_t stream) {
  if (mask == kMaskPagedPrefill)
    return launch_one<D, kMaskPagedPrefill, CTAS>(t, p, grid, stream);
  if (is_packed(mask)) return launch_one<D, kMaskDocument, CTAS>(t, p, grid, stream);
  return launch_one<D, kMaskNone, CTAS>(t, p, grid, stream);
}

// At d = 64 two CTAs fit an SM, each with one S buffer a map. With at most four units an SM one CTA
// with two buffers and longer key tiles ends a unit sooner. One CTA and two, 16 heads: one causal row
// of 1024 14.1 and 18.4 us (0.8 units an SM), two of 1500 29.7 and 34.5 (2.5), two of 2000 43.5 and
// 49.4 (3.4; without a mask 75.3 and 71.6), two of 3000 81.5 and 77.5 (5.1), three of 5003 in a
// window of 1000 150 and 131 (12.6), two of 8192 468 and 428. Documents count the blocks that are
// launched, those without work too (packed_blocks), chunks the tiles that may have rows
// (packed_tiles). 16 heads, documents: 16 of 100 18.0 and 15.8 us (704 blocks, at most 448 tiles), 8 of
// 300 21.9 and 21.0 (544, 416), 4 of 700 24.5 and 25.2 (448, 400). Chunks: 20 of 100 tokens over 2000
// 70.6 and 78.9 (864, 560), 10 of 16 with 32 heads over 8 48.9 and 62.3 (640, 352), 5 of 40 over 3000
// with 64 heads over 4 67 and 100 (640, 384), 12 of 100 with 32 heads 84.7 and 78.7 (1024, 672), 8 of up
// to 1024 over 16K with 64 heads 1030 and 863. Tiles are counted before heads share them: of 32 chunks
// of up to 16 over 500-4000 with 64 heads that is 2176, where about 200 have rows and take 80 and 96,
// but 128 of up to 4 over 100-2000 take 167 and 109 for their 16384 blocks.
int ctas_of(int d, long long units) { return d == 64 && units > 4ll * sms_or_default() ? 2 : 1; }

cudaError_t launch(int d, int ctas, int mask, const DiffMaps& t, const DiffParams& p,
                   cudaStream_t stream) {
  const int grid = p.base.num_units;  // a block a unit: resident ones take over those that wait
  if (d == 128) return launch<128, 1>(mask, t, p, grid, stream);
  return ctas == 2 ? launch<64, 2>(mask, t, p, grid, stream)
                   : launch<64, 1>(mask, t, p, grid, stream);
}

// Query heads of one kv head that may share a tile, as a power of two. Units that the GPU holds at
// once go apart (one prompt of 64 tokens, 32 heads over 8, d = 128: 6.7 us, shared 8.8). Documents
// count the tiles that may have rows (three of 64, 32 heads over 8, d = 128: 192 blocks, at most 128
// tiles, 11.0 us and 13.5 shared; 40 of 64, 16 over 4, d = 64: 25.1 and 22.5), chunks the blocks, since
// heads that share a tile read a context once (three of 16 tokens over 2000, 32 over 8: 192 blocks, 46
// and 32 us).
int head_shift(int group, long long units) {
  int s = 0;
  if (units <= sms_or_default()) return 0;
  while (s < 4 && group % (2 << s) == 0) ++s;
  return s;
}

// Blocks of a packed launch, both halves of every 256-row unit that the segments may have, and the
// 128-row tiles that may have rows, by the numbers that the host has.
long long packed_blocks(int heads, int tokens, int segments) {
  return 2ll * heads * (tokens / kUnitRows + static_cast<long long>(segments));
}
long long packed_tiles(int heads, int tokens, int segments) {
  return static_cast<long long>(heads) * (tokens / 128 + static_cast<long long>(segments));
}

// o and lse are written while other CTAs still read the inputs.
struct Span {
  const void* x;
  size_t n;
};
template <int N>
int diff_outputs(const Span (&in)[N], const Span& o, const Span& lse) {
  bool shared = overlap(o.x, o.n, lse.x, lse.n);
  for (const Span& t : in) shared |= overlap(o.x, o.n, t.x, t.n) || overlap(lse.x, lse.n, t.x, t.n);
  if (shared) return fail(ATTN_ERR_INVALID, "o or lse overlaps another tensor");
  return ATTN_OK;
}

}  // namespace

int diff_checks(const void* q, const void* k, const void* v, const void* o, const float* lse,
                const float* lam, const float* weight, float eps, float out_scale) {
  if (!q || !k || !v || !o || !lse || !lam) return fail(ATTN_ERR_INVALID, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      !aligned16(weight) || (reinterpret_cast<uintptr_t>(lam) & 3u))
    return fail(ATTN_ERR_INVALID, "tensors must be 16-byte aligned, lam 4-byte aligned");
  return diff_numbers(weight, eps, out_scale);
}

int diff_numbers(const float* weight, float eps, float out_scale) {
  if (!std::isfinite(out_scale)) return fail(ATTN_ERR_INVALID, "out_scale is not finite");
  if (weight && !(std::isfinite(eps) && eps >= 0.f))
    return fail(ATTN_ERR_INVALID, "eps must be finite and >= 0");
  return ATTN_OK;
}

int diff_sizes(int B, int Hq, int Hkv, int n, int d, float scale) {
  if (B < 0 || n < 0 || Hq <= 0 || Hkv <= 0)
    return fail(ATTN_ERR_INVALID, "need B >= 0, N >= 0, Hq > 0, Hkv > 0");
  if (Hq % Hkv != 0) return fail(ATTN_ERR_INVALID, "Hq (%d) %% Hkv (%d) != 0", Hq, Hkv);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d (64 or 128)", d);
  if (!std::isfinite(scale)) return fail(ATTN_ERR_INVALID, "scale is not finite");
  if (!(scale > 0.f)) return fail(ATTN_ERR_UNSUPPORTED, "scale must be > 0");
  return ATTN_OK;
}

}  // namespace ta

using namespace ta;

extern "C" {

int attn_fwd_diff(const void* q, const void* k, const void* v, void* o, float* lse,
                  const float* lam, int B, int Hq, int Hkv, int N, int d, float scale,
                  int mask_kind, int window, const int32_t* cu_seqlens, const float* norm_weight,
                  float eps, float out_scale, void* stream) {
  clear_error();
  int rc = diff_sizes(B, Hq, Hkv, N, d, scale);
  if (rc) return rc;
  if (!prefill_kind(mask_kind))
    return fail(ATTN_ERR_INVALID, "mask_kind %d is not a prefill kind", mask_kind);
  if (!window_ok(mask_kind, window))
    return fail(ATTN_ERR_INVALID, "window %d out of range for mask_kind %d", window, mask_kind);
  const bool doc = document_kind(mask_kind);
  if (doc && !cu_seqlens) return fail(ATTN_ERR_INVALID, "cu_seqlens is required");
  if ((rc = diff_numbers(norm_weight, eps, out_scale))) return rc;
  if (B == 0 || N == 0) return ATTN_OK;  // nothing to compute
  if ((rc = diff_checks(q, k, v, o, lse, lam, norm_weight, eps, out_scale))) return rc;
  const long long planes = doc ? Hq : static_cast<long long>(B) * Hq;
  const long long planes_kv = doc ? Hkv : static_cast<long long>(B) * Hkv;
  const int tiles = tiles_for_rows(N);
  long long units = doc ? packed_blocks(Hq, N, B) : planes * tiles;
  if (planes >= (1ll << 31) || units >= (1ll << 31) - 1 || N > INT32_MAX - 512)
    return fail(ATTN_ERR_UNSUPPORTED, "too many work units");
  const size_t q_bytes = static_cast<size_t>(planes) * N * d * 2;
  const size_t kv_bytes = static_cast<size_t>(planes_kv) * N * d * 2;
  const Span in[] = {{q, q_bytes}, {k, kv_bytes}, {v, kv_bytes}, {lam, sizeof(float) * Hq},
                     {norm_weight, norm_weight ? sizeof(float) * d : 0},
                     {cu_seqlens, doc ? sizeof(int32_t) * (B + size_t(1)) : 0}};
  rc = diff_outputs(in, {o, q_bytes}, {lse, static_cast<size_t>(planes) * N * 2 * sizeof(float)});
  if (rc) return rc;
  DiffParams p{};
  if ((rc = status_ptr(&p.base.status))) return rc;
  DiffMaps t;
  if ((rc = encode_3d(&t.q, q, d, N, planes, 128))) return rc;
  if ((rc = encode_3d(&t.o, o, d, N, planes, 32, d / 2))) return rc;
  p.head_shift = head_shift(Hq / Hkv, doc ? packed_tiles(Hq, N, B) : units);
  t.q8 = t.q;
  if (p.head_shift && (rc = encode_3d(&t.q8, q, d, N, planes, 8))) return rc;
  if (!doc)  // units of several heads' last rows
    units -= planes - (planes >> (7 - tile_rows_log2(N - 128 * (tiles - 1), p.head_shift)));
  const int ctas = ctas_of(d, units);
  const uint32_t tile = d == 64 && ctas == 1 ? DiffCfg<64, kMaskNone, 1>::BN : 64;
  if ((rc = encode_3d(&t.k, k, d, N, planes_kv, tile))) return rc;
  if ((rc = encode_3d(&t.v, v, d, N, planes_kv, tile))) return rc;
  p.base.o = o;
  p.base.lse = lse;
  p.base.cu_seqlens = cu_seqlens;
  p.base.B = B;
  p.base.Hq = Hq;
  p.base.Hkv = Hkv;
  p.base.N = N;
  p.base.group = Hq / Hkv;
  p.base.num_units = static_cast<int>(units);
  p.base.window = window;
  p.base.scale_log2 = scale * kLog2e;
  p.base.timeout_ns = kTimeoutNs;
  p.lam = lam;
  p.weight = norm_weight;
  p.eps = eps;
  p.out_scale = out_scale;
  p.mask = mask_kind;
  const cudaError_t e =
      launch(d, ctas, mask_kind, t, p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "differential prefill launch");
  return ATTN_OK;
}

int attn_fwd_diff_paged_prefill(const void* q, const void* k, const void* v, void* o, float* lse,
                                const float* lam, int B, int Hq, int Hkv, int total_q, int d,
                                float scale, const float* norm_weight, float eps,
                                float out_scale, const int32_t* cu_seqlens_q,
                                const int32_t* seqlens_k, const int32_t* block_table,
                                int max_pages, int page_size, int num_pages, void* stream) {
  clear_error();
  int rc = diff_sizes(B, Hq, Hkv, total_q, d, scale);
  if (rc) return rc;
  if (!page_size_ok(page_size))
    return fail(ATTN_ERR_UNSUPPORTED, "page_size %d (16, 32, 64 or 128)", page_size);
  if ((rc = diff_numbers(norm_weight, eps, out_scale))) return rc;
  if (B == 0 || total_q == 0) return ATTN_OK;  // no query rows
  if (!cu_seqlens_q || !seqlens_k || !block_table) return fail(ATTN_ERR_INVALID, "null pointer");
  if ((rc = diff_checks(q, k, v, o, lse, lam, norm_weight, eps, out_scale))) return rc;
  if (max_pages <= 0 || num_pages <= 0)
    return fail(ATTN_ERR_INVALID, "max_pages %d, num_pages %d", max_pages, num_pages);
  const long long keys = static_cast<long long>(max_pages) * page_size;
  if (static_cast<long long>(num_pages) * Hkv >= (1ll << 31) || keys >= (1ll << 30))
    return fail(ATTN_ERR_UNSUPPORTED, "page pool or block table too large");
  const long long units = packed_blocks(Hq, total_q, B);
  if (units >= (1ll << 31) - 1 || total_q >= (1 << 30))
    return fail(ATTN_ERR_UNSUPPORTED, "too many work units");
  const size_t q_bytes = static_cast<size_t>(Hq) * total_q * d * 2;
  const size_t pool = static_cast<size_t>(num_pages) * Hkv * page_size * d * 2;
  const Span in[] = {{q, q_bytes}, {k, pool}, {v, pool}, {lam, sizeof(float) * Hq},
                     {norm_weight, norm_weight ? sizeof(float) * d : 0},
                     {cu_seqlens_q, sizeof(int32_t) * (B + size_t(1))},
                     {seqlens_k, sizeof(int32_t) * B},
                     {block_table, sizeof(int32_t) * B * static_cast<size_t>(max_pages)}};
  rc = diff_outputs(in, {o, q_bytes},
                    {lse, static_cast<size_t>(Hq) * total_q * 2 * sizeof(float)});
  if (rc) return rc;
  DiffParams p{};
  if ((rc = status_ptr(&p.base.status))) return rc;
  DiffMaps t;
  if ((rc = encode_3d(&t.q, q, d, total_q, Hq, 128))) return rc;
  p.head_shift = head_shift(Hq / Hkv, units);
  t.q8 = t.q;
  if (p.head_shift && (rc = encode_3d(&t.q8, q, d, total_q, Hq, 8))) return rc;
  if ((rc = encode_3d(&t.o, o, d, total_q, Hq, 32, d / 2))) return rc;
  const uint64_t planes = static_cast<uint64_t>(num_pages) * Hkv;
  const uint32_t box = page_size < 64 ? page_size : 64;  // rows of a page in one 64-key tile
  if ((rc = encode_3d(&t.k, k, d, page_size, planes, box))) return rc;
  if ((rc = encode_3d(&t.v, v, d, page_size, planes, box))) return rc;
  p.base.o = o;
  p.base.lse = lse;
  p.base.cu_seqlens = cu_seqlens_q;
  p.base.seqlens_k = seqlens_k;
  p.base.table = block_table;
  p.base.max_pages = max_pages;
  p.base.page_size = page_size;
  p.base.page_shift = log2_exact(page_size);
  p.base.num_pages = num_pages;
  p.base.B = B;
  p.base.Hq = Hq;
  p.base.Hkv = Hkv;
  p.base.N = total_q;
  p.base.group = Hq / Hkv;
  p.base.num_units = static_cast<int>(units);
  p.base.scale_log2 = scale * kLog2e;
  p.base.timeout_ns = kTimeoutNs;
  p.lam = lam;
  p.weight = norm_weight;
  p.eps = eps;
  p.out_scale = out_scale;
  p.mask = kMaskPagedPrefill;
  const cudaError_t e = launch(d, ctas_of(d, packed_tiles(Hq, total_q, B)), kMaskPagedPrefill, t, p,
                               static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "differential paged prefill launch");
  return ATTN_OK;
}

}  // extern "C"
