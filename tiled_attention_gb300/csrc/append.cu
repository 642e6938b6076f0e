// append.cu — entry points of the token-row kernels (append.cuh): norm and rotation, append to
// a bf16 or 4-bit paged cache, and 4-bit pages back to bf16.
#include "append.cuh"

#include <cmath>

#include "../../include/attn.h"
#include "api.h"

namespace ta {
namespace {

// Bytes from the first to the last element of token rows.
size_t rows_bytes(int total, int heads, int d, int64_t stride) {
  return total > 0 ? (static_cast<size_t>(total - 1) * stride + static_cast<size_t>(heads) * d) * 2
                   : 0;
}

// Checks and fields common to the row entry points. Sizes of absent tensors (null q or k) are
// passed as 0 heads.
int row_params(RowParams* p, const void* q, const void* k, const void* v, void* q_out, int Hq,
               int Hkv, int total, int N, int d, int64_t q_stride, int64_t k_stride,
               int64_t v_stride, const float* q_weight, const float* k_weight, float eps,
               const float* cos_sin, int max_pos, int rot_dim, int interleaved, int rot_unit) {
  if (total < 0 || N < 1) return fail(ATTN_ERR_INVALID, "need total >= 0 and N >= 1");
  if (Hq < 0 || Hkv < 0 || Hq + static_cast<long long>(Hkv) == 0)
    return fail(ATTN_ERR_INVALID, "Hq %d, Hkv %d", Hq, Hkv);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d (64 or 128)", d);
  if (total % N != 0) return fail(ATTN_ERR_INVALID, "%d tokens are not rows of %d", total, N);
  if (rot_dim < 0 || rot_dim > d) return fail(ATTN_ERR_INVALID, "rot_dim %d", rot_dim);
  if (rot_dim % rot_unit != 0)
    return fail(ATTN_ERR_UNSUPPORTED, "rot_dim %d is not a multiple of %d", rot_dim, rot_unit);
  if (rot_dim > 0 && max_pos < 1) return fail(ATTN_ERR_INVALID, "max_pos %d", max_pos);
  if ((q_weight || k_weight) && !(std::isfinite(eps) && eps >= 0.f))
    return fail(ATTN_ERR_INVALID, "eps must be finite and >= 0");
  const struct { const void* x; int heads; int64_t stride; } in[3] = {
      {q, Hq, q_stride}, {k, Hkv, k_stride}, {v, Hkv, v_stride}};
  for (const auto& i : in) {
    if (!i.x) continue;
    if (i.stride < static_cast<int64_t>(i.heads) * d || i.stride % 8 != 0 ||
        i.stride > (int64_t(1) << 40))
      return fail(ATTN_ERR_INVALID, "token stride %lld (at least the heads' %lld, multiple of 8)",
                  static_cast<long long>(i.stride), static_cast<long long>(i.heads) * d);
    if (!aligned16(i.x)) return fail(ATTN_ERR_INVALID, "tensors must be 16-byte aligned");
  }
  if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(cos_sin) || !aligned16(q_out))
    return fail(ATTN_ERR_INVALID, "tensors must be 16-byte aligned");
  if (rot_dim > 0 && total > 0 && !cos_sin) return fail(ATTN_ERR_INVALID, "cos_sin is required");
  if (q && total > 0 && !q_out) return fail(ATTN_ERR_INVALID, "null pointer");
  // q_out must not touch the rows that other warps may still read.
  const size_t out_bytes = static_cast<size_t>(total) * Hq * d * 2;
  for (const auto& i : in)
    if (q && total > 0 && overlap(q_out, out_bytes, i.x, rows_bytes(total, i.heads, d, i.stride)))
      return fail(ATTN_ERR_INVALID, "an output overlaps an input");
  p->in[0] = static_cast<const uint8_t*>(q);
  p->in[1] = static_cast<const uint8_t*>(k);
  p->in[2] = static_cast<const uint8_t*>(v);
  p->stride[0] = q_stride * 2;
  p->stride[1] = k_stride * 2;
  p->stride[2] = v_stride * 2;
  p->out[0] = static_cast<uint8_t*>(q_out);
  p->weight[0] = q_weight;
  p->weight[1] = k_weight;
  p->cos_sin = rot_dim ? cos_sin : nullptr;
  p->eps = eps;
  p->heads[0] = q ? Hq : 0;
  p->heads[1] = k ? Hkv : 0;
  p->heads[2] = v ? Hkv : 0;
  p->total = total;
  p->N = N;
  p->max_pos = max_pos;
  p->rot = rot_dim;
  p->interleaved = interleaved ? 1 : 0;
  return ATTN_OK;
}

// row_bytes: of one token of one kv head in a pool.
int cache_params(RowParams* p, const void* k, const void* v, void* k_pool, void* v_pool, int B,
                 const int32_t* cu_seqlens_q, const int32_t* seqlens_k,
                 const int32_t* block_table, int max_pages, int page_size, int num_pages, int d,
                 int row_bytes) {
  if (B < 0) return fail(ATTN_ERR_INVALID, "need B >= 0");
  if (!page_size_ok(page_size))
    return fail(ATTN_ERR_UNSUPPORTED, "page_size %d (16, 32, 64 or 128)", page_size);
  if (B == 0 || p->total == 0) return ATTN_OK;
  if (!k || !v || !k_pool || !v_pool || !cu_seqlens_q || !seqlens_k || !block_table)
    return fail(ATTN_ERR_INVALID, "null pointer");
  if (!aligned16(k_pool) || !aligned16(v_pool))
    return fail(ATTN_ERR_INVALID, "tensors must be 16-byte aligned");
  if (max_pages <= 0 || num_pages <= 0)
    return fail(ATTN_ERR_INVALID, "max_pages %d, num_pages %d", max_pages, num_pages);
  if (static_cast<long long>(num_pages) * p->heads[1] >= (1ll << 31) ||
      static_cast<long long>(max_pages) * page_size >= (1ll << 31))
    return fail(ATTN_ERR_UNSUPPORTED, "page pool or block table too large");
  const size_t n = static_cast<size_t>(num_pages) * p->heads[1] * page_size * row_bytes;
  const size_t out_bytes = p->in[0] ? static_cast<size_t>(p->total) * p->heads[0] * d * 2 : 0;
  bool shared = overlap(k_pool, n, v_pool, n);
  for (const void* pool : {k_pool, v_pool}) {
    shared |= overlap(pool, n, p->out[0], out_bytes);
    for (int i = 0; i < 3; ++i)
      shared |= overlap(pool, n, p->in[i], rows_bytes(p->total, p->heads[i], d, p->stride[i] / 2));
  }
  if (shared) return fail(ATTN_ERR_INVALID, "a pool overlaps the other or a tensor of rows");
  p->pool[0] = static_cast<uint8_t*>(k_pool);
  p->pool[1] = static_cast<uint8_t*>(v_pool);
  p->cu = cu_seqlens_q;
  p->lens = seqlens_k;
  p->table = block_table;
  p->B = B;
  p->max_pages = max_pages;
  p->page_shift = log2_exact(page_size);
  p->num_pages = num_pages;
  return ATTN_OK;
}

template <int CACHE>
int launch_rows(RowParams& p, int d, void* stream) {
  int rc = status_ptr(&p.status);
  if (rc) return rc;
  const int rows = 512 / d;  // rows a warp takes at once: 32 lanes over d / 16 lanes a row
  int all = 0;
  for (int i = 0; i < 3; ++i) all += p.groups[i] = (p.heads[i] + rows - 1) / rows;
  // One warp takes all rows of a token once that fills the GPU, so that the position, its
  // angles and its page are found once a token; fewer tokens are split over more warps, down
  // to one row group each, for latency.
  const long long want = 32ll * sms_or_default();
  long long per = (want + p.total - 1) / p.total;
  if (per > all) per = all;
  p.groups_per_task = static_cast<int>((all + per - 1) / per);
  const long long parts = (all + p.groups_per_task - 1) / p.groups_per_task;
  if (parts > 65535) return fail(ATTN_ERR_UNSUPPORTED, "too many heads");
  const int warps = kRowThreads / 32;
  const dim3 grid((static_cast<unsigned>(p.total) + warps - 1) / warps,
                  static_cast<unsigned>(parts));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64)
    rows_kernel<64, CACHE><<<grid, kRowThreads, 0, s>>>(p);
  else
    rows_kernel<128, CACHE><<<grid, kRowThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "row kernel launch");
  return ATTN_OK;
}

// The 4-bit pools' tensor scales: finite, > 0, with a finite reciprocal.
bool pool_scale_ok(float s) { return std::isfinite(s) && s > 0.f && std::isfinite(1.f / s); }

}  // namespace
}  // namespace ta

using namespace ta;

extern "C" {

int attn_norm_rope(const void* q, const void* k, void* q_out, void* k_out, int total, int N,
                   int Hq, int Hkv, int d, int64_t q_stride, int64_t k_stride,
                   const float* q_weight, const float* k_weight, float eps, const float* cos_sin,
                   int max_pos, int rot_dim, int interleaved, const int32_t* positions,
                   void* stream) {
  clear_error();
  RowParams p{};
  int rc = row_params(&p, q, k, nullptr, q_out, Hq, Hkv, total, N, d, q_stride, k_stride, 0,
                      q_weight, k_weight, eps, cos_sin, max_pos, rot_dim, interleaved, 16);
  if (rc) return rc;
  if (total == 0) return ATTN_OK;
  if ((!q && !k) || (k && !k_out)) return fail(ATTN_ERR_INVALID, "null pointer");
  if (p.heads[0] + p.heads[1] == 0) return fail(ATTN_ERR_INVALID, "no heads");
  if (!aligned16(k_out)) return fail(ATTN_ERR_INVALID, "tensors must be 16-byte aligned");
  if (!positions && rot_dim > 0 && N > max_pos)
    return fail(ATTN_ERR_INVALID, "positions of %d rows, a table of %d", N, max_pos);
  if (k) {
    const size_t n = static_cast<size_t>(total) * Hkv * d * 2;
    if (overlap(k_out, n, q, rows_bytes(total, Hq, d, q_stride)) ||
        overlap(k_out, n, k, rows_bytes(total, Hkv, d, k_stride)))
      return fail(ATTN_ERR_INVALID, "an output overlaps an input");
    if (q && overlap(k_out, n, q_out, static_cast<size_t>(total) * Hq * d * 2))
      return fail(ATTN_ERR_INVALID, "q_out and k_out overlap");
  }
  p.out[1] = static_cast<uint8_t*>(k_out);
  p.positions = positions;
  return launch_rows<kCacheNone>(p, d, stream);
}

int attn_append_paged(const void* q, const void* k, const void* v, void* q_out, void* k_pool,
                      void* v_pool, int B, int Hq, int Hkv, int total_q, int N, int d,
                      int64_t q_stride, int64_t k_stride, int64_t v_stride,
                      const float* q_weight, const float* k_weight, float eps,
                      const float* cos_sin, int max_pos, int rot_dim, int interleaved,
                      const int32_t* cu_seqlens_q, const int32_t* seqlens_k,
                      const int32_t* block_table, int max_pages, int page_size, int num_pages,
                      void* stream) {
  clear_error();
  RowParams p{};
  if (Hkv <= 0) return fail(ATTN_ERR_INVALID, "Hkv %d", Hkv);
  int rc = row_params(&p, q, k, v, q_out, Hq, Hkv, total_q, N, d, q_stride, k_stride, v_stride,
                      q_weight, k_weight, eps, cos_sin, max_pos, rot_dim, interleaved, 16);
  if (rc) return rc;
  rc = cache_params(&p, k, v, k_pool, v_pool, B, cu_seqlens_q, seqlens_k, block_table, max_pages,
                    page_size, num_pages, d, 2 * d);
  if (rc) return rc;
  if (B == 0 || total_q == 0) return ATTN_OK;  // no new tokens
  return launch_rows<kCacheBf16>(p, d, stream);
}

int attn_append_paged_fp4(const void* q, const void* k, const void* v, void* q_out, void* k_pool,
                          void* v_pool, float k_scale, float v_scale, int B, int Hq, int Hkv,
                          int total_q, int N, int d, int64_t q_stride, int64_t k_stride,
                          int64_t v_stride, const float* q_weight, const float* k_weight,
                          float eps, const float* cos_sin, int max_pos, int rot_dim,
                          int interleaved, const int32_t* cu_seqlens_q, const int32_t* seqlens_k,
                          const int32_t* block_table, int max_pages, int page_size,
                          int num_pages, void* stream) {
  clear_error();
  RowParams p{};
  if (Hkv <= 0) return fail(ATTN_ERR_INVALID, "Hkv %d", Hkv);
  if (!pool_scale_ok(k_scale) || !pool_scale_ok(v_scale))
    return fail(ATTN_ERR_INVALID, "k_scale and v_scale must be > 0, with finite reciprocals");
  // A 4-bit block is two 8-channel chunks: a half-split rotation pairs whole blocks only if
  // half the rotated channels are a multiple of 16.
  int rc = row_params(&p, q, k, v, q_out, Hq, Hkv, total_q, N, d, q_stride, k_stride, v_stride,
                      q_weight, k_weight, eps, cos_sin, max_pos, rot_dim, interleaved,
                      interleaved ? 16 : 32);
  if (rc) return rc;
  rc = cache_params(&p, k, v, k_pool, v_pool, B, cu_seqlens_q, seqlens_k, block_table, max_pages,
                    page_size, num_pages, d, fp4_row_bytes(d));
  if (rc) return rc;
  if (B == 0 || total_q == 0) return ATTN_OK;
  p.inv_scale[0] = 1.f / k_scale;
  p.inv_scale[1] = 1.f / v_scale;
  return launch_rows<kCacheFp4>(p, d, stream);
}

int attn_unpack_pages_fp4(const void* pool, void* dst, float pool_scale,
                          const int32_t* block_table, const int32_t* seqlens, int B,
                          int max_pages, int Hkv, int page_size, int d, int num_pages,
                          void* stream) {
  clear_error();
  if (B < 0 || max_pages < 0 || Hkv <= 0 || num_pages < 0)
    return fail(ATTN_ERR_INVALID, "bad unpack sizes");
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d (64 or 128)", d);
  if (!page_size_ok(page_size))
    return fail(ATTN_ERR_UNSUPPORTED, "page_size %d (16, 32, 64 or 128)", page_size);
  if (!pool_scale_ok(pool_scale))
    return fail(ATTN_ERR_INVALID, "pool_scale must be > 0, with a finite reciprocal");
  if (B == 0 || max_pages == 0) return ATTN_OK;
  if (!pool || !dst || !block_table || !seqlens) return fail(ATTN_ERR_INVALID, "null pointer");
  if (!aligned16(pool) || !aligned16(dst))
    return fail(ATTN_ERR_INVALID, "pool and dst must be 16-byte aligned");
  if (B > 65535 || static_cast<long long>(max_pages) * page_size >= (1ll << 31) ||
      static_cast<long long>(num_pages) * Hkv >= (1ll << 31) || Hkv > 32768)
    return fail(ATTN_ERR_UNSUPPORTED, "page pool or block table too large");
  const size_t rows = static_cast<size_t>(Hkv) * page_size;
  if (overlap(pool, rows * num_pages * fp4_row_bytes(d), dst,
              rows * B * static_cast<size_t>(max_pages) * d * 2))
    return fail(ATTN_ERR_INVALID, "dst overlaps the pool");
  UnpackParams p{};
  int rc = status_ptr(&p.status);
  if (rc) return rc;
  p.pool = static_cast<const uint8_t*>(pool);
  p.dst = static_cast<uint4*>(dst);
  p.table = block_table;
  p.lens = seqlens;
  p.scale = pool_scale;
  p.max_pages = max_pages;
  p.Hkv = Hkv;
  p.page_shift = log2_exact(page_size);
  p.num_pages = num_pages;
  const long long chunks = static_cast<long long>(Hkv) * page_size * (d / 8);
  const dim3 grid(max_pages, B,
                  static_cast<unsigned>((chunks + 256 * kUnpackBatch - 1) / (256 * kUnpackBatch)));
  if (d == 64)
    unpack_fp4_kernel<64><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  else
    unpack_fp4_kernel<128><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "unpack launch");
  return ATTN_OK;
}

}  // extern "C"
