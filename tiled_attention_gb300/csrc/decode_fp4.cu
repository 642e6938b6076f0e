// decode_fp4.cu — the 4-bit paged decode's instantiations (head dim 64 / 128, one or two
// 8-head column tiles) and its entry points.
#include "decode_fp4.cuh"

#include <cmath>

#include "../../include/attn.h"
#include "api.h"
#include "launch.h"

namespace ta {
namespace {

struct Fp4Layout {
  size_t part_ml, counters, total;
  int chunk_stages, max_splits;
};

// 128-token stages per split-KV CTA.
int fp4_chunk_stages(int B, int Hkv) {
  return static_cast<long long>(B) * Hkv >= sms_or_default() ? 16 : 4;
}

Fp4Layout fp4_layout(int B, int Hq, int Hkv, int N, int d) {
  Fp4Layout L{};
  L.chunk_stages = fp4_chunk_stages(B, Hkv);
  const long long stages = (static_cast<long long>(N) + 127) / 128;
  L.max_splits = static_cast<int>((stages + L.chunk_stages - 1) / L.chunk_stages);
  if (L.max_splits <= 1) return L;  // one CTA per (sequence, kv head): no partials
  const size_t groups = static_cast<size_t>(B) * Hkv;
  const size_t rows = groups * L.max_splits * static_cast<size_t>(Hq / Hkv);
  L.part_ml = align256(rows * d * sizeof(float));
  L.counters = L.part_ml + align256(rows * 2 * sizeof(float));
  L.total = L.counters + align256(groups * sizeof(int));
  return L;
}

template <int D, int NT>
cudaError_t launch_one(const DecodeFp4Params& p, dim3 grid, cudaStream_t stream) {
  static unsigned long long done = 0;
  auto kern = decode_fp4_kernel<D, NT>;
  using C = DecodeFp4Cfg<D, NT>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::kThreads, C::kSmemBytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ta

using namespace ta;

extern "C" {

size_t attn_workspace_bytes_fp4(int B, int Hq, int Hkv, int N, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0) return 0;
  return fp4_layout(B, Hq, Hkv, N, d).total;
}

int attn_fwd_paged_decode_fp4(const void* q, const void* k, const void* v, void* o, float* lse,
                              int B, int Hq, int Hkv, int N, int d, float scale, float k_scale,
                              float v_scale, const int32_t* cu_seqlens,
                              const int32_t* block_table, int page_size, int num_pages,
                              void* workspace, size_t workspace_bytes, void* stream_) {
  clear_error();
  if (B < 0 || N < 0 || Hq <= 0 || Hkv <= 0)
    return fail(ATTN_ERR_INVALID, "need B >= 0, N >= 0, Hq > 0, Hkv > 0");
  if (Hq % Hkv != 0) return fail(ATTN_ERR_INVALID, "Hq (%d) %% Hkv (%d) != 0", Hq, Hkv);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d (64 or 128)", d);
  if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return fail(ATTN_ERR_INVALID, "scale, k_scale or v_scale is not finite");
  if (!(scale > 0.f)) return fail(ATTN_ERR_UNSUPPORTED, "scale must be > 0");
  const float scale_log2 = scale * k_scale * kLog2e;
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(scale_log2))
    return fail(ATTN_ERR_INVALID, "k_scale and v_scale must be > 0, scale * k_scale finite");
  if (!page_size_ok(page_size))
    return fail(ATTN_ERR_UNSUPPORTED, "page_size %d (16, 32, 64 or 128)", page_size);
  const int group = Hq / Hkv;
  if (group > kMaxDecodeGroup)
    return fail(ATTN_ERR_UNSUPPORTED, "query heads per kv head %d (at most %d)", group,
                kMaxDecodeGroup);
  if (B == 0 || N == 0) return ATTN_OK;  // nothing to compute
  if (!q || !k || !v || !o || !lse || !cu_seqlens || !block_table)
    return fail(ATTN_ERR_INVALID, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_INVALID, "tensors must be 16-byte aligned");
  if (num_pages <= 0) return fail(ATTN_ERR_INVALID, "num_pages %d", num_pages);
  if (static_cast<long long>(num_pages) * Hkv >= (1ll << 31) || N > (1 << 30))
    return fail(ATTN_ERR_UNSUPPORTED, "page pool or context too large");
  const Fp4Layout L = fp4_layout(B, Hq, Hkv, N, d);
  if (Hkv > 65535 || B > 65535) return fail(ATTN_ERR_UNSUPPORTED, "decode grid too large");
  if (L.total && (!workspace || workspace_bytes < L.total || !aligned16(workspace)))
    return fail(ATTN_ERR_WORKSPACE, "workspace needs %zu bytes (16-byte aligned)", L.total);
  DecodeFp4Params p{};
  int rc = status_ptr(&p.status);
  if (rc) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const uint4*>(q);
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.cu = cu_seqlens;
  p.table = block_table;
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + L.part_ml);
  p.counters = reinterpret_cast<int*>(ws + L.counters);
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.max_pages = (N + page_size - 1) / page_size;
  p.num_pages = num_pages;
  p.max_splits = L.max_splits;
  p.chunk_stages = L.chunk_stages;
  p.group = group;
  p.page_shift = log2_exact(page_size);
  p.max_len = N;
  p.scale_log2 = scale_log2;
  p.v_scale = v_scale;
  p.timeout_ns = kTimeoutNs;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  cudaError_t e;
  if (L.total) {
    e = cudaMemsetAsync(p.counters, 0, sizeof(int) * static_cast<size_t>(B) * Hkv, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(counters)");
  }
  const dim3 grid(L.max_splits, Hkv, B);
  if (d == 64)
    e = group <= 8 ? launch_one<64, 1>(p, grid, stream) : launch_one<64, 2>(p, grid, stream);
  else
    e = group <= 8 ? launch_one<128, 1>(p, grid, stream) : launch_one<128, 2>(p, grid, stream);
  if (e != cudaSuccess) return cuda_fail(e, "4-bit decode launch");
  return ATTN_OK;
}

}  // extern "C"
