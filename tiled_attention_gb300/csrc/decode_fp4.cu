// decode_fp4.cu — the 4-bit paged decode's instantiations (head dim 64 / 128, one or two
// 8-head column tiles) and its entry points.
#include "decode_fp4.cuh"

#include <cmath>

#include "../../include/attn.h"
#include "api.h"
#include "launch.h"

namespace ta {
namespace {

// CTAs of the decode kernel: as many as the GPU holds at once.
int fp4_slots(int d, int group) {
  const int per = d == 64 ? (group <= 8 ? DecodeFp4Cfg<64, 1>::kCtas : DecodeFp4Cfg<64, 2>::kCtas)
                          : (group <= 8 ? DecodeFp4Cfg<128, 1>::kCtas : DecodeFp4Cfg<128, 2>::kCtas);
  return per * sms_or_default();
}

constexpr int kWorkers = DecodeFp4Cfg<64, 1>::kWarps;  // of a CTA, at most

// Whether this host sees no device at all.
bool no_device() {
  int n = 0;
  const cudaError_t e = cudaGetDeviceCount(&n);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaErrorNoDevice || e == cudaErrorInsufficientDriver;
}

struct Fp4Layout {
  size_t part_ml, joins, total;
  int slots;
};

// Of every worker (up to four a CTA) two partial rows of each query head of a group: O, then
// (max, sum); then what it has to have joined.
Fp4Layout fp4_layout(int Hq, int Hkv, int d) {
  Fp4Layout L{};
  const int group = Hq / Hkv;
  L.slots = fp4_slots(d, group);
  const size_t rows = 2 * static_cast<size_t>(kWorkers * L.slots) * group;
  L.part_ml = align256(rows * d * sizeof(float));
  L.joins = L.part_ml + align256(rows * 2 * sizeof(float));
  L.total = L.joins + align256(static_cast<size_t>(kWorkers * L.slots) * sizeof(int4));
  return L;
}

template <int D, int NT, bool SOLO>
cudaError_t launch_one(const DecodeFp4Params& p, cudaStream_t stream) {
  static unsigned long long done = 0;
  auto kern = decode_fp4_kernel<D, NT, SOLO>;
  using C = DecodeFp4Cfg<D, NT>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  kern<<<p.slots, C::kThreads, C::kSmemBytes, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // The joining kernel may start before the decode kernel has ended (it waits for it).
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = SOLO ? dim3(kWorkers * p.slots) : dim3(p.Hq / p.join_heads, p.B);
  // By contexts: eight threads a column for one head, and as many threads for several (48
  // sequences x 4 kv heads: 73 us, with 128 threads 75); by workers, which have few parts
  // each: 128 (256 sequences x 4 kv heads of 16 at d = 64: 37.7 us, with 256 threads 38.5).
  cfg.blockDim = dim3(SOLO || p.join_heads * D < 128 ? 128 : 256);
  cfg.stream = stream;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_fp4_kernel<D, SOLO>, p);
}

template <bool SOLO>
cudaError_t launch(const DecodeFp4Params& p, int d, cudaStream_t stream) {
  if (d == 64)
    return p.group <= 8 ? launch_one<64, 1, SOLO>(p, stream) : launch_one<64, 2, SOLO>(p, stream);
  return p.group <= 8 ? launch_one<128, 1, SOLO>(p, stream) : launch_one<128, 2, SOLO>(p, stream);
}

}  // namespace
}  // namespace ta

using namespace ta;

extern "C" {

size_t attn_workspace_bytes_fp4(int B, int Hq, int Hkv, int N, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || (d != 64 && d != 128) || Hq < Hkv) return 0;
  return fp4_layout(Hq, Hkv, d).total;
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
  if (B == 0) return ATTN_OK;  // no rows
  // N = 0: every context is empty, and its rows are still the caller's to have: O = 0, LSE =
  // -inf. They come of the lengths alone; q, the pools, the table and the workspace are not used.
  const bool keys = N > 0;
  if (!o || !lse || !cu_seqlens || (keys && (!q || !k || !v || !block_table)))
    return fail(ATTN_ERR_INVALID, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_INVALID, "tensors must be 16-byte aligned");
  if (keys && num_pages <= 0) return fail(ATTN_ERR_INVALID, "num_pages %d", num_pages);
  if (static_cast<long long>(num_pages) * Hkv >= (1ll << 31) || Hkv > 65535 || N > (1 << 30))
    return fail(ATTN_ERR_UNSUPPORTED, "page pool or context too large");
  const long long units = (static_cast<long long>(N) + 63) / 64 + 8;  // of one context, at most
  if (B > 65535 || static_cast<long long>(B) * Hkv >= (1ll << 31) / units)
    return fail(ATTN_ERR_UNSUPPORTED, "decode batch too large");
  if (!keys && no_device()) return ATTN_OK;  // nor are there device rows to fill
  const Fp4Layout L = fp4_layout(Hq, Hkv, d);
  if (keys && (!workspace || workspace_bytes < L.total || !aligned16(workspace)))
    return fail(ATTN_ERR_WORKSPACE, "workspace needs %zu bytes (16-byte aligned)", L.total);
  // Rows are written while other workers still read queries, lengths and pages.
  const int max_pages = (N + page_size - 1) / page_size;
  const size_t rows = static_cast<size_t>(B) * Hq;
  const size_t pool =
      keys ? static_cast<size_t>(num_pages) * Hkv * page_size * fp4_row_bytes(d) : 0;
  const struct { const void* x; size_t bytes; } out[3] = {
      {o, rows * d * 2}, {lse, rows * sizeof(float)}, {workspace, keys ? L.total : 0}}, in[5] = {
      {q, keys ? rows * d * 2 : 0}, {k, pool}, {v, pool},
      {cu_seqlens, sizeof(int32_t) * (B + size_t(1))},
      {block_table, sizeof(int32_t) * B * static_cast<size_t>(max_pages)}};
  for (int i = 0; i < 3; ++i) {
    bool shared = overlap(out[i].x, out[i].bytes, out[(i + 1) % 3].x, out[(i + 1) % 3].bytes);
    for (const auto& t : in) shared |= overlap(out[i].x, out[i].bytes, t.x, t.bytes);
    if (shared) return fail(ATTN_ERR_INVALID, "o, lse or workspace overlaps another tensor");
  }
  DecodeFp4Params p{};
  int rc = status_ptr(&p.status);
  if (rc) return rc;
  p.q = static_cast<const uint4*>(q);
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.cu = cu_seqlens;
  p.table = block_table;
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  if (keys) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + L.part_ml);
    p.joins = reinterpret_cast<int4*>(ws + L.joins);
  }
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.slots = L.slots;
  // The joining kernel: a CTA a group once the groups fill the GPU (48 sequences x 4 kv heads of 16
  // query heads: 4 us less than with a CTA a head), else a CTA a head, with eight threads a
  // column to share the parts (one sequence x 8 kv heads: 12.7 us, with four 13.6).
  p.join_heads = static_cast<long long>(B) * Hkv >= sms_or_default() ? group : 1;
  p.group = group;
  p.page_shift = log2_exact(page_size);
  p.max_len = N;
  p.scale_log2 = scale_log2;
  p.v_scale = v_scale;
  p.timeout_ns = kTimeoutNs;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  // From as many contexts (a sequence and kv head each) on as the GPU holds CTAs, a warp is a
  // worker; below, a CTA. Measured with warps and with CTAs: 64 sequences of 1K-8K tokens x 8 kv
  // heads 66 and 68 us, 256 of 1K 65 and 76, 1000 of 20-400 79 and 169; 24 of 1K-16K 50 and 48,
  // one of 16K 25 and 13. The lengths are not known here, so a batch of that size with its tokens
  // in a few sequences gets warps too: 63 empty ones and one of 16K 26 and 16, 63 of 256 tokens
  // and one of 128K 77 and 46.
  // Without keys CTAs: they find no work and leave the workspace alone, warps would clear `joins`.
  const bool solo = keys && static_cast<long long>(B) * Hkv >= L.slots;
  const cudaError_t e = solo ? launch<true>(p, d, stream) : launch<false>(p, d, stream);
  if (e != cudaSuccess) return cuda_fail(e, "4-bit decode launch");
  return ATTN_OK;
}

}  // extern "C"
