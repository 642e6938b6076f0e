// diff_decode.cu — differential attention's paged decode: instantiations (head dim 64 / 128, one or
// two tiles of eight query heads) and entry points.
#include "diff_decode.cuh"

#include "../../include/attn.h"
#include "api.h"
#include "diff.h"
#include "launch.h"

namespace ta {
namespace {

struct DiffDecodeLayout {
  size_t part_ml, total;
  int slots;
};

// Of every CTA two partial rows of each map and query head of a group: O, then (max, sum).
DiffDecodeLayout diff_layout(int Hq, int Hkv, int d) {
  DiffDecodeLayout L{};
  L.slots = kDiffDecodeCtas * sms_or_default();
  const size_t rows = 4 * static_cast<size_t>(L.slots) * (Hq / Hkv);
  L.part_ml = align256(rows * d * sizeof(float));
  L.total = L.part_ml + align256(rows * 2 * sizeof(float));
  return L;
}

template <int D, int NT>
cudaError_t launch_one(const CUtensorMap& k, const CUtensorMap& v, const DiffDecodeParams& p,
                       cudaStream_t stream) {
  static unsigned long long done = 0;
  auto kern = diff_decode_kernel<D, NT>;
  using C = DiffDecodeCfg<D>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  if (p.max_len > 0) {
    kern<<<p.slots, C::kThreads, C::kSmemBytes, stream>>>(k, v, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  // The joining kernel may start before the decode kernel has ended (it waits for it); alone, it
  // starts after all that is on the stream, since it reads the lengths before it waits.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.join_workers ? p.slots : p.B * p.Hkv, p.group / p.join_heads);
  cfg.blockDim = dim3(kDiffJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = p.max_len > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, diff_join_kernel<D>, p);
}

}  // namespace
}  // namespace ta

using namespace ta;

extern "C" {

size_t attn_workspace_bytes_diff(int B, int Hq, int Hkv, int N, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || (d != 64 && d != 128) || Hq < Hkv) return 0;
  return diff_layout(Hq, Hkv, d).total;
}

int attn_fwd_diff_paged_decode(const void* q, const void* k, const void* v, void* o, float* lse,
                               const float* lam, int B, int Hq, int Hkv, int N, int d,
                               float scale, const float* norm_weight, float eps,
                               float out_scale, const int32_t* cu_seqlens,
                               const int32_t* block_table, int page_size, int num_pages,
                               void* workspace, size_t workspace_bytes, void* stream_) {
  clear_error();
  int rc = diff_sizes(B, Hq, Hkv, N, d, scale);
  if (rc) return rc;
  if (!page_size_ok(page_size))
    return fail(ATTN_ERR_UNSUPPORTED, "page_size %d (16, 32, 64 or 128)", page_size);
  const int group = Hq / Hkv;
  if (group > kMaxDecodeGroup)
    return fail(ATTN_ERR_UNSUPPORTED, "query heads per kv head %d (at most %d)", group,
                kMaxDecodeGroup);
  if ((rc = diff_numbers(norm_weight, eps, out_scale))) return rc;
  if (B == 0) return ATTN_OK;  // no rows
  // N = 0: every context is empty, and its rows are still the caller's to have. They come of the
  // lengths alone; nothing else is used.
  const bool keys = N > 0;
  if (!cu_seqlens || !o || !lse || (keys && !block_table))
    return fail(ATTN_ERR_INVALID, "null pointer");
  if (!aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_INVALID, "tensors must be 16-byte aligned");
  if (keys && (rc = diff_checks(q, k, v, o, lse, lam, norm_weight, eps, out_scale))) return rc;
  if (keys && num_pages <= 0) return fail(ATTN_ERR_INVALID, "num_pages %d", num_pages);
  if (static_cast<long long>(num_pages) * Hkv >= (1ll << 31) || Hkv > 65535 || N > (1 << 30))
    return fail(ATTN_ERR_UNSUPPORTED, "page pool or context too large");
  const long long units =
      (N + DiffShare<64>::kTok - 1ll) / DiffShare<64>::kTok + DiffShare<64>::kStart;
  if (B > 65535 || static_cast<long long>(B) * Hkv >= (1ll << 31) / units)
    return fail(ATTN_ERR_UNSUPPORTED, "decode batch too large");
  if (!keys && no_device()) return ATTN_OK;  // nor are there device rows to fill
  const DiffDecodeLayout L = diff_layout(Hq, Hkv, d);
  if (keys && (!workspace || workspace_bytes < L.total || !aligned16(workspace)))
    return fail(ATTN_ERR_WORKSPACE, "workspace needs %zu bytes (16-byte aligned)", L.total);
  // Rows are written while other workers still read queries, lengths and pages.
  const int max_pages = (N + page_size - 1) / page_size;
  const size_t rows = static_cast<size_t>(B) * Hq;
  const size_t pool = keys ? static_cast<size_t>(num_pages) * Hkv * page_size * d * 2 : 0;
  const struct { const void* x; size_t bytes; } out[3] = {
      {o, rows * d * 2}, {lse, rows * 2 * sizeof(float)}, {workspace, keys ? L.total : 0}}, in[7] = {
      {q, keys ? rows * d * 2 : 0}, {k, pool}, {v, pool}, {lam, keys ? sizeof(float) * Hq : 0},
      {norm_weight, keys ? sizeof(float) * d : 0}, {cu_seqlens, sizeof(int32_t) * (B + size_t(1))},
      {block_table, sizeof(int32_t) * B * static_cast<size_t>(max_pages)}};
  for (int i = 0; i < 3; ++i) {
    bool shared = overlap(out[i].x, out[i].bytes, out[(i + 1) % 3].x, out[(i + 1) % 3].bytes);
    for (const auto& t : in) shared |= overlap(out[i].x, out[i].bytes, t.x, t.bytes);
    if (shared) return fail(ATTN_ERR_INVALID, "o, lse or workspace overlaps another tensor");
  }
  DiffDecodeParams p{};
  if ((rc = status_ptr(&p.status))) return rc;
  // The pools as [num_pages * Hkv][page_size][d], boxes of min(page_size, 64) rows.
  const uint64_t planes = static_cast<uint64_t>(num_pages) * Hkv;
  const uint32_t box = static_cast<uint32_t>(page_size < 64 ? page_size : 64);
  CUtensorMap tk{}, tv{};
  if (keys && (rc = encode_3d(&tk, k, d, page_size, planes, box))) return rc;
  if (keys && (rc = encode_3d(&tv, v, d, page_size, planes, box))) return rc;
  p.q = static_cast<const uint32_t*>(q);
  p.cu = cu_seqlens;
  p.table = block_table;
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.lam = lam;
  p.weight = norm_weight;
  if (keys) {
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.part_ml);
  }
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.group = group;
  p.page_shift = log2_exact(page_size);
  p.max_len = N;
  p.slots = L.slots;
  // The joining kernel: a CTA a group once the groups fill the GPU, else a CTA a head.
  p.join_heads = static_cast<long long>(B) * Hkv >= sms_or_default() ? group : 1;
  p.join_workers = static_cast<long long>(B) * Hkv > L.slots;
  p.scale_log2 = scale * kLog2e;
  p.eps = eps;
  p.out_scale = out_scale;
  p.timeout_ns = kTimeoutNs;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  cudaError_t e;
  if (d == 64)
    e = group <= 8 ? launch_one<64, 1>(tk, tv, p, stream) : launch_one<64, 2>(tk, tv, p, stream);
  else
    e = group <= 8 ? launch_one<128, 1>(tk, tv, p, stream) : launch_one<128, 2>(tk, tv, p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "differential decode launch");
  return ATTN_OK;
}

}  // extern "C"
