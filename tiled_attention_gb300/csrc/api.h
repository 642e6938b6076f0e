// api.h — host helpers shared by the translation units that implement include/attn.h: error
// messages, the device status word and argument checks. Defined in api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace ta {

// Sets the calling thread's message and returns `code`.
int fail(int code, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);
void clear_error();

// Address of the current device's status word.
int status_ptr(int** out);
// Streaming multiprocessors of the current device, or 152 when no device is visible.
int sms_or_default();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Whether two tensors of an and bn bytes share any (a null one shares none).
inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && an && bn && x < y + bn && y < x + an;
}
inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Page sizes of the paged kinds: multiples of the 8-row swizzle atom that divide the
// 128-row prefill tile and either divide or are twice the 64-row decode stage.
inline bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

// log2 of a power of two (the page sizes page_size_ok accepts).
inline int log2_exact(int p) {
  int s = 0;
  while ((1 << s) < p) ++s;
  return s;
}

constexpr unsigned long long kTimeoutNs = 2000000000ull;  // 2 s per pipeline wait
constexpr int kMaxDecodeGroup = 16;    // query heads per kv head: the rows of one MMA tile
constexpr float kLog2e = 1.4426950408889634f;

}  // namespace ta
