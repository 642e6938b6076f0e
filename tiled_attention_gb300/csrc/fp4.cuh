// fp4.cuh — the 4-bit cache format and its conversions.
//
// A pool is [num_pages, Hkv] blocks of page_size tokens: first the tokens' codes, D/2 bytes
// each (channel 2c in the low nibble of byte c, 2c + 1 in the high one), then their scales,
// D/16 bytes each, one E4M3 scale per 16 channels. A value is code * scale * the tensor's fp32
// scale, where a code is E2M1: {0, 0.5, 1, 1.5, 2, 3, 4, 6} and a sign. 4.5 bits an element.
//
// Why this format on GB300: the hardware converts E2M1 pairs and E4M3 pairs to f16 pairs in
// one instruction each, and code * scale (2 + 4 significant bits, magnitudes from 2^-10 to
// 2688) is exact in f16, so a dequantized operand costs one conversion and one packed
// multiply per two elements and loses nothing.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace ta {

constexpr int kFp4Block = 16;  // channels per scale
constexpr float kFp4Large = 4096.f;  // past every value of code * scale (448 * 6 = 2688)

__host__ __device__ constexpr int fp4_code_bytes(int d) { return d / 2; }
__host__ __device__ constexpr int fp4_scale_bytes(int d) { return d / kFp4Block; }
// Bytes of one token of one kv head: 72 at d = 128, 36 at d = 64.
__host__ __device__ constexpr int fp4_row_bytes(int d) {
  return fp4_code_bytes(d) + fp4_scale_bytes(d);
}

// The larger one, or NaN if either is.
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Four E2M1 pairs (the bytes of w, low nibble first) to f16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two E4M3 codes (low byte first) to an f16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t h;
  asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}"
      : "=r"(h)
      : "r"(two));
  return h;
}

// Two fp32 -> two E4M3 codes (lo in the low byte), round to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight fp32 -> eight E2M1 codes, round to nearest even, saturating at 6; x[0].x in the low
// nibble of the low byte.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float2 (&x)[4]) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(r)
      : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y),
        "f"(x[3].x), "f"(x[3].y));
  return r;
}

}  // namespace ta
