// norm.cuh — the norm y / sqrt(mean y^2 + eps) of the token rows and of differential attention's rows,
// for rows of any size that fp32 holds.
//
// Squares in fp32 overflow from |y| = 2^64 on and vanish below 2^-75. A row whose squares would is
// taken times a power of two first, and eps times its square, which leaves the quotient as it is. Other
// rows are not touched: their squares sum to the same bits, and the check is one a row.
#pragma once

namespace ta {

// The power of two for a row whose squares sum to ss. Below 2^-100 a sum may lack squares
// that vanished; from eps = 2^-70 on that is nothing beside D eps.
__device__ __forceinline__ float norm_scale(float ss, float eps) {
  if (!(ss <= 0x1p126f)) return 0x1p-70f;
  return ss < 0x1p-100f && eps < 0x1p-70f ? 0x1p90f : 1.f;
}

// 1 / sqrt(mean + eps) of a row of D channels taken times `by`, its squares summing to ss. A row of
// zeros with eps = 0 stays zero.
template <int D>
__device__ __forceinline__ float norm_factor(float ss, float by, float eps) {
  const float mean = ss * (1.f / D) + eps * by * by;
  return mean == 0.f ? 1.f : rsqrtf(mean);
}

}  // namespace ta
