// diff.h — argument checks the differential attention entry points share (diff.cu).
#pragma once

namespace ta {

int diff_sizes(int B, int Hq, int Hkv, int n, int d, float scale);
// out_scale, and eps where there is a norm.
int diff_numbers(const float* weight, float eps, float out_scale);
// Pointers (weight may be null) and diff_numbers.
int diff_checks(const void* q, const void* k, const void* v, const void* o, const float* lse,
                const float* lam, const float* weight, float eps, float out_scale);

}  // namespace ta
