// Length of a key or query that one wave holds, shared by the gated delta rule's kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "kda_delta.h"

namespace kda {

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d));
  return x;
}
// 1 / sqrt(sum x^2 + eps) over the wave's K values, scaled by their largest power of two so that no finite
// row overflows.
template <int N>
__device__ __forceinline__ float unit_factor(const float (&x)[N]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(x[i]));
  m = wave_max(m);
  const int e = m > 0.f && m < INFINITY ? __builtin_amdgcn_frexp_expf(m) : 0;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float y = __builtin_amdgcn_ldexpf(x[i], -e);
    s += y * y;
  }
  return __builtin_amdgcn_ldexpf(rsqrtf(wave_sum(s) + __builtin_amdgcn_ldexpf(kNormEps, -2 * e)), -e);
}

}  // namespace kda
