// Sums over lanes, and the length of a key or query that one wave holds.
#pragma once

#include <hip/hip_runtime.h>

#include "kda_delta.h"

namespace kda {

template <int kCtrl>
__device__ __forceinline__ float moved(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kCtrl, 0xf, 0xf, true));
}
template <int kCtrl>
__device__ __forceinline__ double moved(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, kCtrl, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), kCtrl, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// x and that of the lane 16 or 32 away, added: exchanges of rows and of half waves.
__device__ __forceinline__ float add_far(float x, int d) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto y = d == 16 ? __builtin_amdgcn_permlane16_swap(u, u, false, false) : __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a = y[0], b = y[1];
  return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}
__device__ __forceinline__ double add_far(double x, int d) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = u, hi = u >> 32;
  const auto l = d == 16 ? __builtin_amdgcn_permlane16_swap(lo, lo, false, false) : __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
  const auto h = d == 16 ? __builtin_amdgcn_permlane16_swap(hi, hi, false, false) : __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
  const uint64_t a = (uint64_t)h[0] << 32 | l[0], b = (uint64_t)h[1] << 32 | l[1];
  return __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b);
}
// The sum over `lanes` neighbours (a power of two), in each of them, without a pass through LDS.
template <typename X>
__device__ __forceinline__ X lane_sum(X x, int lanes) {
  if (lanes > 1) x += moved<0xb1>(x);   // quad_perm 1 0 3 2
  if (lanes > 2) x += moved<0x4e>(x);   // quad_perm 2 3 0 1
  if (lanes > 4) x += moved<0x141>(x);  // half a row mirrored: its quads are uniform by now
  if (lanes > 8) x += moved<0x140>(x);  // a row of 16 mirrored
  if (lanes > 16) x = add_far(x, 16);
  if (lanes > 32) x = add_far(x, 32);
  return x;
}
__device__ __forceinline__ float wave_sum(float x) { return lane_sum(x, 64); }
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
