// Device side of one rotation, shared by the rotary kernel and the linear step.
#pragma once

#include <hip/hip_runtime.h>

#include "kda_linear.h"

namespace kda {

// (factor cos theta, factor sin theta) of token t and frequency i, in 64 bits and rounded once; the sine negated for
// the transposed rotation. In fp32 the angle alone would be off by 0.06 radians at position 10^6, and reduced to a
// fraction of a turn in 64 bits before its rounding it would still add as much to a result's error as the result's own
// arithmetic (5.4e-8 rel-L2 of fp32 results instead of 4.2e-8). All heads of a token share it, so it costs little: 7
// tokens 4.1 us either way, 16384 tokens of 40 heads 65.2 and 65.4 us, of two heads with 128 angles each 15.4 and 16.8.
__device__ __forceinline__ float2 rotation(const RotaryPlan& p, int t, int i, bool inverse) {
  const double pos = p.positions_i64 ? (double)reinterpret_cast<const int64_t*>(p.positions)[t]
                                     : (double)reinterpret_cast<const int32_t*>(p.positions)[t];
  const double turns = pos * p.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
  double s, c;
  sincospi(2.0 * (turns - rint(turns)), &s, &c);
  return float2{(float)(p.factor * c), (float)(p.factor * (inverse ? -s : s))};
}

}  // namespace kda
