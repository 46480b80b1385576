// Device side of one rotation, shared by the rotary kernel and the linear step.
#pragma once

#include <hip/hip_runtime.h>

#include "kda_linear.h"

namespace kda {

// (factor cos theta, factor sin theta) of token t and frequency i; the sine negated for the
// transposed rotation. The angle is a 64-bit product reduced to a fraction of a turn before it
// is rounded to fp32: at position 10^6 its fp32 rounding alone would be off by 0.06 radians.
__device__ __forceinline__ float2 rotation(const RotaryPlan& p, int t, int i, bool inverse) {
  const double pos = p.positions_i64 ? (double)reinterpret_cast<const int64_t*>(p.positions)[t]
                                     : (double)reinterpret_cast<const int32_t*>(p.positions)[t];
  const double turns = pos * p.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
  float s, c;
  sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
  return float2{p.factor * c, p.factor * (inverse ? -s : s)};
}

}  // namespace kda
