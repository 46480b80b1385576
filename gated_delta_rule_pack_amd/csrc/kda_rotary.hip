// Rotary positions.
//
// With theta = pos_t w_i, the pair (a, b) of channels (i, i + r/2), or (2i, 2i + 1) when
// interleaved, becomes f (a cos theta - b sin theta, a sin theta + b cos theta) for i < r/2; the
// other channels pass through. The kernel reads and writes every element once, so it is bound by
// memory; the angles, which all heads of a token share, are made once per workgroup.
#include <hip/hip_runtime.h>

#include "kda_device.h"
#include "kda_linear.h"
#include "kda_rotary.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

template <int DT>
struct Elem;
template <>
struct Elem<kF32> {
  typedef float type;
};
template <>
struct Elem<kF16> {
  typedef _Float16 type;
};
template <>
struct Elem<kBF16> {
  typedef __bf16 type;
};

template <typename E, int VEC>
struct Vec {
  typedef E type __attribute__((ext_vector_type(VEC)));
};
template <typename E>
struct Vec<E, 1> {
  typedef E type;
};
template <int VEC, typename T>
__device__ __forceinline__ float get(const T& v, int i) {
  if constexpr (VEC == 1) return (float)v;
  else return (float)v[i];
}
template <int VEC, typename E, typename T>
__device__ __forceinline__ void set(T& v, int i, float x) {
  if constexpr (VEC == 1) v = (E)x;
  else v[i] = (E)x;
}

// A workgroup takes `tokens` tokens, all their heads. A row (one head of one token) is split into
// items: VEC pairs each (two vectors of VEC elements), then, unless in place, the vectors behind
// the rotated part.
template <int DT, int VEC>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const RotaryPlan p, int tokens, int copies) {
  typedef typename Elem<DT>::type E;
  typedef typename Vec<E, VEC>::type V;
  extern __shared__ float2 turn[];  // [tokens][half]: (c, s)
  const int half = p.rot_dim / 2, pairs = half / VEC, items = pairs + copies;
  const int first = blockIdx.x * tokens, count = min(tokens, p.T - first);
  for (int i = threadIdx.x; i < count * half; i += kThreads)
    turn[i] = rotation(p, first + i / half, i % half, p.inverse != 0);
  __syncthreads();
  const int rows = p.H[0] + p.H[1];
  for (int i = threadIdx.x; i < count * rows * items; i += kThreads) {
    const int u = i % items, row = i / items, t = row / rows, r = row % rows;
    const int which = r >= p.H[0];
    const int h = which ? r - p.H[0] : r;
    const E* in = reinterpret_cast<const E*>(p.in[which]) + (int64_t)(first + t) * p.in_t[which] + h * p.in_h[which];
    E* out = reinterpret_cast<E*>(p.out[which]) + (int64_t)(first + t) * p.out_t[which] + h * p.out_h[which];
    if (u >= pairs) {
      const int d = p.rot_dim + (u - pairs) * VEC;
      *reinterpret_cast<V*>(out + d) = *reinterpret_cast<const V*>(in + d);
      continue;
    }
    const int d0 = p.interleaved ? 2 * u * VEC : u * VEC;
    const int d1 = p.interleaved ? d0 + VEC : d0 + half;
    const V x = *reinterpret_cast<const V*>(in + d0), y = *reinterpret_cast<const V*>(in + d1);
    V xo, yo;
    const float2* cs = turn + t * half + u * VEC;
    if (!p.interleaved || VEC == 1) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float a = get<VEC>(x, j), b = get<VEC>(y, j), c = cs[j].x, s = cs[j].y;
        set<VEC, E>(xo, j, a * c - b * s);
        set<VEC, E>(yo, j, a * s + b * c);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {  // pair j: elements 2j and 2j + 1 of the two vectors in a row
        const int e = 2 * j;
        const float a = e < VEC ? get<VEC>(x, e % VEC) : get<VEC>(y, e % VEC);
        const float b = e < VEC ? get<VEC>(x, (e + 1) % VEC) : get<VEC>(y, (e + 1) % VEC);
        const float c = cs[j].x, s = cs[j].y;
        set<VEC, E>(e < VEC ? xo : yo, e % VEC, a * c - b * s);
        set<VEC, E>(e < VEC ? xo : yo, (e + 1) % VEC, a * s + b * c);
      }
    }
    *reinterpret_cast<V*>(out + d0) = xo;
    *reinterpret_cast<V*>(out + d1) = yo;
  }
}

template <int DT, int VEC>
int launch_vec(const RotaryPlan& p, hipStream_t s) {
  const bool in_place = p.in[0] == p.out[0] && (p.H[1] == 0 || p.in[1] == p.out[1]);
  const int copies = in_place ? 0 : (p.D - p.rot_dim) / VEC;
  const int tokens = p.T >= 4096 ? 4 : 1;
  const int grid = (p.T + tokens - 1) / tokens;
  const size_t lds = (size_t)tokens * (p.rot_dim / 2) * sizeof(float2);
  rotary_kernel<DT, VEC><<<grid, kThreads, lds, s>>>(p, tokens, copies);
  return (int)hipGetLastError();
}

// 16-byte accesses where the rows allow them, single elements otherwise.
template <int DT>
int launch_dt(const RotaryPlan& p, hipStream_t s) {
  constexpr int VEC = DT == kF32 ? 4 : 8;
  bool wide = p.rot_dim / 2 % VEC == 0 && p.D % VEC == 0;
  for (int i = 0; i < 2; ++i) {
    if (p.H[i] == 0) continue;
    wide = wide && (uintptr_t)p.in[i] % 16 == 0 && (uintptr_t)p.out[i] % 16 == 0 && p.in_t[i] % VEC == 0 &&
           p.in_h[i] % VEC == 0 && p.out_t[i] % VEC == 0 && p.out_h[i] % VEC == 0;
  }
  return wide ? launch_vec<DT, VEC>(p, s) : launch_vec<DT, 1>(p, s);
}

}  // namespace

int launch_rotary(const RotaryPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (p.dtype == kF32) return launch_dt<kF32>(p, s);
  if (p.dtype == kF16) return launch_dt<kF16>(p, s);
  return launch_dt<kBF16>(p, s);
}

}  // namespace kda
