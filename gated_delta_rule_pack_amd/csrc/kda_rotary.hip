// Rotary positions.
//
// With theta = pos_t w_i, the pair (a, b) of channels (i, i + r/2), or (2i, 2i + 1) when
// interleaved, becomes f (a cos theta - b sin theta, a sin theta + b cos theta) for i < r/2; the
// other channels pass through. The kernel reads and writes every element once, so in 16-byte
// vectors it is bound by memory; the angles, which all heads of a token share, are made once per workgroup.
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

// Rotates one vector pair: VEC pairs (a, b), x and y as they lie in the row.
template <int VEC, typename E, typename V>
__device__ __forceinline__ void turn_pair(const V& x, const V& y, const float2 (&cs)[VEC], bool interleaved, V& xo, V& yo) {
  if (VEC == 1 || !interleaved) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float a = get<VEC>(x, j), b = get<VEC>(y, j);
      set<VEC, E>(xo, j, a * cs[j].x - b * cs[j].y);
      set<VEC, E>(yo, j, a * cs[j].y + b * cs[j].x);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {  // pair j: elements 2j and 2j + 1 of the two vectors in a row
      const int e = 2 * j;
      const V& from = e < VEC ? x : y;
      V& to = e < VEC ? xo : yo;
      const float a = get<VEC>(from, e % VEC), b = get<VEC>(from, (e + 1) % VEC);
      set<VEC, E>(to, e % VEC, a * cs[j].x - b * cs[j].y);
      set<VEC, E>(to, (e + 1) % VEC, a * cs[j].y + b * cs[j].x);
    }
  }
}

template <typename E>
__device__ __forceinline__ const E* in_row(const RotaryPlan& p, int t, int r) {
  const int which = r >= p.H[0], h = which ? r - p.H[0] : r;
  return reinterpret_cast<const E*>(p.in[which]) + t * p.in_t[which] + h * p.in_h[which];
}
template <typename E>
__device__ __forceinline__ E* out_row(const RotaryPlan& p, int t, int r) {
  const int which = r >= p.H[0], h = which ? r - p.H[0] : r;
  return reinterpret_cast<E*>(p.out[which]) + t * p.out_t[which] + h * p.out_h[which];
}

// 16-byte vectors. A row (one head of one token) is split into items of two vectors: a vector pair
// to rotate, or two that pass through. A thread keeps one item of one token, whose angles it holds in
// registers, and walks the heads `groups` apart, kAhead rows in flight. A workgroup takes `tokens`
// tokens; its angles are made once, by all threads, and meet in LDS. Half of each of 40 heads of 128
// channels at 16384 tokens (336 MB) takes 66 us, 5.1 TB/s.
constexpr int kAhead = 4;
template <int DT, int VEC>
__global__ __launch_bounds__(kThreads) void rotary_wide(const RotaryPlan p, int tokens, int pairs, int items, int groups) {
  typedef typename Elem<DT>::type E;
  typedef typename Vec<E, VEC>::type V;
  extern __shared__ float2 turn[];  // [tokens][half]
  const int half = p.rot_dim / 2, rows = p.H[0] + p.H[1];
  const int first = blockIdx.x * tokens, count = min(tokens, p.T - first);
  for (int i = threadIdx.x; i < count * half; i += kThreads)
    turn[i] = rotation(p, first + i / half, i % half, p.inverse != 0);
  __syncthreads();
  const int u = threadIdx.x % items, r0 = threadIdx.x / items % groups, t = threadIdx.x / items / groups;
  if (t >= count) return;
  const bool rotate = u < pairs;
  int d0, d1;
  if (!rotate) d0 = p.rot_dim + (u - pairs) * 2 * VEC, d1 = d0 + VEC < p.D ? d0 + VEC : d0;
  else if (p.interleaved) d0 = 2 * u * VEC, d1 = d0 + VEC;
  else d0 = u * VEC, d1 = d0 + half;
  float2 cs[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) cs[j] = rotate ? turn[t * half + u * VEC + j] : float2{1.f, 0.f};
  for (int r = r0; r < rows; r += groups * kAhead) {
    V x[kAhead], y[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (r + j * groups >= rows) break;
      const E* in = in_row<E>(p, first + t, r + j * groups);
      x[j] = *reinterpret_cast<const V*>(in + d0);
      y[j] = *reinterpret_cast<const V*>(in + d1);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (r + j * groups >= rows) break;
      E* out = out_row<E>(p, first + t, r + j * groups);
      if (rotate) {
        V xo, yo;
        turn_pair<VEC, E>(x[j], y[j], cs, p.interleaved, xo, yo);
        x[j] = xo, y[j] = yo;
      }
      *reinterpret_cast<V*>(out + d0) = x[j];
      *reinterpret_cast<V*>(out + d1) = y[j];
    }
  }
}

// Single elements, for rows that 16-byte accesses do not fit: a workgroup for each token, items of one
// pair or one channel that passes through. Bound by its instructions, not by memory: 16384 tokens of 40 heads in
// 16 bits take 136 us at D = 80 with 40 channels rotated (1.5 TB/s), 175 us at D = 96 with 24 (1.4 TB/s); 98 and 127
// where a repeated call finds them in the memory-side cache.
template <int DT>
__global__ __launch_bounds__(kThreads) void rotary_narrow(const RotaryPlan p, int copies) {
  typedef typename Elem<DT>::type E;
  extern __shared__ float2 turn[];  // [half]
  const int half = p.rot_dim / 2, items = half + copies, t = blockIdx.x;
  for (int i = threadIdx.x; i < half; i += kThreads) turn[i] = rotation(p, t, i, p.inverse != 0);
  __syncthreads();
  for (int i = threadIdx.x; i < (p.H[0] + p.H[1]) * items; i += kThreads) {
    const int u = i % items, r = i / items;
    const E* in = in_row<E>(p, t, r);
    E* out = out_row<E>(p, t, r);
    if (u >= half) {
      out[p.rot_dim + u - half] = in[p.rot_dim + u - half];
      continue;
    }
    const int d0 = p.interleaved ? 2 * u : u, d1 = p.interleaved ? d0 + 1 : d0 + half;
    const E x = in[d0], y = in[d1];
    E xo, yo;
    const float2 cs[1] = {turn[u]};
    turn_pair<1, E>(x, y, cs, false, xo, yo);
    out[d0] = xo;
    out[d1] = yo;
  }
}

// 16-byte accesses where the rows allow them, single elements otherwise.
template <int DT>
int launch_dt(const RotaryPlan& p, hipStream_t s) {
  constexpr int VEC = DT == kF32 ? 4 : 8;
  const int half = p.rot_dim / 2;
  const bool in_place = p.in[0] == p.out[0] && (p.H[1] == 0 || p.in[1] == p.out[1]);
  bool wide = half % VEC == 0 && p.D % VEC == 0;
  for (int i = 0; i < 2; ++i) {
    if (p.H[i] == 0) continue;
    wide = wide && (uintptr_t)p.in[i] % 16 == 0 && (uintptr_t)p.out[i] % 16 == 0 && p.in_t[i] % VEC == 0 &&
           p.in_h[i] % VEC == 0 && p.out_t[i] % VEC == 0 && p.out_h[i] % VEC == 0;
  }
  const int copies = in_place ? 0 : p.D - p.rot_dim;
  if (!wide) {
    rotary_narrow<DT><<<p.T, kThreads, half * sizeof(float2), s>>>(p, copies);
    return (int)hipGetLastError();
  }
  const int pairs = half / VEC, items = pairs + (copies / VEC + 1) / 2;  // at most 1024 / 4 / 2
  // Four tokens share a workgroup's start where there are enough to fill the chip.
  const int tokens = p.T >= 2048 && items <= kThreads / 4 ? 4 : 1;
  const int groups = kThreads / (items * tokens);
  rotary_wide<DT, VEC><<<(p.T + tokens - 1) / tokens, kThreads, (size_t)tokens * half * sizeof(float2), s>>>(p, tokens, pairs, items, groups);
  return (int)hipGetLastError();
}

}  // namespace

// A launch counts its work-items in 32 bits, so it takes 2^22 tokens at most.
int launch_rotary(const RotaryPlan& whole, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  constexpr int64_t kMost = 1 << 22;
  const int64_t size = whole.dtype == kF32 ? 4 : 2;
  for (int64_t first = 0; first < whole.T; first += kMost) {
    RotaryPlan p = whole;
    p.T = (int)(whole.T - first < kMost ? whole.T - first : kMost);
    for (int i = 0; i < 2; ++i) {
      if (p.H[i] == 0) continue;
      p.in[i] = static_cast<const char*>(p.in[i]) + first * p.in_t[i] * size;
      p.out[i] = static_cast<char*>(p.out[i]) + first * p.out_t[i] * size;
    }
    p.positions = static_cast<const char*>(p.positions) + first * (p.positions_i64 ? 8 : 4);
    const int error = p.dtype == kF32 ? launch_dt<kF32>(p, s) : p.dtype == kF16 ? launch_dt<kF16>(p, s) : launch_dt<kBF16>(p, s);
    if (error) return error;
  }
  return 0;
}

}  // namespace kda
