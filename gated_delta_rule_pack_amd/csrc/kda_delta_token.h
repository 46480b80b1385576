// The gated delta rule's recurrent form for one token of one head: S <- e^g S, S <- S + beta (v - S k) k^T, o = scale S q.
//
// A workgroup reads the V x K state (or a slice of V) once, all its loads issued together, prepares q and k (normalised
// where asked) in LDS meanwhile, and updates the state in registers, in fp32. Both sums over k come from the state as
// it was read, u = S k and w = S q, so that one exchange between lanes serves both: with delta = beta (v - e^g u) the
// new state is e^g S + delta k^T and o = scale (e^g w + delta (k . q)).
#pragma once

#include <hip/hip_runtime.h>

#include "kda_delta.h"
#include "kda_device.h"
#include "kda_unit.h"

namespace kda {

typedef _Float16 halves __attribute__((ext_vector_type(8)));

// 8 neighbouring elements of the state, as they lie in memory.
template <int SDT>
struct StateRaw {
  u32x4 x[SDT == kF32 ? 2 : 1];
};
template <int SDT>
__device__ __forceinline__ StateRaw<SDT> load_raw(const void* base, int64_t at) {
  return *reinterpret_cast<const StateRaw<SDT>*>(reinterpret_cast<const char*>(base) + at * (SDT == kF32 ? 4 : 2));
}
// In fp32, or zeros where `keep` is 0 (all bits set else): a slot that starts anew may hold anything.
template <int SDT>
__device__ __forceinline__ void unpack_raw(const StateRaw<SDT>& r, uint32_t keep, f32x4& a, f32x4& b) {
  if constexpr (SDT == kF32) {
    a = __builtin_bit_cast(f32x4, r.x[0] & keep);
    b = __builtin_bit_cast(f32x4, r.x[1] & keep);
  } else if constexpr (SDT == kF16) {
    const halves h = __builtin_bit_cast(halves, r.x[0] & keep);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = (float)h[j], b[j] = (float)h[4 + j];
  } else {
    const u32x4 u = r.x[0] & keep;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x = u[j], y = u[2 + j];
      a[2 * j] = __builtin_bit_cast(float, x << 16), a[2 * j + 1] = __builtin_bit_cast(float, x & 0xffff0000u);
      b[2 * j] = __builtin_bit_cast(float, y << 16), b[2 * j + 1] = __builtin_bit_cast(float, y & 0xffff0000u);
    }
  }
}
template <int SDT>
__device__ __forceinline__ void store_raw(void* base, int64_t at, f32x4 a, f32x4 b) {
  StateRaw<SDT> r;
  if constexpr (SDT == kF32) {
    r.x[0] = __builtin_bit_cast(u32x4, a), r.x[1] = __builtin_bit_cast(u32x4, b);
  } else if constexpr (SDT == kF16) {
    halves h;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = (_Float16)a[j], h[4 + j] = (_Float16)b[j];
    r.x[0] = __builtin_bit_cast(u32x4, h);
  } else {
    bf16x8 h;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = to_bf16(a[j]), h[4 + j] = to_bf16(b[j]);
    r.x[0] = __builtin_bit_cast(u32x4, h);
  }
  *reinterpret_cast<StateRaw<SDT>*>(reinterpret_cast<char*>(base) + at * (SDT == kF32 ? 4 : 2)) = r;
}
__device__ __forceinline__ float token_float(uint16_t x, int f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, x) : __uint_as_float((uint32_t)x << 16);
}
__device__ __forceinline__ void store_token(void* base, int64_t at, int f16, float x) {
  if (f16) reinterpret_cast<_Float16*>(base)[at] = (_Float16)x;
  else reinterpret_cast<__bf16*>(base)[at] = to_bf16(x);
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return (a[0] * b[0] + a[1] * b[1]) + (a[2] * b[2] + a[3] * b[3]); }

template <int K, int V, int kThreads>
struct TokenShared {
  static constexpr int kWaves = kThreads / 64;
  alignas(16) float q[K], k[K], v[V];
  alignas(16) float part[2 * kWaves][V];  // K-first: the waves' sums
  float kq;
};
template <int K, int V>
constexpr int kTokenRow = (K > V ? K : V) / 64;
// The token's rows on their way, as they are stored: x = q and k in wave 0, x = v in wave 1.
template <int K, int V>
__device__ __forceinline__ void token_rows(const DeltaPlan& p, int64_t token, int h, int v0, int wave, int lane,
                                           uint16_t (&x)[kTokenRow<K, V>], uint16_t (&k)[K / 64]) {
  if (wave > 1) return;
  const uint16_t* row = wave == 0 ? reinterpret_cast<const uint16_t*>(p.q) + token * p.q_t + (h / p.group) * p.q_h
                                  : reinterpret_cast<const uint16_t*>(p.v) + token * p.v_t + h * p.v_h + v0;
#pragma unroll
  for (int j = 0; j < kTokenRow<K, V>; ++j) x[j] = K == V || 64 * j < (wave == 0 ? K : V) ? row[lane + 64 * j] : 0;
  if (wave > 0) return;
  row = reinterpret_cast<const uint16_t*>(p.k) + token * p.k_t + (h / p.group) * p.k_h;
#pragma unroll
  for (int j = 0; j < K / 64; ++j) k[j] = row[lane + 64 * j];
}

// Channels v0 to v0 + V of the token. The state is a plane of rows with adjacent columns, [V][K] or, K-first, [K][V];
// `from` and `to` are the planes' places in state_in and state_out (to < 0: none). Where keep is 0 nothing is kept of
// what was read, and where kMayBeNew is set nothing read.
// V-first: the lanes of a row sum over it. K-first: a lane holds 8 columns and walks rows; lanes and waves are summed, the
// waves through LDS.
template <int K, int V, int SDT, bool kKfirst, int kThreads, bool kMayBeNew>
__device__ __forceinline__ void delta_token(const DeltaPlan& p, TokenShared<K, V, kThreads>& sh, const uint16_t (&x)[kTokenRow<K, V>],
                                            const uint16_t (&kx)[K / 64], int64_t token, int h, int v0, int64_t from, int64_t to, uint32_t keep, int tid) {
  constexpr int kWaves = kThreads / 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  constexpr int kCols = kKfirst ? V : K, kRows = kKfirst ? K : V;
  constexpr int kLanes = kCols / 8;        // lanes per row
  constexpr int kPer = kThreads / kLanes;  // rows at a time
  constexpr int kIters = kRows / kPer;
  static_assert(kRows % kPer == 0, "whole passes");
  const int col = (tid % kLanes) * 8, ld = kKfirst ? p.V : K, step = kPer * ld;
  const int64_t at = (int64_t)(tid / kLanes) * ld + col + (kKfirst ? v0 : v0 * K);
  StateRaw<SDT> raw[kIters] = {};
  if (!kMayBeNew || keep) {
#pragma unroll
    for (int i = 0; i < kIters; ++i) raw[i] = load_raw<SDT>(p.state_in, from + at + i * step);
  }
  float g = 0.f;
  const int64_t ib = token * p.H + h;
  if (p.g) {
    const int64_t i = p.g_per_token ? ib : h;
    g = p.g_bf16 ? (float)reinterpret_cast<const __bf16*>(p.g)[i] : reinterpret_cast<const float*>(p.g)[i];
  }
  float beta = p.beta_bf16 ? (float)reinterpret_cast<const __bf16*>(p.beta)[ib] : reinterpret_cast<const float*>(p.beta)[ib];
  if (!(g <= 0.f)) beta = __builtin_nanf("");
  const float decay = __expf(g);

  if (wave == 0) {
    float q[K / 64], k[K / 64];
#pragma unroll
    for (int j = 0; j < K / 64; ++j) q[j] = token_float(x[j], p.f16), k[j] = token_float(kx[j], p.f16);
    if (p.normalize) {
      const float rq = unit_factor(q), rk = unit_factor(k);
#pragma unroll
      for (int j = 0; j < K / 64; ++j) q[j] *= rq, k[j] *= rk;
    }
    float kq = 0.f;
#pragma unroll
    for (int j = 0; j < K / 64; ++j) {
      sh.q[lane + 64 * j] = q[j];
      sh.k[lane + 64 * j] = k[j];
      kq += k[j] * q[j];
    }
    kq = wave_sum(kq);
    if (lane == 0) sh.kq = kq;
  } else if (wave == 1) {
#pragma unroll
    for (int j = 0; j < V / 64; ++j) sh.v[lane + 64 * j] = token_float(x[j], p.f16);
  }
  __syncthreads();

  const float kq = sh.kq;
  const int64_t out = token * p.o_t + h * p.o_h + v0;
  if constexpr (!kKfirst) {
    const f32x4 k0 = *reinterpret_cast<const f32x4*>(sh.k + col), k1 = *reinterpret_cast<const f32x4*>(sh.k + col + 4);
    const f32x4 q0 = *reinterpret_cast<const f32x4*>(sh.q + col), q1 = *reinterpret_cast<const f32x4*>(sh.q + col + 4);
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int row = tid / kLanes + i * kPer;
      f32x4 a, b;
      unpack_raw<SDT>(raw[i], keep, a, b);
      const float u = lane_sum(dot4(a, k0) + dot4(b, k1), kLanes), w = lane_sum(dot4(a, q0) + dot4(b, q1), kLanes);
      const float delta = beta * (sh.v[row] - decay * u);
      if (to >= 0) store_raw<SDT>(p.state_out, to + at + i * step, a * decay + k0 * delta, b * decay + k1 * delta);
      if (tid % kLanes == 0) store_token(p.out, out + row, p.f16, p.scale * (decay * w + delta * kq));
    }
  } else {
    f32x4 u0 = zero4(), u1 = zero4(), w0 = zero4(), w1 = zero4();
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int row = tid / kLanes + i * kPer;
      const float k = sh.k[row], q = sh.q[row];
      f32x4 a, b;
      unpack_raw<SDT>(raw[i], keep, a, b);
      u0 += a * k, u1 += b * k;
      w0 += a * q, w1 += b * q;
    }
    // Over the lanes of one column: half rows, rows and half waves.
    const auto column_sum = [](float x) __attribute__((always_inline)) {
      if (kLanes == 8) x += moved<0x128>(x);  // row_ror 8
      return add_far(add_far(x, 16), 32);
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u0[j] = column_sum(u0[j]), u1[j] = column_sum(u1[j]);
      w0[j] = column_sum(w0[j]), w1[j] = column_sum(w1[j]);
    }
    if (lane < kLanes) {
      *reinterpret_cast<f32x4*>(&sh.part[wave][col]) = u0, *reinterpret_cast<f32x4*>(&sh.part[wave][col + 4]) = u1;
      *reinterpret_cast<f32x4*>(&sh.part[kWaves + wave][col]) = w0, *reinterpret_cast<f32x4*>(&sh.part[kWaves + wave][col + 4]) = w1;
    }
    __syncthreads();
    f32x4 d0, d1;
    u0 = u1 = zero4();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      u0 += *reinterpret_cast<const f32x4*>(&sh.part[w][col]);
      u1 += *reinterpret_cast<const f32x4*>(&sh.part[w][col + 4]);
    }
    d0 = (*reinterpret_cast<const f32x4*>(sh.v + col) - u0 * decay) * beta;
    d1 = (*reinterpret_cast<const f32x4*>(sh.v + col + 4) - u1 * decay) * beta;
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const float k = sh.k[tid / kLanes + i * kPer];
      f32x4 a, b;
      unpack_raw<SDT>(raw[i], keep, a, b);
      if (to >= 0) store_raw<SDT>(p.state_out, to + at + i * step, a * decay + d0 * k, b * decay + d1 * k);
    }
    if (tid < V) {
      float u = 0.f, w = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) u += sh.part[i][tid], w += sh.part[kWaves + i][tid];
      store_token(p.out, out + tid, p.f16, p.scale * (decay * w + beta * (sh.v[tid] - decay * u) * kq));
    }
  }
}

}  // namespace kda
