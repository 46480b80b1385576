// The gated delta rule with one decay for each head, recurrent form for single tokens:
// S <- e^g S, S <- S + beta (v - S k) k^T, o = scale S q, one token for each row of the call.
//
// A row reads and writes its V x K state once and little else, so the kernel is bound by memory. A workgroup takes
// one row's one head, issues all its state loads, prepares q and k (normalised where asked) in LDS meanwhile, and
// updates the state in registers, in fp32. Both sums over k come from the state as it was read,
// u = S k and w = S q, so that one exchange between lanes serves both: with delta = beta (v - e^g u) the new state is
// e^g S + delta k^T and o = scale (e^g w + delta (k . q)).
#include <hip/hip_runtime.h>

#include "kda_delta.h"
#include "kda_device.h"
#include "kda_unit.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 8 neighbouring elements of the state, as they lie in memory.
template <int SDT>
struct Raw8 {
  u32x4 x[SDT == kF32 ? 2 : 1];
};
template <int SDT>
__device__ __forceinline__ Raw8<SDT> load8(const void* base, int64_t at) {
  return *reinterpret_cast<const Raw8<SDT>*>(reinterpret_cast<const char*>(base) + at * (SDT == kF32 ? 4 : 2));
}
// In fp32, or zeros where `keep` is 0 (all bits set else): a slot that starts anew may hold anything.
template <int SDT>
__device__ __forceinline__ void unpack8(const Raw8<SDT>& r, uint32_t keep, f32x4& a, f32x4& b) {
  if constexpr (SDT == kF32) {
    a = __builtin_bit_cast(f32x4, r.x[0] & keep);
    b = __builtin_bit_cast(f32x4, r.x[1] & keep);
  } else if constexpr (SDT == kF16) {
    const f16x8 h = __builtin_bit_cast(f16x8, r.x[0] & keep);
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
__device__ __forceinline__ void store8(void* base, int64_t at, f32x4 a, f32x4 b) {
  Raw8<SDT> r;
  if constexpr (SDT == kF32) {
    r.x[0] = __builtin_bit_cast(u32x4, a), r.x[1] = __builtin_bit_cast(u32x4, b);
  } else if constexpr (SDT == kF16) {
    f16x8 h;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = (_Float16)a[j], h[4 + j] = (_Float16)b[j];
    r.x[0] = __builtin_bit_cast(u32x4, h);
  } else {
    bf16x8 h;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = to_bf16(a[j]), h[4 + j] = to_bf16(b[j]);
    r.x[0] = __builtin_bit_cast(u32x4, h);
  }
  *reinterpret_cast<Raw8<SDT>*>(reinterpret_cast<char*>(base) + at * (SDT == kF32 ? 4 : 2)) = r;
}
__device__ __forceinline__ float load_token(const void* base, int64_t at, int f16) {
  return f16 ? (float)reinterpret_cast<const _Float16*>(base)[at] : (float)reinterpret_cast<const __bf16*>(base)[at];
}
__device__ __forceinline__ void store_token(void* base, int64_t at, int f16, float x) {
  if (f16) reinterpret_cast<_Float16*>(base)[at] = (_Float16)x;
  else reinterpret_cast<__bf16*>(base)[at] = to_bf16(x);
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return (a[0] * b[0] + a[1] * b[1]) + (a[2] * b[2] + a[3] * b[3]); }

// The state as stored is a plane of kRows x kCols, columns adjacent: [V][K] or, K-first, [K][V].
// V-first: the lanes of a row sum over it. K-first: a lane holds 8 columns and walks rows; lanes and
// waves are summed, the waves through LDS.
template <int K, int V, int SDT, bool kKfirst>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(const DeltaPlan p) {
  __shared__ __align__(16) float sq[K], sk[K], sv[V];
  __shared__ __align__(16) float part[kKfirst ? 2 * kWaves : 1][V];
  __shared__ float skq;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n = blockIdx.x / p.H, h = blockIdx.x % p.H;
  // The row's own loads go out before its slot is known. Wave 0: q and k. Wave 1: v.
  constexpr int kOf = K / 64;
  float q[kOf], k[kOf], v[V / 64];
  if (wave == 0) {
#pragma unroll
    for (int j = 0; j < kOf; ++j) {
      q[j] = load_token(p.q, n * p.q_t + (h / p.group) * p.q_h + lane + 64 * j, p.f16);
      k[j] = load_token(p.k, n * p.k_t + (h / p.group) * p.k_h + lane + 64 * j, p.f16);
    }
  } else if (wave == 1) {
#pragma unroll
    for (int j = 0; j < V / 64; ++j) v[j] = load_token(p.v, n * p.v_t + h * p.v_h + lane + 64 * j, p.f16);
  }
  const int64_t slot = p.indices ? p.indices[n] : n;
  if (slot < 0 || slot >= p.num_slots) return;  // padding
  const uint32_t keep = !p.flags || p.flags[n] ? ~0u : 0u;
  const int64_t plane = slot * p.stride0 + (int64_t)h * K * V;

  constexpr int kCols = kKfirst ? V : K, kRows = kKfirst ? K : V;
  constexpr int kLanes = kCols / 8;        // lanes per row
  constexpr int kPer = kThreads / kLanes;  // rows at a time
  constexpr int kIters = kRows / kPer;
  static_assert(kRows % kPer == 0, "whole passes");
  const int col = (tid % kLanes) * 8;
  const int64_t at = plane + tid / kLanes * kCols + col;
  constexpr int kStep = kPer * kCols;
  Raw8<SDT> raw[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) raw[i] = load8<SDT>(p.state_in, at + i * kStep);
  float g = 0.f;
  if (p.g) {
    const int64_t i = p.g_per_token ? (int64_t)n * p.H + h : h;
    g = p.g_bf16 ? (float)reinterpret_cast<const __bf16*>(p.g)[i] : reinterpret_cast<const float*>(p.g)[i];
  }
  const int64_t ib = (int64_t)n * p.H + h;
  float beta = p.beta_bf16 ? (float)reinterpret_cast<const __bf16*>(p.beta)[ib] : reinterpret_cast<const float*>(p.beta)[ib];
  if (!(g <= 0.f)) beta = __builtin_nanf("");
  const float decay = __expf(g);

  if (wave == 0) {
    if (p.normalize) {
      const float rq = unit_factor(q), rk = unit_factor(k);
#pragma unroll
      for (int j = 0; j < kOf; ++j) q[j] *= rq, k[j] *= rk;
    }
    float kq = 0.f;
#pragma unroll
    for (int j = 0; j < kOf; ++j) {
      sq[lane + 64 * j] = q[j];
      sk[lane + 64 * j] = k[j];
      kq += k[j] * q[j];
    }
    kq = wave_sum(kq);
    if (lane == 0) skq = kq;
  } else if (wave == 1) {
#pragma unroll
    for (int j = 0; j < V / 64; ++j) sv[lane + 64 * j] = v[j];
  }
  __syncthreads();

  const float kq = skq;
  const int64_t out = n * p.o_t + h * p.o_h;
  if constexpr (!kKfirst) {
    const f32x4 k0 = *reinterpret_cast<const f32x4*>(sk + col), k1 = *reinterpret_cast<const f32x4*>(sk + col + 4);
    const f32x4 q0 = *reinterpret_cast<const f32x4*>(sq + col), q1 = *reinterpret_cast<const f32x4*>(sq + col + 4);
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int row = tid / kLanes + i * kPer;
      f32x4 a, b;
      unpack8<SDT>(raw[i], keep, a, b);
      const float u = lane_sum(dot4(a, k0) + dot4(b, k1), kLanes), w = lane_sum(dot4(a, q0) + dot4(b, q1), kLanes);
      const float delta = beta * (sv[row] - decay * u);
      store8<SDT>(p.state_out, at + i * kStep, a * decay + k0 * delta, b * decay + k1 * delta);
      if (tid % kLanes == 0) store_token(p.out, out + row, p.f16, p.scale * (decay * w + delta * kq));
    }
  } else {
    f32x4 u0 = zero4(), u1 = zero4(), w0 = zero4(), w1 = zero4();
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int row = tid / kLanes + i * kPer;
      const float k = sk[row], q = sq[row];
      f32x4 a, b;
      unpack8<SDT>(raw[i], keep, a, b);
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
      *reinterpret_cast<f32x4*>(&part[wave][col]) = u0, *reinterpret_cast<f32x4*>(&part[wave][col + 4]) = u1;
      *reinterpret_cast<f32x4*>(&part[kWaves + wave][col]) = w0, *reinterpret_cast<f32x4*>(&part[kWaves + wave][col + 4]) = w1;
    }
    __syncthreads();
    f32x4 d0, d1;
    u0 = u1 = zero4();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      u0 += *reinterpret_cast<const f32x4*>(&part[w][col]);
      u1 += *reinterpret_cast<const f32x4*>(&part[w][col + 4]);
    }
    d0 = (*reinterpret_cast<const f32x4*>(sv + col) - u0 * decay) * beta;
    d1 = (*reinterpret_cast<const f32x4*>(sv + col + 4) - u1 * decay) * beta;
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const float k = sk[tid / kLanes + i * kPer];
      f32x4 a, b;
      unpack8<SDT>(raw[i], keep, a, b);
      store8<SDT>(p.state_out, at + i * kStep, a * decay + d0 * k, b * decay + d1 * k);
    }
    if (tid < V) {
      float u = 0.f, w = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) u += part[i][tid], w += part[kWaves + i][tid];
      store_token(p.out, out + tid, p.f16, p.scale * (decay * w + beta * (sv[tid] - decay * u) * kq));
    }
  }
}

template <int K, int V, int SDT>
int launch_sdt(const DeltaPlan& p, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.N * p.H);
  if (p.kfirst) delta_step_kernel<K, V, SDT, true><<<grid, kThreads, 0, s>>>(p);
  else delta_step_kernel<K, V, SDT, false><<<grid, kThreads, 0, s>>>(p);
  return (int)hipGetLastError();
}

template <int K, int V>
int launch_kv(const DeltaPlan& p, hipStream_t s) {
  if (p.state_dtype == kF32) return launch_sdt<K, V, kF32>(p, s);
  if (p.state_dtype == kF16) return launch_sdt<K, V, kF16>(p, s);
  return launch_sdt<K, V, kBF16>(p, s);
}

}  // namespace

int launch_delta_step(const DeltaPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (p.K == 128) return p.V == 128 ? launch_kv<128, 128>(p, s) : launch_kv<128, 64>(p, s);
  return p.V == 128 ? launch_kv<64, 128>(p, s) : launch_kv<64, 64>(p, s);
}

}  // namespace kda
