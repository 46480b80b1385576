// Linear attention with a decay for each head, recurrent form for single tokens:
// S <- e^g S + v k^T, o = scale S q, one token for each row of the call.
//
// A row reads and writes its V x K state once and little else, so the kernel is bound by memory.
// A workgroup takes one row's one head, issues all its state loads, prepares q and k (rotated in
// fp32 where the call has positions) in LDS meanwhile, and updates the state in registers, in fp32.
// 500 rows at H = 32, fp32 (2.1 GB): 415 us, 5.1 TB/s, the rate of a large copy; 512 rows at H = 12,
// bf16 (402 MB): 68 us, 5.9 TB/s, K-first 66 us; 64 rows at H = 12, fp32: 20 us, 5.1 TB/s.
#include <hip/hip_runtime.h>

#include "kda_device.h"
#include "kda_linear.h"
#include "kda_rotary.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// Eight adjacent state elements.
template <int SDT>
__device__ __forceinline__ void load8(const void* base, int64_t at, f32x4& a, f32x4& b) {
  a = load_state4<SDT>(base, at);
  b = load_state4<SDT>(base, at + 4);
}
template <int SDT>
__device__ __forceinline__ void store8(void* base, int64_t at, f32x4 a, f32x4 b) {
  store_state4<SDT>(base, at, a);
  store_state4<SDT>(base, at + 4, b);
}

// The state as stored is a plane of kRows x kCols, columns adjacent: [V][K] or, K-first, [K][V].
// V-first: the lanes of a row sum over it. K-first: a lane holds 8 columns and walks rows; lanes and
// waves are summed, the waves through LDS.
template <int K, int V, int SDT, bool kKfirst>
__global__ __launch_bounds__(kThreads) void linear_step_kernel(const LinearPlan p) {
  __shared__ __align__(16) float sq[K], sk[K], sv[V];
  __shared__ __align__(16) float part[kKfirst ? kWaves : 1][V];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int64_t slot = p.indices ? p.indices[n] : n;
  if (slot < 0 || slot >= p.num_slots) return;  // padding
  const bool old = !p.flags || p.flags[n];
  const int64_t plane = slot * p.stride0 + (int64_t)h * K * V;

  constexpr int kCols = kKfirst ? V : K, kRows = kKfirst ? K : V;
  constexpr int kLanes = kCols / 8;        // lanes per row
  constexpr int kPer = kThreads / kLanes;  // rows at a time
  constexpr int kIters = kRows / kPer;
  static_assert(kRows % kPer == 0, "whole passes");
  const int col = (tid % kLanes) * 8;
  const int64_t at = plane + tid / kLanes * kCols + col;
  constexpr int kStep = kPer * kCols;
  f32x4 a[kIters], b[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) a[i] = b[i] = zero4();
  if (old) {
#pragma unroll
    for (int i = 0; i < kIters; ++i) load8<SDT>(p.state_in, at + i * kStep, a[i], b[i]);
  }

  const __bf16* q = reinterpret_cast<const __bf16*>(p.q) + n * p.q_t + (h / p.group) * p.q_h;
  const __bf16* k = reinterpret_cast<const __bf16*>(p.k) + n * p.k_t + (h / p.group) * p.k_h;
  const __bf16* v = reinterpret_cast<const __bf16*>(p.v) + n * p.v_t + h * p.v_h;
  for (int d = tid; d < 2 * K; d += kThreads) {
    const __bf16* src = d < K ? q : k;
    const int e = d < K ? d : d - K;
    float x = from_bf16(src[e]);
    if (p.rot.inv_freq && e < p.rot.rot_dim) {
      const int half = p.rot.rot_dim / 2;
      const bool second = p.rot.interleaved ? (e & 1) : e >= half;
      const int i = p.rot.interleaved ? e >> 1 : (second ? e - half : e);
      const int other = p.rot.interleaved ? e ^ 1 : (second ? e - half : e + half);
      const float y = from_bf16(src[other]);
      const float2 cs = rotation(p.rot, n, i, false);
      x = second ? y * cs.y + x * cs.x : x * cs.x - y * cs.y;
    }
    (d < K ? sq : sk)[e] = x;
  }
  if (tid < V) sv[tid] = from_bf16(v[tid]);
  float g = 0.f;
  if (p.g) {
    const int64_t i = p.g_per_token ? (int64_t)n * p.H + h : h;
    g = p.g_bf16 ? (float)reinterpret_cast<const __bf16*>(p.g)[i] : reinterpret_cast<const float*>(p.g)[i];
  }
  const float decay = __expf(g);
  __syncthreads();

  __bf16* out = reinterpret_cast<__bf16*>(p.out) + n * p.o_t + h * p.o_h;
  if constexpr (!kKfirst) {
    const f32x4 k0 = *reinterpret_cast<const f32x4*>(sk + col), k1 = *reinterpret_cast<const f32x4*>(sk + col + 4);
    const f32x4 q0 = *reinterpret_cast<const f32x4*>(sq + col), q1 = *reinterpret_cast<const f32x4*>(sq + col + 4);
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int row = tid / kLanes + i * kPer;
      const float x = sv[row];
      a[i] = a[i] * decay + k0 * x;
      b[i] = b[i] * decay + k1 * x;
      store8<SDT>(p.state_out, at + i * kStep, a[i], b[i]);
      const f32x4 m = a[i] * q0 + b[i] * q1;
      float o = (m[0] + m[1]) + (m[2] + m[3]);
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) o += __shfl_xor(o, d);
      if (tid % kLanes == 0) out[row] = to_bf16(p.scale * o);
    }
  } else {
    const f32x4 v0 = *reinterpret_cast<const f32x4*>(sv + col), v1 = *reinterpret_cast<const f32x4*>(sv + col + 4);
    f32x4 o0 = zero4(), o1 = zero4();
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int row = tid / kLanes + i * kPer;
      a[i] = a[i] * decay + v0 * sk[row];
      b[i] = b[i] * decay + v1 * sk[row];
      store8<SDT>(p.state_out, at + i * kStep, a[i], b[i]);
      o0 += a[i] * sq[row];
      o1 += b[i] * sq[row];
    }
#pragma unroll
    for (int d = kLanes; d < 64; d <<= 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o0[j] += __shfl_xor(o0[j], d);
        o1[j] += __shfl_xor(o1[j], d);
      }
    }
    if (lane < kLanes) {
      *reinterpret_cast<f32x4*>(&part[wave][col]) = o0;
      *reinterpret_cast<f32x4*>(&part[wave][col + 4]) = o1;
    }
    __syncthreads();
    if (tid < V) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) o += part[w][tid];
      out[tid] = to_bf16(p.scale * o);
    }
  }
}

template <int K, int V, int SDT>
int launch_sdt(const LinearPlan& p, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.N * p.H);
  if (p.kfirst) linear_step_kernel<K, V, SDT, true><<<grid, kThreads, 0, s>>>(p);
  else linear_step_kernel<K, V, SDT, false><<<grid, kThreads, 0, s>>>(p);
  return (int)hipGetLastError();
}

template <int K, int V>
int launch_kv(const LinearPlan& p, hipStream_t s) {
  if (p.state_dtype == kF32) return launch_sdt<K, V, kF32>(p, s);
  if (p.state_dtype == kF16) return launch_sdt<K, V, kF16>(p, s);
  return launch_sdt<K, V, kBF16>(p, s);
}

}  // namespace

int launch_linear_step(const LinearPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (p.K == 128) return p.V == 128 ? launch_kv<128, 128>(p, s) : launch_kv<128, 64>(p, s);
  return p.V == 128 ? launch_kv<64, 128>(p, s) : launch_kv<64, 64>(p, s);
}

}  // namespace kda
