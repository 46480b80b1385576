// Norms of q and k for each head, with the position rotation in the same pass, and their gradient.
//
// For a row x of D channels, r = 1 / sqrt(m sum x^2 + eps) (m = 1 / D or 1), w the offset weight and R the rotation:
//   forward   y = R (x r w)
//   backward  z = R^T dy;  dw = sum over rows of z x r;  u = z w;  dx = r (u - m x r sum(u x r)).
// Every element is read and written once, so in 16-byte vectors both are bound by memory. A row's sums are taken over
// the lanes that hold it before anything of it is written, so a result may take its input's place. Squares are
// summed in 64 bits: their sum overflows in 32 from |x| = 1.8e19 on, and these kernels wait for memory anyway.
#include <hip/hip_runtime.h>

#include "kda_delta.h"
#include "kda_device.h"
#include "kda_rotary.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

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

__device__ __forceinline__ double xor_lanes(double x, int d) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __shfl_xor((int)u, d), hi = __shfl_xor((int)(u >> 32), d);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// 1 / sqrt(s) for s = m sum x^2 + eps, which may lie outside fp32 where its root does not.
__device__ __forceinline__ float inverse_root(double s) {
  if (!(s < 1e300)) return __builtin_nanf("");  // a row that is not finite
  const int e = __builtin_amdgcn_frexp_exp(s) & ~1;
  return __builtin_amdgcn_ldexpf(rsqrtf((float)__builtin_amdgcn_ldexp(s, -e)), -e / 2);
}

template <typename E>
__device__ __forceinline__ float weight_at(const NormPlan& p, int c, int d) {
  const void* w = p.weight[c];
  if (!w) return 1.f;
  return p.offset + (p.weight_f32 ? reinterpret_cast<const float*>(w)[d] : (float)reinterpret_cast<const E*>(w)[d]);
}
template <typename E>
__device__ __forceinline__ E* row_at(const void* base, int64_t t, int h, int64_t stride_t, int64_t stride_h) {
  return reinterpret_cast<E*>(const_cast<void*>(base)) + t * stride_t + h * stride_h;
}

// 16-byte vectors. A row is held by `lanes` lanes (a power of two), two vectors each: a pair that is rotated, or two
// that pass through. A workgroup takes `tokens` tokens at a time, whose angles meet in LDS, and its groups of lanes
// walk their q rows and then their k rows. The backward pass keeps the sums of its lanes' weight gradients in
// registers over all its tokens, and leaves them in the workspace.
template <int DT, int VEC, bool kInterleaved, bool kBack>
__global__ __launch_bounds__(kThreads) void norm_wide(const NormPlan p, int tokens, int pairs, int items, int lanes) {
  typedef typename Elem<DT>::type E;
  typedef E V __attribute__((ext_vector_type(VEC)));
  extern __shared__ __align__(16) char shared[];
  float2* turn = reinterpret_cast<float2*>(shared);  // [tokens][half]
  const int half = p.rot_dim / 2, u = threadIdx.x % lanes, group = threadIdx.x / lanes, groups = kThreads / lanes;
  const auto place = [&](int u, int& d0, int& d1) {
    if (u >= pairs) d0 = p.rot_dim + (u - pairs) * 2 * VEC, d1 = d0 + VEC;
    else if (kInterleaved) d0 = 2 * u * VEC, d1 = d0 + VEC;
    else d0 = u * VEC, d1 = d0 + half;
  };
  int d0, d1;
  place(u, d0, d1);
  const bool rotate = u < pairs, here = u < items, second = here && d1 < p.D;
  const float share = p.l2 ? 1.f : 1.f / (float)p.D;
  const double m = p.l2 ? 1. : 1. / p.D;
  float w[2][2 * VEC], sum[kBack ? 2 : 1][2 * VEC];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[c][j] = here ? weight_at<E>(p, c, d0 + j) : 1.f;
      w[c][VEC + j] = second ? weight_at<E>(p, c, d1 + j) : 1.f;
      if constexpr (kBack) sum[c][j] = sum[c][VEC + j] = 0.f;
    }
  const int64_t step = (int64_t)gridDim.x * tokens;
  for (int64_t first = (int64_t)blockIdx.x * tokens; first < p.T; first += step) {
    const int count = (int)min((int64_t)tokens, p.T - first);
    if (half > 0) {
      __syncthreads();
      for (int i = threadIdx.x; i < count * half; i += kThreads) turn[i] = rotation(p, (int)first + i / half, i % half, kBack);
      __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      for (int row = group; row < count * p.H[c]; row += groups) {
        const int t = row / p.H[c], h = row - t * p.H[c];
        const E* in = row_at<E>(p.in[c], first + t, h, p.in_t[c], p.in_h[c]);
        V x0 = {}, x1 = {}, z0 = {}, z1 = {};
        if (here) x0 = *reinterpret_cast<const V*>(in + d0);
        if (second) x1 = *reinterpret_cast<const V*>(in + d1);
        if constexpr (kBack) {
          const E* grad = row_at<E>(p.grad[c], first + t, h, p.grad_t[c], p.grad_h[c]);
          if (here) z0 = *reinterpret_cast<const V*>(grad + d0);
          if (second) z1 = *reinterpret_cast<const V*>(grad + d1);
        }
        float x[2 * VEC], z[2 * VEC];
        double s = 0.;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          x[j] = (float)x0[j], x[VEC + j] = (float)x1[j];
          s += (double)x[j] * x[j];
          s += (double)x[VEC + j] * x[VEC + j];
        }
        for (int d = 1; d < lanes; d <<= 1) s += xor_lanes(s, d);
        const float r = inverse_root(m * s + p.eps);
#pragma unroll
        for (int j = 0; j < 2 * VEC; ++j) {
          x[j] *= r;
          z[j] = kBack ? (float)(j < VEC ? z0[j % VEC] : z1[j % VEC]) : x[j] * w[c][j];
        }
        if (rotate) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float2 cs = turn[t * half + u * VEC + j];
            float &a = z[kInterleaved ? 2 * j : j], &b = z[kInterleaved ? 2 * j + 1 : VEC + j];
            const float ao = a * cs.x - b * cs.y, bo = a * cs.y + b * cs.x;
            a = ao, b = bo;
          }
        }
        if constexpr (kBack) {
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < 2 * VEC; ++j) {
            sum[c][j] += z[j] * x[j];
            z[j] *= w[c][j];
            dot += z[j] * x[j];
          }
          for (int d = 1; d < lanes; d <<= 1) dot += __shfl_xor(dot, d);
          dot *= share;
#pragma unroll
          for (int j = 0; j < 2 * VEC; ++j) z[j] = r * (z[j] - x[j] * dot);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) x0[j] = (E)z[j], x1[j] = (E)z[VEC + j];
        E* out = row_at<E>(p.out[c], first + t, h, p.out_t[c], p.out_h[c]);
        if (here) *reinterpret_cast<V*>(out + d0) = x0;
        if (second) *reinterpret_cast<V*>(out + d1) = x1;
      }
    }
  }
  if constexpr (kBack) {
    if (!p.sums) return;
    float* all = reinterpret_cast<float*>(shared);  // [groups][lanes][2 VEC]
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2 * VEC; ++j) all[(size_t)threadIdx.x * 2 * VEC + j] = sum[c][j];
      __syncthreads();
      for (int i = threadIdx.x; i < items * 2 * VEC; i += kThreads) {
        int a, b;
        place(i / (2 * VEC), a, b);
        const int j = i % (2 * VEC), d = j < VEC ? a + j : b + j - VEC;
        if (d >= p.D) continue;
        float x = 0.f;
        for (int g = 0; g < groups; ++g) x += all[g * lanes * 2 * VEC + i];
        p.sums[((int64_t)blockIdx.x * 2 + c) * p.D + d] = x;
      }
    }
  }
}

// Orders a wave's own LDS accesses: its lanes read what others of them wrote.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Single elements, for rows that 16-byte accesses do not fit: a workgroup for each token at a time, a wave for each of its
// rows. The row passes through the wave's LDS, where its lanes find the other halves of their pairs.
template <int DT, bool kBack>
__global__ __launch_bounds__(kThreads) void norm_narrow(const NormPlan p) {
  typedef typename Elem<DT>::type E;
  extern __shared__ __align__(16) char shared[];
  const int half = p.rot_dim / 2, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, D = p.D;
  float2* turn = reinterpret_cast<float2*>(shared);           // [half]
  float* buf = reinterpret_cast<float*>(turn + half) + wave * D;  // [waves][D]
  float* all = reinterpret_cast<float*>(turn + half) + kWaves * D;  // backward: [waves][2][D]
  float* sums = all + wave * 2 * D;
  const float share = p.l2 ? 1.f : 1.f / (float)D;
  const double m = p.l2 ? 1. : 1. / D;
  if constexpr (kBack)
    for (int d = lane; d < 2 * D; d += 64) sums[d] = 0.f;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    if (half > 0) {
      __syncthreads();
      for (int i = threadIdx.x; i < half; i += kThreads) turn[i] = rotation(p, (int)t, i, kBack);
      __syncthreads();
    }
    for (int row = wave; row < p.H[0] + p.H[1]; row += kWaves) {
      const int c = row >= p.H[0], h = c ? row - p.H[0] : row;
      const E* in = row_at<E>(p.in[c], t, h, p.in_t[c], p.in_h[c]);
      const E* grad = kBack ? row_at<E>(p.grad[c], t, h, p.grad_t[c], p.grad_h[c]) : nullptr;
      double s = 0.;
      for (int d = lane; d < D; d += 64) {
        const float x = (float)in[d];
        s += (double)x * x;
        if constexpr (kBack) buf[d] = (float)grad[d];
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) s += xor_lanes(s, d);
      const float r = inverse_root(m * s + p.eps);
      if constexpr (!kBack)
        for (int d = lane; d < D; d += 64) buf[d] = (float)in[d] * r * weight_at<E>(p, c, d);
      wave_sync();
      // Element d of the row in buf, rotated.
      const auto turned = [&](int d) {
        const float a = buf[d];
        if (d >= p.rot_dim) return a;
        const bool low = p.interleaved ? !(d & 1) : d < half;
        const int i = p.interleaved ? d >> 1 : (low ? d : d - half);
        const float2 cs = turn[i];
        const float b = buf[p.interleaved ? d ^ 1 : (low ? d + half : d - half)];
        return low ? a * cs.x - b * cs.y : b * cs.y + a * cs.x;
      };
      E* out = row_at<E>(p.out[c], t, h, p.out_t[c], p.out_h[c]);
      if constexpr (!kBack) {
        for (int d = lane; d < D; d += 64) out[d] = (E)turned(d);
      } else {
        float dot = 0.f;
        for (int d = lane; d < D; d += 64) {
          const float z = turned(d), x = (float)in[d] * r;
          sums[c * D + d] += z * x;
          dot += z * weight_at<E>(p, c, d) * x;
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d);
        dot *= share;
        for (int d = lane; d < D; d += 64) out[d] = (E)(r * (turned(d) * weight_at<E>(p, c, d) - (float)in[d] * r * dot));
      }
      wave_sync();
    }
  }
  if constexpr (kBack) {
    if (!p.sums) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      float x = 0.f;
      for (int w = 0; w < kWaves; ++w) x += all[w * 2 * D + i];
      p.sums[(int64_t)blockIdx.x * 2 * D + i] = x;
    }
  }
}

// The workgroups' sums of weight gradients, joined: 16 channels to a workgroup, 16 threads to a channel.
template <int DT>
__global__ __launch_bounds__(kThreads) void norm_sums(const NormPlan p) {
  typedef typename Elem<DT>::type E;
  __shared__ float part[16][17];
  const int c = blockIdx.y, lane = threadIdx.x & 15, way = threadIdx.x >> 4, d = blockIdx.x * 16 + lane;
  float x = 0.f;
  if (d < p.D)
    for (int i = way; i < p.groups; i += 16) x += p.sums[((int64_t)i * 2 + c) * p.D + d];
  part[way][lane] = x;
  __syncthreads();
  void* to = p.grad_weight[c];
  if (way != 0 || d >= p.D || !to) return;
  x = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) x += part[i][lane];
  if (p.weight_f32) reinterpret_cast<float*>(to)[d] = x;
  else reinterpret_cast<E*>(to)[d] = (E)x;
}

template <int DT, int VEC, bool kBack>
int launch_wide(const NormPlan& p, unsigned grid, int tokens, int pairs, int items, int lanes, hipStream_t s) {
  size_t shared = (size_t)tokens * (p.rot_dim / 2) * sizeof(float2);
  if (kBack && shared < (size_t)kThreads * 2 * VEC * sizeof(float)) shared = (size_t)kThreads * 2 * VEC * sizeof(float);
  if (p.interleaved) norm_wide<DT, VEC, true, kBack><<<grid, kThreads, shared, s>>>(p, tokens, pairs, items, lanes);
  else norm_wide<DT, VEC, false, kBack><<<grid, kThreads, shared, s>>>(p, tokens, pairs, items, lanes);
  return (int)hipGetLastError();
}

// 16-byte accesses where the rows allow them, single elements otherwise.
template <int DT, bool kBack>
int launch_dt(const NormPlan& p, hipStream_t s) {
  constexpr int VEC = DT == kF32 ? 4 : 8;
  const int half = p.rot_dim / 2;
  const auto fits = [](const void* at, int64_t st, int64_t sh) { return (uintptr_t)at % 16 == 0 && st % VEC == 0 && sh % VEC == 0; };
  bool wide = half % VEC == 0 && p.D % VEC == 0;
  for (int c = 0; c < 2; ++c) {
    if (p.H[c] == 0) continue;
    wide = wide && fits(p.in[c], p.in_t[c], p.in_h[c]) && fits(p.out[c], p.out_t[c], p.out_h[c]);
    if (kBack) wide = wide && fits(p.grad[c], p.grad_t[c], p.grad_h[c]);
  }
  const int pairs = half / VEC, items = pairs + ((p.D - p.rot_dim) / VEC + 1) / 2;
  int lanes = 1;
  while (lanes < items) lanes *= 2;
  if (!wide || lanes > 64) {
    const unsigned grid = kBack ? (unsigned)p.groups : (unsigned)(p.T < (1 << 20) ? p.T : 1 << 20);
    const size_t shared = (size_t)half * sizeof(float2) + (size_t)kWaves * p.D * sizeof(float) * (kBack ? 3 : 1);
    norm_narrow<DT, kBack><<<grid, kThreads, shared, s>>>(p);
    return (int)hipGetLastError();
  }
  // Four tokens share a workgroup's start where there are enough to fill the chip.
  const int tokens = p.T >= 2048 ? 4 : 1;
  const int batches = (p.T + tokens - 1) / tokens;
  const unsigned grid = kBack ? (unsigned)p.groups : (unsigned)(batches < (1 << 20) ? batches : 1 << 20);
  return launch_wide<DT, VEC, kBack>(p, grid, tokens, pairs, items, lanes, s);
}

template <int DT>
int launch_back(const NormPlan& p, hipStream_t s) {
  if (p.T > 0) {
    const int error = launch_dt<DT, true>(p, s);
    if (error) return error;
  }
  if (!p.grad_weight[0] && !p.grad_weight[1]) return 0;
  norm_sums<DT><<<dim3((unsigned)(p.D + 15) / 16, 2), kThreads, 0, s>>>(p);
  return (int)hipGetLastError();
}

}  // namespace

int norm_groups(int T) { return T < 1024 ? T : 1024; }

int launch_qk_norm(const NormPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return p.dtype == kF32 ? launch_dt<kF32, false>(p, s) : p.dtype == kF16 ? launch_dt<kF16, false>(p, s) : launch_dt<kBF16, false>(p, s);
}

int launch_qk_norm_backward(const NormPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return p.dtype == kF32 ? launch_back<kF32>(p, s) : p.dtype == kF16 ? launch_back<kF16>(p, s) : launch_back<kBF16>(p, s);
}

}  // namespace kda
