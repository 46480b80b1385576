// Norms of q and k for each head, with the position rotation in the same pass, and their gradient.
//
// For a row x of D channels, r = 1 / sqrt(m sum x^2 + eps) (m = 1 / D or 1), w the offset weight and R the rotation:
//   forward   y = R (x r w)
//   backward  z = R^T dy;  dw = sum over rows of z x r;  u = z w;  dx = r (u - m x r sum(u x r)).
// Every element is read and written once, so in vectors both are bound by memory: bf16 tokens of 32 + 8 heads of 128,
// 16384 forward in 67 us, 5.0 TB/s, and 8192 backward in 54 to 57, 4.5 TB/s with the weight gradients' sums; a few tokens wait
// for their angles, 6 us. A row's sums are taken over the lanes that hold it before anything of it is
// written, so a result may take its input's place. Squares are summed in 64 bits: their sum overflows in 32 from
// |x| = 1.8e19 on, and these kernels wait for memory anyway.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kda_delta.h"
#include "kda_device.h"
#include "kda_rotary.h"
#include "kda_unit.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
// As many workgroups as the registers of their 16-byte form let stay on the chip, each walking its share of the tokens
// (16384 tokens of 32 + 8 heads of 128, backward 8192, bf16: 1024 and 512 took 67 and 54 us; 2048 and 1024 67 and 59, 512
// and 256 groups of a backward pass 54 and 77, 768 with their uneven share 61).
constexpr int kForwardGroups = 1024, kBackwardGroups = 512;

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

// Vectors of VEC elements. A row is held by `lanes` lanes (a power of two), two vectors each: a pair that is rotated, or
// two that pass through. A workgroup takes `tokens` tokens at a time, whose angles meet in LDS beside the weights, and
// its groups of lanes walk their q rows and then their k rows, each row's loads issued while the one before is worked on.
// The backward pass keeps the sums of its lanes' weight gradients in registers over all its tokens, and leaves
// them in the workspace.
template <int DT, int VEC, bool kBack>
__global__ __launch_bounds__(kThreads) void norm_wide(const NormPlan p, int tokens, int pairs, int items, int lanes) {
  typedef typename Elem<DT>::type E;
  typedef E V __attribute__((ext_vector_type(VEC)));
  typedef float FV __attribute__((ext_vector_type(VEC)));
  typedef float TV __attribute__((ext_vector_type(2 * VEC)));
  extern __shared__ __align__(64) char shared[];
  const int half = p.rot_dim / 2, u = threadIdx.x % lanes, group = threadIdx.x / lanes, groups = kThreads / lanes;
  float2* turn = reinterpret_cast<float2*>(shared);                    // [tokens][half]
  float* weights = reinterpret_cast<float*>(turn + tokens * half);     // [2][D]
  const auto place = [&](int u, int& d0, int& d1) __attribute__((always_inline)) {
    if (u >= pairs) d0 = p.rot_dim + (u - pairs) * 2 * VEC, d1 = d0 + VEC;
    else if (p.interleaved) d0 = 2 * u * VEC, d1 = d0 + VEC;
    else d0 = u * VEC, d1 = d0 + half;
  };
  int d0, d1;
  place(u, d0, d1);
  const bool rotate = u < pairs, here = u < items, second = here && d1 < p.D;
  // Lanes without a vector load the row's first, which counts in no sum and is not written.
  d0 = here ? d0 : 0, d1 = second ? d1 : 0;
  const float share = p.l2 ? 1.f : 1.f / (float)p.D;
  const double m = p.l2 ? 1. : 1. / p.D;
  float sum[kBack ? 2 : 1][2 * VEC];
  if constexpr (kBack)
#pragma unroll
    for (int j = 0; j < 2 * VEC; ++j) sum[0][j] = sum[1][j] = 0.f;

  // A turn of the walk: each group's i-th row of the tokens from `first` on, all of q or all of k.
  struct Turn {
    int64_t first;
    int i;
  };
  struct Row {
    V x0, x1, z0, z1;
  };
  const int64_t step = (int64_t)gridDim.x * tokens;
  const auto count_of = [&](const Turn& w) __attribute__((always_inline)) { return (int)min((int64_t)tokens, p.T - w.first); };
  const auto turns_of = [&](int count, int c) __attribute__((always_inline)) { return (count * p.H[c] + groups - 1) / groups; };
  const auto next_of = [&](Turn w) __attribute__((always_inline)) {
    const int count = count_of(w);
    if (++w.i == turns_of(count, 0) + turns_of(count, 1)) w.i = 0, w.first += step;
    return w;
  };
  // Its tensor, token and head, and whether there is such a row (the last one else). At most 8 tokens of at most 2^16
  // heads: the quotient is off by less than its distance from a whole number.
  const auto row_of = [&](const Turn& w, int& c, int& t, int& h) __attribute__((always_inline)) {
    const int count = count_of(w), of_q = turns_of(count, 0);
    c = w.i >= of_q;
    const int heads = p.H[c], row = (c ? w.i - of_q : w.i) * groups + group, at = min(row, count * heads - 1);
    t = (int)(((float)at + 0.5f) * __builtin_amdgcn_rcpf((float)heads));
    h = at - t * heads;
    return row == at;
  };
  const auto fetch = [&](Row& r, const Turn& w) __attribute__((always_inline)) {
    int c, t, h;
    row_of(w, c, t, h);
    const E* in = row_at<E>(p.in[c], w.first + t, h, p.in_t[c], p.in_h[c]);
    r.x0 = *reinterpret_cast<const V*>(in + d0);
    r.x1 = *reinterpret_cast<const V*>(in + d1);
    if constexpr (kBack) {
      const E* grad = row_at<E>(p.grad[c], w.first + t, h, p.grad_t[c], p.grad_h[c]);
      r.z0 = *reinterpret_cast<const V*>(grad + d0);
      r.z1 = *reinterpret_cast<const V*>(grad + d1);
    }
  };
  const auto angles = [&](const Turn& w) __attribute__((always_inline)) {
    if (w.i > 0) return;
    __syncthreads();
    for (int i = threadIdx.x; i < count_of(w) * half; i += kThreads) turn[i] = rotation(p, (int)w.first + i / half, i % half, kBack);
    __syncthreads();
  };
  const auto work = [&](const Row& row, const Turn& w) __attribute__((always_inline)) {
    int c, t, h;
    const bool real = row_of(w, c, t, h);
    float x[2 * VEC], z[2 * VEC], wt[2 * VEC];
    double s0 = 0., s1 = 0.;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      x[j] = (float)row.x0[j], x[VEC + j] = (float)row.x1[j];
      s0 += (double)x[j] * x[j];
      s1 += (double)x[VEC + j] * x[VEC + j];
    }
    const double s = lane_sum((here ? s0 : 0.) + (second ? s1 : 0.), lanes);
    const float r = inverse_root(m * s + p.eps);
    const FV w0 = *reinterpret_cast<const FV*>(weights + c * p.D + d0), w1 = *reinterpret_cast<const FV*>(weights + c * p.D + d1);
#pragma unroll
    for (int j = 0; j < VEC; ++j) wt[j] = w0[j], wt[VEC + j] = w1[j];
#pragma unroll
    for (int j = 0; j < 2 * VEC; ++j) {
      x[j] *= r;
      z[j] = kBack ? (float)(j < VEC ? row.z0[j % VEC] : row.z1[j % VEC]) : x[j] * wt[j];
    }
    if (rotate) {
      const TV cs = *reinterpret_cast<const TV*>(turn + t * half + u * VEC);
      const auto rotated = [&](float& a, float& b, int j) __attribute__((always_inline)) {
        const float ao = a * cs[2 * j] - b * cs[2 * j + 1], bo = a * cs[2 * j + 1] + b * cs[2 * j];
        a = ao, b = bo;
      };
      if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) rotated(z[2 * j], z[2 * j + 1], j);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) rotated(z[j], z[VEC + j], j);
      }
    }
    if constexpr (kBack) {
      if (real) {
        if (c == 0) {
#pragma unroll
          for (int j = 0; j < 2 * VEC; ++j) sum[0][j] += z[j] * x[j];
        } else {
#pragma unroll
          for (int j = 0; j < 2 * VEC; ++j) sum[1][j] += z[j] * x[j];
        }
      }
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        z[j] *= wt[j], z[VEC + j] *= wt[VEC + j];
        a += z[j] * x[j], b += z[VEC + j] * x[VEC + j];
      }
      const float dot = share * lane_sum((here ? a : 0.f) + (second ? b : 0.f), lanes);
#pragma unroll
      for (int j = 0; j < 2 * VEC; ++j) z[j] = r * (z[j] - x[j] * dot);
    }
    V y0, y1;
#pragma unroll
    for (int j = 0; j < VEC; ++j) y0[j] = (E)z[j], y1[j] = (E)z[VEC + j];
    E* out = row_at<E>(p.out[c], w.first + t, h, p.out_t[c], p.out_h[c]);
    if (real && here) *reinterpret_cast<V*>(out + d0) = y0;
    if (real && second) *reinterpret_cast<V*>(out + d1) = y1;
  };

  Turn w = {(int64_t)blockIdx.x * tokens, 0};
  if (w.first < p.T) {
    Row a, b;
    fetch(a, w);
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) weights[i] = weight_at<E>(p, i >= p.D, i >= p.D ? i - p.D : i);
    for (;;) {
      angles(w);
      Turn n = next_of(w);
      if (n.first >= p.T) {
        work(a, w);
        break;
      }
      fetch(b, n);
      work(a, w);
      w = n;
      angles(w);
      n = next_of(w);
      if (n.first >= p.T) {
        work(b, w);
        break;
      }
      fetch(a, n);
      work(b, w);
      w = n;
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
        float part[4] = {0.f, 0.f, 0.f, 0.f};  // (groups: a power of two, 4 or more)
        for (int g = 0; g < groups; g += 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[e] += all[(g + e) * lanes * 2 * VEC + i];
        const float x = (part[0] + part[1]) + (part[2] + part[3]);
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

// Single elements, for rows of more than 64 pairs of the vectors that fit them (more than 128 channels with an odd half
// or at an odd address, more than 512 in fp32): a workgroup for each token at a time, a wave for each of its
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
      s = lane_sum(s, 64);
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
        dot = share * lane_sum(dot, 64);
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

// The workgroups' sums of weight gradients, joined: 16 channels to a workgroup, 64 threads to a channel, four loads in
// flight at a time (512 workgroups' sums of 128 channels: 4.1 us; 16 threads to a channel and one load at a time took 20 for 1024),
// summed in pairs: the 64 threads' sums one after another would add 3.3 2^-24 to a gradient's error, pairs of pairs 1.4.
template <int DT>
__global__ __launch_bounds__(1024) void norm_sums(const NormPlan p) {
  typedef typename Elem<DT>::type E;
  constexpr int kWays = 64, kParts = 1024 / 64;
  __shared__ float part[kParts][16];
  const int c = blockIdx.y, lane = threadIdx.x & 15, way = threadIdx.x >> 4, wave = threadIdx.x >> 6, d = blockIdx.x * 16 + lane;
  const float* from = p.sums + c * p.D + min(d, p.D - 1);
  float x = 0.f;
  for (int i = way; i < p.groups; i += 4 * kWays) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = from[(int64_t)min(i + j * kWays, p.groups - 1) * 2 * p.D];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = i + j * kWays < p.groups ? y[j] : 0.f;
    x += (y[0] + y[1]) + (y[2] + y[3]);
  }
  x = add_far(add_far(x, 16), 32);  // a wave's four ways
  if ((threadIdx.x & 63) < 16) part[wave][lane] = x;
  __syncthreads();
  if (wave > 0) return;
  const int first = threadIdx.x >> 4;
  x = (part[first][lane] + part[first + 4][lane]) + (part[first + 8][lane] + part[first + 12][lane]);
  x = add_far(add_far(x, 16), 32);
  void* to = p.grad_weight[c];
  if (first > 0 || d >= p.D || !to) return;
  if (p.weight_f32) reinterpret_cast<float*>(to)[d] = x;
  else reinterpret_cast<E*>(to)[d] = (E)x;
}

// The widest vectors that the rows allow, 16 bytes at most; rows of more than 64 pairs of vectors take single elements.
template <int DT, int VEC, bool kBack>
int launch_vec(const NormPlan& p, hipStream_t s) {
  const int half = p.rot_dim / 2;
  constexpr int kBytes = VEC * (DT == kF32 ? 4 : 2);
  const auto fits = [](const void* at, int64_t st, int64_t sh) { return (uintptr_t)at % kBytes == 0 && st % VEC == 0 && sh % VEC == 0; };
  bool wide = half % VEC == 0 && p.D % VEC == 0;
  for (int c = 0; c < 2; ++c) {
    if (p.H[c] == 0) continue;
    wide = wide && fits(p.in[c], p.in_t[c], p.in_h[c]) && fits(p.out[c], p.out_t[c], p.out_h[c]);
    if (kBack) wide = wide && fits(p.grad[c], p.grad_t[c], p.grad_h[c]);
  }
  if constexpr (VEC > 1) {
    if (!wide) return launch_vec<DT, VEC / 2, kBack>(p, s);
  }
  const int pairs = half / VEC, items = pairs + ((p.D - p.rot_dim) / VEC + 1) / 2;
  int lanes = 1;
  while (lanes < items) lanes *= 2;
  if (lanes > 64) {
    const unsigned grid = kBack ? (unsigned)p.groups : (unsigned)(p.T < (1 << 20) ? p.T : 1 << 20);
    const size_t shared = (size_t)half * sizeof(float2) + (size_t)kWaves * p.D * sizeof(float) * (kBack ? 3 : 1);
    norm_narrow<DT, kBack><<<grid, kThreads, shared, s>>>(p);
    return (int)hipGetLastError();
  }
  // Angles are made, between two barriers, for four tokens at a time, and for up to eight where that lets each group of
  // lanes walk five rows behind them; for fewer where the workgroups would run out of tokens (16384 tokens of 32 + 8
  // heads, 64 of 128 channels rotated: 1, 2, 4, 8 tokens 86, 71, 67, 71 us; of 8 + 2 heads of 256: 4 and 8 tokens
  // 40 and 37 us, backward 68 and 60).
  const int most = kBack ? p.groups : kForwardGroups, even = (int)(((int64_t)p.T + most - 1) / most);
  const int heads = p.H[0] + p.H[1], long_enough = (5 * (kThreads / lanes) + heads - 1) / heads;
  const int tokens = std::min(even, std::max(4, std::min(8, long_enough)));
  const int batches = (p.T + tokens - 1) / tokens;
  const unsigned grid = kBack ? (unsigned)p.groups : (unsigned)(batches < most ? batches : most);
  size_t shared = (size_t)tokens * half * sizeof(float2) + 2 * p.D * sizeof(float);
  if (kBack && shared < (size_t)kThreads * 2 * VEC * sizeof(float)) shared = (size_t)kThreads * 2 * VEC * sizeof(float);
  norm_wide<DT, VEC, kBack><<<grid, kThreads, shared, s>>>(p, tokens, pairs, items, lanes);
  return (int)hipGetLastError();
}
template <int DT, bool kBack>
int launch_dt(const NormPlan& p, hipStream_t s) {
  return launch_vec<DT, DT == kF32 ? 4 : 8, kBack>(p, s);
}

template <int DT>
int launch_back(const NormPlan& p, hipStream_t s) {
  if (p.T > 0) {
    const int error = launch_dt<DT, true>(p, s);
    if (error) return error;
  }
  if (!p.grad_weight[0] && !p.grad_weight[1]) return 0;
  norm_sums<DT><<<dim3((unsigned)(p.D + 15) / 16, 2), 1024, 0, s>>>(p);
  return (int)hipGetLastError();
}

}  // namespace

int norm_groups(int T) { return std::min(T, kBackwardGroups); }

int launch_qk_norm(const NormPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return p.dtype == kF32 ? launch_dt<kF32, false>(p, s) : p.dtype == kF16 ? launch_dt<kF16, false>(p, s) : launch_dt<kBF16, false>(p, s);
}

int launch_qk_norm_backward(const NormPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return p.dtype == kF32 ? launch_back<kF32>(p, s) : p.dtype == kF16 ? launch_back<kF16>(p, s) : launch_back<kBF16>(p, s);
}

}  // namespace kda
