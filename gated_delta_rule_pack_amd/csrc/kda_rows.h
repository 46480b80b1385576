// Host helpers for rows in memory, shared by the entry points that take strided tensors of tokens and heads.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cstdlib>

#include "kda.h"

namespace kda {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t state_bytes(kda_dtype d) { return d == KDA_F32 ? 4 : 2; }

// Bytes [lo, hi) of rows t < T, heads h < H of D adjacent elements (strides are not negative).
struct Range {
  uintptr_t lo = 0, hi = 0;
};
inline Range range_of(const void* p, int64_t T, int64_t H, int64_t D, int64_t st, int64_t sh, size_t es) {
  Range r;
  if (T < 1 || H < 1) return r;
  r.lo = (uintptr_t)p;
  r.hi = r.lo + (uintptr_t)((T - 1) * st + (H - 1) * sh + D) * es;
  return r;
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Strides 0, 0 mean dense.
struct Strides {
  int64_t t, h;
};
inline Strides strides_of(int64_t t, int64_t h, int64_t H, int64_t D) {
  return t == 0 && h == 0 ? Strides{H * D, D} : Strides{t, h};
}
// Largest stride: far above any real row, and far below what would overflow 64-bit offsets.
constexpr int64_t kMaxStride = int64_t(1) << 31;
constexpr int64_t kMaxTokenStride = int64_t(1) << 23;
// Workgroups of 256 threads in one launch: its work-items are counted in 32 bits.
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;
inline bool stride_ok(Strides s) { return s.t >= 0 && s.h >= 0 && s.t <= kMaxStride && s.h <= kMaxStride; }
// No two rows of an output overlap: heads inside tokens, or tokens inside heads.
inline bool distinct_rows(Strides s, int64_t T, int64_t H, int64_t D) {
  if (T < 1 || H < 1) return true;
  const int64_t heads = (H - 1) * s.h + D, tokens = (T - 1) * s.t + D;
  const bool h_ok = H == 1 || s.h >= D, t_ok = T == 1 || s.t >= D;
  return h_ok && t_ok && (T == 1 || H == 1 || s.t >= heads || s.h >= tokens);
}

// T tokens of H rows of D elements of es bytes at `at`.
struct Rows {
  const void* at;
  int64_t T, H, D;
  Strides s;
  size_t es;
};
inline bool overlap(const Rows& a, const Rows& b) {
  return overlap(range_of(a.at, a.T, a.H, a.D, a.s.t, a.s.h, a.es), range_of(b.at, b.T, b.H, b.D, b.s.t, b.s.h, b.es));
}
inline bool same_rows(const Rows& a, const Rows& b) {
  return a.at == b.at && a.H == b.H && (a.T == 1 || a.s.t == b.s.t) && (a.H == 1 || a.s.h == b.s.h);
}
// Whether no element belongs to both (of equal T, D and es), where their byte ranges may interleave: in the rows of
// one projection, or of one buffer whose heads hold both in turn. Different token strides are not looked into.
inline bool disjoint(const Rows& a, const Rows& b) {
  if (!overlap(a, b)) return true;
  if (a.T > 1 && (a.s.t != b.s.t || a.s.t < 1)) return false;
  const auto mod = [](int64_t x, int64_t m) { return (x % m + m) % m; };
  const int64_t D = a.D, gap = ((intptr_t)b.at - (intptr_t)a.at) / (intptr_t)a.es;
  const int64_t wa = (a.H - 1) * a.s.h + D, wb = (b.H - 1) * b.s.h + D;
  // All heads of one beside those of the other.
  if (a.T > 1 && mod(gap, a.s.t) >= wa && mod(gap, a.s.t) + wb <= a.s.t) return true;
  // A head of one beside a head of the other.
  const int64_t h = a.H > 1 ? a.s.h : b.s.h;
  if ((a.H == 1 || b.H == 1 || a.s.h == b.s.h) && h > 0 && (a.T == 1 || a.s.t % h == 0) && mod(gap, h) >= D && mod(gap, h) + D <= h)
    return true;
  // Each pair of heads: the tokens that come nearest.
  if (a.H * b.H > 1024) return false;
  for (int64_t i = 0; i < a.H; ++i)
    for (int64_t j = 0; j < b.H; ++j) {
      const int64_t off = gap + j * b.s.h - i * a.s.h;
      int64_t far = off;
      if (a.T > 1) {
        const int64_t k = std::min(std::max(-off / a.s.t, 1 - a.T), a.T - 1);
        for (int64_t t : {k - 1, k, k + 1})
          if (std::abs(t) < a.T && std::abs(off + t * a.s.t) < std::abs(far)) far = off + t * a.s.t;
      }
      if (std::abs(far) < D) return false;
    }
  return true;
}

}  // namespace kda
