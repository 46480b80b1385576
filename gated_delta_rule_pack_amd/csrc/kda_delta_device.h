// Device side that the gated delta rule's prompt kernels share: operands in fp16 terms, scaled rows, a chunk's
// numbers, and the triangular inverse T. kda_delta.hip has the mathematics.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "kda_delta.h"
#include "kda_device.h"
#include "kda_unit.h"
#include "kda_walk.h"

namespace kda {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
// fp32 operands: A row l % 16, B column l % 16, both k = l / 16.
__device__ __forceinline__ f32x4 mfma32(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }
__device__ __forceinline__ float ldexp2(float x, int e) { return __builtin_amdgcn_ldexpf(x, e); }

// Two fp32 values as fp16, low first, rounded to nearest.
__device__ __forceinline__ uint32_t pair_f16(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  uint32_t r = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
  asm("" : "+v"(r));
  return r;
}
// What two values leave of those, exactly, rounded to fp16: one instruction each. (Written as conversions and differences
// the compiler takes three; and where a and b are a product or a sum it makes the first term of the exact value in one
// instruction and this one of the rounded value: where those fall on two sides of a middle, both terms miss it by 2^-10.)
__device__ __forceinline__ uint32_t rest_pair(float a, float b, uint32_t first, float minus = -1.f) {
  const f16x2 h = __builtin_bit_cast(f16x2, first);
  asm("" : "+s"(minus));  // a known factor would become a difference, which has no such instruction
  const f16x2 r = {(_Float16)__builtin_fmaf((float)h[0], minus, a), (_Float16)__builtin_fmaf((float)h[1], minus, b)};
  return __builtin_bit_cast(uint32_t, r);
}
// Two tiles (rows 4g + i and 16 + 4g + i) as an operand, in two terms.
__device__ __forceinline__ f16x8 to_f16(f32x4 a, f32x4 b) {
  return __builtin_bit_cast(f16x8, u32x4{pair_f16(a[0], a[1]), pair_f16(a[2], a[3]), pair_f16(b[0], b[1]), pair_f16(b[2], b[3])});
}
__device__ __forceinline__ f16x8 rest_f16(f32x4 a, f32x4 b, f16x8 hi) {
  const u32x4 h = __builtin_bit_cast(u32x4, hi);
  return __builtin_bit_cast(f16x8, u32x4{rest_pair(a[0], a[1], h[0]), rest_pair(a[2], a[3], h[1]), rest_pair(b[0], b[1], h[2]),
                                         rest_pair(b[2], b[3], h[3])});
}
// Second terms times 2^12, as large as the first ones: fp16's least step then stands for 2^-37. Their products are summed by
// themselves and taken back by 2^-12. (Of the state alone the second term stands as it is: its largest value is kept near 1.)
constexpr float kUp = 0x1p12f, kDown = 0x1p-12f;
__device__ __forceinline__ uint32_t rest_up(float a, float b, uint32_t first) {
  return rest_pair(a * kUp, b * kUp, first, -kUp);
}
__device__ __forceinline__ f16x8 rest_up(f32x4 a, f32x4 b, f16x8 hi) {
  const u32x4 h = __builtin_bit_cast(u32x4, hi);
  return __builtin_bit_cast(f16x8, u32x4{rest_up(a[0], a[1], h[0]), rest_up(a[2], a[3], h[1]), rest_up(b[0], b[1], h[2]), rest_up(b[2], b[3], h[3])});
}
// One tile (rows 4g + i) as half a fragment, in two terms.
template <bool kRestUp>
__device__ __forceinline__ void put_half(char* high, char* low, int at, f32x4 x) {
  const u32x2 h = {pair_f16(x[0], x[1]), pair_f16(x[2], x[3])};
  *reinterpret_cast<u32x2*>(high + at) = h;
  *reinterpret_cast<u32x2*>(low + at) = kRestUp ? u32x2{rest_up(x[0], x[1], h[0]), rest_up(x[2], x[3], h[1])}
                                                : u32x2{rest_pair(x[0], x[1], h[0]), rest_pair(x[2], x[3], h[1])};
}
// P stands 64 times as large as it is (it is at most 2^9, by the longest rows). Its second term has 8 bits, five of exponent and two of
// fraction, fp16's upper byte: with them P is within 2^-14 of itself, an eighth of the half step of outputs in fp16, or within 2^-34, and its
// records keep their size. It is stored times 2^11, and read times 2^12.
constexpr float kTimesP = 64.f;
__device__ __forceinline__ uint32_t p_rest(f32x4 x, u32x2 first) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const float up = kUp / 2;
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const u16x2 r = __builtin_bit_cast(u16x2, rest_pair(x[2 * j] * up, x[2 * j + 1] * up, first[j], -up));
    w[j] = __builtin_bit_cast(uint32_t, (u16x2)(r + (u16x2){0x80, 0x80}));  // to nearest
  }
  return __builtin_amdgcn_perm(w[1], w[0], 0x07050301);
}
__device__ __forceinline__ f16x8 p_rest_operand(u32x2 x) {
  const u32x4 w = {__builtin_amdgcn_perm(0, x[0], 0x010c000c), __builtin_amdgcn_perm(0, x[0], 0x030c020c),
                   __builtin_amdgcn_perm(0, x[1], 0x010c000c), __builtin_amdgcn_perm(0, x[1], 0x030c020c)};
  return __builtin_bit_cast(f16x8, w) * (_Float16)2.f;
}

// A token's element of a 16-bit word, by type.
template <bool kF16In>
__device__ __forceinline__ float token_value(uint32_t half) {
  if constexpr (kF16In) return (float)__builtin_bit_cast(_Float16, (uint16_t)half);
  else return __uint_as_float(half << 16);
}
template <bool kF16In>
__device__ __forceinline__ float low_value(uint32_t w) {
  return kF16In ? token_value<true>(w & 0xffff) : __uint_as_float(w << 16);
}
template <bool kF16In>
__device__ __forceinline__ float high_value(uint32_t w) {
  return kF16In ? token_value<true>(w >> 16) : __uint_as_float(w & 0xffff0000u);
}

// A decay's or step size's bits on their way, fp32 or bf16: widened where they are used, not where they land.
__device__ __forceinline__ uint32_t load_bits(const void* base, int64_t at, int bf16) {
  return bf16 ? (uint32_t)reinterpret_cast<const uint16_t*>(base)[at] : reinterpret_cast<const uint32_t*>(base)[at];
}
__device__ __forceinline__ float bits_value(uint32_t x, int bf16) { return __uint_as_float(bf16 ? x << 16 : x); }

// Maximum and sum over the 8 or 16 lanes of a row: quads, halves, whole rows.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, dpp<0xb1>(x));   // quad_perm [1, 0, 3, 2]
  x = max(x, dpp<0x4e>(x));   // quad_perm [2, 3, 0, 1]
  x = max(x, dpp<0x141>(x));  // row_half_mirror
  if constexpr (kLanes == 16) x = max(x, dpp<0x140>(x));  // row_mirror
  return x;
}
// The exponent of x >= 0: x < 2^e.
constexpr int kNoExponent = -4096;
__device__ __forceinline__ int exponent(float x) { return x > 0.f && x < INFINITY ? __builtin_amdgcn_frexp_expf(x) : kNoExponent; }
// Over the four lanes that hold one channel: exchanges of half waves and of rows, without LDS.
__device__ __forceinline__ int channel_max(int x) {
  const auto a = __builtin_amdgcn_permlane32_swap((unsigned)x, (unsigned)x, false, false);
  x = max((int)a[0], (int)a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap((unsigned)x, (unsigned)x, false, false);
  return max((int)b[0], (int)b[1]);
}

// Two exponents in one word, and the larger of each.
typedef short i16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ int pair_max(int a, int b) {
  return __builtin_bit_cast(int, __builtin_elementwise_max(__builtin_bit_cast(i16x2, a), __builtin_bit_cast(i16x2, b)));
}
__device__ __forceinline__ i16x2 channel_max(i16x2 of) {
  unsigned x = __builtin_bit_cast(unsigned, of);
  const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  x = pair_max((int)a[0], (int)a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  return __builtin_bit_cast(i16x2, pair_max((int)b[0], (int)b[1]));
}

constexpr int kBadRow = 1 << 20;  // exponent of a row that is not finite
// A scaled row's exponent and the sum of its scaled squares.
struct RowInfo {
  int e;
  float squares;
};

// The sequence of a rank, the longest first: where workgroups wait for a place on the chip, those of long sequences start
// early, so that none of them runs alone at the end (128 prompts of 0 to 2048 tokens at H = 12: 930 us in the call's order,
// 810 ranked). Lengths count by their half octave of chunks, and the call's order inside one: with 8 waves' ballots
// that takes 0.7 us of a workgroup, where ranks by comparison with every length took 7 for 256 sequences.
constexpr int kRankWaves = kMostRanked / 64, kRankClasses = 32;
struct Ranking {
  alignas(16) int count[kRankClasses * kRankWaves];  // of a class in a wave
  int sequence;
};
__device__ __forceinline__ int ranked_sequence(const DeltaPlan& p, Ranking& r, int rank, int tid) {
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const bool here = tid < p.N;
  const int chunks = here ? (max(bound(p, tid + 1) - bound(p, tid), 0) + kC - 1) / kC : 0;
  // An exponent and one bit of its fraction, from one chunk on.
  const int octave = (int)(__float_as_uint((float)chunks) >> 22) - 2 * 127, own = kRankClasses - 1 - min(max(octave, 0), kRankClasses - 1);
  if (tid < kRankClasses * kRankWaves) r.count[tid] = 0;
  uint64_t same = __ballot(here);
#pragma unroll
  for (int b = 0; b < 5; ++b) {
    const uint64_t set = __ballot(own >> b & 1);
    same &= own >> b & 1 ? set : ~set;
  }
  const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
  barrier_lds();
  if (here && before == 0) r.count[own * kRankWaves + wave] = __builtin_popcountll(same);
  barrier_lds();
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  const i32x4 c = *reinterpret_cast<const i32x4*>(r.count + 4 * lane);
  const int total = c[0] + c[1] + c[2] + c[3];
  int sum = total;
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) {
    const int x = __shfl_up(sum, i);
    sum += lane >= i ? x : 0;
  }
  int rest = rank - (sum - total), cell = 4 * lane;
  const uint64_t found = __ballot(rest >= 0 && rest < total);
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    const bool on = cell == 4 * lane + e && rest >= c[e];
    rest -= on ? c[e] : 0, cell += on;
  }
  const int from = __builtin_ctzll(found | 1ull << 63);
  cell = __builtin_amdgcn_readlane(cell, from), rest = __builtin_amdgcn_readlane(rest, from);
  if (here && own * kRankWaves + wave == cell && before == rest) r.sequence = tid;
  barrier_lds();
  return __builtin_amdgcn_readfirstlane(r.sequence);
}

// Rows of q or k on their way to LDS as fp16, each scaled by 2^-e: e = 0 for rows whose length is between 1/2 and 16, where all
// that counts of them fits as it stands, else what brings their largest element into [1/4, 1/2), or below 2 at bf16's end: 2^e has to be finite.
// (Two rows of the largest length, 2 sqrt(128), make P 2^15 at most.)
template <int D, int kThreads, bool kF16In>
struct ScaledRows {
  typedef Rows<D, kThreads> R;
  static constexpr float kLeast = 0x1p-2f, kMost = 0x1p8f;
  R rows;
  RowInfo info[R::kPasses];

  // All rows side by side, so that their chains of sums run beside each other; one look for rows out of the ordinary.
  __device__ __forceinline__ void squares(const u32x4 (&x)[R::kPasses], float (&s)[R::kPasses]) {
#pragma unroll
    for (int i = 0; i < R::kPasses; ++i) s[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < R::kPasses; ++i) {
        const uint32_t word = x[i][j];
        const f16x2 h = __builtin_bit_cast(f16x2, word);
        s[i] = __builtin_amdgcn_fdot2(h, h, s[i], false);
      }
#pragma unroll
    for (int i = 0; i < R::kPasses; ++i) s[i] += __uint_as_float(dpp<0xb1>(__float_as_uint(s[i])));
#pragma unroll
    for (int i = 0; i < R::kPasses; ++i) s[i] += __uint_as_float(dpp<0x4e>(__float_as_uint(s[i])));
#pragma unroll
    for (int i = 0; i < R::kPasses; ++i) s[i] += __uint_as_float(dpp<0x141>(__float_as_uint(s[i])));
    if constexpr (R::kUnits == 16) {
#pragma unroll
      for (int i = 0; i < R::kPasses; ++i) s[i] += __uint_as_float(dpp<0x140>(__float_as_uint(s[i])));
    }
  }
  __device__ __forceinline__ void scale() {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u32x4 out[R::kPasses];
    float s[R::kPasses];
#pragma unroll
    for (int i = 0; i < R::kPasses; ++i) {
      out[i] = rows.w[i];
      if constexpr (!kF16In) {
#pragma unroll
        for (int j = 0; j < 4; ++j) out[i][j] = pair_f16(low_value<false>(rows.w[i][j]), high_value<false>(rows.w[i][j]));
      }
    }
    squares(out, s);
    // (Elements that fp16 does not hold make the sum large or not finite.)
    float least = s[0], most = s[0];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < R::kPasses; ++i) {
      least = fminf(least, s[i]), most = fmaxf(most, s[i]);
      nan = nan || s[i] != s[i];
      info[i] = RowInfo{0, s[i]};
    }
    if (__ballot(nan || !(least >= kLeast && most <= kMost))) {
#pragma unroll
      for (int i = 0; i < R::kPasses; ++i) {
        const bool plain = s[i] >= kLeast && s[i] <= kMost;
        u16x2 top = {0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, rows.w[i][j] & 0x7fff7fffu));
        const uint32_t largest = row_max<R::kUnits>(max((uint32_t)top[0], (uint32_t)top[1]));
        const bool bad = largest >= (kF16In ? 0x7c00u : 0x7f80u);
        const int e = largest == 0 || bad || plain ? 0 : min(__builtin_amdgcn_frexp_expf(token_value<kF16In>(largest)) + 1, 127);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t word = bad ? 0u : rows.w[i][j];
          out[i][j] = pair_f16(ldexp2(low_value<kF16In>(word), -e), ldexp2(high_value<kF16In>(word), -e));
        }
        info[i].e = bad ? kBadRow : e;
      }
      squares(out, s);
#pragma unroll
      for (int i = 0; i < R::kPasses; ++i) info[i].squares = s[i];
    }
#pragma unroll
    for (int i = 0; i < R::kPasses; ++i) rows.w[i] = out[i];
  }
  __device__ __forceinline__ void put(char* tile, RowInfo* to, int tid) const {
    rows.put(tile, tid);
    const unsigned u = (unsigned)local_copy(tid);
    if (u % R::kUnits == 0) {
#pragma unroll
      for (int i = 0; i < R::kPasses; ++i) to[u / R::kUnits + i * R::kRows] = info[i];
    }
  }
};

// What the walk needs of a chunk beside its tiles; t, s are tokens.
//   K'_t, Q'_t: scaled rows; rk_t, rq_t: what takes them to the keys and queries of the rule. The rule of K' has the step
// sizes beta rk^2 and the values V / rk, and the same states: what rk holds of a key's length stays in fp32.
struct Factors {
  float b[kC];  // beta rk: the share of V in what is to be learnt
  float h[kC];  // beta rk^2 e^G: that of K' S0
  float c[kC];  // e^{G_C - G}: what of D reaches the chunk's end
  float e[kC];  // e^G times 64, as P
  float f[kC];  // scale rq / 64: outputs; NaN from the first bad token on
  float s[kC];  // beta rk^2, for a walk by tokens
  float total;  // e^{G_C}; NaN with a bad token
  int steps;    // |b| < 2^steps
  int reach;    // |h K'| < 2^reach
};
// For the making of T and P alone.
struct Making {
  alignas(16) float G[kC];    // inclusive cumsum of g, and what its rounding left
  alignas(16) float rest[kC];
  alignas(16) float step[kC]; // beta rk^2
};

__device__ __forceinline__ int wave_max(int x) {
  x = max(x, (int)dpp<0xb1>((uint32_t)x));
  x = max(x, (int)dpp<0x4e>((uint32_t)x));
  x = max(x, (int)dpp<0x141>((uint32_t)x));
  x = max(x, (int)dpp<0x140>((uint32_t)x));
  return channel_max(x);
}
// A token's decays, one lane for each token: what does not wait for the chunk's rows.
struct Decays {
  float own;      // e^g
  float e, c;     // e^G, e^{G_C - G}
  float total;    // e^{G_C}
  uint64_t bad;   // tokens whose log decay is not allowed
};
__device__ __forceinline__ Decays put_decays(Making& mk, float g, int lane) {
  Decays d;
  const bool bad = !(g <= 0.f);
  d.bad = __ballot(bad);
  if (bad) g = 0.f;
  g = g < kMinLogDecay ? kMinLogDecay : g;
  d.own = __expf(g);
  const double G = prefix_sum((double)g);
  const uint64_t u = __builtin_bit_cast(uint64_t, G);
  const double end = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63) << 32 |
                                                    (uint32_t)__builtin_amdgcn_readlane((int)u, 63));
  d.e = __expf((float)G);
  d.c = __expf((float)(end - G));
  d.total = __expf((float)end);
  mk.G[lane] = (float)G;
  mk.rest[lane] = (float)(G - (double)(float)G);
  return d;
}
// A token's part of the chunk's numbers, one lane for each token, in two steps: what the making of T waits for, and what the chain does.
struct Numbers {
  float share, step, rq, length, beta;  // rq: f without its NaN
  int long_by;      // the chunk's longest raw key, as a power of two
  uint64_t all_bad;
  bool bad_q;
  __device__ __forceinline__ void put_steps(Making& mk, const DeltaPlan& p, const Decays& d, RowInfo k, RowInfo q, float of, int lane) {
    beta = of;
    const bool bad = k.e == kBadRow || !(fabsf(beta) < INFINITY);
    all_bad = __ballot(bad) | d.bad;
    bad_q = q.e == kBadRow;
    if (all_bad >> lane & 1) beta = 0.f, k = RowInfo{0, 0.f};
    if (k.squares == 0.f) beta = 0.f;  // nothing is learnt of a zero key, whatever its step size
    length = k.squares;
    if (p.normalize) {
      const float rk = rsqrtf(k.squares + ldexp2(kNormEps, -2 * k.e));
      rq = p.scale / kTimesP * rsqrtf(q.squares + ldexp2(kNormEps, -2 * q.e));
      share = beta * rk;
      step = share * rk;
      long_by = 0;
    } else {
      share = ldexp2(beta, k.e);
      step = ldexp2(beta, 2 * k.e);
      rq = ldexp2(p.scale / kTimesP, q.e);
      long_by = k.squares > 0.f ? k.e : -1000;
    }
    mk.step[lane] = step;
  }
  __device__ __forceinline__ void put_factors(Factors& to, const DeltaPlan& p, const Decays& d, int lane) const {
    int longest = 0;
    if (!p.normalize) {
      const int top = wave_max(long_by);
      longest = top == -1000 ? 0 : top;
    }
    // Step sizes that break |beta| |k|^2 <= 2 so far that the products' fp16 would: outputs and the final state are not finite.
    const bool wide = __ballot(!(fabsf(ldexp2(beta, 2 * longest)) < 0x1p28f)) != 0;
    const int first = all_bad ? __builtin_ctzll(all_bad) : kC;
    const float h = step * d.e;
    to.b[lane] = share;
    to.h[lane] = h;
    to.c[lane] = d.c;
    to.e[lane] = d.e * kTimesP;
    to.s[lane] = step;
    to.f[lane] = wide || lane >= first || bad_q ? __builtin_nanf("") : rq;
    const int steps = wave_max(exponent(fabsf(share))), reach = wave_max(exponent(fabsf(h) * __builtin_amdgcn_sqrtf(length)));
    if (lane == 0) {
      to.total = wide || all_bad ? __builtin_nanf("") : d.total;
      to.steps = steps;
      to.reach = reach;
    }
  }
};

// A's ten causal 16 x 16 blocks in fp32, each as [s][t] with rows of 20 floats; T's take their places.
constexpr int kBlockRow = 20, kBlock = 16 * kBlockRow;
__device__ __forceinline__ constexpr int block_at(int tt, int st) { return (tt * (tt + 1) / 2 + st) * kBlock; }

// Fragment (token tile tt, sources 32 b ..) of P or one term of T.
__device__ __forceinline__ f16x8 read_fragment(const char* p, int lane, int tt, int b) { return __builtin_bit_cast(f16x8, read_p(p, lane, tt, b)); }
// Tile (tt, st) of it, of which a lane holds token l % 16 and sources 4g + i.
__device__ __forceinline__ void put_fragment(char* p, int lane, int tt, int st, f16x4 x) {
  const int b = st >> 1;
  *reinterpret_cast<f16x4*>(p + fragment(tt, b) + (half_fragment(tt, b) ? lane * 8 : lane * 16 + (st & 1) * 8)) = x;
}

// The same of P's second term, a byte for each value.
constexpr int kRestP = kTermP / 2;
__device__ __forceinline__ f16x8 read_rest(const char* p, int lane, int tt, int b) {
  if (!half_fragment(tt, b)) return p_rest_operand(*reinterpret_cast<const u32x2*>(p + fragment(tt, b) / 2 + lane * 8));
  return p_rest_operand(u32x2{*reinterpret_cast<const uint32_t*>(p + fragment(tt, b) / 2 + lane * 4), 0u});
}
__device__ __forceinline__ void put_rest(char* p, int lane, int tt, int st, uint32_t x) {
  const int b = st >> 1;
  *reinterpret_cast<uint32_t*>(p + fragment(tt, b) / 2 + (half_fragment(tt, b) ? lane * 4 : lane * 8 + (st & 1) * 4)) = x;
}

// Making T and P, by four waves. The ten tiles (tt, st <= tt) of K' K'^T and K' Q'^T, rows s = 4g + i, column t = l % 16, are dealt
// out as rows of tiles: 0 and 1, 2, 3 but its last, and that one, by the wave that makes the chunk's numbers in the walk. Each wave has
// code of its own, in which all places are constants.
constexpr int kTileJobs = 3;
template <int W>
struct TileJobs {
  static constexpr int kCount = W < 3 ? 3 : 1;
  static constexpr int tt(int j) { return W == 0 ? (j > 0) : W == 1 ? 2 : 3; }
  static constexpr int st(int j) { return W == 0 ? (j == 2) : W < 3 ? j : 3; }
};
template <typename F>
__device__ __forceinline__ void by_wave(int w, F f) {
  if (w == 0) f(std::integral_constant<int, 0>());
  else if (w == 1) f(std::integral_constant<int, 1>());
  else if (w == 2) f(std::integral_constant<int, 2>());
  else f(std::integral_constant<int, 3>());
}
struct TileProducts {
  f32x4 kk[kTileJobs], kq[kTileJobs];
};
template <int K, int W>
__device__ __forceinline__ void tile_products(const char* k, const char* q, int lane, TileProducts& t) {
  typedef TileJobs<W> Jobs;
  constexpr int KB = K / 32;
#pragma unroll
  for (int j = 0; j < Jobs::kCount; ++j) t.kk[j] = t.kq[j] = zero4();
#pragma unroll
  for (int m = 0; m < KB; ++m) {
    f16x8 own_k, own_q;
#pragma unroll
    for (int j = 0; j < Jobs::kCount; ++j) {
      if (j == 0 || Jobs::tt(j) != Jobs::tt(j - 1)) {
        own_k = __builtin_bit_cast(f16x8, read_row<K>(k, lane, 16 * Jobs::tt(j), m));
        own_q = __builtin_bit_cast(f16x8, read_row<K>(q, lane, 16 * Jobs::tt(j), m));
      }
      const f16x8 s = Jobs::st(j) == Jobs::tt(j) ? own_k : __builtin_bit_cast(f16x8, read_row<K>(k, lane, 16 * Jobs::st(j), m));
      t.kk[j] = mfma(s, own_k, t.kk[j]);
      t.kq[j] = mfma(s, own_q, t.kq[j]);
    }
  }
}
// The decays between a tile's tokens, e^{G_t - G_s}. A difference of prefix sums is taken of their two parts each: exact but for 2^-24 of
// itself.
struct TileDecays {
  f32x4 of[kTileJobs];
};
template <int W>
__device__ __forceinline__ void tile_decays(const Making& mk, int lane, TileDecays& d) {
  typedef TileJobs<W> Jobs;
  f32x4 Gs[kTileJobs], rest_s[kTileJobs];
  float Gt[kTileJobs], rest[kTileJobs];
#pragma unroll
  for (int j = 0; j < Jobs::kCount; ++j) {
    const int t = 16 * Jobs::tt(j) + (lane & 15), s0 = 16 * Jobs::st(j) + 4 * (lane >> 4);
    Gt[j] = mk.G[t], rest[j] = mk.rest[t];
    Gs[j] = *reinterpret_cast<const f32x4*>(&mk.G[s0]), rest_s[j] = *reinterpret_cast<const f32x4*>(&mk.rest[s0]);
  }
#pragma unroll
  for (int j = 0; j < Jobs::kCount; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) d.of[j][i] = __expf((Gt[j] - Gs[j][i]) + (rest[j] - rest_s[j][i]));
}
// A's blocks and P's tiles; put_p(tt, st, x, rest) takes a tile of P.
template <int W, typename PutP>
__device__ __forceinline__ void put_tiles(float* blocks, const Making& mk, int lane, const TileProducts& p, const TileDecays& d, PutP put_p) {
  typedef TileJobs<W> Jobs;
  const int g4 = lane >> 4, l16 = lane & 15;
  float step[kTileJobs];
#pragma unroll
  for (int j = 0; j < Jobs::kCount; ++j) step[j] = mk.step[16 * Jobs::tt(j) + l16];
  float* const at = blocks + 4 * g4 * kBlockRow + l16;
#pragma unroll
  for (int j = 0; j < Jobs::kCount; ++j) {
    float* to = at + block_at(Jobs::tt(j), Jobs::st(j));
    const bool diagonal = Jobs::tt(j) == Jobs::st(j);
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = p.kk[j][i] * (d.of[j][i] * step[j]);
      x[i] = p.kq[j][i] * (d.of[j][i] * kTimesP);
      to[i * kBlockRow] = diagonal && 4 * g4 + i >= l16 ? 0.f : a;
      if (diagonal && 4 * g4 + i > l16) x[i] = 0.f;
    }
    const u32x2 first = {pair_f16(x[0], x[1]), pair_f16(x[2], x[3])};
    put_p(Jobs::tt(j), Jobs::st(j), __builtin_bit_cast(f16x4, first), p_rest(x, first));
  }
}

// The diagonal blocks of T, one for each 16 lanes, a column to a lane.
__device__ __forceinline__ void invert_diagonal(float* blocks, int lane) {
  float* a = blocks + block_at(lane >> 4, lane >> 4);
  const int j = lane & 15;
  float x[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) x[t] = t == j ? 1.f : 0.f;
#pragma unroll
  for (int part = 0; part < 3; ++part) {  // a part's reads first: one wait for LDS each
    constexpr int kFrom[4] = {0, 3, 8, 15};
    f32x4 col[15][4];
#pragma unroll
    for (int s = kFrom[part]; s < kFrom[part + 1]; ++s)
#pragma unroll
      for (int c = (s + 1) / 4; c < 4; ++c) col[s][c] = *reinterpret_cast<const f32x4*>(a + s * kBlockRow + 4 * c);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = kFrom[part]; s < kFrom[part + 1]; ++s)
#pragma unroll
      for (int t = s + 1; t < 16; ++t) x[t] -= col[s][t / 4][t % 4] * x[s];
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) *reinterpret_cast<f32x4*>(a + j * kBlockRow + 4 * c) = f32x4{x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]};
}
// d + L^T R^T for blocks stored as [s][t]: of L (r, u) at [u][r] is the left operand, row u; of R (t, r) the right one.
__device__ __forceinline__ f32x4 left_block(const float* at, int lane) { return *reinterpret_cast<const f32x4*>(at + (lane & 15) * kBlockRow + 4 * (lane >> 4)); }
__device__ __forceinline__ f32x4 right_block(const float* at, int lane) {
  f32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = at[(4 * (lane >> 4) + i) * kBlockRow + (lane & 15)];
  return y;
}
__device__ __forceinline__ f32x4 product(f32x4 left, f32x4 right, f32x4 d) {
#pragma unroll
  for (int i = 0; i < 4; ++i) d = mfma32(left[i], right[i], d);
  return d;
}
// T's blocks below the diagonal, in two parts with a barrier of the four waves between them (and one before each): those
// beside the diagonal (and the diagonal's own as fragments), then the square of four. put_t(tt, st, x) takes a block, rows s = 4g + i,
// column t = l % 16. The first wave, which inverts the diagonal, has no part in them.
template <typename PutT>
__device__ __forceinline__ void near_blocks(float* blocks, int lane, int w, PutT put_t) {
  if (w == 0) return;
  const auto block = [&](int tt, int st) { return blocks + block_at(tt, st); };
  if (w == 3) {
    f32x4 y[4];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) y[tt] = right_block(block(tt, tt), lane);
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) put_t(tt, tt, y[tt]);
    return;
  }
  const auto make = [&](int t, int s) __attribute__((always_inline)) {
    float* at = block(t, s);
    const f32x4 low = left_block(at, lane), right = right_block(block(t, t), lane), top = left_block(block(s, s), lane);
    const f32x4 y = -product(top, product(low, right, zero4()), zero4());
    put_t(t, s, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) at[(4 * (lane >> 4) + i) * kBlockRow + (lane & 15)] = y[i];
  };
  if (w == 1) make(1, 0);
  else make(3, 2);
}
template <typename PutT>
__device__ __forceinline__ void far_blocks(const float* blocks, int lane, int w, PutT put_t) {
  if (w == 0) return;
  const auto block = [&](int tt, int st) { return blocks + block_at(tt, st); };
  const f32x4 t22 = right_block(block(2, 2), lane), t32 = right_block(block(3, 2), lane), t33 = right_block(block(3, 3), lane);
  const f32x4 a21 = left_block(block(2, 1), lane), a31 = left_block(block(3, 1), lane);
  if (w == 3) {  // (2, 1) and (3, 1)
    const f32x4 t11 = left_block(block(1, 1), lane);
    f32x4 z2 = zero4(), z3 = zero4(), y2 = zero4(), y3 = zero4();
#pragma unroll
    for (int i = 0; i < 4; ++i) z3 = mfma32(a21[i], t32[i], z3), z2 = mfma32(a21[i], t22[i], z2);
    z3 = product(a31, t33, z3);
#pragma unroll
    for (int i = 0; i < 4; ++i) y2 = mfma32(t11[i], z2[i], y2), y3 = mfma32(t11[i], z3[i], y3);
    put_t(2, 1, -y2);
    put_t(3, 1, -y3);
    return;
  }
  const f32x4 a20 = left_block(block(2, 0), lane), a30 = left_block(block(3, 0), lane);
  const f32x4 t00 = left_block(block(0, 0), lane), t10 = left_block(block(1, 0), lane);
  f32x4 z0 = zero4(), z1 = zero4(), y0 = zero4(), y1 = zero4();
  if (w == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) z0 = mfma32(a20[i], t32[i], z0), z1 = mfma32(a21[i], t32[i], z1);
#pragma unroll
    for (int i = 0; i < 4; ++i) z0 = mfma32(a30[i], t33[i], z0), z1 = mfma32(a31[i], t33[i], z1);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) z0 = mfma32(a20[i], t22[i], z0), z1 = mfma32(a21[i], t22[i], z1);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y0 = mfma32(t00[i], z0[i], y0), y1 = mfma32(t10[i], z1[i], y1);
  const f32x4 y = -(y0 + y1);
  if (w == 1) put_t(3, 0, y);
  else put_t(2, 0, y);
}
// A block of T in two terms.
struct Terms {
  f16x4 hi, lo;
};
__device__ __forceinline__ Terms t_terms(f32x4 x) {
  const u32x2 hi = {pair_f16(x[0], x[1]), pair_f16(x[2], x[3])}, lo = {rest_up(x[0], x[1], hi[0]), rest_up(x[2], x[3], hi[1])};
  return Terms{__builtin_bit_cast(f16x4, hi), __builtin_bit_cast(f16x4, lo)};
}

// Powers of two that hold one value channel in fp16's range: the state S' = S 2^s, what is to be learnt X' = X 2^x. X' is
// kept in [1, 16) before the keys' products (|X'| is then at most 2^7.6, and no stable rule makes more than 64 times that of it: below
// fp16's largest number, 2^16), and S' at the same power where that leaves it in [2^-9, 2^12): else it has a power of its own.
struct Ranges {
  int s, x;
};
// state: exponent of the largest |S'| at 2^now; learnt: of the largest X. kNoExponent or less: none.
__device__ __forceinline__ Ranges ranges_of(int now, int state, int learnt) {
  constexpr int kNone = kNoExponent / 2, kMost = 120, kTop = 3;
  Ranges r = {now, now};
  if (learnt > kNone && (learnt + now > 4 || learnt + now < 1)) r.x = min(max(kTop - learnt, -kMost), kMost);
  const int there = state + r.x - now;
  r.s = state > kNone && (there > 12 || there < -8) ? min(max(now + kTop - state, -kMost), kMost) : r.x;
  // What is this far below the other is nothing beside it, or is found too small (fades).
  r.x = min(r.x, r.s + 60);
  r.s = min(r.s, r.x + 100);
  return r;
}
// Whether both may stay where they are (a plain sight: some that may stay are not seen).
__device__ __forceinline__ bool stays(int now, int state, int learnt) { return (unsigned)(learnt + now - 1) <= 3u && (unsigned)(state + 8) <= 20u; }
// A channel's powers of two.
struct Scale {
  int ex;          // of the state
  int apart;       // X's less the state's; the state takes X's with the chunk
  float v;         // X's
  f32x4 out;       // its inverse, of the channels 4g + i, for tiles that hold channels as rows
  __device__ __forceinline__ void set(int lane, int to) {
    v = ldexp2(1.f, to);
    const float back = ldexp2(1.f, -to);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __shfl(back, 4 * (lane >> 4) + i);
  }
};

// What a token's output and state are made of: of the state before the chunk and of what it and those before it learn, each as far as
// it has decayed, the largest, L_t = max(e^{g_t} L_{t-1}, |X'_t|). Beside the share of 2^-22 of itself that a term may be off, T and what is to be
// learnt may be off by 2^-37 and P by 2^-34, wherever the range's top (2^4) stands; where every L_t is at least kLeastShare that is little of
// what the token is made of: over 7500 random batches (values and steps of 2^+-30, resets, raw keys) states were within 2^-16 of L_t, and outputs too,
// beside their rounding. A chunk in which some L_t is less (a large value behind small ones, small ones behind a large one that
// was forgotten) is walked token by token. With random values that is one chunk and wave in 10^5, where decays are steepest.
template <bool kF16In>
constexpr float kLeastShare = kF16In ? 0x1p-17f : 0x1p-18f;

// The plan read again from the kernel's arguments, for what is rare: with one copy of it for all the walk spills scalars (2 %).
__device__ __forceinline__ const DeltaPlan& plan_again() {
  typedef const __attribute__((address_space(4))) DeltaPlan* Arguments;
  Arguments arguments = (Arguments)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(arguments));
  return *(const DeltaPlan*)arguments;
}
// The decays of tokens `first` to first + 3, of which `count` are the chunk's, as the chunks count them.
__device__ __forceinline__ f32x4 decays_at(const DeltaPlan& p, int64_t first, int count, int h) {
  f32x4 d = {1.f, 1.f, 1.f, 1.f};
  if (!p.g || count <= 0) return d;
  uint32_t bits[4];
  const int64_t at = p.g_per_token ? first * p.H + h : h, step = p.g_per_token ? p.H : 0;
  if (p.g_bf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) bits[i] = (uint32_t)reinterpret_cast<const uint16_t*>(p.g)[at + min(i, count - 1) * step] << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) bits[i] = reinterpret_cast<const uint32_t*>(p.g)[at + min(i, count - 1) * step];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float g = __uint_as_float(bits[i]);
    if (i < count && g <= 0.f) d[i] = __expf(fmaxf(g, kMinLogDecay));
  }
  return d;
}
// L over a run of four tokens: out = max(in * all, own).
struct Fading {
  f32x4 decay, x;
  float all, own;
  __device__ __forceinline__ void set(f32x4 decays, f32x4 of) {
    decay = decays;
    all = 1.f, own = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = of[i] == of[i] ? fabsf(of[i]) : INFINITY;  // not finite: not to be found too small
      all *= decay[i];
      own = fmaxf(own * decay[i], x[i]);
    }
  }
  // The four runs of 16 tokens follow each other in the lanes of a channel: L before this lane's, and, in `through`, behind the last.
  __device__ __forceinline__ float before(float& through, int lane) const {
    float mine = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float a = __shfl(all, (lane & 15) + 16 * g), o = __shfl(own, (lane & 15) + 16 * g);
      if (lane >> 4 == g) mine = through;
      through = fmaxf(through * a, o);
    }
    return mine;
  }
  // Whether some L is too small. (Where nothing at all is left the chunk's products are zeros too.)
  __device__ __forceinline__ bool fades(float L, float least) const {
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      L = fmaxf(L * decay[i], x[i]);
      found = found || (L > 0.f && L < least);
    }
    return found;
  }
};
// A lower bound of L before the chunk, and whether the state alone holds L up to the chunk's end.
__device__ __forceinline__ float state_share(int state, int apart) { return state > kNoExponent / 2 ? ldexp2(0.5f, state + apart) : 0.f; }
__device__ __forceinline__ bool state_lasts(int state, int apart, float total) { return state + apart + exponent(total) >= -12; }  // 2^-14

}  // namespace kda
