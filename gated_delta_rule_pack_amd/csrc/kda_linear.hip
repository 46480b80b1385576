// Linear attention with a decay for each head, chunked form for prompts.
//
// Per sequence and value head, S_t = e^{g_t} S_{t-1} + v_t k_t^T and o_t = scale S_t q_t. A chunk
// of 64 tokens with G the inclusive cumsum of g in it and S0 the state before it gives
//
//   P[t, s] = scale (q_t . k_s) e^{G_t - G_s}  (s <= t)
//   O = P V + diag(scale e^G) Q S0^T
//   S = e^{G_C} S0 + (diag(e^{G_C - G}) V)^T K
//
// Every factor inside a chunk is the exponential of a sum of log decays over a run of its tokens,
// taken of the difference of 64-bit prefix sums: nothing is divided, so no decay is too steep. From
// chunk to chunk the state is an fp32 recurrence: a chunk's product with e^{G_C}, that factor's own
// rounding and the sum leave at most 3 2^-24 of its terms, which add up where the decay is slow (40000 tokens at
// g = -1e-5 in one segment, terms of one sign: 1.1e-5 rel-L2, in the policy's segments 2e-6).
//
// Split. The tokens of all sequences lie on one axis (LinearPlan) that is cut into equal
// segments; a workgroup walks one segment of one value head. With more than one segment,
// linear_maps walks the part of each segment whose sequence crosses the segment's end, for the
// state there; linear_combine chains those states along each sequence; linear_output walks
// every segment with its true start states. Nothing but the bounds' own values decides which
// tokens a workgroup takes, so a call needs no host tables.
//
// A workgroup takes all V state rows, or a slice of 64 of them where there are few segments and
// heads. Each wave holds 16 of its rows in fp32 MFMA accumulators, S^T[k][v], for the whole walk.
// Lanes (l, g = l / 16): an accumulator tile of K^T U holds column l % 16 (v), rows 4g + i. Tile 2m is
// made of channels 32m + 8g + i and tile 2m + 1 of 32m + 8g + 4 + i (i < 4), so that a lane's two
// tiles are eight channels in a row: an operand of Q S^T as it stands, and 16 or 32 bytes of a stored
// state. P, made as K Q^T, meets V in the order (4g + i, 16 + 4g + i) of its tiles. Neither the state
// nor P is ever transposed.
//
// What bounds it. A long prompt reads k and v twice (map and output), q once, and writes the outputs:
// 1 x 32768 tokens at H = 32, fp32 state, move 1.7 GB in 410 us (map 121, combine 10, output 253),
// 4.1 TB/s. The map walk is bound by memory. The output walk is by both: with one term each for P and the state it took
// 237 us, as long as without any arithmetic, and their second terms, for which it can not wait less, add 16. 128 ragged
// prompts (131 K tokens at H = 12, bf16 pool) take 475 us (map 57, output 395). A workgroup alone on a compute
// unit takes 3 us for a chunk, 2 us in the map walk, by the length of its chain of LDS reads, products and three
// barriers: 1 x 4096 at H = 12 takes 41 us that way.
#include <hip/hip_runtime.h>

#include "kda_device.h"
#include "kda_linear.h"
#include "kda_walk.h"

namespace kda {
namespace {

// bf16 is the upper half of fp32: the upper halves of a and b, a below.
constexpr uint32_t kTop = 0xffff0000u;
__device__ __forceinline__ uint32_t top_halves(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
}

// Both rounded to nearest, a below.
__device__ __forceinline__ uint32_t both_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 r = {to_bf16(a), to_bf16(b)};
  return __builtin_bit_cast(uint32_t, r);
}

// a and b in two bf16 terms for a product with bf16 values: the first cut off, the second what that leaves,
// rounded. The first leaves less than 2^-7 of the value and the second 2^-8 of that: 2^-15 in all. (Both rounded
// leave 2^-17 and take 407 instead of 403 us for 32768 tokens at H = 32.)
struct TwoTerms {
  uint32_t hi, lo;
};
__device__ __forceinline__ TwoTerms two_terms(float a, float b) {
  return TwoTerms{top_halves(a, b), both_bf16(a - __uint_as_float(__float_as_uint(a) & kTop), b - __uint_as_float(__float_as_uint(b) & kTop))};
}

template <int K, int V, bool kOut>
struct Shared {
  alignas(16) char k[kC * kRowBytes<K>];
  alignas(16) char v[kC * kRowBytes<V>];  // then, once every wave has its columns, the outputs
  alignas(16) char q[kOut ? kC * kRowBytes<K> : 16];
  // P (terms()), and between a sequence's chunks and the next one's, when no wave reads P, 1 KB of each
  // wave's for its state. K = 128, V = 64 has P in the q tile, which takes a barrier more and leaves room for a
  // third workgroup on a compute unit (64 ragged prompts at H = 24 take 354 instead of 383 us; 168 K tokens at
  // H = 1, which leave one to a unit, 91 instead of 86).
  static constexpr bool kTermsInQ = kOut && K == 128 && V == 64;
  static constexpr int kStage = 1024 * kWavesOf<V>;
  alignas(16) char p[kOut && !kTermsInQ && 2 * kTermP > kStage ? 2 * kTermP : kStage];
  __device__ __forceinline__ char* terms() { return kTermsInQ ? q : p; }
  struct Decays {
    double G[kC];             // inclusive cumsum of g
    alignas(16) float c[kC];  // e^{G_C - G}
    float e[kC];              // scale e^G
    float total;              // e^{G_C}
  } decays[2];                // of this chunk and the next
};

template <typename D>
__device__ __forceinline__ void put_decays(D& d, float g, float scale, int lane) {
  lane = local_copy(lane);
  const double G = prefix_sum((double)(g < kMinLogDecay ? kMinLogDecay : g));
  const uint64_t u = __builtin_bit_cast(uint64_t, G);
  const double end = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63) << 32 |
                                                    (uint32_t)__builtin_amdgcn_readlane((int)u, 63));
  d.G[lane] = G;
  d.c[lane] = __expf((float)(end - G));
  d.e[lane] = scale * __expf((float)G);
  if (lane == 0) d.total = __expf((float)end);
}

// Whether a wave's columns of V are finite, by their largest exponent.
template <int VT>
__device__ __forceinline__ bool all_finite(const bf16x8 (&raw)[2][VT]) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  u16x2 top = {0, 0};
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      const u32x4 w = __builtin_bit_cast(u32x4, raw[b][vt]);
#pragma unroll
      for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    }
  return __ballot(top[0] >= 0x7f80 || top[1] >= 0x7f80) == 0;
}
// Zeros for what is not finite in a column's tokens t0 + i and t0 + 16 + i (i < 4); first: the earliest such token.
__device__ __forceinline__ void take_finite(bf16x8& x, int t0, int& first) {
  u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t half = i & 1 ? kTop : ~kTop;
    if ((w[i / 2] & half & 0x7f807f80u) == (half & 0x7f807f80u)) {
      w[i / 2] &= ~half;
      first = min(first, t0 + (i & 3) + (i & 4) * 4);
    }
  }
  x = __builtin_bit_cast(bf16x8, w);
}

// One chunk of `count` tokens: P and the outputs (kOut), then the state.
// next(i) issues the loads of part i of the next chunk (0: k, 1: v, 2: q), spread over the work: issued
// at once they hold every wave for the 48 KB to pass.
template <int K, int V, bool kOut, int kTerms, typename Next>
__device__ __forceinline__ void chunk(const LinearPlan& p, Shared<K, V, kOut>& sh, const typename Shared<K, V, kOut>::Decays& dec,
                                      Walk<K, V>& walk, int wave, int lane_, Next next) {
  const int lane = local_copy(lane_);
  constexpr int VT = Walk<K, V>::VT, KT = Walk<K, V>::KT, KB = K / 32;
  const int g = lane >> 4, l16 = lane & 15;
  bf16x8 raw[2][VT];
  next(0);
  if constexpr (kOut) {
    // P^T tiles (token tile tt, source tile st <= tt), rows s = 4 g + i, column t: ten, dealt out
    // over the waves. Two terms each: the product with V is a bf16 MFMA with fp32 sums.
    constexpr int kDeal = (10 + kWavesOf<V> - 1) / kWavesOf<V>;
    u32x2 hi[kDeal], lo[kDeal];
    const auto put_p = [&](int j) {
      const int tile = j * kWavesOf<V> + wave, tt = tile_t(tile), st = tile_s(tile), b = st >> 1;
      char* at = sh.terms() + fragment(tt, b) + (half_fragment(tt, b) ? lane * 8 : lane * 16 + (st & 1) * 8);
      *reinterpret_cast<u32x2*>(at) = hi[j];
      *reinterpret_cast<u32x2*>(at + kTermP) = lo[j];
    };
#pragma unroll
    for (int j = 0; j < kDeal; ++j) {
      const int tile = j * kWavesOf<V> + wave;
      if (tile >= 10) break;
      const int tt = tile_t(tile), st = tile_s(tile), t = 16 * tt + l16;
      f32x4 d = zero4();
#pragma unroll
      for (int m = 0; m < KB; ++m)
        d = mfma(read_row<K>(sh.k, lane, 16 * st, m), read_row<K>(sh.q, lane, 16 * tt, m), d);
      const double Gt = dec.G[t];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = 16 * st + 4 * g + i;
        float x = d[i] * p.scale * __expf((float)(Gt - dec.G[s]));
        asm("" : "+v"(x));  // a select, not a branch around the exponential
        d[i] = s <= t ? x : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const TwoTerms w = two_terms(d[2 * i], d[2 * i + 1]);
        hi[j][i] = w.hi, lo[j][i] = w.lo;
      }
      if constexpr (!Shared<K, V, kOut>::kTermsInQ) put_p(j);
    }
    next(1);
    // Q S^T, transposed: rows v = 4 g + i, column t. The fp32 state goes in as two terms:
    // with one each for it and P the outputs are off by 2.35e-3 (rel-L2), with two by the 1.66e-3 that their own
    // rounding to bf16 makes (32768 tokens at H = 32: 378 and 405 us).
    f32x4 acc[VT][4];
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) acc[vt][tt] = zero4();
#pragma unroll
    for (int m = 0; m < KB; ++m) {
      bf16x8 hi[VT], lo[VT];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        u32x4 h, l;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 x = walk.S[vt][2 * m + i / 2];
          const TwoTerms w = two_terms(x[2 * i & 3], x[(2 * i + 1) & 3]);
          h[i] = w.hi, l[i] = w.lo;
        }
        hi[vt] = __builtin_bit_cast(bf16x8, h), lo[vt] = __builtin_bit_cast(bf16x8, l);
      }
      // Two token tiles at a time, term by term: no product waits for the one before it.
#pragma unroll
      for (int tt = 0; tt < 4; tt += 2) {
        const bf16x8 b0 = read_row<K>(sh.q, lane, 16 * tt, m), b1 = read_row<K>(sh.q, lane, 16 * tt + 16, m);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          acc[vt][tt] = mfma(lo[vt], b0, acc[vt][tt]);
          acc[vt][tt + 1] = mfma(lo[vt], b1, acc[vt][tt + 1]);
          acc[vt][tt] = mfma(hi[vt], b0, acc[vt][tt]);
          acc[vt][tt + 1] = mfma(hi[vt], b1, acc[vt][tt + 1]);
        }
      }
    }
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      const float e = dec.e[16 * tt + l16];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) acc[vt][tt] *= e;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) raw[b][vt] = read_col<V, false>(sh.v, lane, 32 * b, wave * VT + vt);
    if (!all_finite<VT>(raw)) {
      // The zeros of P would make NaN of such a value in the tokens before it too. Its channel becomes NaN from its
      // token on and in the state; the products go on with the finite values.
      const int lane = local_copy(lane_), g = lane >> 4, l16 = lane & 15;
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        int first = kC;
#pragma unroll
        for (int b = 0; b < 2; ++b) take_finite(raw[b][vt], 32 * b + 4 * g, first);
        first = min(first, __shfl_xor(first, 16));
        first = min(first, __shfl_xor(first, 32));
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
          if (first < kC) walk.S[vt][kt] = zero4() + __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t0 = __shfl(first, 4 * g + i);
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
            if (16 * tt + l16 >= t0) acc[vt][tt][i] = __builtin_nanf("");
        }
      }
    }
    next(2);
    if constexpr (Shared<K, V, kOut>::kTermsInQ) {
      barrier_lds();  // q
#pragma unroll
      for (int j = 0; j < kDeal; ++j)
        if (j * kWavesOf<V> + wave < 10) put_p(j);
    }
    barrier_lds();  // P
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
      for (int b = 0; b <= tt / 2; ++b) {
        const bf16x8 lo = read_p(sh.terms() + kTermP, lane, tt, b), hi = read_p(sh.terms(), lane, tt, b);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) acc[vt][tt] = mfma(raw[b][vt], lo, acc[vt][tt]);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) acc[vt][tt] = mfma(raw[b][vt], hi, acc[vt][tt]);
      }
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        const f32x4 o = acc[vt][tt];
        const bf16x4 b = {to_bf16(o[0]), to_bf16(o[1]), to_bf16(o[2]), to_bf16(o[3])};
        *reinterpret_cast<bf16x4*>(sh.v + row_at<V>(16 * tt + l16) + ((wave * VT + vt) * 16 + 4 * g) * 2) = b;
      }
    }
  } else {
    next(1);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) raw[b][vt] = read_col<V, false>(sh.v, lane, 32 * b, wave * VT + vt);
  }
  // State. The decayed values x (fp32) go in as bf16 terms against the stored keys, which are bf16.
  // Three terms of 8 bits each, cut off rather than rounded, are x exactly: the state keeps fp32
  // accuracy. Two rounded terms leave 2^-17 of x (8e-6) at most, which serves where the state is stored in 16
  // bits (fp16: 2^-12 of it) or, without one, goes into outputs alone.
  const float total = dec.total;
#pragma unroll
  for (int vt = 0; vt < VT; ++vt)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) walk.S[vt][kt] *= total;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    bf16x8 term[kTerms][VT];  // the largest last
    const f32x4 c0 = *reinterpret_cast<const f32x4*>(&dec.c[32 * b + 4 * g]);
    const f32x4 c1 = *reinterpret_cast<const f32x4*>(&dec.c[32 * b + 16 + 4 * g]);
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      const u32x4 w = __builtin_bit_cast(u32x4, raw[b][vt]);
      u32x4 t[kTerms];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 c = i < 2 ? c0 : c1;
        const float x0 = __uint_as_float(w[i] << 16) * c[2 * i & 3], x1 = __uint_as_float(w[i] & kTop) * c[(2 * i + 1) & 3];
        if constexpr (kTerms == 3) {
          const float r0 = x0 - __uint_as_float(__float_as_uint(x0) & kTop), r1 = x1 - __uint_as_float(__float_as_uint(x1) & kTop);
          const float s0 = r0 - __uint_as_float(__float_as_uint(r0) & kTop), s1 = r1 - __uint_as_float(__float_as_uint(r1) & kTop);
          t[2][i] = top_halves(x0, x1);
          t[1][i] = top_halves(r0, r1);
          t[0][i] = top_halves(s0, s1);
        } else {
          t[1][i] = both_bf16(x0, x1);
          t[0][i] = both_bf16(x0 - __uint_as_float(t[1][i] << 16), x1 - __uint_as_float(t[1][i] & kTop));
        }
      }
#pragma unroll
      for (int j = 0; j < kTerms; ++j) term[j][vt] = __builtin_bit_cast(bf16x8, t[j]);
    }
    // Two tiles of K at a time, term by term: no product waits for the one before it.
#pragma unroll
    for (int kt = 0; kt < KT; kt += 2) {
      const bf16x8 k0 = read_col<K, true>(sh.k, lane, 32 * b, kt), k1 = read_col<K, true>(sh.k, lane, 32 * b, kt + 1);
#pragma unroll
      for (int j = 0; j < kTerms; ++j) {
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          walk.S[vt][kt] = mfma(k0, term[j][vt], walk.S[vt][kt]);
          walk.S[vt][kt + 1] = mfma(k1, term[j][vt], walk.S[vt][kt + 1]);
        }
      }
    }
  }
}

// A sequence of one token: the recurrent step on the walk's registers, in fp32. No wave waits for
// another, so a batch's single tokens run as 8 KB of state in flight for every wave.
template <int K, int V>
__device__ __forceinline__ void single(const LinearPlan& p, Walk<K, V>& walk, const __bf16* q, const __bf16* k, const __bf16* v,
                                       __bf16* out, int64_t token, int h, int wave, int lane_) {
  constexpr int VT = Walk<K, V>::VT, KT = Walk<K, V>::KT;
  const int lane = local_copy(lane_), g = lane >> 4, row = wave * VT * 16 + (lane & 15);
  float decay = 1.f;
  if (p.g) {
    const int64_t at = p.g_per_token ? token * p.H + h : h;
    decay = __expf(p.g_bf16 ? (float)reinterpret_cast<const __bf16*>(p.g)[at] : reinterpret_cast<const float*>(p.g)[at]);
  }
  float x[VT], o[VT];
#pragma unroll
  for (int vt = 0; vt < VT; ++vt) x[vt] = from_bf16(v[token * p.v_t + row + 16 * vt]), o[vt] = 0.f;
#pragma unroll
  for (int m = 0; m < KT / 2; ++m) {
    const bf16x8 kk = *reinterpret_cast<const bf16x8*>(k + token * p.k_t + 32 * m + 8 * g);
    const bf16x8 qq = *reinterpret_cast<const bf16x8*>(q + token * p.q_t + 32 * m + 8 * g);
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f32x4& S = walk.S[vt][2 * m + j / 4];
        S[j % 4] = S[j % 4] * decay + x[vt] * (float)kk[j];
        o[vt] += S[j % 4] * (float)qq[j];
      }
  }
#pragma unroll
  for (int vt = 0; vt < VT; ++vt) {
    o[vt] += __shfl_xor(o[vt], 16);
    o[vt] += __shfl_xor(o[vt], 32);
    if (g == 0) out[token * p.o_t + row + 16 * vt] = to_bf16(p.scale * o[vt]);
  }
}

// Walks segment `seg` of head h. kOut: every token, with outputs and final states; else only
// the sequence that crosses the segment's end, for its map.
template <int K, int V, bool kOut, int kTerms>
__global__ __launch_bounds__(64 * kWavesOf<V>, V == 128 ? 4 : 3) void linear_walk(const LinearPlan p) {
  constexpr int kThreads = 64 * kWavesOf<V>;
  __shared__ Shared<K, V, kOut> sh;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int slice = blockIdx.x % p.slices, unit = blockIdx.x / p.slices;
  const int seg = unit / p.H, h = unit % p.H, v0 = slice * V;
  const int64_t a = (int64_t)seg * p.seg_len, b = a + p.seg_len;
  const int64_t plane = (int64_t)K * V;  // of the slice
  const int64_t border = ((int64_t)unit * p.slices + slice) * plane;  // this segment's entry in maps and initials
  const __bf16* q = reinterpret_cast<const __bf16*>(p.q) + (h / p.group) * p.q_h;
  const __bf16* k = reinterpret_cast<const __bf16*>(p.k) + (h / p.group) * p.k_h;
  const __bf16* v = reinterpret_cast<const __bf16*>(p.v) + h * p.v_h + v0;
  __bf16* out = reinterpret_cast<__bf16*>(p.out) + h * p.o_h + v0;

  int n = find_sequence(p, kOut ? a : b - 1, lane);
  int begin = bound(p, n), end = bound(p, n + 1);
  Slots slots = slots_of(p, n);
  if constexpr (!kOut) {
    const int64_t start = begin + (int64_t)n * p.head_cost;
    const bool crosses = end > begin && start < b && start + (end - begin) > b;
    if (h == 0 && slice == 0 && tid == 0) p.spans[seg] = crosses ? (start >= a ? 1 : 2) : 0;
    if (!crosses) return;
  }
  char* stage = sh.p + wave * 1024;
  Walk<K, V> walk;
  Rows<K, kThreads> rq, rk;
  Rows<V, kThreads> rv;
  float g_next = 0.f;  // this lane's token of the next chunk
  auto fetch = [&](int part, int64_t first, int count) {
    if (part == 0) {
      g_next = 0.f;
      if (wave == 3 && p.g && lane < count) {
        const int64_t at = p.g_per_token ? (first + lane) * p.H + h : h;
        g_next = p.g_bf16 ? (float)reinterpret_cast<const __bf16*>(p.g)[at] : reinterpret_cast<const float*>(p.g)[at];
      }
      rk.load(k, p.k_t, first, count, tid);
    } else if (part == 1) {
      rv.load(v, p.v_t, first, count, tid);
    } else if constexpr (kOut) {
      rq.load(q, p.q_t, first, count, tid);
    }
  };
  while (true) {
    // The next sequence's bound and slots are on their way while this one is walked.
    const bool last = !kOut || n + 1 >= p.N;
    const int next_end = last ? end : bound(p, n + 2);
    const Slots next_slots = last ? slots : slots_of(p, n + 1);
    const int len = max(end - begin, 0);
    const int64_t start = begin + (int64_t)n * p.head_cost;
    const int t0 = (int)max((int64_t)0, a - start), t1 = (int)min((int64_t)len, b - start);
    if (kOut && len <= 1) {
      // An empty sequence stands in the stretch before its place, from which find_sequence finds it.
      const int64_t place = start - (len == 0 && n > 0);
      if (place >= a && place < b) {
        walk.zero();
        if (slots.from >= 0) walk.load_plane(p, stage, plane_at(p, slots.from, h), v0, wave, lane);
        if (len == 1) single<K, V>(p, walk, q, k, v, out, begin, h, wave, lane);
        if (slots.to >= 0) walk.store_plane(p, stage, plane_at(p, slots.to, h), v0, wave, lane);
      }
    } else if (t0 < t1) {
      int64_t first = (int64_t)begin + t0;
      int left = t1 - t0;
      for (int part = 0; part < 3; ++part) fetch(part, first, min(left, kC));
      // Start state. A sequence that goes on after this segment leaves its final state from
      // another workgroup, perhaps in the plane it starts from: the output walk starts it from
      // the copy that the map walk made.
      walk.zero();
      if (t0 == 0) {
        if (slots.from >= 0) {
          if (kOut && t1 < len) {
            walk.load(p.initials + border, wave, lane);
          } else {
            walk.load_plane(p, stage, plane_at(p, slots.from, h), v0, wave, lane);
            if (!kOut) walk.store(p.initials + border, wave, lane);
          }
        }
      } else if (kOut) {
        walk.load(p.maps + border - p.H * p.slices * plane, wave, lane);
      }
      float decay = 1.f;
      int turn = 0;
      if (wave == 3) put_decays(sh.decays[0], g_next, p.scale, lane);
      while (left > 0) {
        const int count = min(left, kC);
        if constexpr (kOut) rq.put(sh.q, tid);
        rk.put(sh.k, tid);
        rv.put(sh.v, tid);
        barrier_lds();
        const int64_t here = first;
        first += count;
        left -= count;
        chunk<K, V, kOut, kTerms>(p, sh, sh.decays[turn], walk, wave, lane, [&](int part) {
          if (left > 0) fetch(part, first, min(left, kC));
        });
        decay *= sh.decays[turn].total;
        turn ^= 1;
        // Wave 3 has few tiles of P.
        if (wave == 3 && left > 0) put_decays(sh.decays[turn], g_next, p.scale, lane);
        barrier_lds();
        if constexpr (kOut) Rows<V, kThreads>::store(sh.v, out, p.o_t, here, count, tid);
      }
      if constexpr (kOut) {
        if (t1 == len && slots.to >= 0) walk.store_plane(p, stage, plane_at(p, slots.to, h), v0, wave, lane);
      } else {
        walk.store(p.maps + border, wave, lane);
        if (slice == 0 && tid == 0) p.decays[(int64_t)seg * p.H + h] = decay;
      }
    }
    if (last) break;
    ++n;
    begin = end, end = next_end, slots = next_slots;
    if (begin + (int64_t)n * p.head_cost - 1 >= b) break;
  }
}

// Chains the segments' states: map s becomes the true state at the end of segment s. The chain
// runs along each element by itself: a thread owns kWidth elements and loads kAhead segments at a
// time, so that it waits for memory once for each kAhead. Four elements and 16 segments move 16
// bytes a lane; where that leaves most compute units without work (a few heads), one element and 32, in
// workgroups of a wave: 168 K tokens at H = 1, K = 128, V = 64 in 658 segments take 108 instead of 145 us.
template <int kWidth, int kAhead, int kCombineThreads>
__global__ __launch_bounds__(kCombineThreads) void linear_combine(const LinearPlan p) {
  typedef float Elems __attribute__((ext_vector_type(kWidth)));
  const int per_head = p.K * p.V / (kWidth * kCombineThreads), lane = threadIdx.x & 63;
  const int h = blockIdx.x / per_head;
  const int64_t plane = (int64_t)p.K * p.V, step = p.H * plane;
  float* at = p.maps + h * plane + (int64_t)((blockIdx.x % per_head) * kCombineThreads + threadIdx.x) * kWidth;
  const int n = p.n_seg - 1;
  Elems cur = 0.f;
  for (int s0 = 0; s0 < n; s0 += kAhead) {
    const int mine = min(s0 + lane % kAhead, n - 1);
    const float decay = p.decays[(int64_t)mine * p.H + h];
    const int span = p.spans[mine];
    Elems m[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) m[j] = *reinterpret_cast<const Elems*>(at + min(s0 + j, n - 1) * step);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (s0 + j >= n) break;
      const int kind = __builtin_amdgcn_readlane(span, j);
      if (kind == 1) cur = m[j];
      if (kind == 2) {
        cur = m[j] + cur * __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, decay), j));
        *reinterpret_cast<Elems*>(at + (s0 + j) * step) = cur;
      }
    }
  }
}

template <bool kOut, int kTerms>
int launch_walk(const LinearPlan& p, int segments, hipStream_t s) {
  const int V = p.V / p.slices;
  const dim3 grid((unsigned)((int64_t)segments * p.H * p.slices)), threads(64 * (V == 128 ? kWavesOf<128> : kWavesOf<64>));
  if (p.K == 128 && V == 128) linear_walk<128, 128, kOut, kTerms><<<grid, threads, 0, s>>>(p);
  else if (p.K == 128) linear_walk<128, 64, kOut, kTerms><<<grid, threads, 0, s>>>(p);
  else if (V == 128) linear_walk<64, 128, kOut, kTerms><<<grid, threads, 0, s>>>(p);
  else linear_walk<64, 64, kOut, kTerms><<<grid, threads, 0, s>>>(p);
  return (int)hipGetLastError();
}
template <bool kOut>
int launch_walk(const LinearPlan& p, int segments, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool exact = p.out_mode != kStateNone && p.state_dtype == kF32;
  return exact ? launch_walk<kOut, 3>(p, segments, s) : launch_walk<kOut, 2>(p, segments, s);
}

}  // namespace

int launch_linear_maps(const LinearPlan& p, void* stream) { return launch_walk<false>(p, p.n_seg - 1, stream); }
int launch_linear_output(const LinearPlan& p, void* stream) { return launch_walk<true>(p, p.n_seg, stream); }
int launch_linear_combine(const LinearPlan& p, void* stream) {
  const int64_t elems = (int64_t)p.H * p.K * p.V;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (elems >= (1 << 17)) linear_combine<4, 16, 256><<<(unsigned)(elems / 1024), 256, 0, s>>>(p);
  else linear_combine<1, 32, 64><<<(unsigned)(elems / 64), 64, 0, s>>>(p);
  return (int)hipGetLastError();
}

}  // namespace kda
