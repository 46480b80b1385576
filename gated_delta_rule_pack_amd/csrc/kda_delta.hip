// The gated delta rule with one decay for each head, chunked form for prompts.
//
// Per sequence and value head, S <- e^g S, S <- S + beta (v - S k) k^T, o = scale S q. Over a chunk of 64 tokens, with
// G the inclusive cumsum of g in it, S0 the state before it and d_t = beta_t (v_t - e^{g_t} S_{t-1} k_t):
//
//   A[t, s] = beta_t (k_t . k_s) e^{G_t - G_s}  (s < t)      T = (I + A)^{-1}
//   D = T diag(beta) (V - diag(e^G) K S0^T)                  P[t, s] = (q_t . k_s) e^{G_t - G_s}  (s <= t)
//   O = scale (diag(e^G) Q S0^T + P D)                       S = e^{G_C} S0 + (diag(e^{G_C - G}) D)^T K
//
// Every factor is the exponential of a sum of log decays over a run of tokens, taken of the difference of 64-bit prefix
// sums: nothing is divided, so no decay is too steep. T is made of 16 x 16 blocks: those on the diagonal by forward
// substitution, those below it by products of blocks, all in fp32.
//
// Number formats. MFMA operands are fp16, whose 11 bits make two terms 22: every operand but keys and queries enters in two,
// where bf16 would take three. Keys and queries are exact in one: 8 bits of bf16 (11 of fp16) fit, and rows far from unit length
// are scaled by a power of two of their own (ScaledRows). The state and what is to be learnt of one value channel are held in a range
// by powers of two of that channel's own (Scale); step sizes and what the keys' scaling left of their lengths stay in
// fp32 (Factors), so that T's diagonal is 1. P's second term has 8 bits (p_rest). What decays further within a chunk
// than two terms reach is walked token by token in fp32 (by_tokens).
//
// A workgroup walks one sequence of one value head, or a slice of 64 of its state rows, with four chain waves and four
// making waves. The chain waves hold the state as S^T[k][v] in fp32 MFMA accumulators, 32 or 16 value channels each. Lanes
// (l, g = l / 16): an accumulator tile holds column l % 16, rows 4g + i. The chain K S0^T -> D -> state keeps the columns
// v, so that every accumulator is the next product's operand as it stands (rows t in the order 4g + i, 16 + 4g + i of two tiles),
// and no chain wave waits for another's values. Meanwhile the making waves turn the next chunk's rows into operands, T and P in
// the other half of LDS.
//
// Measured: a turn takes 16500 cycles at V = 128 (12750 for slices of 64). The making waves work for up to 14200 of them and the
// chain waves, each beside one of those on its SIMD, for 13300 to 13900 (12100 and 9300); the longest of each of the six parts come to
// 16100 and 12500. 128 ragged prompts (135060 tokens) at H = 12 with bf16 states take 805 us: vector instructions 46 % of the time, the matrix
// unit 27 %, LDS 25 %, memory 1.16 GB at 1.4 TB/s; what is left is one part waiting for the next. (With one term of what is learnt
// and of the state they took 664, and with all eight waves making and walking in turn 1507.) A chunk that is walked by tokens adds
// 32 us at 64 channels and 110 at 128.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "kda_delta.h"
#include "kda_delta_device.h"
#include "kda_delta_token.h"

namespace kda {
namespace {

// A chunk's operands in LDS.
template <int K, int V>
struct Slot {
  alignas(16) char k[kC * kRowBytes<K>];
  alignas(16) char q[kC * kRowBytes<K>];
  alignas(16) char v[kC * kRowBytes<V>];  // then, once its chain wave has its columns, the outputs
  alignas(16) char t[2 * kTermP];
  alignas(16) char p[kTermP + kRestP];
  alignas(16) Factors factors;
  alignas(16) float decay[kC];  // e^g
};
template <int K, int V>
struct DeltaShared {
  Slot<K, V> slot[2];
  alignas(16) float blocks[10 * kBlock];
  Making making;
  RowInfo info[2][kC];
};
constexpr int kChainWaves = 4, kMakingWaves = 4, kWalkThreads = 64 * (kChainWaves + kMakingWaves);
// Barriers of a chunk: the making waves' parts meet at them, and the chain waves pass them on their way.
constexpr int kBarriers = 6;
constexpr int kNumbersWave = 3;  // of the making waves, one with few tiles

template <int K, int V, bool kF16In>
struct Chain {
  typedef Walk<K, V, kChainWaves> State;
  static constexpr int VT = State::VT, KT = K / 16, KB = K / 32;
  State state;
  Scale scale[VT];

  __device__ __forceinline__ void ldexp_state(int vt, int by) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) state.S[vt][kt][i] = ldexp2(state.S[vt][kt][i], by);
  }

  // One chunk; passes kBarriers - 1 barriers.
  __device__ __forceinline__ void step(Slot<K, V>& slot, int wave, int lane_, int count) {
    const int lane = local_copy(lane_), g4 = lane >> 4, l16 = lane & 15;
    constexpr uint32_t kInf = kF16In ? 0x7c00u : 0x7f80u;
    const Factors& fa = slot.factors;
    // V's columns, tokens 4g + i of each tile; finite values alone.
    u32x2 raw[VT][4];
    int first_bad[VT];
    bool any_bad = false;
    const int steps = fa.steps, reach = fa.reach;
    int state_top[VT];
    bool apart = false;
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      uint32_t most = 0;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const u32x4 w = __builtin_bit_cast(u32x4, read_col<V, false>(slot.v, lane, 32 * b, wave * VT + vt));
        raw[vt][2 * b] = u32x2{w[0], w[1]}, raw[vt][2 * b + 1] = u32x2{w[2], w[3]};
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int j = 0; j < 2; ++j) most = max(most, max(raw[vt][tt][j] & 0x7fffu, (raw[vt][tt][j] >> 16) & 0x7fffu));
      first_bad[vt] = kC;
      if (__ballot(most >= kInf)) {
        any_bad = true;
        most = 0;
        int bad = kC;
#pragma unroll
        for (int tt = 3; tt >= 0; --tt)
#pragma unroll
          for (int j = 3; j >= 0; --j) {
            const uint32_t x = (raw[vt][tt][j / 2] >> (16 * (j & 1))) & 0x7fffu;
            if (x >= kInf) {
              bad = 16 * tt + 4 * g4 + j;
              raw[vt][tt][j / 2] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
            } else {
              most = max(most, x);
            }
          }
        first_bad[vt] = -channel_max(-bad);
      }
      // The channel's scale.
      float top = 0.f;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(state.S[vt][kt][i]));
      Scale& sc = scale[vt];
      const int own = exponent(top);
      const i16x2 tops = channel_max(i16x2{(short)own, (short)max(own - sc.ex + reach, exponent(token_value<kF16In>(most)) + steps)});
      state_top[vt] = tops[0];
      sc.apart = 0;
      if (__ballot(!stays(sc.ex, tops[0], tops[1]))) {  // each channel by itself: none depends on the others of its wave
        const Ranges r = ranges_of(sc.ex, tops[0], tops[1]);
        ldexp_state(vt, r.s - sc.ex);
        state_top[vt] += r.s - sc.ex;
        sc.ex = r.s;
        sc.apart = r.x - r.s;
        sc.set(lane, r.x);
        apart = apart || __ballot(sc.apart != 0);
      }
    }
    barrier_lds();
    // K' S0^T, rows t = 4g + i, column v; S0 Q'^T, rows v, column t.
    f32x4 x[VT][4], o[VT][4];
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) x[vt][tt] = o[vt][tt] = zero4();
#pragma unroll
    for (int m = 0; m < KB; ++m) {
      f16x8 hi[VT], lo[VT];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        hi[vt] = to_f16(state.S[vt][2 * m], state.S[vt][2 * m + 1]);
        lo[vt] = rest_f16(state.S[vt][2 * m], state.S[vt][2 * m + 1], hi[vt]);
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const f16x8 kk = __builtin_bit_cast(f16x8, read_row<K>(slot.k, lane, 16 * tt, m));
        const f16x8 qq = __builtin_bit_cast(f16x8, read_row<K>(slot.q, lane, 16 * tt, m));
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          x[vt][tt] = mfma(kk, lo[vt], x[vt][tt]);
          o[vt][tt] = mfma(lo[vt], qq, o[vt][tt]);
        }
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          x[vt][tt] = mfma(kk, hi[vt], x[vt][tt]);
          o[vt][tt] = mfma(hi[vt], qq, o[vt][tt]);
        }
      }
      if (m == KB / 2 - 1) barrier_lds();
      else __builtin_amdgcn_sched_barrier(0);
    }
    barrier_lds();
    // What is to be learnt, b V - h K' S.
    if (apart) {
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        const float by = ldexp2(1.f, scale[vt].apart);
        f32x4 rows;
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = __shfl(by, 4 * g4 + i);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) x[vt][tt] *= by, o[vt][tt] *= rows;
      }
    }
    f16x8 xh[VT][2], xl[VT][2];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      const f32x4 hh = *reinterpret_cast<const f32x4*>(&fa.h[16 * tt + 4 * g4]), bb = *reinterpret_cast<const f32x4*>(&fa.b[16 * tt + 4 * g4]);
      const float e = fa.e[16 * tt + l16];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = i & 1 ? high_value<kF16In>(raw[vt][tt][i / 2]) : low_value<kF16In>(raw[vt][tt][i / 2]);
          x[vt][tt][i] = y * (bb[i] * scale[vt].v) - hh[i] * x[vt][tt][i];
          o[vt][tt][i] *= e;
        }
    }
    uint64_t small[VT], any_small = 0;
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      float least = INFINITY;
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) least = fminf(least, fabsf(x[vt][tt][i]));
      small[vt] = __ballot(least < kLeastShare<kF16In> && !state_lasts(state_top[vt], scale[vt].apart, fa.total));
      any_small |= small[vt];
    }
    if (__builtin_expect(any_small != 0, 0) && __builtin_expect(fades(slot, x, small, state_top, lane), 0)) {
      by_tokens(slot, wave, lane, count);
      barrier_lds();
      barrier_lds();
      return;
    }
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        xh[vt][b] = to_f16(x[vt][2 * b], x[vt][2 * b + 1]);
        xl[vt][b] = rest_up(x[vt][2 * b], x[vt][2 * b + 1], xh[vt][b]);
      }
    // D = T x, rows t, column v.
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      f16x8 th[2];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) x[vt][tt] = zero4();
#pragma unroll
      for (int b = 0; b <= tt / 2; ++b) {
        th[b] = read_fragment(slot.t, lane, tt, b);
        const f16x8 tl = read_fragment(slot.t + kTermP, lane, tt, b);
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          x[vt][tt] = mfma(tl, xh[vt][b], x[vt][tt]);
          x[vt][tt] = mfma(th[b], xl[vt][b], x[vt][tt]);
        }
      }
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        x[vt][tt] *= kDown;
#pragma unroll
        for (int b = 0; b <= tt / 2; ++b) x[vt][tt] = mfma(th[b], xh[vt][b], x[vt][tt]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    barrier_lds();
    // O^T += D^T P^T, and the outputs, rows v = 4g + i, column t, to V's tile.
    {
      f16x8 dh[VT][2], dl[VT][2];
#pragma unroll
      for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          dh[vt][b] = to_f16(x[vt][2 * b], x[vt][2 * b + 1]);
          dl[vt][b] = rest_up(x[vt][2 * b], x[vt][2 * b + 1], dh[vt][b]);
        }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const float f = fa.f[16 * tt + l16];
        f16x8 pp[2];
        f32x4 rest[VT];
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) rest[vt] = zero4();
#pragma unroll
        for (int b = 0; b <= tt / 2; ++b) {
          pp[b] = read_fragment(slot.p, lane, tt, b);
          const f16x8 pl = read_rest(slot.p + kTermP, lane, tt, b);
#pragma unroll
          for (int vt = 0; vt < VT; ++vt) {
            rest[vt] = mfma(dl[vt][b], pp[b], rest[vt]);
            rest[vt] = mfma(dh[vt][b], pl, rest[vt]);
          }
        }
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
          o[vt][tt] += rest[vt] * kDown;
#pragma unroll
          for (int b = 0; b <= tt / 2; ++b) o[vt][tt] = mfma(dh[vt][b], pp[b], o[vt][tt]);
        }
        __builtin_amdgcn_sched_barrier(0);  // one row of tiles at a time: with all reads first the walk spills
#pragma unroll
        for (int vt = 0; vt < VT; ++vt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[vt][tt][i] *= f * scale[vt].out[i];
      }
    }
    if (any_bad) {
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int from = __shfl(first_bad[vt], 4 * g4 + i);
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
            if (16 * tt + l16 >= from) o[vt][tt][i] = __builtin_nanf("");
        }
        if (first_bad[vt] < kC)
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) state.S[vt][kt] = zero4() + __builtin_nanf("");
      }
    }
#pragma unroll
    for (int tt = 0; tt < 4; ++tt)
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        char* at = slot.v + row_at<V>(16 * tt + l16) + ((wave * VT + vt) * 16 + 4 * g4) * 2;
        const f32x4 y = o[vt][tt];
        if constexpr (kF16In) *reinterpret_cast<f16x4*>(at) = f16x4{(_Float16)y[0], (_Float16)y[1], (_Float16)y[2], (_Float16)y[3]};
        else *reinterpret_cast<bf16x4*>(at) = bf16x4{to_bf16(y[0]), to_bf16(y[1]), to_bf16(y[2]), to_bf16(y[3])};
      }
    barrier_lds();
    // The state.
    f16x8 dh[VT][2], dl[VT][2];
    float total[VT];
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      total[vt] = ldexp2(fa.total, 12 + scale[vt].apart);
      scale[vt].ex += scale[vt].apart;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const f32x4 c0 = *reinterpret_cast<const f32x4*>(&fa.c[32 * b + 4 * g4]), c1 = *reinterpret_cast<const f32x4*>(&fa.c[32 * b + 16 + 4 * g4]);
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        const f32x4 y0 = x[vt][2 * b] * c0, y1 = x[vt][2 * b + 1] * c1;
        dh[vt][b] = to_f16(y0, y1);
        dl[vt][b] = rest_up(y0, y1, dh[vt][b]);
      }
    }
#pragma unroll
    for (int kt = 0; kt < KT; kt += 2) {
      f16x8 k0[2], k1[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        k0[b] = __builtin_bit_cast(f16x8, read_col<K, true>(slot.k, lane, 32 * b, kt));
        k1[b] = __builtin_bit_cast(f16x8, read_col<K, true>(slot.k, lane, 32 * b, kt + 1));
      }
#pragma unroll
      for (int vt = 0; vt < VT; ++vt) {
        f32x4 &s0 = state.S[vt][kt], &s1 = state.S[vt][kt + 1];
        s0 *= total[vt], s1 *= total[vt];
#pragma unroll
        for (int b = 0; b < 2; ++b) s0 = mfma(k0[b], dl[vt][b], s0), s1 = mfma(k1[b], dl[vt][b], s1);
        s0 *= kDown, s1 *= kDown;
#pragma unroll
        for (int b = 0; b < 2; ++b) s0 = mfma(k0[b], dh[vt][b], s0), s1 = mfma(k1[b], dh[vt][b], s1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  __device__ __forceinline__ bool fades(const Slot<K, V>& slot, const f32x4 (&x)[VT][4], const uint64_t (&small)[VT], const int (&state_top)[VT],
                                        int lane) const {
    bool found = false;
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      if (!small[vt]) continue;
      float through = state_share(state_top[vt], scale[vt].apart);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        Fading f;
        f.set(*reinterpret_cast<const f32x4*>(&slot.decay[16 * tt + 4 * (lane >> 4)]), x[vt][tt]);
        const float before = f.before(through, lane);
        found = found || f.fades(before, kLeastShare<kF16In>);
      }
    }
    return __ballot(found) != 0;
  }
  // The chunk token by token in fp32, for this wave's channels.
  __device__ __forceinline__ void by_tokens(Slot<K, V>& slot, int wave, int lane, int count) {
    const Factors& fa = slot.factors;
    const auto channel_sum = [](f32x4 x) __attribute__((always_inline)) { return add_far(add_far((x[0] + x[1]) + (x[2] + x[3]), 16), 32); };
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      f32x4 (&S)[KT] = state.S[vt];
      ldexp_state(vt, -scale[vt].ex);
      scale[vt].ex = scale[vt].apart = 0;
      scale[vt].set(lane, 0);
      const auto over_keys = [&](const char* row, auto use) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < KB; ++m) {
          const f16x8 k = *reinterpret_cast<const f16x8*>(row + m * 64 + (lane >> 4) * 16);
#pragma unroll
          for (int j = 0; j < 8; ++j) use(2 * m + j / 4, j % 4, (float)k[j]);
        }
      };
#pragma unroll 1
      for (int t = 0; t < count; ++t) {
        const float decay = slot.decay[t];
        uint16_t* const at = reinterpret_cast<uint16_t*>(slot.v + row_at<V>(t)) + (wave * VT + vt) * 16 + (lane & 15);
        f32x4 us = zero4(), os = zero4();
        over_keys(slot.k + row_at<K>(t), [&](int kt, int i, float k) __attribute__((always_inline)) { us[i] += S[kt][i] * k; });
        float u = channel_sum(us);
        u = fa.b[t] * token_value<kF16In>(*at) - fa.s[t] * (decay * u);
        over_keys(slot.k + row_at<K>(t), [&](int kt, int i, float k) __attribute__((always_inline)) { S[kt][i] = S[kt][i] * decay + u * k; });
        over_keys(slot.q + row_at<K>(t), [&](int kt, int i, float q) __attribute__((always_inline)) { os[i] += S[kt][i] * q; });
        const float o = fa.f[t] * channel_sum(os) * kTimesP;
        if (lane < 16) *at = kF16In ? __builtin_bit_cast(uint16_t, (_Float16)o) : __builtin_bit_cast(uint16_t, to_bf16(o));
      }
      if (fa.total != fa.total) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = zero4() + __builtin_nanf("");
      }
    }
  }
};

// A sequence of one token, in fp32 as a step of its own. (As a chunk it would take as long
// as 64 tokens: 16 prompts of 256 among 240 single tokens at H = 12, with fp32 states, 226 instead of 127 us.)
template <int K, int V>
__device__ __forceinline__ void one_token(DeltaShared<K, V>& shared, int begin, int h, int v0, Slots slots, int tid) {
  const DeltaPlan& p = plan_again();
  auto& sh = *reinterpret_cast<TokenShared<K, V, kWalkThreads>*>(&shared);
  static_assert(sizeof(TokenShared<K, V, kWalkThreads>) <= sizeof(shared), "fits");
  uint16_t x[kTokenRow<K, V>], k[K / 64];
  token_rows<K, V>(p, begin, h, v0, __builtin_amdgcn_readfirstlane(tid >> 6), tid & 63, x, k);
  const int64_t from = slots.from >= 0 ? plane_at(p, slots.from, h) : 0, to = slots.to >= 0 ? plane_at(p, slots.to, h) : -1;
  const uint32_t keep = slots.from >= 0 ? ~0u : 0u;
  const auto of = [&](auto sdt) __attribute__((always_inline)) {
    constexpr int SDT = decltype(sdt)::value;
    if (p.kfirst) delta_token<K, V, SDT, true, kWalkThreads, true>(p, sh, x, k, begin, h, v0, from, to, keep, tid);
    else delta_token<K, V, SDT, false, kWalkThreads, true>(p, sh, x, k, begin, h, v0, from, to, keep, tid);
  };
  if (p.state_dtype == kF32) of(std::integral_constant<int, kF32>());
  else if (p.state_dtype == kF16) of(std::integral_constant<int, kF16>());
  else of(std::integral_constant<int, kBF16>());
}

template <int K, int V, bool kF16In>
__global__ __launch_bounds__(kWalkThreads, 2) void delta_walk(const DeltaPlan p) {
  constexpr int kThreads = 64 * kMakingWaves;
  __shared__ DeltaShared<K, V> sh;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int slice = blockIdx.x % p.slices, unit = blockIdx.x / p.slices;
  __shared__ Ranking ranking;
  const int h = unit % p.H, v0 = slice * V, n = p.ranked ? ranked_sequence(p, ranking, unit / p.H, threadIdx.x) : unit / p.H;
  const int begin = __builtin_amdgcn_readfirstlane(bound(p, n));
  const int len = __builtin_amdgcn_readfirstlane(max(bound(p, n + 1) - begin, 0)), chunks = (len + kC - 1) / kC;
  const Slots slots = slots_of(p, n);
  if (len == 1) {
    one_token<K, V>(sh, begin, h, v0, slots, threadIdx.x);
    return;
  }
  if (wave < kChainWaves) {
    Chain<K, V, kF16In> chain;
    char* const stage = sh.slot[1].k + wave * 1024;  // no row stands there yet
    chain.state.zero();
    if (slots.from >= 0) chain.state.load_plane(p, stage, plane_at(p, slots.from, h), v0, wave, lane);
#pragma unroll
    for (int vt = 0; vt < chain.VT; ++vt) {
      chain.scale[vt].ex = 0;
      chain.scale[vt].set(lane, 0);
    }
    if (chunks > 0) {
      for (int i = 0; i <= kBarriers; ++i) barrier_lds();
      for (int i = 0; i < chunks; ++i) {
        chain.step(sh.slot[i & 1], wave, lane, min(len - i * kC, kC));
        barrier_lds();
      }
    }
    if (slots.to >= 0) {
#pragma unroll
      for (int vt = 0; vt < chain.VT; ++vt) chain.ldexp_state(vt, -chain.scale[vt].ex);
      chain.state.store_plane(p, sh.slot[chunks & 1].k + wave * 1024, plane_at(p, slots.to, h), v0, wave, lane);
    }
    return;
  }
  if (chunks == 0) return;
  const int tid = threadIdx.x - 64 * kChainWaves, w = wave - kChainWaves;
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + (h / p.group) * p.q_h;
  const uint16_t* k = reinterpret_cast<const uint16_t*>(p.k) + (h / p.group) * p.k_h;
  const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v) + h * p.v_h + v0;
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + h * p.o_h + v0;
  ScaledRows<K, kThreads, kF16In> rq, rk;
  Rows<V, kThreads> rv;
  uint32_t g_next = 0, beta_next = 0;  // this lane's token of the next chunk as it is stored, in one wave
  Decays decays = {};
  TileDecays between;
  const auto count_of = [&](int i) { return min(len - i * kC, kC); };
  // (Not a running pointer: the compiler would keep that in vector registers, and take every lane's buffer by itself.)
  const auto first_of = [&](int i) { return (int64_t)__builtin_amdgcn_readfirstlane(begin + i * kC); };
  const auto fetch = [&](int i) __attribute__((always_inline)) {
    const int64_t first = first_of(i);
    const int count = count_of(i);
    if (w == kNumbersWave) {
      g_next = beta_next = 0;
      if (lane < count) {
        const int64_t at = (first + lane) * p.H + h;
        if (p.g) g_next = load_bits(p.g, p.g_per_token ? at : h, p.g_bf16);
        beta_next = load_bits(p.beta, at, p.beta_bf16);
      }
    }
    rk.rows.load(reinterpret_cast<const __bf16*>(k), p.k_t, first, count, tid);
    rq.rows.load(reinterpret_cast<const __bf16*>(q), p.q_t, first, count, tid);
  };
  const auto fetch_v = [&](int i) __attribute__((always_inline)) {
    rv.load(reinterpret_cast<const __bf16*>(v), p.v_t, first_of(i), count_of(i), tid);
  };
  const auto scale_rows = [&]() __attribute__((always_inline)) {
    rk.scale();
    rq.scale();
  };
  const auto make_decays = [&]() __attribute__((always_inline)) { decays = put_decays(sh.making, bits_value(g_next, p.g_bf16), lane); };
  const auto store = [&](int i) __attribute__((always_inline)) {
    Rows<V, kThreads>::store(sh.slot[i & 1].v, reinterpret_cast<__bf16*>(out), p.o_t, first_of(i), count_of(i), tid);
  };
  fetch(0);
  fetch_v(0);
  if (w == kNumbersWave) make_decays();
  scale_rows();
  barrier_lds();
  const auto make_between = [&](int l) __attribute__((always_inline)) {
    by_wave(w, [&](auto W) { tile_decays<decltype(W)::value>(sh.making, l, between); });
  };
  make_between(local_copy(lane));
  // In turn i the chain waves walk chunk i - 1 and these make chunk i, in the place of chunk i - 2, whose outputs leave first. What
  // of chunk i + 1 waits for no tile, its rows' scales and its decays, is made where a turn leaves waves without work.
  // (Loads and stores are spread over a turn, and none stands in a branch, so that a wait counts what is behind its own.)
  // The last chunk has code of its own, without the next one's (in one form with the others it made the
  // last again: 37 tokens 13 us of kernel instead of 11).
  const auto make = [&](int i, auto last) __attribute__((always_inline)) {
    constexpr bool kNext = !decltype(last)::value;
    Slot<K, V>& slot = sh.slot[i & 1];
    rk.put(slot.k, sh.info[0], tid);
    rq.put(slot.q, sh.info[1], tid);
    barrier_lds();
    const int l = local_copy(lane);
    Numbers numbers;
    if (w == kNumbersWave) numbers.put_steps(sh.making, p, decays, sh.info[0][l], sh.info[1][l], bits_value(beta_next, p.beta_bf16), l);
    TileProducts products;
    by_wave(w, [&](auto W) { tile_products<K, decltype(W)::value>(slot.k, slot.q, l, products); });
    if constexpr (kNext) fetch(i + 1);
    barrier_lds();
    by_wave(w, [&](auto W) {
      put_tiles<decltype(W)::value>(sh.blocks, sh.making, l, products, between, [&](int tt, int st, f16x4 x, uint32_t rest) {
        put_fragment(slot.p, l, tt, st, x);
        put_rest(slot.p + kTermP, l, tt, st, rest);
      });
    });
    if (w == kNumbersWave) {
      numbers.put_factors(slot.factors, p, decays, l);
      slot.decay[l] = decays.own;
    }
    {
      // The outputs of chunk i - 2; for the first two a buffer of no rows.
      const __amdgpu_buffer_rsrc_t to = i < 2 ? __builtin_amdgcn_make_buffer_rsrc(out, (short)0, 0, kBufWord3)
                                              : rows_buffer<V>(reinterpret_cast<__bf16*>(out), first_of(i - 2), p.o_t, kC);
      Rows<V, kThreads>::store(slot.v, to, p.o_t, tid);
    }
    barrier_lds();
    if (w == 0) invert_diagonal(sh.blocks, l);
    if (kNext && w != 0) scale_rows();  // the first wave's in the next two parts, in which it has none
    barrier_lds();
    const auto put_t = [&](int tt, int st, f32x4 x) {
      const Terms y = t_terms(x);
      put_fragment(slot.t, l, tt, st, y.hi);
      put_fragment(slot.t + kTermP, l, tt, st, y.lo);
    };
    near_blocks(sh.blocks, l, w, put_t);
    rv.put(slot.v, tid);
    if constexpr (kNext) fetch_v(i + 1);
    if (kNext && w == 0) rk.scale();
    if (kNext && w == kNumbersWave) make_decays();
    barrier_lds();
    far_blocks(sh.blocks, l, w, put_t);
    if (kNext && w == 0) rq.scale();
    if constexpr (kNext) make_between(l);
    barrier_lds();
  };
  for (int i = 0; i + 1 < chunks; ++i) make(i, std::false_type());
  make(chunks - 1, std::true_type());
  if (chunks >= 2) store(chunks - 2);
  for (int j = 0; j < kBarriers; ++j) barrier_lds();
  store(chunks - 1);
}

template <int K, int V>
int launch_kv(const DeltaPlan& p, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.N * p.H * p.slices);
  if (p.f16) delta_walk<K, V, true><<<grid, kWalkThreads, 0, s>>>(p);
  else delta_walk<K, V, false><<<grid, kWalkThreads, 0, s>>>(p);
  return (int)hipGetLastError();
}

}  // namespace

int launch_delta_walk(const DeltaPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int V = p.V / p.slices;
  if (p.K == 128) return V == 128 ? launch_kv<128, 128>(p, s) : launch_kv<128, 64>(p, s);
  return V == 128 ? launch_kv<64, 128>(p, s) : launch_kv<64, 64>(p, s);
}

}  // namespace kda
