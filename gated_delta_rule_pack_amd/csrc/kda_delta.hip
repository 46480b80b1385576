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
// Number formats. MFMA operands are fp16, whose 11 bits make two terms 22: the state keeps nearly fp32's accuracy in two
// products where bf16 would take three. Keys and queries are exact in one term: each row is scaled by the power of two
// that brings its largest element into [1/4, 1/2), near unit length, and 8 bits of bf16 (11 of fp16) fit. What else becomes an operand is held in a
// range by exact powers of two: the state and V of one value channel by a power of two of that channel's own (Scale), step
// sizes by one of the chunk (Chunk::shift). One term serves for outputs in bf16.
//
// A workgroup walks one sequence of one value head, or a slice of 64 of its state rows; each wave holds 16 of them as
// S^T[k][v] in fp32 MFMA accumulators. Lanes (l, g = l / 16): an accumulator tile holds column l % 16, rows 4g + i. The
// chain K S0^T -> D -> state keeps the columns v, so that every accumulator is the next product's operand as it stands
// (rows t in the order 4g + i, 16 + 4g + i of two tiles), and no wave waits for another's values.
#include <hip/hip_runtime.h>

#include "kda_delta.h"
#include "kda_delta_device.h"

namespace kda {
namespace {

template <int K, int V>
struct DeltaShared {
  static constexpr int kTileV = kC * kRowBytes<V>, kBlocks = 10 * kBlock * 4;
  alignas(16) char k[kC * kRowBytes<K>];
  alignas(16) char q[kC * kRowBytes<K>];
  // V's rows, then A's and T's blocks, then the outputs' rows.
  alignas(16) char v[kTileV > kBlocks ? kTileV : kBlocks];
  // T in two terms; between a sequence's chunks and the next one's, 1 KB of each wave's for its state.
  alignas(16) char t[2 * kTermP > 1024 * kWavesOf<V> ? 2 * kTermP : 1024 * kWavesOf<V>];
  alignas(16) char p[kTermP];
  Chunk chunk;
  RowInfo info[2][kC];
};

template <int K, int V, int kTerms, bool kF16In>
__global__ __launch_bounds__(64 * kWavesOf<V>, 2) void delta_walk(const DeltaPlan p) {
  constexpr int kWaves = kWavesOf<V>, kThreads = 64 * kWaves, KT = K / 16, KB = K / 32;
  __shared__ DeltaShared<K, V> sh;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g4 = lane >> 4, l16 = lane & 15;
  const int slice = blockIdx.x % p.slices, unit = blockIdx.x / p.slices;
  const int n = unit / p.H, h = unit % p.H, v0 = slice * V;
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + (h / p.group) * p.q_h;
  const uint16_t* k = reinterpret_cast<const uint16_t*>(p.k) + (h / p.group) * p.k_h;
  const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v) + h * p.v_h + v0;
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + h * p.o_h + v0;
  const int begin = bound(p, n), len = max(bound(p, n + 1) - begin, 0);
  const Slots slots = slots_of(p, n);
  char* stage = sh.t + wave * 1024;
  Walk<K, V> walk;
  f32x4* S = walk.S[0];
  Rows<K, kThreads> rq, rk;
  Rows<V, kThreads> rv;
  float g_next = 0.f, beta_next = 0.f;  // this lane's token of the next chunk, in the last wave
  const auto fetch = [&](int64_t first, int count) {
    if (wave == kWaves - 1) {
      g_next = beta_next = 0.f;
      if (lane < count) {
        const int64_t at = (first + lane) * p.H + h;
        if (p.g) {
          const int64_t ag = p.g_per_token ? at : h;
          g_next = p.g_bf16 ? (float)reinterpret_cast<const __bf16*>(p.g)[ag] : reinterpret_cast<const float*>(p.g)[ag];
        }
        beta_next = p.beta_bf16 ? (float)reinterpret_cast<const __bf16*>(p.beta)[at] : reinterpret_cast<const float*>(p.beta)[at];
      }
    }
    rk.load(reinterpret_cast<const __bf16*>(k), p.k_t, first, count, tid);
    rv.load(reinterpret_cast<const __bf16*>(v), p.v_t, first, count, tid);
    rq.load(reinterpret_cast<const __bf16*>(q), p.q_t, first, count, tid);
  };
  int64_t first = begin;
  int left = len;
  if (left > 0) fetch(first, min(left, kC));
  walk.zero();
  if (slots.from >= 0) walk.load_plane(p, stage, plane_at(p, slots.from, h), v0, wave, lane);
  Scale scale;
  scale.shift = 0;
  scale.set(lane, 0);
  while (left > 0) {
    const int count = min(left, kC);
    put_scaled<K, kThreads, kF16In>(rk, sh.k, sh.info[0], tid, true);
    put_scaled<K, kThreads, kF16In>(rq, sh.q, sh.info[1], tid, p.normalize);
    rv.put(sh.v, tid);
    barrier_lds();
    if (wave == kWaves - 1) put_chunk(sh.chunk, p, sh.info[0][lane], sh.info[1][lane], g_next, beta_next, lane);
    const int64_t here = first;
    first += count;
    left -= count;
    if (left > 0) fetch(first, min(left, kC));

    // V's column of this lane, tokens 4g + i of each tile, finite values alone.
    u32x2 raw[4];
    uint32_t most = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const u32x4 w = __builtin_bit_cast(u32x4, read_col<V, false>(sh.v, lane, 32 * b, wave));
      raw[2 * b] = u32x2{w[0], w[1]}, raw[2 * b + 1] = u32x2{w[2], w[3]};
    }
#pragma unroll
    for (int tt = 0; tt < 4; ++tt)
#pragma unroll
      for (int j = 0; j < 2; ++j) most = max(most, max(raw[tt][j] & 0x7fffu, (raw[tt][j] >> 16) & 0x7fffu));
    constexpr uint32_t kInf = kF16In ? 0x7c00u : 0x7f80u;
    int first_bad = kC;  // of this lane's channel
    if (__ballot(most >= kInf)) {
      most = 0;
#pragma unroll
      for (int tt = 3; tt >= 0; --tt)
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          const uint32_t x = (raw[tt][j / 2] >> (16 * (j & 1))) & 0x7fffu;
          if (x >= kInf) {
            first_bad = 16 * tt + 4 * g4 + j;
            raw[tt][j / 2] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
          } else {
            most = max(most, x);
          }
        }
      first_bad = min(first_bad, __shfl_xor(first_bad, 16));
      first_bad = min(first_bad, __shfl_xor(first_bad, 32));
    }
    barrier_lds();  // the chunk's numbers; V's tile has been read

    // The channel's scale.
    const Chunk& ch = sh.chunk;
    if (ch.shift != scale.shift) {
      const int by = ch.shift - scale.shift;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[kt][i] = ldexp2(S[kt][i], by);
      scale.shift = ch.shift;
    }
    float top = 0.f;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(S[kt][i]));
    const int e = channel_max(max(exponent(top), exponent(token_value<kF16In>(most)) + scale.ex));
    if (__ballot(e > 4 || (e < 1 && e > kNoExponent / 2))) {
      const int by = e > kNoExponent / 2 ? min(max(scale.ex + 4 - e, -120), 120) - scale.ex : 0;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[kt][i] = ldexp2(S[kt][i], by);
      scale.set(lane, scale.ex + by);
    }

    // A's and P's tiles, dealt over the waves.
#pragma unroll
    for (int j = 0; j < (20 + kWaves - 1) / kWaves; ++j) {
      const int job = j * kWaves + wave;
      if (job >= 20) break;
      const int tile = job < 10 ? job : job - 10, tt = tile_t(tile), st = tile_s(tile);
      const int t = 16 * tt + l16;
      const f32x4 decay = tile_decay(ch, lane, tt, st);
      if (job < 10) {
        const f32x4 d = tile_product<K>(sh.k, sh.k, lane, tt, st) * decay;
        const f32x4 r = *reinterpret_cast<const f32x4*>(&ch.rk[16 * st + 4 * g4]);
        const float bk = ch.bk[t];
        float* to = reinterpret_cast<float*>(sh.v) + block_at(tt, st) + 4 * g4 * kBlockRow + l16;
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i * kBlockRow] = 16 * st + 4 * g4 + i < t ? d[i] * (bk * r[i]) : 0.f;
      } else {
        const f32x4 d = tile_product<K>(sh.k, sh.q, lane, tt, st) * decay;
        const f32x4 r = *reinterpret_cast<const f32x4*>(&ch.rk[16 * st + 4 * g4]);
        f16x4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (_Float16)(16 * st + 4 * g4 + i <= t ? d[i] * r[i] : 0.f);
        put_fragment(sh.p, lane, tt, st, x);
      }
    }
    barrier_lds();
    float* blocks = reinterpret_cast<float*>(sh.v);
    if (wave == 0) invert_diagonal(blocks, lane);

    // K' S0^T, rows t = 4g + i, column v; S0 Q'^T, rows v, column t.
    f32x4 x[4], o[4];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) x[tt] = o[tt] = zero4();
#pragma unroll
    for (int m = 0; m < KB; ++m) {
      const f16x8 hi = to_f16(S[2 * m], S[2 * m + 1]);
      if constexpr (kTerms == 2) {
        const f16x8 lo = rest_f16(S[2 * m], S[2 * m + 1], hi);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          x[tt] = mfma(__builtin_bit_cast(f16x8, read_row<K>(sh.k, lane, 16 * tt, m)), lo, x[tt]);
          if constexpr (kF16In) o[tt] = mfma(lo, __builtin_bit_cast(f16x8, read_row<K>(sh.q, lane, 16 * tt, m)), o[tt]);
        }
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        x[tt] = mfma(__builtin_bit_cast(f16x8, read_row<K>(sh.k, lane, 16 * tt, m)), hi, x[tt]);
        o[tt] = mfma(hi, __builtin_bit_cast(f16x8, read_row<K>(sh.q, lane, 16 * tt, m)), o[tt]);
      }
    }
    // What is to be learnt, V' - h K' S.
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      const f32x4 hh = *reinterpret_cast<const f32x4*>(&ch.h[16 * tt + 4 * g4]);
      const float e = ch.e[16 * tt + l16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = i & 1 ? high_value<kF16In>(raw[tt][i / 2]) : low_value<kF16In>(raw[tt][i / 2]);
        x[tt][i] = y * scale.v - hh[i] * x[tt][i];
        o[tt][i] *= e;
      }
    }
    barrier_lds();
    // T below the diagonal: first beside it, then the square of four blocks.
    const auto block = [&](int tt, int st) { return blocks + block_at(tt, st); };
    const auto read_block = [&](int tt, int st) {
      f32x4 y;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = block(tt, st)[(4 * g4 + i) * kBlockRow + l16];
      return y;
    };
    if (wave < 2) {
      const int t = 2 * wave + 1, s = 2 * wave;
      const f32x4 y = -block_product(block(s, s), block_product(block(t, s), block(t, t), lane, zero4()), lane, zero4());
      put_t(sh.t, ch, lane, t, s, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) block(t, s)[(4 * g4 + i) * kBlockRow + l16] = y[i];
    } else if (wave == 2) {
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) put_t(sh.t, ch, lane, tt, tt, read_block(tt, tt));
    }
    barrier_lds();
    if (wave < 2) {
      const int t = 2 + wave;
      f32x4 z0 = block_product(block(2, 0), block(t, 2), lane, zero4()), z1 = block_product(block(2, 1), block(t, 2), lane, zero4());
      if (wave == 1) z0 = block_product(block(3, 0), block(3, 3), lane, z0), z1 = block_product(block(3, 1), block(3, 3), lane, z1);
      put_t(sh.t, ch, lane, t, 0, -block_product(block(1, 0), z1, lane, block_product(block(0, 0), z0, lane, zero4())));
      put_t(sh.t, ch, lane, t, 1, -block_product(block(1, 1), z1, lane, zero4()));
    }
    barrier_lds();

    // D = T x, rows t, column v.
    f32x4 d[4];
    {
      f16x8 hi[2], lo[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        hi[b] = to_f16(x[2 * b], x[2 * b + 1]);
        if constexpr (kTerms == 2) lo[b] = rest_f16(x[2 * b], x[2 * b + 1], hi[b]);
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        d[tt] = zero4();
#pragma unroll
        for (int b = 0; b <= tt / 2; ++b) {
          const f16x8 th = read_fragment(sh.t, lane, tt, b);
          if constexpr (kTerms == 2) {
            d[tt] = mfma(read_fragment(sh.t + kTermP, lane, tt, b), hi[b], d[tt]);
            d[tt] = mfma(th, lo[b], d[tt]);
          }
          d[tt] = mfma(th, hi[b], d[tt]);
        }
      }
    }
    // O^T += D^T P^T, and the outputs, rows v = 4g + i, column t, to V's tile.
    {
      f16x8 dh[2], dl[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        dh[b] = to_f16(d[2 * b], d[2 * b + 1]);
        if constexpr (kF16In) dl[b] = rest_f16(d[2 * b], d[2 * b + 1], dh[b]);
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
        for (int b = 0; b <= tt / 2; ++b) {
          const f16x8 pp = read_fragment(sh.p, lane, tt, b);
          if constexpr (kF16In) o[tt] = mfma(dl[b], pp, o[tt]);
          o[tt] = mfma(dh[b], pp, o[tt]);
        }
        const float f = ch.f[16 * tt + l16];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[tt][i] *= f * scale.out[i];
      }
    }
    if (__ballot(first_bad < kC)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int from = __shfl(first_bad, 4 * g4 + i);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
          if (16 * tt + l16 >= from) o[tt][i] = __builtin_nanf("");
      }
      if (first_bad < kC)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = zero4() + __builtin_nanf("");
    }
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      char* at = sh.v + row_at<V>(16 * tt + l16) + (wave * 16 + 4 * g4) * 2;
      if constexpr (kF16In) {
        *reinterpret_cast<f16x4*>(at) = f16x4{(_Float16)o[tt][0], (_Float16)o[tt][1], (_Float16)o[tt][2], (_Float16)o[tt][3]};
      } else {
        *reinterpret_cast<bf16x4*>(at) = bf16x4{to_bf16(o[tt][0]), to_bf16(o[tt][1]), to_bf16(o[tt][2]), to_bf16(o[tt][3])};
      }
    }
    // The state.
    const float total = ch.total;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] *= total;
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) d[tt] *= *reinterpret_cast<const f32x4*>(&ch.c[16 * tt + 4 * g4]);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const f16x8 hi = to_f16(d[2 * b], d[2 * b + 1]);
      f16x8 lo;
      if constexpr (kTerms == 2) lo = rest_f16(d[2 * b], d[2 * b + 1], hi);
#pragma unroll
      for (int kt = 0; kt < KT; kt += 2) {
        const f16x8 k0 = __builtin_bit_cast(f16x8, read_col<K, true>(sh.k, lane, 32 * b, kt));
        const f16x8 k1 = __builtin_bit_cast(f16x8, read_col<K, true>(sh.k, lane, 32 * b, kt + 1));
        if constexpr (kTerms == 2) S[kt] = mfma(k0, lo, S[kt]), S[kt + 1] = mfma(k1, lo, S[kt + 1]);
        S[kt] = mfma(k0, hi, S[kt]), S[kt + 1] = mfma(k1, hi, S[kt + 1]);
      }
    }
    barrier_lds();
    Rows<V, kThreads>::store(sh.v, reinterpret_cast<__bf16*>(out), p.o_t, here, count, tid);
  }
  if (slots.to >= 0) {
    const int by = -(scale.ex + scale.shift);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[kt][i] = ldexp2(S[kt][i], by);
    walk.store_plane(p, stage, plane_at(p, slots.to, h), v0, wave, lane);
  }
}

template <int K, int V, int kTerms>
int launch_kv(const DeltaPlan& p, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.N * p.H * p.slices);
  if (p.f16) delta_walk<K, V, kTerms, true><<<grid, 64 * kWavesOf<V>, 0, s>>>(p);
  else delta_walk<K, V, kTerms, false><<<grid, 64 * kWavesOf<V>, 0, s>>>(p);
  return (int)hipGetLastError();
}
template <int kTerms>
int launch_terms(const DeltaPlan& p, hipStream_t s) {
  const int V = p.V / p.slices;
  if (p.K == 128) return V == 128 ? launch_kv<128, 128, kTerms>(p, s) : launch_kv<128, 64, kTerms>(p, s);
  return V == 128 ? launch_kv<64, 128, kTerms>(p, s) : launch_kv<64, 64, kTerms>(p, s);
}

}  // namespace

int launch_delta_walk(const DeltaPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return one_term(p) ? launch_terms<1>(p, s) : launch_terms<2>(p, s);
}

}  // namespace kda
