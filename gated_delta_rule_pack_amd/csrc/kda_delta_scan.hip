// The gated delta rule's prompts where there are few sequences and heads: the chunks' own work in one parallel kernel, and a
// walk over the chunks that many workgroups share. kda_delta.hip has the mathematics, and the walk for many units.
//
// delta_prep takes one chunk of one value head to a workgroup and leaves its record: T and P as operand fragments,
// and the chunk's factors; the first head of a group leaves the scaled rows K' and Q', in fragment order too.
//
// delta_scan walks a sequence's chunks for 16 value channels to a workgroup. A chunk's chain (K' S -> what is to be learnt -> D
// -> S) is cut over four waves, one for each 16 tokens and, of the state, for each quarter of the key channels; they meet
// three times a chunk in LDS, where every value passes as an operand fragment. Four more waves make the outputs behind them.
// All read their fragments straight from memory, a few chunks ahead, each fragment in one wave alone.
//
// Measured: delta_prep is bound by memory, 0.87 GB in 195 us for 32768 tokens at H = 32 (4.5 TB/s) and 50 us for 16384 at
// H = 12; a chunk of delta_scan takes 1.33 us, 3200 cycles, most of it its three dependent products with what lies between
// them: 342 us for 16384 tokens at H = 12, where the walk takes 1270 for all. V comes by the outputs' waves, through LDS and a
// transposing read: by the chain's own, two bytes a lane, the scan took 308 us where it took 274, and with K' by the outputs'
// waves too 300. A chunk that is walked by tokens adds 20 us.
#include <hip/hip_runtime.h>

#include <cstddef>
#include <type_traits>

#include "kda_delta_device.h"

namespace kda {
namespace {

// A record: T in two terms, P's first, fragments as the walk has them in LDS, P's second, then the factors.
constexpr int kRecP = 2 * kTermP, kRecRest = 3 * kTermP, kRecFactors = 3 * kTermP + kRestP;
static_assert(kRecFactors + sizeof(Factors) <= kDeltaRecord, "record size");

// Sequence n's chunks have the places floor(cu[n] / 64) + n on: at least as many as it has chunks.
__device__ __forceinline__ int chunk_place(const DeltaPlan& p, int n) { return bound(p, n) / kC + n; }
// The last sequence that starts at or before a place.
__device__ __forceinline__ int find_chunk(const DeltaPlan& p, int place, int lane) {
  int lo = 0, hi = p.N;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6;
    const int at = lo + lane * step;
    const uint64_t mask = __ballot(at < hi && chunk_place(p, at) <= place) | 1;
    lo += __builtin_amdgcn_readfirstlane(63 - __builtin_clzll(mask)) * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// A tile's rows in LDS to memory as operand fragments: 16 rows and 32 channels to 1 KB.
template <int D, int kThreads>
__device__ __forceinline__ void store_fragments(const char* tile, char* to, int tid) {
#pragma unroll
  for (int i = 0; i < kC * D * 2 / 16 / kThreads; ++i) {
    const int unit = i * kThreads + tid, lane = unit & 63, m = (unit >> 6) % (D / 32), tt = (unit >> 6) / (D / 32);
    *reinterpret_cast<u32x4*>(to + unit * 16) =
        *reinterpret_cast<const u32x4*>(tile + row_at<D>(16 * tt + (lane & 15)) + m * 64 + (lane >> 4) * 16);
  }
}

template <int K, bool kF16In>
__global__ __launch_bounds__(256, 3) void delta_prep(const DeltaPlan p) {
  constexpr int kThreads = 256;
  __shared__ struct {
    alignas(16) char k[kC * kRowBytes<K>];
    alignas(16) char q[kC * kRowBytes<K>];
    alignas(16) float blocks[10 * kBlock];
    Making making;
    RowInfo info[2][kC];
  } sh;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int place = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int n = find_chunk(p, place, lane);
  const int begin = bound(p, n), len = bound(p, n + 1) - begin;
  const int in = (place - chunk_place(p, n)) * kC;
  if (len <= 1 || in < 0 || in >= len) return;  // no chunk stands here (or the bounds fall)
  const int count = min(len - in, kC);
  const int64_t first = begin + in;
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + (h / p.group) * p.q_h;
  const uint16_t* k = reinterpret_cast<const uint16_t*>(p.k) + (h / p.group) * p.k_h;
  ScaledRows<K, kThreads, kF16In> rq, rk;
  rk.rows.load(reinterpret_cast<const __bf16*>(k), p.k_t, first, count, tid);
  rq.rows.load(reinterpret_cast<const __bf16*>(q), p.q_t, first, count, tid);
  float g = 0.f, beta = 0.f;
  if (wave == 0 && lane < count) {
    const int64_t at = (first + lane) * p.H + h;
    if (p.g) {
      const int64_t ag = p.g_per_token ? at : h;
      g = p.g_bf16 ? (float)reinterpret_cast<const __bf16*>(p.g)[ag] : reinterpret_cast<const float*>(p.g)[ag];
    }
    beta = p.beta_bf16 ? (float)reinterpret_cast<const __bf16*>(p.beta)[at] : reinterpret_cast<const float*>(p.beta)[at];
  }
  Decays decays = {};
  if (wave == 0) decays = put_decays(sh.making, g, lane);
  rk.scale();
  rq.scale();
  rk.put(sh.k, sh.info[0], tid);
  rq.put(sh.q, sh.info[1], tid);
  barrier_lds();
  char* rec = p.records + ((int64_t)place * p.H + h) * kDeltaRecord;
  if (h % p.group == 0) {
    const int64_t at = ((int64_t)place * (p.H / p.group) + h / p.group) * (kC * K * 2);
    store_fragments<K, kThreads>(sh.k, p.keys + at, tid);
    store_fragments<K, kThreads>(sh.q, p.queries + at, tid);
  }
  if (wave == 0) {
    Numbers numbers;
    numbers.put_steps(sh.making, p, decays, sh.info[0][lane], sh.info[1][lane], beta, lane);
    numbers.put_factors(*reinterpret_cast<Factors*>(rec + kRecFactors), p, decays, lane);
  }
  TileDecays between;
  TileProducts products;
  by_wave(wave, [&](auto W) {
    tile_decays<decltype(W)::value>(sh.making, lane, between);
    tile_products<K, decltype(W)::value>(sh.k, sh.q, lane, products);
  });
  barrier_lds();
  by_wave(wave, [&](auto W) {
    put_tiles<decltype(W)::value>(sh.blocks, sh.making, lane, products, between, [&](int tt, int st, f16x4 x, uint32_t rest) {
      put_fragment(rec + kRecP, lane, tt, st, x);
      put_rest(rec + kRecRest, lane, tt, st, rest);
    });
  });
  barrier_lds();
  if (wave == 0) invert_diagonal(sh.blocks, lane);
  barrier_lds();
  const auto put_t = [&](int tt, int st, f32x4 x) {
    const Terms y = t_terms(x);
    put_fragment(rec, lane, tt, st, y.hi);
    put_fragment(rec + kTermP, lane, tt, st, y.lo);
  };
  near_blocks(sh.blocks, lane, wave, put_t);
  barrier_lds();
  far_blocks(sh.blocks, lane, wave, put_t);
}

constexpr int kBadTop = 1 << 14;  // exponent that stands for a value that is not finite
template <int K>
struct ScanShared {
  static constexpr int KB = K / 32;
  alignas(16) char s[KB][2][1024];   // the state's fragments, two terms
  alignas(16) char x[2][2][1024];    // what is to be learnt
  alignas(16) char d[2][2][1024];    // D times its decay to the chunk's end
  alignas(16) char dh[2][2][1024];   // D
  alignas(16) char k[kC * kRowBytes<K>];
  alignas(16) char v[2][kC * 32];    // V of this chunk and of the next, 16 channels
  alignas(16) float factors[2][3][kC];  // b, h and c of both
  alignas(16) uint32_t numbers[2][4];   // total, steps, reach
  alignas(16) int top[16][4];        // largest exponents of a channel, of its state and of what is to be learnt, by wave
  alignas(16) int bad[16][4];        // its first token whose value is not finite
  alignas(16) uint32_t small[2][4];  // whether a wave found what is to be learnt too small: at first sight; looked into
  alignas(16) float sum[2][4][16];
  // For a chunk that is walked token by token.
  alignas(16) float run[2][4][16];   // what a wave's tokens leave of L before them, and their own L
  alignas(16) float token[4][kC];    // b, s and f, and the decays
  alignas(16) char q[kC * kRowBytes<K>];
};

// A wave's share of a chunk on its way from memory, in the same registers for both kinds of wave.
template <int K>
struct Fetch {
  u32x4 rows[K / 32];  // 16 tokens of K' (chain) or Q' (outputs)
  u32x4 frag[2][2];    // [term][b] of T's or P's row of tiles
  u32x4 v;             // outputs: V of the next chunk, a token's 8 channels in half the lanes
  // The outputs' alone.
  float e, f;          // factors of token l % 16
  uint32_t factor;     // of the next chunk, as V: b, h or c of token l % 16, or one of the chunk's numbers
};

template <int K, bool kF16In>
__global__ __launch_bounds__(512, 2) void delta_scan(const DeltaPlan p) {
  constexpr int KB = K / 32, KTW = K / 64;  // tiles of a chain wave's state
  __shared__ ScanShared<K> sh;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
  // The slices of a unit run on one XCD, whose L2 then reads a record once.
  const int slices = p.V / 16, j = blockIdx.x >> 3, slice = j % slices, unit = (j / slices) * 8 + (blockIdx.x & 7);
  if (unit >= p.N * p.H) return;
  __shared__ Ranking ranking;
  const int h = unit % p.H, v0 = slice * 16, n = p.ranked ? ranked_sequence(p, ranking, unit / p.H, tid) : unit / p.H;
  const bool chain = wave < 4;
  const int w = wave & 3;  // token tile; a chain wave's part of the state too
  const int begin = __builtin_amdgcn_readfirstlane(bound(p, n));
  const int len = __builtin_amdgcn_readfirstlane(max(bound(p, n + 1) - begin, 0));
  const Slots slots = slots_of(p, n);
  const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v) + h * p.v_h + v0;
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + h * p.o_h + v0;

  // The state: S[j] holds channel v0 + l16 and keys k0 + 4 j + i.
  const int k0 = KTW == 2 ? 32 * w + 8 * g4 : 32 * (w >> 1) + 8 * g4 + 4 * (w & 1);
  f32x4 S[KTW];
#pragma unroll
  for (int kt = 0; kt < KTW; ++kt) S[kt] = zero4();
  if (chain && slots.from >= 0) {
    const int64_t plane = plane_at(p, slots.from, h);
#pragma unroll
    for (int kt = 0; kt < KTW; ++kt) {
      if (!p.kfirst) {
        const int64_t at = plane + (int64_t)(v0 + l16) * K + k0 + 4 * kt;
        if (p.state_dtype == kF32) S[kt] = load_state4<kF32>(p.state_in, at);
        else if (p.state_dtype == kF16) S[kt] = load_state4<kF16>(p.state_in, at);
        else S[kt] = load_state4<kBF16>(p.state_in, at);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t at = plane + (int64_t)(k0 + 4 * kt + i) * p.V + v0 + l16;
          if (p.state_dtype == kF32) S[kt][i] = load_state1<kF32>(p.state_in, at);
          else if (p.state_dtype == kF16) S[kt][i] = load_state1<kF16>(p.state_in, at);
          else S[kt][i] = load_state1<kBF16>(p.state_in, at);
        }
      }
    }
  }
  const auto store_state = [&]() __attribute__((always_inline)) {
    if (!chain || slots.to < 0) return;
    const int64_t plane = plane_at(p, slots.to, h);
#pragma unroll
    for (int kt = 0; kt < KTW; ++kt) {
      if (!p.kfirst) {
        const int64_t at = plane + (int64_t)(v0 + l16) * K + k0 + 4 * kt;
        if (p.state_dtype == kF32) store_state4<kF32>(p.state_out, at, S[kt]);
        else if (p.state_dtype == kF16) store_state4<kF16>(p.state_out, at, S[kt]);
        else store_state4<kBF16>(p.state_out, at, S[kt]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t at = plane + (int64_t)(k0 + 4 * kt + i) * p.V + v0 + l16;
          if (p.state_dtype == kF32) store_state1<kF32>(p.state_out, at, S[kt][i]);
          else if (p.state_dtype == kF16) store_state1<kF16>(p.state_out, at, S[kt][i]);
          else store_state1<kBF16>(p.state_out, at, S[kt][i]);
        }
      }
    }
  };
  if (len == 0) {
    store_state();
    return;
  }
  if (len == 1) {  // the recurrent step, in fp32
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + (int64_t)begin * p.q_t + (h / p.group) * p.q_h;
    const uint16_t* k = reinterpret_cast<const uint16_t*>(p.k) + (int64_t)begin * p.k_t + (h / p.group) * p.k_h;
    const int64_t at = (int64_t)begin * p.H + h;
    float g = 0.f;
    if (p.g) {
      const int64_t ag = p.g_per_token ? at : h;
      g = p.g_bf16 ? (float)reinterpret_cast<const __bf16*>(p.g)[ag] : reinterpret_cast<const float*>(p.g)[ag];
    }
    float beta = p.beta_bf16 ? (float)reinterpret_cast<const __bf16*>(p.beta)[at] : reinterpret_cast<const float*>(p.beta)[at];
    if (!(g <= 0.f)) beta = __builtin_nanf("");
    const float decay = __expf(g);
    // Every wave takes the whole rows: two channels a lane at K = 128.
    float kk[KTW], qq[KTW];
#pragma unroll
    for (int i = 0; i < KTW; ++i) kk[i] = token_value<kF16In>(k[lane + 64 * i]), qq[i] = token_value<kF16In>(q[lane + 64 * i]);
    float rk = 1.f, rq = 1.f;
    if (p.normalize) rk = unit_factor(kk), rq = unit_factor(qq);
    float kq = 0.f;
#pragma unroll
    for (int i = 0; i < KTW; ++i) kq += (kk[i] * rk) * (qq[i] * rq);
    kq = wave_sum(kq);
    float u = 0.f, o = 0.f, key[4 * KTW];
    if (chain) {
#pragma unroll
      for (int i = 0; i < 4 * KTW; ++i) {
        key[i] = token_value<kF16In>(k[k0 + i]) * rk;
        u += S[i / 4][i % 4] * key[i];
        o += S[i / 4][i % 4] * (token_value<kF16In>(q[k0 + i]) * rq);
      }
      u += __shfl_xor(u, 16), o += __shfl_xor(o, 16);
      u += __shfl_xor(u, 32), o += __shfl_xor(o, 32);
      if (g4 == 0) sh.sum[0][w][l16] = u, sh.sum[1][w][l16] = o;
    }
    barrier_lds();
    if (!chain) return;
    u = o = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) u += sh.sum[0][i][l16], o += sh.sum[1][i][l16];
    const float delta = beta * (token_value<kF16In>(v[(int64_t)begin * p.v_t + l16]) - decay * u);
#pragma unroll
    for (int i = 0; i < 4 * KTW; ++i) S[i / 4][i % 4] = S[i / 4][i % 4] * decay + delta * key[i];
    store_state();
    if (w == 0 && g4 == 0) {
      const float x = p.scale * (decay * o + delta * kq);
      out[(int64_t)begin * p.o_t + l16] = kF16In ? __builtin_bit_cast(uint16_t, (_Float16)x) : __builtin_bit_cast(uint16_t, to_bf16(x));
    }
    return;
  }

  const int chunks = (len + kC - 1) / kC, place = chunk_place(p, n);
  const int H_qk = p.H / p.group, hq = h / p.group;
  const auto whole = [](const char* at, int bytes) __attribute__((always_inline)) { return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), (short)0, bytes, kBufWord3); };
  // Rows of V or the outputs, 16 channels: those behind the sequence's end are out of range.
  const auto buffer = [&](const uint16_t* at, int64_t stride, int left) __attribute__((always_inline)) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(at), (short)0, ((min(left, kC) - 1) * (int)stride + 16) * 2, kBufWord3);
  };
  constexpr int kAhead = 3;
  Fetch<K> fetched[kAhead];
  const auto load = [](__amdgpu_buffer_rsrc_t r, int at, int uniform) __attribute__((always_inline)) { return __builtin_amdgcn_raw_buffer_load_b128(r, at, uniform, 0); };
  // Where the next chunk to be fetched lies. Behind the last chunk it is fetched again, without a branch, so that a wait can count
  // the loads behind its own.
  const char* next_record = p.records + ((int64_t)place * p.H + h) * kDeltaRecord;
  const char* next_rows = (chain ? p.keys : p.queries) + ((int64_t)place * H_qk + hq) * (kC * K * 2);
  const char* next_factors = next_record;
  const uint16_t* next_v = v + (int64_t)begin * p.v_t;
  int next_left = len, left_v = len;
  const int at16 = lane * 16, at_row = l16 * 4;
  // The last fragment of a row of tiles: with one tile (half_fragment) a lane has 8 bytes of it, and reads 16; what is its neighbour's goes.
  const int last_unit = w & 1 ? 16 : 8;
  const uint32_t keep[2] = {w == 0 ? 0u : ~0u, w == 2 ? 0u : ~0u};
  const auto operand = [&](u32x4 x, int b) __attribute__((always_inline)) {
    x[2] &= keep[b], x[3] &= keep[b];
    return __builtin_bit_cast(f16x8, x);
  };
  const auto rest_operand = [&](u32x4 x, int b) __attribute__((always_inline)) { return p_rest_operand(u32x2{x[0], x[1] & keep[b]}); };
  const auto advance = [&]() __attribute__((always_inline)) {
    const bool more = next_left > kC;
    next_record += more ? (int64_t)p.H * kDeltaRecord : 0;
    next_rows += more ? (int64_t)H_qk * (kC * K * 2) : 0;
    next_left -= more ? kC : 0;
  };
  const auto fetch_rows = [&](Fetch<K>& f) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t row = whole(next_rows, kC * K * 2);
#pragma unroll
    for (int m = 0; m < KB; ++m) f.rows[m] = load(row, at16 + m * 1024, w * (KB * 1024));
  };
  const auto fetch_record = [&](Fetch<K>& f, auto for_chain) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t rec = whole(next_record, kDeltaRecord);
#pragma unroll
    for (int b = 0; b < 2; ++b) {  // the first two rows of tiles have one fragment
      const int from = fragment(w, w < 2 ? 0 : b), at = lane * (b == w >> 1 || w < 2 ? last_unit : 16);
      f.frag[0][b] = load(rec, at, (for_chain ? 0 : kRecP) + from);
      if constexpr (for_chain) {
        f.frag[1][b] = load(rec, at, kTermP + from);
      } else {
        const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(rec, at / 2, kRecRest + from / 2, 0);
        f.frag[1][b][0] = x[0], f.frag[1][b][1] = x[1];
      }
    }
    if constexpr (!for_chain) {
      f.e = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rec, at_row, kRecFactors + (int)offsetof(Factors, e) + 64 * w, 0));
      f.f = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rec, at_row, kRecFactors + (int)offsetof(Factors, f) + 64 * w, 0));
    }
  };
  // V of one chunk, by the outputs' waves: token 16 w + l / 2, channels 8 (l % 2) on, twice. (All of a row's offset is the
  // lane's: the uniform one is not compared with the buffer's end.)
  const auto fetch_v = [&]() __attribute__((always_inline)) {
    const int v_row = (int)p.v_t * 2;
    return load(buffer(next_v, p.v_t, left_v), (16 * w + ((lane & 31) >> 1)) * v_row + (lane & 1) * 16, 0);
  };
  const auto advance_v = [&]() __attribute__((always_inline)) {
    const bool more = left_v > kC;
    next_v += more ? p.v_t * kC : 0;
    next_factors += more ? (int64_t)p.H * kDeltaRecord : 0;
    left_v -= more ? kC : 0;
  };
  const auto put_v = [&](u32x4 x, int i) __attribute__((always_inline)) { *reinterpret_cast<u32x4*>(sh.v[i & 1] + 16 * w * 32 + (lane & 31) * 16) = x; };
  // The factors that the chain takes: b, h and c of tokens 16 w + l % 16 in 48 lanes, the chunk's numbers behind them.
  static_assert(offsetof(Factors, b) == 0 && offsetof(Factors, h) == 4 * kC && offsetof(Factors, c) == 8 * kC &&
                offsetof(Factors, steps) == offsetof(Factors, total) + 4 && offsetof(Factors, reach) == offsetof(Factors, total) + 8, "as they are fetched");
  const int number = min(lane - 48, 2), at_factor = lane < 48 ? 4 * kC * g4 + 64 * w + 4 * l16 : (int)offsetof(Factors, total) + 4 * number;
  const auto fetch_factor = [&]() __attribute__((always_inline)) { return __builtin_amdgcn_raw_buffer_load_b32(whole(next_factors, kDeltaRecord), at_factor, kRecFactors, 0); };
  const auto put_factor = [&](uint32_t x, int i) __attribute__((always_inline)) {
    if (lane < 48) sh.factors[i & 1][g4][16 * w + l16] = __uint_as_float(x);
    else if (w == 0) sh.numbers[i & 1][number] = x;
  };
  struct OwnFactors {
    f32x4 b, h, c;  // of tokens 16 w + 4g + i
    uint32_t total, steps, reach;
  };
  const auto read_factors = [&](int i) __attribute__((always_inline)) {
    const auto of = [&](int j) __attribute__((always_inline)) { return *reinterpret_cast<const f32x4*>(&sh.factors[i & 1][j][16 * w + 4 * g4]); };
    const u32x4 n = *reinterpret_cast<const u32x4*>(sh.numbers[i & 1]);
    return OwnFactors{of(0), of(1), of(2), n[0], n[1], n[2]};
  };
  // Tokens 16 w + 4g + i of channel l % 16.
  const auto read_v = [&](int i) __attribute__((always_inline)) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(sh.v[i & 1] + (16 * w + 4 * g4 + (l16 >> 2)) * 32 + (lane & 3) * 8));
  };
  Scale scale;
  scale.ex = scale.apart = 0;
  scale.set(lane, 0);
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  const auto largest = [&]() __attribute__((always_inline)) {
    const i32x4 t = *reinterpret_cast<const i32x4*>(sh.top[l16]);
    return __builtin_bit_cast(i16x2, pair_max(pair_max(t[0], t[1]), pair_max(t[2], t[3])));
  };
  const auto least_bad = [&]() __attribute__((always_inline)) {
    const i32x4 t = *reinterpret_cast<const i32x4*>(sh.bad[l16]);
    return min(min(t[0], t[1]), min(t[2], t[3]));
  };
  const auto any_small = [&](int i) __attribute__((always_inline)) {
    const u32x4 t = *reinterpret_cast<const u32x4*>(sh.small[i]);
    return __builtin_amdgcn_readfirstlane(t[0] | t[1] | t[2] | t[3]) != 0;
  };
  const auto moves = [&](i16x2 tops) __attribute__((always_inline)) { return !stays(scale.ex, tops[0], tops[1]); };
  // Takes the ranges' powers; how far the state moves.
  const auto move = [&](i16x2 tops) __attribute__((always_inline)) {
    const Ranges r = ranges_of(scale.ex, tops[0], tops[1]);
    const int by = r.s - scale.ex;
    scale.ex = r.s;
    scale.apart = r.x - r.s;
    scale.set(lane, r.x);
    return by;
  };
  // (One way out of the loop: from each of its steps the compiler would see a way back to the first, and wait there for all loads.)
  const auto walk_chunks = [&](auto step) __attribute__((always_inline)) {
    static_assert(kAhead == 3, "as written out");
    int i = 0;
    for (; i + 3 <= chunks; i += 3) {
      step(fetched[0], i);
      step(fetched[1], i + 1);
      step(fetched[2], i + 2);
    }
    if (i < chunks) step(fetched[0], i);
    if (i + 1 < chunks) step(fetched[1], i + 1);
  };
  // Both kinds of wave take the same barriers: three a chunk; three more where a channel's scale has to move or a value
  // is not finite, which all of them see in sh.top; and two more where what is to be learnt is small, which they see in sh.small, and
  // three where it is too small.
  // A chunk token by token in fp32, by the chain's waves: K / 8 lanes to a channel, 8 keys to a lane. The state is in sh.s, [channel][K].
  const auto by_tokens = [&](int i, int count, float total) __attribute__((always_inline)) {
    constexpr int kLanes = K / 8;
    const int channel = tid / kLanes, j = tid % kLanes;
    if (channel >= 16) return;
    float* const plain = reinterpret_cast<float*>(sh.s) + channel * K + 8 * j;
    f32x4 a = *reinterpret_cast<const f32x4*>(plain), b = *reinterpret_cast<const f32x4*>(plain + 4);
    const DeltaPlan& p = plan_again();
    uint16_t* to = reinterpret_cast<uint16_t*>(p.out) + h * p.o_h + v0 + (begin + (int64_t)i * kC) * p.o_t + channel;
    const auto row = [&](const char* tile, int t, f32x4& x, f32x4& y) __attribute__((always_inline)) {
      const f16x8 r = *reinterpret_cast<const f16x8*>(tile + row_at<K>(t) + 16 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = (float)r[e], y[e] = (float)r[4 + e];
    };
    const auto dot = [&](f32x4 x, f32x4 y) __attribute__((always_inline)) {
      x *= a, y *= b;
      return lane_sum(((x[0] + x[1]) + (x[2] + x[3])) + ((y[0] + y[1]) + (y[2] + y[3])), kLanes);
    };
#pragma unroll 1
    for (int t = 0; t < count; ++t) {
      f32x4 k0, k1, q0, q1;
      row(sh.k, t, k0, k1);
      row(sh.q, t, q0, q1);
      const float decay = sh.token[3][t], v = token_value<kF16In>(*reinterpret_cast<const uint16_t*>(sh.v[i & 1] + t * 32 + channel * 2));
      const float x = sh.token[0][t] * v - sh.token[1][t] * (decay * dot(k0, k1));
      a = a * decay + k0 * x, b = b * decay + k1 * x;
      const float o = sh.token[2][t] * dot(q0, q1) * kTimesP;
      if (j == 0) to[t * p.o_t] = kF16In ? __builtin_bit_cast(uint16_t, (_Float16)o) : __builtin_bit_cast(uint16_t, to_bf16(o));
    }
    if (total != total) a = b = zero4() + __builtin_nanf("");
    *reinterpret_cast<f32x4*>(plain) = a, *reinterpret_cast<f32x4*>(plain + 4) = b;
  };
  if (chain) {
    constexpr uint32_t kInf = kF16In ? 0x7c00u : 0x7f80u;
    const auto put_state = [&]() __attribute__((always_inline)) {
      if constexpr (KTW == 2) {
        const f16x8 hi = to_f16(S[0], S[1]);
        *reinterpret_cast<f16x8*>(sh.s[w][0] + lane * 16) = hi;
        *reinterpret_cast<f16x8*>(sh.s[w][1] + lane * 16) = rest_f16(S[0], S[1], hi);
      } else {
        put_half<false>(sh.s[w >> 1][0], sh.s[w >> 1][1], lane * 16 + (w & 1) * 8, S[0]);
      }
    };
    const auto state_top = [&]() __attribute__((always_inline)) {
      float m = 0.f;
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(S[kt][i]));
      return exponent(m);
    };
    char* const k_rows = sh.k + 16 * w * kRowBytes<K> + row_at<K>(l16) + g4 * 16;
    __builtin_amdgcn_s_setprio(3);  // the outputs' waves fill its gaps
    barrier_lds();  // the first chunk's V and factors
    s16x4 values = read_v(0);
    OwnFactors own = read_factors(0);
    const auto step = [&](Fetch<K>& f, int i) __attribute__((always_inline)) {
      const int steps = (int)__builtin_amdgcn_readfirstlane(own.steps), reach = (int)__builtin_amdgcn_readfirstlane(own.reach);
      const float total = __uint_as_float(__builtin_amdgcn_readfirstlane(own.total));
      // The state's fragments and the channel's largest exponents.
      put_state();
      uint32_t value[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) value[e] = (uint16_t)values[e];
      uint32_t most = max(max(value[0] & 0x7fffu, value[1] & 0x7fffu), max(value[2] & 0x7fffu, value[3] & 0x7fffu));
      const auto tops_of = [&](uint32_t most) __attribute__((always_inline)) {
        const int state = state_top(), learnt = max(state - scale.ex + reach, exponent(token_value<kF16In>(most)) + steps);
        return __builtin_bit_cast(int, channel_max(i16x2{(short)state, (short)(most >= kInf ? kBadTop : learnt)}));
      };
      sh.top[l16][w] = tops_of(most);
      barrier_lds();
      f16x8 hi[KB], lo[KB];
      i16x2 tops = largest();
      const auto read_state = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < KB; ++m) {
          hi[m] = *reinterpret_cast<const f16x8*>(sh.s[m][0] + at16);
          lo[m] = *reinterpret_cast<const f16x8*>(sh.s[m][1] + at16);
        }
      };
      // K' S0, tokens 4g + i, channel l % 16.
      f32x4 a, b;
      const auto products = [&]() __attribute__((always_inline)) {
        a = b = zero4();
#pragma unroll
        for (int m = 0; m < KB; ++m) {
          const f16x8 k = __builtin_bit_cast(f16x8, f.rows[m]);
          a = mfma(k, hi[m], a);
          b = mfma(k, lo[m], b);
        }
      };
      read_state();
      __builtin_amdgcn_sched_barrier(0);  // all reads before the first wait
      products();
#pragma unroll
      for (int m = 0; m < KB; ++m) *reinterpret_cast<u32x4*>(k_rows + m * 64) = f.rows[m];
      int first_bad = kC;
      scale.apart = 0;
      f32x4 x;  // what is to be learnt, b V - h K' S
      bool lasts;
      const auto own_part = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = token_value<kF16In>(value[e]) * (own.b[e] * scale.v);
        lasts = state_lasts(tops[0], scale.apart, total);
      };
      own_part();
      if (__builtin_expect(__ballot(moves(tops)) != 0, 0)) {
        barrier_lds();
        int bad = kC;
        most = 0;
#pragma unroll
        for (int x = 3; x >= 0; --x) {
          if ((value[x] & 0x7fffu) >= kInf) bad = 16 * w + 4 * g4 + x, value[x] = 0;
          most = max(most, value[x] & 0x7fffu);
        }
        sh.top[l16][w] = tops_of(most);
        sh.bad[l16][w] = -channel_max(-bad);
        barrier_lds();
        first_bad = least_bad();
        tops = largest();
        const int by = move(tops);
        tops[0] += by;
#pragma unroll
        for (int kt = 0; kt < KTW; ++kt)
#pragma unroll
          for (int x = 0; x < 4; ++x) S[kt][x] = ldexp2(S[kt][x], by);
        put_state();
        barrier_lds();
        read_state();
        products();
        const float apart = ldexp2(1.f, scale.apart);
        a *= apart, b *= apart;
        own_part();
      }
      {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] -= own.h[e] * (a[e] + b[e]);
        const float least = fminf(fminf(fabsf(x[0]), fabsf(x[1])), fminf(fabsf(x[2]), fabsf(x[3])));
        const uint32_t small = __ballot(least < kLeastShare<kF16In> && !lasts) != 0;
        put_half<true>(sh.x[w >> 1][0], sh.x[w >> 1][1], at16 + (w & 1) * 8, x);
        sh.small[0][w] = small;
      }
      const f16x8 t0 = operand(f.frag[0][0], 0), t1 = operand(f.frag[1][0], 0), u0 = operand(f.frag[0][1], 1), u1 = operand(f.frag[1][1], 1);
      barrier_lds();
      f16x8 kk[2][KTW];
      u32x4 smalls;
      {
        smalls = *reinterpret_cast<const u32x4*>(sh.small[0]);
        f16x8 xh[2], xl[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          xh[s] = *reinterpret_cast<const f16x8*>(sh.x[s][0] + at16);
          xl[s] = *reinterpret_cast<const f16x8*>(sh.x[s][1] + at16);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt) kk[s][kt] = __builtin_bit_cast(f16x8, read_col<K, true>(sh.k, lane, 32 * s, w * KTW + kt));
        fetch_rows(f);
        __builtin_amdgcn_sched_barrier(0);
        f32x4 a = mfma(t0, xh[0], zero4()), b = mfma(t1, xh[0], zero4()), c = mfma(t0, xl[0], zero4());
        if (w >= 2) {
          a = mfma(u0, xh[1], a);
          b = mfma(u1, xh[1], b);
          c = mfma(u0, xl[1], c);
        }
        f32x4 d = a + (b + c) * kDown, decayed = d * own.c;
        put_half<true>(sh.d[w >> 1][0], sh.d[w >> 1][1], at16 + (w & 1) * 8, decayed);
        put_half<true>(sh.dh[w >> 1][0], sh.dh[w >> 1][1], at16 + (w & 1) * 8, d);
      }
      barrier_lds();
      const bool found_small = __builtin_amdgcn_readfirstlane(smalls[0] | smalls[1] | smalls[2] | smalls[3]) != 0;
      bool walked = false;  // the next chunk's loads stand behind both ways, which then have the same loads behind each other
      if (__builtin_expect(found_small, 0)) {
        Fading own_run;
        const int count = min(len - i * kC, kC), t = 16 * w + 4 * g4;
        own_run.set(decays_at(plan_again(), begin + (int64_t)i * kC + t, count - t, h), x);
        float through = 0.f, all = own_run.all;
        own_run.before(through, lane);
        all *= __shfl_xor(all, 16), all *= __shfl_xor(all, 32);
        if (lane < 16) sh.run[0][w][lane] = all, sh.run[1][w][lane] = through;
        barrier_lds();
        through = state_share(tops[0], scale.apart);
        for (int j = 0; j < w; ++j) through = fmaxf(through * sh.run[0][j][l16], sh.run[1][j][l16]);
        const float before = own_run.before(through, lane);
        const uint32_t found = __ballot(own_run.fades(before, kLeastShare<kF16In>)) != 0;
        if (lane == 0) sh.small[1][w] = found;
        barrier_lds();
        if (any_small(1)) {
          float* const plain = reinterpret_cast<float*>(sh.s);  // the state, [channel][K]
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt)
#pragma unroll
            for (int e = 0; e < 4; ++e) plain[l16 * K + k0 + 4 * kt + e] = ldexp2(S[kt][e], -scale.ex);
          scale.ex = scale.apart = 0;
          scale.set(lane, 0);
          barrier_lds();
          by_tokens(i, count, total);
          barrier_lds();
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt) S[kt] = *reinterpret_cast<const f32x4*>(plain + l16 * K + k0 + 4 * kt);
          barrier_lds();
          walked = true;
        }
      }
      if (__builtin_expect(!walked, 1)) {
#pragma unroll
        for (int kt = 0; kt < KTW; ++kt) S[kt] *= ldexp2(total, scale.apart);
        scale.ex += scale.apart;
      }
      {
        f16x8 dh[2], dl[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          dh[s] = *reinterpret_cast<const f16x8*>(sh.d[s][0] + at16);
          dl[s] = *reinterpret_cast<const f16x8*>(sh.d[s][1] + at16);
        }
        values = read_v(i + 1);
        own = read_factors(i + 1);
        fetch_record(f, std::true_type());
        advance();
        __builtin_amdgcn_sched_barrier(0);
        if (__builtin_expect(!walked, 1)) {
          f32x4 rest[KTW];
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt) rest[kt] = mfma(kk[0][kt], dl[0], zero4());
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt) S[kt] = mfma(kk[0][kt], dh[0], S[kt]);
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt) rest[kt] = mfma(kk[1][kt], dl[1], rest[kt]);
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt) S[kt] = mfma(kk[1][kt], dh[1], S[kt]);
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt) S[kt] += rest[kt] * kDown;
          if (first_bad < kC)
#pragma unroll
            for (int kt = 0; kt < KTW; ++kt) S[kt] = zero4() + __builtin_nanf("");
        }
      }
    };
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      fetch_rows(fetched[a]);
      fetch_record(fetched[a], std::true_type());
      advance();
      __builtin_amdgcn_sched_barrier(0);  // in this order, for the first chunks' waits
    }
    walk_chunks(step);
#pragma unroll
    for (int kt = 0; kt < KTW; ++kt)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[kt][e] = ldexp2(S[kt][e], -scale.ex);
    store_state();
  } else {
    const int at_out = ((16 * w + l16) * (int)p.o_t + 4 * g4) * 2;
    put_v(fetch_v(), 0);
    put_factor(fetch_factor(), 0);
    advance_v();
    const auto step = [&](Fetch<K>& f, int i) __attribute__((always_inline)) {
      barrier_lds();
      // S0 Q', channels 4g + i, token l % 16.
      f32x4 o, low;
      const auto products = [&]() __attribute__((always_inline)) {
        o = low = zero4();
#pragma unroll
        for (int m = 0; m < KB; ++m) {
          const f16x8 q = __builtin_bit_cast(f16x8, f.rows[m]);
          o = mfma(*reinterpret_cast<const f16x8*>(sh.s[m][0] + lane * 16), q, o);
          low = mfma(*reinterpret_cast<const f16x8*>(sh.s[m][1] + lane * 16), q, low);
        }
      };
      const i16x2 tops = largest();
      products();
      put_v(f.v, i + 1);
      put_factor(f.factor, i + 1);
      int first_bad = kC;
      scale.apart = 0;
      f32x4 by_apart = zero4() + 1.f;
      if (__builtin_expect(__ballot(moves(tops)) != 0, 0)) {
        barrier_lds();
        barrier_lds();
        first_bad = least_bad();
        move(largest());
        const float by = ldexp2(1.f, scale.apart);
#pragma unroll
        for (int e = 0; e < 4; ++e) by_apart[e] = __shfl(by, 4 * g4 + e);
        barrier_lds();
        products();
      }
      o = (o + low) * (f.e * by_apart);
      barrier_lds();
      const bool found_small = any_small(0);
      const f16x8 p0 = operand(f.frag[0][0], 0), p1 = operand(f.frag[0][1], 1), rest0 = rest_operand(f.frag[1][0], 0), rest1 = rest_operand(f.frag[1][1], 1);
      fetch_rows(f);
      barrier_lds();
      bool walked = false;
      if (__builtin_expect(found_small, 0)) {
        barrier_lds();
        barrier_lds();
        if (any_small(1)) {
          scale.ex = scale.apart = 0;
          scale.set(lane, 0);
          // The rows of Q' and the tokens' factors, for the chain's waves.
          const DeltaPlan& p = plan_again();
          const char* rows = p.queries + (((int64_t)place + i) * H_qk + hq) * (kC * K * 2) + w * (KB * 1024) + at16;
#pragma unroll
          for (int m = 0; m < KB; ++m)
            *reinterpret_cast<u32x4*>(sh.q + 16 * w * kRowBytes<K> + row_at<K>(l16) + g4 * 16 + m * 64) = *reinterpret_cast<const u32x4*>(rows + m * 1024);
          const Factors& fa = *reinterpret_cast<const Factors*>(p.records + (((int64_t)place + i) * p.H + h) * kDeltaRecord + kRecFactors);
          sh.token[w][lane] = w == 3 ? decays_at(p, begin + (int64_t)i * kC + lane, min(len - i * kC - lane, 1), h)[0]
                                     : (w == 0 ? fa.b : w == 1 ? fa.s : fa.f)[lane];
          barrier_lds();
          barrier_lds();
          barrier_lds();
          walked = true;
        }
      }
      u32x2 packed = {0, 0};
      if (__builtin_expect(!walked, 1)) {
        scale.ex += scale.apart;
        const auto d = [&](int s, int term) __attribute__((always_inline)) { return *reinterpret_cast<const f16x8*>(sh.dh[s][term] + lane * 16); };
        const f16x8 d0 = d(0, 0);
        o = mfma(d0, p0, o);
        f32x4 rest = mfma(d(0, 1), p0, zero4()), other = mfma(d0, rest0, zero4());
        if (w >= 2) {
          const f16x8 d1 = d(1, 0);
          o = mfma(d1, p1, o);
          rest = mfma(d(1, 1), p1, rest);
          other = mfma(d1, rest1, other);
        }
        o += (rest + other) * kDown;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= f.f * scale.out[e];
        if (__ballot(first_bad < kC)) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * w + l16 >= __shfl(first_bad, 4 * g4 + e)) o[e] = __builtin_nanf("");
        }
        if constexpr (kF16In) packed = __builtin_bit_cast(u32x2, f16x4{(_Float16)o[0], (_Float16)o[1], (_Float16)o[2], (_Float16)o[3]});
        else packed = __builtin_bit_cast(u32x2, bf16x4{to_bf16(o[0]), to_bf16(o[1]), to_bf16(o[2]), to_bf16(o[3])});
      }
      fetch_record(f, std::false_type());
      advance();
      f.v = fetch_v();
      f.factor = fetch_factor();
      advance_v();
      // (Of no row where the chunk was walked.)
      __builtin_amdgcn_raw_buffer_store_b64(packed, walked ? whole(reinterpret_cast<const char*>(out), 0) : buffer(out + (begin + (int64_t)i * kC) * p.o_t, p.o_t, len - i * kC), at_out, 0, 0);
    };
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      fetch_rows(fetched[a]);
      fetch_record(fetched[a], std::false_type());
      advance();
      fetched[a].v = fetch_v();
      fetched[a].factor = fetch_factor();
      advance_v();
      __builtin_amdgcn_sched_barrier(0);
    }
    barrier_lds();
    walk_chunks(step);
  }
}

template <int K, bool kF16In>
int launch_prep(const DeltaPlan& p, hipStream_t s) {
  delta_prep<K, kF16In><<<(unsigned)((int64_t)p.places * p.H), 256, 0, s>>>(p);
  return (int)hipGetLastError();
}
template <int K, bool kF16In>
int launch_scan(const DeltaPlan& p, hipStream_t s) {
  const int64_t units = (int64_t)p.N * p.H;
  delta_scan<K, kF16In><<<(unsigned)((units + 7) / 8 * 8 * (p.V / 16)), 512, 0, s>>>(p);
  return (int)hipGetLastError();
}

}  // namespace

int launch_delta_prep(const DeltaPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (p.K == 128) return p.f16 ? launch_prep<128, true>(p, s) : launch_prep<128, false>(p, s);
  return p.f16 ? launch_prep<64, true>(p, s) : launch_prep<64, false>(p, s);
}

int launch_delta_scan(const DeltaPlan& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (p.K == 128) return p.f16 ? launch_scan<128, true>(p, s) : launch_scan<128, false>(p, s);
  return p.f16 ? launch_scan<64, true>(p, s) : launch_scan<64, false>(p, s);
}

}  // namespace kda
