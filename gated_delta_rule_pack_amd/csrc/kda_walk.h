// Device side that the walks over packed prompts share (linear attention, the gated delta rule): tiles of 64 rows in
// LDS, the state's registers, bounds and slots.
#pragma once

#include <hip/hip_runtime.h>

#include "kda_device.h"
#include "kda_linear.h"

namespace kda {

constexpr int kC = kLinChunk;
// Waves of a walk's workgroup, 16 state rows each.
template <int V>
constexpr int kWavesOf = V / 16;
constexpr float kMinLogDecay = -120.f;  // e^-120 is 0 in fp32; keeps -inf out of the differences

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// Keeps what is derived from x inside the loop it is used in: left to itself the compiler makes all
// the walk's LDS and state addresses once, and then spills them around every chunk.
__device__ __forceinline__ int local_copy(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// LDS tile of 64 rows of D bf16. A row takes 16 bytes more than its elements, and inside 16 rows
// row r stands at place 2 (r % 8) + r / 8: the 16 rows of an operand read then start on different
// banks, and the 8 rows of half a plain transposing read do not meet. Every read is a lane's own place and
// a constant offset, and these take 9 cycles a wave (a transposing read moves half as much in them). The
// spread reads of k do meet: a lane's 8 bytes lie 16 from the next lane's, so rows r and r + 1, 8 banks apart,
// share every other pair of banks, two lanes to each. SQ_LDS_BANK_CONFLICT is 34 % of SQ_LDS_IDX_ACTIVE in the map walk
// and 37 % in the output walk of 32768 tokens at H = 32.
template <int D>
constexpr int kRowBytes = 2 * D + 16;
template <int D>
__device__ __forceinline__ int row_at(int row) {
  return ((row & ~15) | ((row & 7) << 1) | ((row >> 3) & 1)) * kRowBytes<D>;
}
// Operand rows: row r0 + l % 16 (r0 a multiple of 16), elements 32 m + 8 g + j.
template <int D>
__device__ __forceinline__ bf16x8 read_row(const char* tile, int lane, int r0, int m) {
  return *reinterpret_cast<const bf16x8*>(tile + r0 * kRowBytes<D> + m * 64 + row_at<D>(lane & 15) + (lane >> 4) * 16);
}
// Operand columns: of rows t0 + 4 g + i and t0 + 16 + 4 g + i (t0 a multiple of 32), by two transposing
// reads: 16 lanes give the addresses of four groups of four columns in four rows, lane j of row j / 4
// and group j % 4. Plain: columns 16 c + l % 16. Spread (k): the channels of state tile c.
template <int D, bool kSpread>
__device__ __forceinline__ bf16x8 read_col(const char* tile, int lane, int t0, int c) {
  const char* p = tile + t0 * kRowBytes<D> + (kSpread ? (c >> 1) * 64 + (c & 1) * 8 : c * 32) +
                  row_at<D>(4 * (lane >> 4) + ((lane & 15) >> 2)) + (lane & 3) * (kSpread ? 16 : 8);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + 16 * kRowBytes<D>));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Token bound n inside [0, T], whatever the device bounds hold.
__device__ __forceinline__ int bound(const LinearPlan& p, int n) { return min(max(p.cu[n], 0), p.T); }
// Where sequence n's tokens start on the axis, and the first place that is its own: an empty
// sequence takes that place (in the stretch that stands for its state).
__device__ __forceinline__ int64_t axis_start(const LinearPlan& p, int n) { return bound(p, n) + (int64_t)n * p.head_cost; }
__device__ __forceinline__ int64_t axis_own(const LinearPlan& p, int n) { return axis_start(p, n) - (n > 0); }

// The last sequence whose own place is at or before x: every wave probes 64 places at a time.
__device__ __forceinline__ int find_sequence(const LinearPlan& p, int64_t x, int lane) {
  int lo = 0, hi = p.N;  // own(lo) <= x; own(hi) > x or hi == N
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6;
    const int at = lo + lane * step;
    const bool before = at < hi && axis_own(p, at) <= x;
    const uint64_t mask = __ballot(before) | 1;
    const int last = __builtin_amdgcn_readfirstlane(63 - __builtin_clzll(mask));
    lo += last * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// Slots that sequence n starts from and leaves its final state in; -1: none.
struct Slots {
  int from, to;
};
__device__ __forceinline__ Slots slots_of(const LinearPlan& p, int n) {
  if (p.in_mode != kStatePaged) return Slots{p.in_mode == kStateDense ? n : -1, p.out_mode == kStateDense ? n : -1};
  const int s = p.indices[n];
  const bool old = p.flags[n], inside = s >= 0 && s < p.num_slots;
  return Slots{inside && old ? s : -1, inside ? s : -1};
}
__device__ __forceinline__ int64_t plane_at(const LinearPlan& p, int slot, int h) {
  return slot * p.stride0 + (int64_t)h * p.K * p.V;
}

// Eight elements of a state in a row.
template <int SDT>
__device__ __forceinline__ void load8(const void* base, size_t at, f32x4& a, f32x4& b) {
  a = load_state4<SDT>(base, at);
  b = load_state4<SDT>(base, at + 4);
}
template <int SDT>
__device__ __forceinline__ void store8(void* base, size_t at, f32x4 a, f32x4 b) {
  store_state4<SDT>(base, at, a);
  store_state4<SDT>(base, at + 4, b);
}

// The walk's state registers: S[vt][2 m + h] holds v = 16 vt + l % 16 of the wave's rows and
// k = 32 m + 8 g + 4 h + i.
template <int K, int V, int kWaves = kWavesOf<V>>
struct Walk {
  static constexpr int VT = V / (16 * kWaves);  // 16-row tiles of V per wave
  static constexpr int KT = K / 16;
  f32x4 S[VT][KT];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) S[vt][kt] = zero4();
  }
  // Plain workspace planes: register order, 1 KB per tile.
  __device__ __forceinline__ void load(const float* plane, int wave, int lane) {
    lane = local_copy(lane);
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        S[vt][kt] = *reinterpret_cast<const f32x4*>(plane + (((wave * VT + vt) * KT + kt) * 64 + lane) * 4);
  }
  __device__ __forceinline__ void store(float* plane, int wave, int lane) const {
    lane = local_copy(lane);
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        *reinterpret_cast<f32x4*>(plane + (((wave * VT + vt) * KT + kt) * 64 + lane) * 4) = S[vt][kt];
  }
  // The caller's planes, [V][K] or [K][V], from row (column) v0 on. 16-bit K-first planes pass through
  // 1 KB of the wave's LDS (stage), 32 rows of its 16 columns at a time, and the transposing read: 16
  // bytes a lane instead of 2 from memory (512 single tokens at H = 12: 100 instead of 231 us).
  __device__ __forceinline__ void load_plane(const LinearPlan& p, char* stage, int64_t at, int v0, int wave, int lane_) {
    const int lane = local_copy(lane_), g = lane >> 4;
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      const int v = v0 + (wave * VT + vt) * 16;
      if (p.kfirst && p.state_dtype != kF32) {
        u32x4 w[KT / 2];
#pragma unroll
        for (int m = 0; m < KT / 2; ++m)
          w[m] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p.state_in) + at +
                                                 (int64_t)(32 * m + (lane >> 1)) * p.V + v + (lane & 1) * 8);
#pragma unroll
        for (int m = 0; m < KT / 2; ++m) {
          *reinterpret_cast<u32x4*>(stage + lane * 16) = w[m];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4)(stage + (8 * g + 4 * h + ((lane & 15) >> 2)) * 32 + (lane & 3) * 8));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              S[vt][2 * m + h][i] = p.state_dtype == kF16 ? (float)__builtin_bit_cast(_Float16, (short)x[i])
                                                          : (float)__builtin_bit_cast(__bf16, (short)x[i]);
          }
        }
        continue;
      }
#pragma unroll
      for (int m = 0; m < KT / 2; ++m) {
        const int row = v + (lane & 15), k = m * 32 + 8 * g;
        f32x4 &a = S[vt][2 * m], &b = S[vt][2 * m + 1];
        if (!p.kfirst) {
          const size_t off = (size_t)(at + (int64_t)row * K + k);
          if (p.state_dtype == kF32) load8<kF32>(p.state_in, off, a, b);
          else if (p.state_dtype == kF16) load8<kF16>(p.state_in, off, a, b);
          else load8<kBF16>(p.state_in, off, a, b);
        } else {
          const float* from = reinterpret_cast<const float*>(p.state_in) + at + (int64_t)k * p.V + row;
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = from[i * p.V], b[i] = from[(4 + i) * p.V];
        }
      }
    }
  }
  __device__ __forceinline__ void store_plane(const LinearPlan& p, char* stage, int64_t at, int v0, int wave, int lane_) const {
    const int lane = local_copy(lane_), g = lane >> 4;
#pragma unroll
    for (int vt = 0; vt < VT; ++vt) {
      const int v = v0 + (wave * VT + vt) * 16;
#pragma unroll
      for (int m = 0; m < KT / 2; ++m) {
        const int row = v + (lane & 15), k = m * 32 + 8 * g;
        const f32x4 a = S[vt][2 * m], b = S[vt][2 * m + 1];
        if (!p.kfirst) {
          const size_t off = (size_t)(at + (int64_t)row * K + k);
          if (p.state_dtype == kF32) store8<kF32>(p.state_out, off, a, b);
          else if (p.state_dtype == kF16) store8<kF16>(p.state_out, off, a, b);
          else store8<kBF16>(p.state_out, off, a, b);
        } else if (p.state_dtype == kF32) {
          float* to = reinterpret_cast<float*>(p.state_out) + at + (int64_t)k * p.V + row;
#pragma unroll
          for (int i = 0; i < 4; ++i) to[i * p.V] = a[i], to[(4 + i) * p.V] = b[i];
        } else {
          uint16_t* to = reinterpret_cast<uint16_t*>(stage) + 8 * g * 16 + (lane & 15);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = j < 4 ? a[j & 3] : b[j & 3];
            to[j * 16] = p.state_dtype == kF16 ? __builtin_bit_cast(uint16_t, (_Float16)x) : __builtin_bit_cast(uint16_t, to_bf16(x));
          }
          *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p.state_out) + at + (int64_t)(32 * m + (lane >> 1)) * p.V + v +
                                    (lane & 1) * 8) = *reinterpret_cast<const u32x4*>(stage + lane * 16);
        }
      }
    }
  }
};

// Buffer over `count` rows of D bf16, `stride` elements apart, from row `first` of a tensor: a row
// behind them is out of range (rows do not overlap), so loads of it give zeros and stores are dropped.
template <int D>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const __bf16* base, int64_t first, int64_t stride, int count) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<__bf16*>(base + first * stride), (short)0,
                                           ((count - 1) * (int)stride + D) * 2, kBufWord3);
}

// 64 rows of D bf16 on their way from memory to an LDS tile: loaded a chunk ahead into
// registers, rows past the chunk's end as zeros.
template <int D, int kThreads>
struct Rows {
  static constexpr int kUnits = D / 8;             // 16-byte units of a row
  static constexpr int kRows = kThreads / kUnits;  // rows per pass
  static constexpr int kPasses = kC / kRows;
  u32x4 w[kPasses];
  __device__ __forceinline__ void load(const __bf16* base, int64_t stride, int64_t first, int count, int tid) {
    const __amdgpu_buffer_rsrc_t r = rows_buffer<D>(base, first, stride, count);
    const unsigned u = (unsigned)local_copy(tid);
    const int at = (int)(u / kUnits) * (int)stride * 2 + (int)(u % kUnits) * 16;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      w[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at + i * kRows * (int)stride * 2, 0, 0));
  }
  // Rows of a tile to memory, `count` of them, whole rows to a wave (parts of rows
  // leave their merging to L2: 32768 tokens at H = 32 took 405 us so when this way took 379) and past the caches,
  // which have no use for them (385 us without the hint then). A thread reads the bytes that its own put writes
  // next, so no barrier stands between.
  static __device__ __forceinline__ void store(const char* tile, __bf16* base, int64_t stride, int64_t first, int count, int tid) {
    store(tile, rows_buffer<D>(base, first, stride, count), stride, tid);
  }
  static __device__ __forceinline__ void store(const char* tile, __amdgpu_buffer_rsrc_t r, int64_t stride, int tid) {
    const unsigned u = (unsigned)local_copy(tid);
    const int at = (int)(u / kUnits) * (int)stride * 2 + (int)(u % kUnits) * 16;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(tile + row_at<D>((int)(u / kUnits)) + i * kRows * kRowBytes<D> + (u % kUnits) * 16);
      __builtin_amdgcn_raw_buffer_store_b128(x, r, at + i * kRows * (int)stride * 2, 0, kStreamLoad);
    }
  }
  __device__ __forceinline__ void put(char* tile, int tid) const {
    const unsigned u = (unsigned)local_copy(tid);
    static_assert(kRows % 16 == 0, "whole groups of rows");
    char* at = tile + row_at<D>((int)(u / kUnits)) + (u % kUnits) * 16;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) *reinterpret_cast<u32x4*>(at + i * kRows * kRowBytes<D>) = w[i];
  }
};

// Where the fragment of P with token tile tt and sources 32 b .. 32 b + 31 stands: the causal ones alone.
// The two that hold one tile of 16 sources take half as much, and their lanes' other half is zero.
__device__ __forceinline__ constexpr bool half_fragment(int tt, int b) { return tt == 2 * b; }
__device__ __forceinline__ constexpr int fragment(int tt, int b) { return 256 * tt * (tt + 1) + 1024 * b; }
constexpr int kTermP = 5120;  // bytes of one term of P; all first terms stand before the second ones
// Tile 0 .. 9 of P: token tile and source tile.
__device__ __forceinline__ int tile_t(int tile) { return (0x0112223333ull >> (4 * tile)) & 15; }
__device__ __forceinline__ int tile_s(int tile) { return (0x0102103210ull >> (4 * tile)) & 15; }

// Fragment of one term of P.
__device__ __forceinline__ bf16x8 read_p(const char* p, int lane, int tt, int b) {
  if (!half_fragment(tt, b)) return *reinterpret_cast<const bf16x8*>(p + fragment(tt, b) + lane * 16);
  const u32x2 x = *reinterpret_cast<const u32x2*>(p + fragment(tt, b) + lane * 8);
  return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], 0u, 0u});  // the tile past the diagonal is not made
}

// Sum over lanes 0 .. l: row shifts inside 16 lanes, then the rows' last lanes broadcast on.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xf, false);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double prefix_sum(double x) {
  x = add_dpp<0x111, 0xf>(x);  // row_shr:1, 2, 4, 8; lanes without a source add 0
  x = add_dpp<0x112, 0xf>(x);
  x = add_dpp<0x114, 0xf>(x);
  x = add_dpp<0x118, 0xf>(x);
  x = add_dpp<0x142, 0xa>(x);  // row_bcast:15 into rows 1 and 3
  x = add_dpp<0x143, 0xc>(x);  // row_bcast:31 into rows 2 and 3
  return x;
}

}  // namespace kda
