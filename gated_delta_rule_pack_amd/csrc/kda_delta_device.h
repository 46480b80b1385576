// Device side that the gated delta rule's prompt kernels share: operands in fp16 terms, scaled rows, a chunk's
// numbers, and the triangular inverse T. kda_delta.hip has the mathematics.
#pragma once

#include <hip/hip_runtime.h>

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
__device__ __forceinline__ uint32_t rest_pair(float a, float b, uint32_t first) {
  const f16x2 h = __builtin_bit_cast(f16x2, first);
  float minus = -1.f;
  asm("" : "+s"(minus));  // a known factor would become a difference, which has no such instruction
  const f16x2 r = {(_Float16)__builtin_fmaf((float)h[0], minus, a), (_Float16)__builtin_fmaf((float)h[1], minus, b)};
  return __builtin_bit_cast(uint32_t, r);
}
// Two tiles (rows 4g + i and 16 + 4g + i) as an operand, in one or two terms.
__device__ __forceinline__ f16x8 to_f16(f32x4 a, f32x4 b) {
  return __builtin_bit_cast(f16x8, u32x4{pair_f16(a[0], a[1]), pair_f16(a[2], a[3]), pair_f16(b[0], b[1]), pair_f16(b[2], b[3])});
}
__device__ __forceinline__ f16x8 rest_f16(f32x4 a, f32x4 b, f16x8 hi) {
  const u32x4 h = __builtin_bit_cast(u32x4, hi);
  return __builtin_bit_cast(f16x8, u32x4{rest_pair(a[0], a[1], h[0]), rest_pair(a[2], a[3], h[1]), rest_pair(b[0], b[1], h[2]),
                                         rest_pair(b[2], b[3], h[3])});
}
// One tile (rows 4g + i) as half a fragment, in one or two terms.
__device__ __forceinline__ void put_half(char* high, char* low, int at, f32x4 x) {
  const u32x2 h = {pair_f16(x[0], x[1]), pair_f16(x[2], x[3])};
  *reinterpret_cast<u32x2*>(high + at) = h;
  if (low) *reinterpret_cast<u32x2*>(low + at) = u32x2{rest_pair(x[0], x[1], h[0]), rest_pair(x[2], x[3], h[1])};
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
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
  x += __uint_as_float(dpp<0xb1>(__float_as_uint(x)));
  x += __uint_as_float(dpp<0x4e>(__float_as_uint(x)));
  x += __uint_as_float(dpp<0x141>(__float_as_uint(x)));
  if constexpr (kLanes == 16) x += __uint_as_float(dpp<0x140>(__float_as_uint(x)));
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

constexpr int kBadRow = 1 << 20;  // exponent of a row that is not finite
// A scaled row's exponent and the sum of its scaled squares.
struct RowInfo {
  int e;
  float squares;
};

// Rows of a tile of q or k in LDS as fp16, each scaled by 2^-e.
template <int D, int kThreads, bool kF16In>
__device__ __forceinline__ void put_scaled(const Rows<D, kThreads>& rows, char* tile, RowInfo* info, int tid, bool squares) {
  typedef Rows<D, kThreads> R;
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  tid = local_copy(tid);
  char* at = tile + row_at<D>(tid / R::kUnits) + (tid % R::kUnits) * 16;
#pragma unroll
  for (int i = 0; i < R::kPasses; ++i) {
    const u32x4 w = rows.w[i];
    u16x2 top = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[j] & 0x7fff7fffu));
    const uint32_t most = row_max<R::kUnits>(max((uint32_t)top[0], (uint32_t)top[1]));
    const bool bad = most >= (kF16In ? 0x7c00u : 0x7f80u);
    const int e = most == 0 || bad ? 0 : __builtin_amdgcn_frexp_expf(token_value<kF16In>(most)) + 1;
    u32x4 out = {0, 0, 0, 0};
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = ldexp2(low_value<kF16In>(w[j]), -e), b = ldexp2(high_value<kF16In>(w[j]), -e);
      s += a * a;
      s += b * b;
      const f16x2 h = {(_Float16)a, (_Float16)b};
      out[j] = bad ? 0u : __builtin_bit_cast(uint32_t, h);
    }
    *reinterpret_cast<u32x4*>(at + i * R::kRows * kRowBytes<D>) = out;
    if (squares) s = row_sum<R::kUnits>(s);
    if (tid % R::kUnits == 0) info[tid / R::kUnits + i * R::kRows] = RowInfo{bad ? kBadRow : e, s};
  }
}

// What the walk needs of a chunk beside its tiles; t, s are tokens.
//   K'_t, Q'_t: scaled rows; rk_t, rq_t: what takes them to the keys and queries of the rule, as it is scaled here:
// keys by 2^-X, step sizes by 2^{2X}, states by 2^X, with X other than 0 only for keys far from unit length; states
// are scaled by 2^Y more, with Y other than 0 only where all step sizes are small.
struct Factors {
  float h[kC];  // rk e^G 2^-Y: the share of K' S in what is to be learnt
  float c[kC];  // rk e^{G_C - G}: what of D reaches the chunk's end
  float e[kC];  // e^G
  float f[kC];  // scale rq 2^-Y: outputs; NaN from the first bad token on
  float total;  // e^{G_C}; NaN with a bad token
  int shift;    // X + Y
};
// For the making of T and P alone.
struct Making {
  double G[kC];               // inclusive cumsum of g
  alignas(16) float bk[kC];   // beta rk
  alignas(16) float rk[kC];
  alignas(16) float col[kC];  // beta 2^Y: the columns of T
};

__device__ __forceinline__ int wave_max(int x) {
  x = max(x, (int)dpp<0xb1>((uint32_t)x));
  x = max(x, (int)dpp<0x4e>((uint32_t)x));
  x = max(x, (int)dpp<0x141>((uint32_t)x));
  x = max(x, (int)dpp<0x140>((uint32_t)x));
  return channel_max(x);
}
// One lane for each token.
__device__ __forceinline__ void put_chunk(Making& mk, Factors& to, const DeltaPlan& p, RowInfo k, RowInfo q, float g, float beta, int lane) {
  const bool bad = k.e == kBadRow || !(g <= 0.f) || !(fabsf(beta) < INFINITY);
  const uint64_t all_bad = __ballot(bad);
  const int first = all_bad ? __builtin_ctzll(all_bad) : kC;
  if (bad) beta = 0.f, g = 0.f, k = RowInfo{0, 0.f};
  // Exponents of the chunk. A row's largest element is 2^-1 of its power of two at most: unit length means -2 to 2.
  int X = 0;
  float rk = 1.f, rq = 1.f;
  if (p.normalize) {
    rk = rsqrtf(k.squares + ldexp2(kNormEps, -2 * k.e));
    rq = rsqrtf(q.squares + ldexp2(kNormEps, -2 * q.e));
  } else {
    const int top = wave_max(k.squares > 0.f ? k.e : -1000);
    X = top < -2 || top > 2 ? (top == -1000 ? 0 : top) : 0;
    rk = ldexp2(1.f, k.e - X);
    rq = ldexp2(1.f, q.e - X);
  }
  beta = ldexp2(beta, 2 * X);
  const int big = wave_max(beta != 0.f ? __builtin_amdgcn_frexp_expf(beta) : -1000);  // |beta| < 2^big
  const int Y = big == -1000 || (big >= -1 && big <= 2) ? 0 : -big;
  const double G = prefix_sum((double)(g < kMinLogDecay ? kMinLogDecay : g));
  const uint64_t u = __builtin_bit_cast(uint64_t, G);
  const double end = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63) << 32 |
                                                    (uint32_t)__builtin_amdgcn_readlane((int)u, 63));
  const float eG = __expf((float)G);
  mk.G[lane] = G;
  mk.bk[lane] = beta * rk;
  mk.rk[lane] = rk;
  mk.col[lane] = ldexp2(beta, Y);
  to.h[lane] = ldexp2(rk * eG, -Y);
  to.c[lane] = rk * __expf((float)(end - G));
  to.e[lane] = eG;
  to.f[lane] = lane >= first || q.e == kBadRow ? __builtin_nanf("") : p.scale * ldexp2(rq, -Y);
  if (lane == 0) {
    to.total = all_bad ? __builtin_nanf("") : __expf((float)end);
    to.shift = X + Y;
  }
}

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

// Making T and P, by four waves of which wave w takes the token tile w: the tiles (w, st <= w) of K' K'^T and K' Q'^T, rows
// s = 4g + i, column t = l % 16. A tile of sources is read once for both.
template <int K>
__device__ __forceinline__ void tile_products(const char* k, const char* q, int lane, int w, f32x4 (&kk)[4], f32x4 (&kq)[4]) {
  constexpr int KB = K / 32;
  f16x8 own_k[KB], own_q[KB];
#pragma unroll
  for (int m = 0; m < KB; ++m) {
    own_k[m] = __builtin_bit_cast(f16x8, read_row<K>(k, lane, 16 * w, m));
    own_q[m] = __builtin_bit_cast(f16x8, read_row<K>(q, lane, 16 * w, m));
  }
#pragma unroll
  for (int st = 0; st < 4; ++st) {
    if (st > w) break;
    kk[st] = kq[st] = zero4();
#pragma unroll
    for (int m = 0; m < KB; ++m) {
      const f16x8 s = __builtin_bit_cast(f16x8, read_row<K>(k, lane, 16 * st, m));
      kk[st] = mfma(s, own_k[m], kk[st]);
      kq[st] = mfma(s, own_q[m], kq[st]);
    }
  }
}
// A's blocks and P's tiles from them; put_p(st, x) takes a tile of P.
template <typename PutP>
__device__ __forceinline__ void put_tiles(float* blocks, const Making& mk, int lane, int w, f32x4 (&kk)[4], f32x4 (&kq)[4], PutP put_p) {
  const int g4 = lane >> 4, t = 16 * w + (lane & 15);
  const double Gt = mk.G[t];
  const float bk = mk.bk[t];
#pragma unroll
  for (int st = 0; st < 4; ++st) {
    if (st > w) break;
    const int s0 = 16 * st + 4 * g4;
    const f32x4 r = *reinterpret_cast<const f32x4*>(&mk.rk[s0]);
    float* to = blocks + block_at(w, st) + 4 * g4 * kBlockRow + (lane & 15);
    f16x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float factor = r[i] * __expf((float)(Gt - mk.G[s0 + i]));
      to[i * kBlockRow] = s0 + i < t ? kk[st][i] * (factor * bk) : 0.f;
      x[i] = (_Float16)(s0 + i <= t ? kq[st][i] * factor : 0.f);
    }
    put_p(st, x);
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
  for (int s = 0; s < 15; ++s) {
#pragma unroll
    for (int c = (s + 1) / 4; c < 4; ++c) {
      const f32x4 col = *reinterpret_cast<const f32x4*>(a + s * kBlockRow + 4 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * c + i > s) x[4 * c + i] -= col[i] * x[s];
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) *reinterpret_cast<f32x4*>(a + j * kBlockRow + 4 * c) = f32x4{x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]};
}
// d + L^T R^T for blocks stored as [s][t]: L's (r, u) at [u][r] is the left operand, row u; R's (t, r) the right one.
__device__ __forceinline__ f32x4 block_product(const float* left, const float* right, int lane, f32x4 d) {
  const int g = lane >> 4, l16 = lane & 15;
  const f32x4 a = *reinterpret_cast<const f32x4*>(left + l16 * kBlockRow + 4 * g);
#pragma unroll
  for (int i = 0; i < 4; ++i) d = mfma32(a[i], right[(4 * g + i) * kBlockRow + l16], d);
  return d;
}
__device__ __forceinline__ f32x4 block_product(const float* left, f32x4 right, int lane, f32x4 d) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(left + (lane & 15) * kBlockRow + 4 * (lane >> 4));
#pragma unroll
  for (int i = 0; i < 4; ++i) d = mfma32(a[i], right[i], d);
  return d;
}
// T's blocks below the diagonal, in two parts with a barrier of the four waves between them (and one before each): those
// beside the diagonal, then the square of four. put_t(tt, st, x) takes a block, rows s = 4g + i, column t = l % 16.
template <typename PutT>
__device__ __forceinline__ void near_blocks(float* blocks, int lane, int w, PutT put_t) {
  const int g4 = lane >> 4, l16 = lane & 15;
  if (w < 2) {
    const int t = 2 * w + 1, s = 2 * w;
    float* at = blocks + block_at(t, s);
    const f32x4 y = -block_product(blocks + block_at(s, s), block_product(at, blocks + block_at(t, t), lane, zero4()), lane, zero4());
    put_t(t, s, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) at[(4 * g4 + i) * kBlockRow + l16] = y[i];
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tt = 2 * (w - 2) + j;
      const float* at = blocks + block_at(tt, tt);
      f32x4 y;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = at[(4 * g4 + i) * kBlockRow + l16];
      put_t(tt, tt, y);
    }
  }
}
template <typename PutT>
__device__ __forceinline__ void far_blocks(const float* blocks, int lane, int w, PutT put_t) {
  if (w >= 2) return;
  const int t = 2 + w;
  const auto block = [&](int tt, int st) { return blocks + block_at(tt, st); };
  f32x4 z0 = block_product(block(2, 0), block(t, 2), lane, zero4()), z1 = block_product(block(2, 1), block(t, 2), lane, zero4());
  if (w == 1) z0 = block_product(block(3, 0), block(3, 3), lane, z0), z1 = block_product(block(3, 1), block(3, 3), lane, z1);
  put_t(t, 0, -block_product(block(1, 0), z1, lane, block_product(block(0, 0), z0, lane, zero4())));
  put_t(t, 1, -block_product(block(1, 1), z1, lane, zero4()));
}
// A block of T with its columns' factors, in two terms.
struct Terms {
  f16x4 hi, lo;
};
__device__ __forceinline__ Terms t_terms(const Making& mk, int lane, int st, f32x4 x) {
  x *= *reinterpret_cast<const f32x4*>(&mk.col[16 * st + 4 * (lane >> 4)]);
  const u32x2 hi = {pair_f16(x[0], x[1]), pair_f16(x[2], x[3])}, lo = {rest_pair(x[0], x[1], hi[0]), rest_pair(x[2], x[3], hi[1])};
  return Terms{__builtin_bit_cast(f16x4, hi), __builtin_bit_cast(f16x4, lo)};
}

// Powers of two that hold one value channel's state and V in fp16's range: S' = S 2^{ex + shift}, V' = V 2^ex. The larger of
// both is kept in [1, 16): fp16's least step, 2^-24, is then nothing beside it, and what 64 tokens learn stays below fp16's largest
// number, 2^16: |v' - S' k| is at most 2^7.6, and no stable rule makes more than 64 times that of it.
struct Scale {
  int ex, shift;
  float v;         // 2^ex
  f32x4 out;       // 2^-ex of the channels 4g + i, for tiles that hold channels as rows
  __device__ __forceinline__ void set(int lane, int to) {
    ex = to;
    v = ldexp2(1.f, to);
    const float back = ldexp2(1.f, -to);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __shfl(back, 4 * (lane >> 4) + i);
  }
};

}  // namespace kda
