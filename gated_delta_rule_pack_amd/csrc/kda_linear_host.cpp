// Host side of linear attention with a decay for each head and of rotary positions:
// argument checks, the segment policy, workspace layout and the launch sequence. No metadata
// is built or uploaded: the kernels find their tokens from the device bounds.

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "kda.h"
#include "kda_linear.h"
#include "kda_rows.h"

namespace kda {


int32_t heads_qk(const kda_linear_args* a) { return a->H_qk > 0 ? a->H_qk : a->H; }

kda_status check_rotation(int32_t rot_dim, int32_t D, const double* inv_freq, const void* positions,
                          int32_t positions_i64, int32_t interleaved, float factor, int32_t T) {
  if (rot_dim < 2 || rot_dim > D || rot_dim % 2 != 0 || !std::isfinite(factor)) return KDA_ERR_INVALID_ARG;
  if ((positions_i64 != 0 && positions_i64 != 1) || (interleaved != 0 && interleaved != 1)) return KDA_ERR_INVALID_ARG;
  if (!inv_freq || !aligned(inv_freq, 8)) return KDA_ERR_INVALID_ARG;
  if (T > 0 && (!positions || !aligned(positions, positions_i64 ? 8 : 4))) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

// Everything the two linear entry points have in common.
kda_status check_linear(const kda_linear_args* a) {
  if (!a) return KDA_ERR_INVALID_ARG;
  if (a->N < 1 || a->T < 0 || a->H < 1 || a->N > (1 << 20) || a->H > (1 << 16)) return KDA_ERR_INVALID_ARG;
  if (a->T > INT32_MAX - (1 << 20)) return KDA_ERR_UNSUPPORTED;
  if ((a->K != 64 && a->K != 128) || (a->V != 64 && a->V != 128)) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(a->scale)) return KDA_ERR_INVALID_ARG;
  if (a->H_qk < 0 || a->H_qk > a->H || (a->H_qk > 0 && a->H % a->H_qk != 0)) return KDA_ERR_INVALID_ARG;
  if (a->state_k_first != 0 && a->state_k_first != 1) return KDA_ERR_INVALID_ARG;
  if (a->g_per_token != 0 && a->g_per_token != 1) return KDA_ERR_INVALID_ARG;
  if (a->g && a->g_dtype != KDA_F32 && a->g_dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
  if (a->g && !aligned(a->g, state_bytes(a->g_dtype))) return KDA_ERR_INVALID_ARG;
  if (a->state_dtype != KDA_F32 && a->state_dtype != KDA_F16 && a->state_dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
  const int32_t H_qk = heads_qk(a);
  const Strides sq = strides_of(a->q_stride_t, a->q_stride_h, H_qk, a->K);
  const Strides sk = strides_of(a->k_stride_t, a->k_stride_h, H_qk, a->K);
  const Strides sv = strides_of(a->v_stride_t, a->v_stride_h, a->H, a->V);
  const Strides so = strides_of(a->out_stride_t, a->out_stride_h, a->H, a->V);
  // The kernels hold a chunk's 64 rows in 32-bit byte offsets, and rows do not overlap.
  const int64_t least[4] = {a->K, a->K, a->V, a->V};
  int i = 0;
  for (const Strides& s : {sq, sk, sv, so}) {
    if (!stride_ok(s) || s.t % 8 != 0 || s.h % 8 != 0 || s.t > kMaxTokenStride) return KDA_ERR_INVALID_ARG;
    if (a->T > 1 && s.t < least[i]) return KDA_ERR_INVALID_ARG;
    ++i;
  }
  if (!distinct_rows(so, a->T, a->H, a->V)) return KDA_ERR_ALIAS;
  if (a->T > 0) {
    if (!a->q || !a->k || !a->v || !a->out) return KDA_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->out, 16)) return KDA_ERR_INVALID_ARG;
    const Range out = range_of(a->out, a->T, a->H, a->V, so.t, so.h, 2);
    if (overlap(out, range_of(a->q, a->T, H_qk, a->K, sq.t, sq.h, 2)) ||
        overlap(out, range_of(a->k, a->T, H_qk, a->K, sk.t, sk.h, 2)) ||
        overlap(out, range_of(a->v, a->T, a->H, a->V, sv.t, sv.h, 2)))
      return KDA_ERR_ALIAS;
  }
  const bool dense = a->initial_state || a->final_state;
  if (dense && a->state_cache) return KDA_ERR_STATE_MODE;
  const int64_t plane = (int64_t)a->H * a->K * a->V;
  if (a->state_cache) {
    if (a->num_slots < 1) return KDA_ERR_INVALID_ARG;
    if (a->state_cache_stride0 < plane) return KDA_ERR_STRIDE;
    if (!aligned(a->state_cache, 16) || (size_t)a->state_cache_stride0 * state_bytes(a->state_dtype) % 16 != 0)
      return KDA_ERR_INVALID_ARG;
  }
  if (dense) {
    if ((a->initial_state && !aligned(a->initial_state, 16)) || (a->final_state && !aligned(a->final_state, 16)))
      return KDA_ERR_INVALID_ARG;
    const size_t es = state_bytes(a->state_dtype);
    if (a->initial_state && a->final_state && a->initial_state != a->final_state &&
        overlap(range_of(a->initial_state, a->N, 1, plane, plane, 0, es), range_of(a->final_state, a->N, 1, plane, plane, 0, es)))
      return KDA_ERR_ALIAS;
  }
  if (a->inv_freq)
    return check_rotation(a->rot_dim, a->K, a->inv_freq, a->positions, a->positions_i64, a->interleaved, a->rot_factor, a->T);
  return KDA_OK;
}

// Fields both kernels' plans take from the arguments as they are.
LinearPlan plan_of(const kda_linear_args* a) {
  LinearPlan p{};
  p.T = a->T;
  p.N = a->N;
  p.H = a->H;
  p.group = a->H / heads_qk(a);
  p.K = a->K;
  p.V = a->V;
  p.scale = a->scale;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.out = a->out;
  const Strides sq = strides_of(a->q_stride_t, a->q_stride_h, heads_qk(a), a->K);
  const Strides sk = strides_of(a->k_stride_t, a->k_stride_h, heads_qk(a), a->K);
  const Strides sv = strides_of(a->v_stride_t, a->v_stride_h, a->H, a->V);
  const Strides so = strides_of(a->out_stride_t, a->out_stride_h, a->H, a->V);
  p.q_t = sq.t, p.q_h = sq.h, p.k_t = sk.t, p.k_h = sk.h, p.v_t = sv.t, p.v_h = sv.h, p.o_t = so.t, p.o_h = so.h;
  p.g = a->g;
  p.g_bf16 = a->g_dtype == KDA_BF16;
  p.g_per_token = a->g_per_token;
  p.cu = a->cu_seqlens;
  p.state_dtype = a->state_dtype == KDA_F32 ? kda::kF32 : (a->state_dtype == KDA_F16 ? kda::kF16 : kda::kBF16);
  p.kfirst = a->state_k_first;
  if (a->state_cache) {
    p.state_in = a->state_cache;
    p.state_out = a->state_cache;
    p.in_mode = p.out_mode = kda::kStatePaged;
    p.stride0 = a->state_cache_stride0;
    p.num_slots = a->num_slots;
  } else {
    p.state_in = a->initial_state;
    p.in_mode = a->initial_state ? kda::kStateDense : kda::kStateNone;
    p.state_out = a->final_state;
    p.out_mode = a->final_state ? kda::kStateDense : kda::kStateNone;
    p.stride0 = (int64_t)a->H * a->K * a->V;
    p.num_slots = a->N;
  }
  p.indices = a->state_indices;
  p.flags = a->has_initial_state;
  p.rot.inv_freq = a->inv_freq;
  p.rot.positions = a->positions;
  p.rot.positions_i64 = a->positions_i64;
  p.rot.rot_dim = a->rot_dim;
  p.rot.interleaved = a->interleaved;
  p.rot.factor = a->rot_factor;
  return p;
}

int launch(kda_ctx* ctx, int kernel, const void* plan, void* stream) {
  const kda_runtime& rt = kda::context_runtime(ctx);
  return rt.launch(rt.user, kernel, plan, stream, nullptr, nullptr);
}

}  // namespace kda

namespace {

using namespace kda;

// A sequence's state, read and written once, in tokens' worth of q, k, v and out bytes.
int32_t head_cost_of(const kda_linear_args* a) {
  const bool state = a->initial_state || a->final_state || a->state_cache;
  if (!state) return 2;
  return (int32_t)((size_t)a->K * a->V * state_bytes(a->state_dtype) * 2 / ((size_t)(a->K + a->V) * 2 * 2));
}

int64_t axis_of(const kda_linear_args* a) {
  return std::max<int64_t>(a->T, 1) + (int64_t)head_cost_of(a) * (a->N - 1);
}

// Segment length. A long segment costs its own walk (5 us for each 64 tokens of K = V = 128, map and
// output, one workgroup on a compute unit); every segment costs a step of the combine's chain (0.06 us)
// and, for each head, a state that is written, chained and read back (0.059 us at K = V = 128). The sum
// is least at a length that grows with the root of the tokens: measured best at H = 12 for 1024 tokens
// 128 (24.6 us; 64: 28.4, 192: 27.8), 4096 tokens 192 (40.9 us; 128: 48.8, 384: 50.5), 8192 tokens 384; at H = 32
// for 1536 tokens 192, 6144 tokens 384; at H = 1 for 168 K tokens (V = 64) 384 to 768 (94 us; 256: 110). Work for
// more workgroups than the chip holds at once (two of 128 state rows on a compute unit, three of 64) takes
// as many: 32768 tokens at H = 32, 2048 (415 us; 1024: 436). Little work takes one segment and one
// kernel: 128 tokens 12.6 us, 15.0 in two segments; 192 tokens 16.5 and 18.9, 256 tokens 20.4 and 20.1;
// two sequences of 10 tokens 15.1 and 14.1, three 20.9 and 14.3. (Replays of a captured call.)
int32_t seg_len_of(const kda_linear_args* a) {
  if (a->seg_len > 0) return a->seg_len;
  constexpr int64_t C = kda::kLinChunk;
  const int64_t axis = axis_of(a), units = a->V == 64 ? 768 : 512;
  const int64_t fit = std::max<int64_t>(1, units / a->H), fill = (axis + fit - 1) / fit;
  const double per_segment = 0.06 + 0.059 * a->H * a->K * a->V / (128 * 128), per_token = 5.0 / C;
  const int64_t root = (int64_t)(std::sqrt(per_segment * (double)axis / per_token) / C + 0.5) * C;
  const auto whole = [](int64_t n) { return (std::max<int64_t>(n, 1) + C - 1) / C * C; };
  const auto count = [axis](int64_t l) { return (axis + l - 1) / l; };
  int64_t len = whole(a->T + 128 * ((int64_t)a->N - 1) <= 224 ? axis : std::max(fill, root));
  // Workgroups for more than one on each of 256 compute units, and for two at most: the units with two decide the
  // time. As many whole segments as leave one to a unit are taken instead where that is an eighth less by these
  // costs (3 us for each 64 tokens of a single segment, which has no map). 65536 tokens at H = 2: 342 workgroups 97
  // us, 256: 85; 16384 at H = 192: 384 in two segments 1183 us, 192 in one 1015; at H = 256: 1397 and 1196. Where the
  // two ways cost as much, two to a unit run faster, one working while the other waits: 16384 at H = 48: 480
  // workgroups 349 us, 240: 371; at H = 160: 480 in three segments 966 us, 160 in one 1004.
  const int64_t n = count(len), most = std::max<int64_t>(1, 256 / a->H), alone = whole((axis + most - 1) / most);
  if (n * a->H > 264 && n * a->H <= 512 && count(alone) < n) {
    const double two = 2 * (double)len * per_token + (double)n * per_segment;
    const double one = (double)alone * (count(alone) == 1 ? 0.6 : 1.0) * per_token + (double)count(alone) * per_segment;
    if (one < 0.875 * two) len = alone;
  }
  return (int32_t)std::min<int64_t>(len, 1 << 30);
}
int32_t segments_of(const kda_linear_args* a) {
  const int64_t L = seg_len_of(a);
  return (int32_t)((axis_of(a) + L - 1) / L);
}

struct LinearWs {
  size_t maps = 0, initials = 0, decays = 0, spans = 0, rot_q = 0, rot_k = 0, total = 0;
};
LinearWs workspace_of(const kda_linear_args* a) {
  LinearWs w;
  const size_t borders = (size_t)segments_of(a) - 1;
  const size_t plane = (size_t)a->H * a->K * a->V * sizeof(float);
  auto take = [&](size_t bytes) {
    const size_t at = w.total;
    w.total += (bytes + 255) / 256 * 256;
    return at;
  };
  w.maps = take(borders * plane);
  w.initials = take(a->initial_state || a->state_cache ? borders * plane : 0);
  w.decays = take(borders * a->H * sizeof(float));
  w.spans = take(borders * sizeof(int32_t));
  if (a->inv_freq) {
    const size_t rows = (size_t)a->T * heads_qk(a) * a->K * 2;
    w.rot_q = take(rows);
    w.rot_k = take(rows);
  }
  return w;
}

}  // namespace

extern "C" {

kda_status kda_linear_fwd_validate(const kda_linear_args* a) {
  if (kda_status st = check_linear(a)) return st;
  if (!a->cu_seqlens || !aligned(a->cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
  if (a->seg_len < 0 || a->seg_len % kda::kLinChunk != 0 || a->seg_len > (1 << 30)) return KDA_ERR_INVALID_ARG;
  if (a->state_cache && (!a->state_indices || !a->has_initial_state)) return KDA_ERR_INVALID_ARG;
  if (axis_of(a) > INT32_MAX - (1 << 20)) return KDA_ERR_UNSUPPORTED;
  if ((int64_t)segments_of(a) * a->H > kMaxGroups / 2) return KDA_ERR_UNSUPPORTED;  // of 512 threads
  if (const int32_t* cu = a->cu_seqlens_host) {
    if (cu[0] != 0 || cu[a->N] > a->T) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < a->N; ++i)
      if (cu[i + 1] < cu[i]) return KDA_ERR_INVALID_ARG;
  }
  return KDA_OK;
}

size_t kda_linear_fwd_workspace_bytes(const kda_linear_args* a) {
  return kda_linear_fwd_validate(a) == KDA_OK ? workspace_of(a).total : 0;
}

int32_t kda_linear_seg_len(const kda_linear_args* a) {
  return kda_linear_fwd_validate(a) == KDA_OK ? seg_len_of(a) : 0;
}

kda_status kda_linear_fwd(kda_ctx* ctx, const kda_linear_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (!ctx) return KDA_ERR_INVALID_ARG;
  if (kda_status st = kda_linear_fwd_validate(a)) return st;
  const LinearWs w = workspace_of(a);
  if (w.total > 0 && (!ws || ws_bytes < w.total || !aligned(ws, 256))) return KDA_ERR_WORKSPACE;
  LinearPlan p = plan_of(a);
  char* base = reinterpret_cast<char*>(ws);
  p.seg_len = seg_len_of(a);
  p.head_cost = head_cost_of(a);
  p.n_seg = segments_of(a);
  // Slices of 64 state rows where they still get a compute unit each: 37 tokens at H = 12 take 8.7
  // instead of 9.8 us; 4096 tokens (264 units) would take 46.8 instead of 43.0.
  p.slices = a->V == 128 && (int64_t)p.n_seg * a->H <= 128 ? 2 : 1;
  p.maps = reinterpret_cast<float*>(base + w.maps);
  p.initials = reinterpret_cast<float*>(base + w.initials);
  p.decays = reinterpret_cast<float*>(base + w.decays);
  p.spans = reinterpret_cast<int32_t*>(base + w.spans);
  if (a->inv_freq && a->T > 0) {
    const int32_t H_qk = heads_qk(a);
    RotaryPlan r = p.rot;
    r.T = a->T;
    r.D = a->K;
    r.dtype = kda::kBF16;
    r.H[0] = r.H[1] = H_qk;
    r.in[0] = p.q, r.in_t[0] = p.q_t, r.in_h[0] = p.q_h;
    r.in[1] = p.k, r.in_t[1] = p.k_t, r.in_h[1] = p.k_h;
    for (int i = 0; i < 2; ++i) {
      r.out[i] = base + (i ? w.rot_k : w.rot_q);
      r.out_t[i] = (int64_t)H_qk * a->K;
      r.out_h[i] = a->K;
    }
    if (launch(ctx, 9, &r, stream)) return KDA_ERR_HIP;
    p.q = r.out[0], p.k = r.out[1];
    p.q_t = p.k_t = (int64_t)H_qk * a->K;
    p.q_h = p.k_h = a->K;
  }
  if (p.n_seg > 1) {
    if (launch(ctx, 5, &p, stream) || launch(ctx, 6, &p, stream)) return KDA_ERR_HIP;
  }
  return launch(ctx, 7, &p, stream) ? KDA_ERR_HIP : KDA_OK;
}

kda_status kda_linear_step_validate(const kda_linear_args* a) {
  if (kda_status st = check_linear(a)) return st;
  if (a->T != a->N || !a->state_cache) return KDA_ERR_INVALID_ARG;
  if (!a->state_indices && a->num_slots < a->N) return KDA_ERR_INVALID_ARG;
  if ((int64_t)a->N * a->H > kMaxGroups) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status kda_linear_step(kda_ctx* ctx, const kda_linear_args* a, void* stream) {
  if (!ctx) return KDA_ERR_INVALID_ARG;
  if (kda_status st = kda_linear_step_validate(a)) return st;
  LinearPlan p = plan_of(a);
  return launch(ctx, 8, &p, stream) ? KDA_ERR_HIP : KDA_OK;
}

kda_status kda_rotary_validate(const kda_rotary_args* a) {
  if (!a) return KDA_ERR_INVALID_ARG;
  if (a->T < 0 || a->H_q < 1 || a->H_k < 0 || a->D < 1) return KDA_ERR_INVALID_ARG;
  if (a->D > 1024 || a->H_q > (1 << 16) || a->H_k > (1 << 16)) return KDA_ERR_UNSUPPORTED;
  if (a->dtype != KDA_F32 && a->dtype != KDA_F16 && a->dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
  if (a->inverse != 0 && a->inverse != 1) return KDA_ERR_INVALID_ARG;
  if (kda_status st = check_rotation(a->rot_dim, a->D, a->inv_freq, a->positions, a->positions_i64, a->interleaved, a->factor, a->T))
    return st;
  const size_t es = state_bytes(a->dtype);
  const void* in[2] = {a->q, a->k};
  void* out[2] = {a->out_q, a->out_k};
  const int64_t H[2] = {a->H_q, a->H_k};
  const Strides si[2] = {strides_of(a->q_stride_t, a->q_stride_h, a->H_q, a->D), strides_of(a->k_stride_t, a->k_stride_h, a->H_k, a->D)};
  const Strides so[2] = {strides_of(a->out_q_stride_t, a->out_q_stride_h, a->H_q, a->D),
                         strides_of(a->out_k_stride_t, a->out_k_stride_h, a->H_k, a->D)};
  Rows r[4];  // q, k, and their results
  int n = 0;
  for (int i = 0; i < 2; ++i) {
    if (H[i] == 0 || a->T == 0) continue;
    if (!in[i] || !out[i] || !aligned(in[i], es) || !aligned(out[i], es)) return KDA_ERR_INVALID_ARG;
    if (!stride_ok(si[i]) || !stride_ok(so[i])) return KDA_ERR_INVALID_ARG;
    if (!distinct_rows(so[i], a->T, H[i], a->D)) return KDA_ERR_ALIAS;
    r[n++] = Rows{in[i], a->T, H[i], a->D, si[i], es};
    r[n++] = Rows{out[i], a->T, H[i], a->D, so[i], es};
  }
  // A result may take its input's place, and share no element with anything else.
  for (int o = 1; o < n; o += 2)
    for (int x = 0; x < n; ++x)
      if (x != o && !(x == o - 1 && same_rows(r[x], r[o])) && !disjoint(r[o], r[x])) return KDA_ERR_ALIAS;
  return KDA_OK;
}

kda_status kda_rotary(kda_ctx* ctx, const kda_rotary_args* a, void* stream) {
  if (!ctx) return KDA_ERR_INVALID_ARG;
  if (kda_status st = kda_rotary_validate(a)) return st;
  if (a->T == 0) return KDA_OK;
  RotaryPlan r{};
  r.T = a->T;
  r.D = a->D;
  r.rot_dim = a->rot_dim;
  r.dtype = a->dtype == KDA_F32 ? kda::kF32 : (a->dtype == KDA_F16 ? kda::kF16 : kda::kBF16);
  r.H[0] = a->H_q;
  r.H[1] = a->H_k;
  const Strides si[2] = {strides_of(a->q_stride_t, a->q_stride_h, a->H_q, a->D), strides_of(a->k_stride_t, a->k_stride_h, a->H_k, a->D)};
  const Strides so[2] = {strides_of(a->out_q_stride_t, a->out_q_stride_h, a->H_q, a->D),
                         strides_of(a->out_k_stride_t, a->out_k_stride_h, a->H_k, a->D)};
  const void* in[2] = {a->q, a->k};
  void* out[2] = {a->out_q, a->out_k};
  for (int i = 0; i < 2; ++i) {
    r.in[i] = in[i], r.out[i] = out[i];
    r.in_t[i] = si[i].t, r.in_h[i] = si[i].h;
    r.out_t[i] = so[i].t, r.out_h[i] = so[i].h;
  }
  r.positions = a->positions;
  r.positions_i64 = a->positions_i64;
  r.inv_freq = a->inv_freq;
  r.factor = a->factor;
  r.interleaved = a->interleaved;
  r.inverse = a->inverse;
  return launch(ctx, 9, &r, stream) ? KDA_ERR_HIP : KDA_OK;
}

size_t kda_linear_args_size(void) { return sizeof(kda_linear_args); }
size_t kda_rotary_args_size(void) { return sizeof(kda_rotary_args); }

}  // extern "C"
