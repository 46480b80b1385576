// Host side of the gated delta rule with one decay for each head and of the norms of q and k: argument checks,
// workspaces and the launch sequence.

#include <algorithm>
#include <cmath>

#include "kda.h"
#include "kda_delta.h"
#include "kda_rows.h"

namespace {

using namespace kda;

int dtype_of(kda_dtype d) { return d == KDA_F32 ? kF32 : (d == KDA_F16 ? kF16 : kBF16); }

kda_status check_delta(const kda_gated_delta_args* a) {
  if (!a) return KDA_ERR_INVALID_ARG;
  if (kda_status st = check_linear(&a->lin)) return st;
  if (a->lin.inv_freq || a->lin.seg_len != 0) return KDA_ERR_INVALID_ARG;
  if (a->dtype != KDA_BF16 && a->dtype != KDA_F16) return KDA_ERR_UNSUPPORTED;
  if (a->beta_dtype != KDA_F32 && a->beta_dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
  if (a->normalize != 0 && a->normalize != 1) return KDA_ERR_INVALID_ARG;
  if (a->path < KDA_DELTA_POLICY || a->path > KDA_DELTA_SCAN) return KDA_ERR_INVALID_ARG;
  if (a->lin.T > 0 && (!a->beta || !aligned(a->beta, state_bytes(a->beta_dtype)))) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

DeltaPlan delta_plan_of(const kda_gated_delta_args* a) {
  DeltaPlan p{};
  static_cast<LinearPlan&>(p) = plan_of(&a->lin);
  p.beta = a->beta;
  p.beta_bf16 = a->beta_dtype == KDA_BF16;
  p.f16 = a->dtype == KDA_F16;
  p.normalize = a->normalize;
  return p;
}

int32_t places_of(const kda_gated_delta_args* a) { return a->lin.T / kLinChunk + a->lin.N; }
// One launch counts its work-items in 32 bits.
bool fits_scan(const kda_gated_delta_args* a) {
  const kda_linear_args& l = a->lin;
  return (int64_t)places_of(a) * l.H <= kMaxGroups && ((int64_t)l.N * l.H + 7) * (l.V / 16) <= kMaxGroups / 2;
}
// Whether a call makes its chunks' records in one kernel and scans them with workgroups of 16 value channels, or
// walks every sequence of a head in one workgroup. Times in turns of the scan (1.4 us); a chunk of the walk takes four.
// Both wait for the longest sequence, or for all of them where there are more workgroups than 256: the walk has one for
// each sequence and head, whose start takes about a chunk; the scan V / 16, whose start takes about two turns,
// and its records are made 75 to a turn. Tokens that are their sequence's only one are a step in both. Without bounds on
// the host all sequences count as equally long.
//
// Measured at K = V = 128 with 32-bit states, in a graph, walk and scan: prompts of 1024 tokens at 12, 48, 64, 96, 128, 192 sequences
// and heads 92 and 43, 93 and 80, 93 and 89, 94 and 121, 97 and 155, 125 and 228 us; one prompt of 64, 128, 192 at H = 12 17.3
// and 18.3, 22.3 and 20.4, 27.5 and 22.4; one of 4096 among 31 single tokens 437 and 122, one of 512 among 127 at
// H = 24 102 and 451; eight from 64 to 8192 644 and 231. K = V = 64, 1024 tokens at 96, 128, 144: 82 and 79, 83 and 89, 83 and 112.
bool scans(const kda_gated_delta_args* a) {
  const kda_linear_args& l = a->lin;
  if (a->path != KDA_DELTA_POLICY) return a->path == KDA_DELTA_SCAN;
  if (!fits_scan(a)) return false;
  const auto chunks_of = [](int64_t len) { return len > 1 ? (len + kLinChunk - 1) / kLinChunk : 0; };
  int64_t longest = 0, chunks = 0;
  if (const int32_t* cu = l.cu_seqlens_host) {
    for (int i = 0; i < l.N; ++i) {
      const int64_t c = chunks_of(cu[i + 1] - cu[i]);
      longest = std::max(longest, c), chunks += c;
    }
  } else if (l.N > 0) {
    longest = chunks_of((l.T + l.N - 1) / l.N), chunks = longest * l.N;
  }
  const double heads = l.H, walk = 4 * std::max(longest + 1., (double)(chunks + l.N) * heads / 256);
  const double scan = std::max(longest + 2., (double)(chunks + 2 * (int64_t)l.N) * heads * l.V / 4096) + chunks * heads / 75 + 8;
  return scan < walk;
}

struct DeltaWs {
  size_t records = 0, keys = 0, queries = 0, total = 0;
};
DeltaWs workspace_of(const kda_gated_delta_args* a) {
  DeltaWs w;
  if (!scans(a)) return w;
  const size_t places = (size_t)places_of(a), rows = places * heads_qk(&a->lin) * kLinChunk * a->lin.K * 2;
  const auto take = [&](size_t bytes) {
    const size_t at = w.total;
    w.total += (bytes + 255) / 256 * 256;
    return at;
  };
  w.records = take(places * a->lin.H * kDeltaRecord);
  w.keys = take(rows);
  w.queries = take(rows);
  return w;
}

// The rows of one tensor of a norm's call: x, its result, or a gradient.
struct NormRows {
  const void* at;
  Strides s;
};

kda_status check_norm(const kda_qk_norm_args* a, bool back) {
  if (!a) return KDA_ERR_INVALID_ARG;
  if (a->T < 0 || a->H_q < 1 || a->H_k < 0 || a->D < 1) return KDA_ERR_INVALID_ARG;
  if (a->D > 1024 || a->H_q > (1 << 16) || a->H_k > (1 << 16)) return KDA_ERR_UNSUPPORTED;
  // Rows of one workgroup's tokens are counted in 32 bits, and so are the tokens and a last step behind them.
  if (a->T > INT32_MAX - (1 << 20)) return KDA_ERR_UNSUPPORTED;
  if (a->dtype != KDA_F32 && a->dtype != KDA_F16 && a->dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
  if (a->kind != KDA_NORM_RMS && a->kind != KDA_NORM_L2) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(a->eps) || !(a->eps > 0.f) || !std::isfinite(a->weight_offset)) return KDA_ERR_INVALID_ARG;
  if (a->rot_dim != 0 || a->inv_freq) {
    if (kda_status st = check_rotation(a->rot_dim, a->D, a->inv_freq, a->positions, a->positions_i64, a->interleaved, 1.f, a->T))
      return st;
  } else if (a->interleaved != 0 && a->interleaved != 1) {
    return KDA_ERR_INVALID_ARG;
  }
  if (a->q_weight || a->k_weight) {
    if (a->weight_dtype != KDA_F32 && a->weight_dtype != a->dtype) return KDA_ERR_UNSUPPORTED;
    const size_t ws = state_bytes(a->weight_dtype);
    if (!aligned(a->q_weight, ws) || !aligned(a->k_weight, ws)) return KDA_ERR_INVALID_ARG;
    if (back && (!aligned(a->grad_q_weight, ws) || !aligned(a->grad_k_weight, ws))) return KDA_ERR_INVALID_ARG;
  }
  if (a->k_weight && a->H_k == 0) return KDA_ERR_INVALID_ARG;
  if (back ? (!a->q_weight != !a->grad_q_weight || !a->k_weight != !a->grad_k_weight) : (a->grad_q_weight || a->grad_k_weight))
    return KDA_ERR_INVALID_ARG;
  const size_t es = state_bytes(a->dtype);
  const int64_t H[2] = {a->H_q, a->H_k}, D = a->D;
  const NormRows in[2] = {{a->q, strides_of(a->q_stride_t, a->q_stride_h, H[0], D)}, {a->k, strides_of(a->k_stride_t, a->k_stride_h, H[1], D)}};
  const NormRows out[2] = {{a->out_q, strides_of(a->out_q_stride_t, a->out_q_stride_h, H[0], D)},
                           {a->out_k, strides_of(a->out_k_stride_t, a->out_k_stride_h, H[1], D)}};
  const NormRows grad[2] = {{a->grad_q, strides_of(a->grad_q_stride_t, a->grad_q_stride_h, H[0], D)},
                            {a->grad_k, strides_of(a->grad_k_stride_t, a->grad_k_stride_h, H[1], D)}};
  Rows r[6], o[2];
  int own[2], n = 0, m = 0;  // own: the input whose place the result may take
  for (int c = 0; c < 2; ++c) {
    if (H[c] == 0 || a->T == 0) continue;
    for (const NormRows* x : {&in[c], &out[c], back ? &grad[c] : nullptr}) {
      if (!x) continue;
      if (!x->at || !aligned(x->at, es) || !stride_ok(x->s)) return KDA_ERR_INVALID_ARG;
    }
    if (!distinct_rows(out[c].s, a->T, H[c], D)) return KDA_ERR_ALIAS;
    own[m] = back ? n + 1 : n;
    r[n++] = Rows{in[c].at, a->T, H[c], D, in[c].s, es};
    if (back) r[n++] = Rows{grad[c].at, a->T, H[c], D, grad[c].s, es};
    o[m++] = Rows{out[c].at, a->T, H[c], D, out[c].s, es};
  }
  if (m == 2 && !disjoint(o[0], o[1])) return KDA_ERR_ALIAS;
  for (int i = 0; i < m; ++i)
    for (int x = 0; x < n; ++x)
      if (!(x == own[i] && same_rows(r[x], o[i])) && !disjoint(o[i], r[x])) return KDA_ERR_ALIAS;
  // Weights and their gradients share no byte with a result or each other.
  const size_t wb = (size_t)D * state_bytes(a->weight_dtype);
  const auto bytes = [&](const void* at) { return at ? Range{(uintptr_t)at, (uintptr_t)at + wb} : Range{}; };
  const Range small[4] = {bytes(a->grad_q_weight), bytes(a->grad_k_weight), bytes(a->q_weight), bytes(a->k_weight)};
  for (int i = 0; i < 4; ++i) {
    if (small[i].lo == small[i].hi) continue;
    for (int x = 0; x < m; ++x)
      if (overlap(small[i], range_of(o[x].at, o[x].T, o[x].H, D, o[x].s.t, o[x].s.h, es))) return KDA_ERR_ALIAS;
    if (i >= 2) continue;
    for (int x = 0; x < n; ++x)
      if (overlap(small[i], range_of(r[x].at, r[x].T, r[x].H, D, r[x].s.t, r[x].s.h, es))) return KDA_ERR_ALIAS;
    for (int x = 0; x < 4; ++x)
      if (x != i && small[x].lo != small[x].hi && overlap(small[i], small[x])) return KDA_ERR_ALIAS;
  }
  return KDA_OK;
}

NormPlan norm_plan_of(const kda_qk_norm_args* a) {
  NormPlan p{};
  p.T = a->T;
  p.D = a->D;
  p.rot_dim = a->rot_dim;
  p.dtype = dtype_of(a->dtype);
  p.H[0] = a->H_q;
  p.H[1] = a->H_k;
  const auto put = [&](const void* at, int64_t t, int64_t h, int c, const void** to, int64_t* to_t, int64_t* to_h) {
    const Strides s = strides_of(t, h, p.H[c], p.D);
    to[c] = at, to_t[c] = s.t, to_h[c] = s.h;
  };
  put(a->q, a->q_stride_t, a->q_stride_h, 0, p.in, p.in_t, p.in_h);
  put(a->k, a->k_stride_t, a->k_stride_h, 1, p.in, p.in_t, p.in_h);
  put(a->grad_q, a->grad_q_stride_t, a->grad_q_stride_h, 0, p.grad, p.grad_t, p.grad_h);
  put(a->grad_k, a->grad_k_stride_t, a->grad_k_stride_h, 1, p.grad, p.grad_t, p.grad_h);
  const void* out[2];
  put(a->out_q, a->out_q_stride_t, a->out_q_stride_h, 0, out, p.out_t, p.out_h);
  put(a->out_k, a->out_k_stride_t, a->out_k_stride_h, 1, out, p.out_t, p.out_h);
  p.out[0] = a->out_q, p.out[1] = a->out_k;
  p.positions = a->positions;
  p.positions_i64 = a->positions_i64;
  p.inv_freq = a->inv_freq;
  p.factor = 1.f;
  p.interleaved = a->interleaved;
  p.weight[0] = a->q_weight, p.weight[1] = a->k_weight;
  p.grad_weight[0] = a->grad_q_weight, p.grad_weight[1] = a->grad_k_weight;
  p.weight_f32 = a->weight_dtype == KDA_F32;
  p.l2 = a->kind == KDA_NORM_L2;
  p.eps = a->eps;
  p.offset = a->weight_offset;
  p.groups = norm_groups(a->T);
  return p;
}

size_t sums_bytes(const kda_qk_norm_args* a) {
  return a->q_weight || a->k_weight ? (size_t)norm_groups(a->T) * 2 * a->D * sizeof(float) : 0;
}

}  // namespace

extern "C" {

kda_status kda_gated_delta_fwd_validate(const kda_gated_delta_args* a) {
  if (kda_status st = check_delta(a)) return st;
  const kda_linear_args& l = a->lin;
  if (!l.cu_seqlens || !aligned(l.cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
  if (l.state_cache && (!l.state_indices || !l.has_initial_state)) return KDA_ERR_INVALID_ARG;
  if (const int32_t* cu = l.cu_seqlens_host) {
    if (cu[0] != 0 || cu[l.N] > l.T) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < l.N; ++i)
      if (cu[i + 1] < cu[i]) return KDA_ERR_INVALID_ARG;
  }
  // A launch counts its work-items in 32 bits: two slices of up to 512 threads.
  if (scans(a) ? !fits_scan(a) : (int64_t)l.N * l.H > kMaxGroups / 4) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

size_t kda_gated_delta_fwd_workspace_bytes(const kda_gated_delta_args* a) {
  return kda_gated_delta_fwd_validate(a) == KDA_OK ? workspace_of(a).total : 0;
}

kda_status kda_gated_delta_fwd(kda_ctx* ctx, const kda_gated_delta_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (!ctx) return KDA_ERR_INVALID_ARG;
  if (kda_status st = kda_gated_delta_fwd_validate(a)) return st;
  const DeltaWs w = workspace_of(a);
  if (w.total > 0 && (!ws || ws_bytes < w.total || !aligned(ws, 256))) return KDA_ERR_WORKSPACE;
  DeltaPlan p = delta_plan_of(a);
  const int64_t units = (int64_t)p.N * p.H;
  // Ranking is for calls of more workgroups than run at once, and of as many sequences as a workgroup can rank.
  const auto rank = [&](int64_t groups) { p.ranked = p.N > 1 && p.N <= kMostRanked && groups > 256; };
  if (!scans(a)) {
    p.slices = p.V == 128 && units <= 128 ? 2 : 1;
    rank(units * p.slices);
    return launch(ctx, 10, &p, stream) ? KDA_ERR_HIP : KDA_OK;
  }
  char* base = reinterpret_cast<char*>(ws);
  p.places = places_of(a);
  rank(units * (p.V / 16));
  p.records = base + w.records;
  p.keys = base + w.keys;
  p.queries = base + w.queries;
  return launch(ctx, 14, &p, stream) || launch(ctx, 15, &p, stream) ? KDA_ERR_HIP : KDA_OK;
}

kda_status kda_gated_delta_step_validate(const kda_gated_delta_args* a) {
  if (kda_status st = check_delta(a)) return st;
  const kda_linear_args& l = a->lin;
  if (l.T != l.N || !l.state_cache) return KDA_ERR_INVALID_ARG;
  if (!l.state_indices && l.num_slots < l.N) return KDA_ERR_INVALID_ARG;
  if ((int64_t)l.N * l.H > kMaxGroups) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status kda_gated_delta_step(kda_ctx* ctx, const kda_gated_delta_args* a, void* stream) {
  if (!ctx) return KDA_ERR_INVALID_ARG;
  if (kda_status st = kda_gated_delta_step_validate(a)) return st;
  const DeltaPlan p = delta_plan_of(a);
  return launch(ctx, 11, &p, stream) ? KDA_ERR_HIP : KDA_OK;
}

kda_status kda_qk_norm_validate(const kda_qk_norm_args* a) { return check_norm(a, false); }

kda_status kda_qk_norm(kda_ctx* ctx, const kda_qk_norm_args* a, void* stream) {
  if (!ctx) return KDA_ERR_INVALID_ARG;
  if (kda_status st = check_norm(a, false)) return st;
  if (a->T == 0) return KDA_OK;
  const NormPlan p = norm_plan_of(a);
  return launch(ctx, 12, &p, stream) ? KDA_ERR_HIP : KDA_OK;
}

kda_status kda_qk_norm_backward_validate(const kda_qk_norm_args* a) { return check_norm(a, true); }

size_t kda_qk_norm_backward_workspace_bytes(const kda_qk_norm_args* a) {
  return check_norm(a, true) == KDA_OK ? sums_bytes(a) : 0;
}

kda_status kda_qk_norm_backward(kda_ctx* ctx, const kda_qk_norm_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (!ctx) return KDA_ERR_INVALID_ARG;
  if (kda_status st = check_norm(a, true)) return st;
  const size_t need = sums_bytes(a);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 256))) return KDA_ERR_WORKSPACE;
  if (a->T == 0 && !a->q_weight && !a->k_weight) return KDA_OK;
  NormPlan p = norm_plan_of(a);
  p.sums = need > 0 ? reinterpret_cast<float*>(ws) : nullptr;
  return launch(ctx, 13, &p, stream) ? KDA_ERR_HIP : KDA_OK;
}

size_t kda_gated_delta_args_size(void) { return sizeof(kda_gated_delta_args); }
size_t kda_qk_norm_args_size(void) { return sizeof(kda_qk_norm_args); }

}  // extern "C"
