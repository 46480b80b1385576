// Internal declarations of the linear-attention and rotary kernels: launch data and
// launchers, shared by their host side and their .hip files.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kda.h"
#include "kda_internal.h"

namespace kda {

constexpr int kLinChunk = 64;  // tokens per chunk of the linear walk

// Rotation of one kernel's q and k (inv_freq null: none).
struct RotaryPlan {
  int T, D, rot_dim, dtype;
  int H[2];                    // q heads, k heads (0: no k)
  const void* in[2];
  void* out[2];
  int64_t in_t[2], in_h[2];    // element strides
  int64_t out_t[2], out_h[2];
  const void* positions;
  int positions_i64;
  const double* inv_freq;
  float factor;
  int interleaved, inverse;
};

// Segments. The tokens of a call lie on one axis on which sequence n starts at
// cu[n] + n * head_cost: its state's read and write count as head_cost tokens, so cutting the
// axis into equal pieces of seg_len cuts the work into equal pieces. At most one sequence
// crosses the border between segments s and s + 1; it has entry s of the arrays below.
struct LinearPlan {
  int T, N, H, group, K, V;  // group = H / H_qk
  float scale;
  const void* q;
  const void* k;
  const void* v;
  void* out;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;  // element strides
  const void* g;  // null: no decay
  int g_bf16;
  int g_per_token;
  const int32_t* cu;  // [N+1], device; null for the step
  int state_dtype, kfirst;
  const void* state_in;
  int in_mode;  // StateMode
  void* state_out;
  int out_mode;
  int64_t stride0, num_slots;
  const int32_t* indices;
  const uint8_t* flags;
  int seg_len, head_cost, n_seg;
  int slices;       // workgroups that share a segment of a head, V / slices state rows each
  float* maps;      // [n_seg - 1][H][slices][V / slices * K]: state at the end of segment s, as if its start were
                    // zero; after the combine the true state. Register order of the walk.
  float* initials;  // as maps: copy of the initial state of a sequence that
                    // starts in segment s and crosses its end
  float* decays;    // [n_seg - 1][H]: e^{sum of g} over the crossing sequence's part of s, as the fp32
                    // product of its chunks' factors
  int32_t* spans;   // [n_seg - 1]: 0 nothing crosses the end of s, 1 a sequence that starts in
                    // s, 2 one that came from before
  RotaryPlan rot;   // step: rotation in the kernel
};

int launch_linear_maps(const LinearPlan& p, void* stream);
int launch_linear_combine(const LinearPlan& p, void* stream);
int launch_linear_output(const LinearPlan& p, void* stream);
int launch_linear_step(const LinearPlan& p, void* stream);
int launch_rotary(const RotaryPlan& p, void* stream);

// Argument checks and plan fields that the linear and gated delta entry points have in common, and the rotation's.
kda_status check_linear(const kda_linear_args* a);
LinearPlan plan_of(const kda_linear_args* a);
kda_status check_rotation(int32_t rot_dim, int32_t D, const double* inv_freq, const void* positions, int32_t positions_i64,
                          int32_t interleaved, float factor, int32_t T);
int32_t heads_qk(const kda_linear_args* a);
// Runs one kernel through the context's runtime table.
int launch(kda_ctx* ctx, int kernel, const void* plan, void* stream);

// The context's runtime table (kda_host.cpp owns the context's definition).
const kda_runtime& context_runtime(kda_ctx* ctx);

}  // namespace kda
