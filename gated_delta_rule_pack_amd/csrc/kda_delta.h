// Internal declarations of the gated delta rule's and the q/k norms' kernels: launch data and launchers,
// shared by their host side and their .hip files.
#pragma once

#include "kda_linear.h"

namespace kda {

constexpr float kNormEps = 1e-6f;  // of normalised q and k, as in kda_chunk_fwd

// The linear plan's fields (its segments aside) and what the delta rule adds.
struct DeltaPlan : LinearPlan {
  const void* beta;  // [T, H]
  int beta_bf16;
  int f16;           // q, k, v and out are fp16, not bf16
  int normalize;
  int ranked;        // workgroups take their sequences longest first
  // The chunks' records, for the scan. A chunk has a place: sequence n's are floor(cu[n] / 64) + n on.
  int places;
  char* records;     // [places][H] of kDeltaRecord bytes
  char* keys;        // [places][H_qk] of 64 K fp16 values, in operand order
  char* queries;
};
constexpr int kDeltaRecord = 19712;
constexpr int kMostRanked = 512;  // sequences that a workgroup of the walk or the scan can rank, one to a thread

int launch_delta_walk(const DeltaPlan& p, void* stream);
int launch_delta_prep(const DeltaPlan& p, void* stream);
int launch_delta_scan(const DeltaPlan& p, void* stream);
int launch_delta_step(const DeltaPlan& p, void* stream);

// Norms of q and k: the rotation's fields (in: x, out: y or dx) and the norm's.
struct NormPlan : RotaryPlan {
  const void* grad[2];
  int64_t grad_t[2], grad_h[2];
  const void* weight[2];       // null: none
  void* grad_weight[2];
  float* sums;                 // backward with weights: [groups][2][D], a workgroup's sums of weight gradients
  int groups;
  int weight_f32;              // else of dtype
  int l2;
  float eps, offset;
};

// Workgroups of the backward pass that leave sums, for T tokens.
int norm_groups(int T);

int launch_qk_norm(const NormPlan& p, void* stream);
int launch_qk_norm_backward(const NormPlan& p, void* stream);

}  // namespace kda
