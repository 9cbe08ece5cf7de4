// Launch interfaces of the router's training kernels (losses and gradient).
#pragma once
#include "common.cuh"

namespace moe {

// Workspace of the losses: one row of per-expert sums and counts per block of
// the first kernel, and its sum of squared normalisers and token count.
int64_t router_loss_workspace_bytes(int32_t T, int32_t E);

struct RouterLossArgs {
  const void* logits;   // [T][E], fp32 or bf16
  const uint8_t* mask;  // [T] or null: 0 marks padding
  int32_t T, E, k;
  int32_t* topk_idx;    // [T][k]
  float* topk_prob;     // [T][k]
  float* lse;           // [T]
  int32_t* counts;      // [E]
  float* prob_sums;     // [E]
  int32_t* tokens;      // [1]
  float* losses;        // [2]
};
cudaError_t launch_router_losses(const RouterLossArgs& a, bool bf16, void* ws, cudaStream_t st);

struct RouterBwdArgs {
  const void* logits;
  const uint8_t* mask;
  int32_t T, E, k;
  const int32_t* topk_idx;
  const float* topk_prob;
  const float* lse;
  const int32_t* counts;
  const int32_t* tokens;
  const float* dprob;    // [T][k] or null (zero)
  const float* dlosses;  // [2] or null (zero)
  void* dlogits;         // [T][E], the logits' type
};
cudaError_t launch_router_bwd(const RouterBwdArgs& a, bool bf16, cudaStream_t st);

}  // namespace moe
