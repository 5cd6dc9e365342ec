// Launchers of the policy and preference losses (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gpt {

// Rows of logits and of their gradient: bf16 or fp32, M rows of V values,
// row strides in elements.  dlogits null: no gradient.
struct LossRows {
  const void* logits;
  void* dlogits;
  long long ld, ld_d;
  const int* targets;   // [M], -1: not counted
  int M, V;
  bool fp32;
};

struct PolicyArgs {
  const float* old_logp;   // [M] or null: the present ones (ratio 1)
  const float* ref_logp;   // [M] or null: no KL term
  const float* advantage;  // [M]
  const float* weight;     // [M], 0: not counted
  double clip_low, clip_high, kl_coef;
  float* stats;   // [4]
  float* logp;    // [M]
};

struct PreferenceArgs {
  const int* cu;           // [2 n_pairs + 1]
  int n_pairs;
  const float* ref_logp;   // [2 n_pairs] or null: zero
  double beta, smoothing;
  float* loss;       // [1]
  float* margin;     // [n_pairs]
  float* seq_logp;   // [2 n_pairs]
  float* logp;       // [M]
  bool clear_past;   // zeros in the gradient's rows past the last sequence
};

size_t policy_loss_scratch(int M);
size_t preference_loss_scratch(int M, int n_pairs);
cudaError_t launch_policy_loss(const LossRows& r, const PolicyArgs& a, void* scratch, int* err, cudaStream_t s);
cudaError_t launch_preference_loss(const LossRows& r, const PreferenceArgs& a, void* scratch, int* err,
                                   cudaStream_t s);

}  // namespace gpt
