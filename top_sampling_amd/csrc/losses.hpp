// Host-side interfaces of the scoring and loss kernels (losses.hip), used by
// the entry points in api_losses.hip.  Every launcher assumes its arguments
// were validated there and returns the hipError_t of its launches.
#pragma once

#include "ts_internal.hpp"

namespace ts {

// Logits rows, each with one token whose log-probability is asked for.
struct TokenRows {
  const void* x;          // fp32 or bf16 [rows, vocab], leading dimension ld
  int64_t ld;
  int bf16;
  int rows, vocab;
  const int32_t* tokens;  // [rows]; negative: the row is left out
  const float* weights;   // [rows] or null; 0: the row is left out
  double temperature;
};

// Gradient rows in the logits' type; x null: no gradient is written.
struct GradRows {
  void* x;
  int64_t ld;
};

struct ScoreOut {
  float* logprobs;
  float* entropies;     // may be null
  float* row_stats;     // [rows, 2], may be null
  int32_t* row_status;  // may be null
};

struct ScoreGrad {
  const float* row_stats;
  const float* logprobs;        // may be null
  const float* grad_logprobs;
  const float* entropies;       // null iff grad_entropies is
  const float* grad_entropies;
};

struct PolicyArgs {
  double clip_low, clip_high, kl_coef;
  const float* old_logprobs;
  const float* ref_logprobs;  // null: no KL term, kl rows are 0
  const float* advantages;
  const float* grad_loss;     // null: 1
  float* loss;
  float* logprobs;            // these four may be null
  float* ratios;
  float* kl;
  int32_t* row_status;
};

struct PreferenceArgs {
  double beta, label_smoothing, margin;
  int mean;
  int n_pairs;
  const int32_t* seq_offsets;  // [2 n_pairs + 1]
  const float* ref_logprobs;   // null: zeros
  const float* pair_weights;   // null: 1 / n_pairs
  const float* grad_loss;      // null: 1
  float* loss;
  float* pair_losses;          // these four may be null
  float* rewards;
  float* logprobs;
  int32_t* row_status;
};

size_t token_rows_workspace_size(int64_t rows, int64_t vocab, int64_t n_pairs);
hipError_t launch_token_logprobs(const TokenRows& t, const ScoreOut& o, void* ws,
                                 hipStream_t stream);
hipError_t launch_token_logprobs_backward(const TokenRows& t, const ScoreGrad& g,
                                          const GradRows& d, hipStream_t stream);
hipError_t launch_policy_loss(const TokenRows& t, const PolicyArgs& p, const GradRows& d, void* ws,
                              hipStream_t stream);
hipError_t launch_preference_loss(const TokenRows& t, const PreferenceArgs& p, const GradRows& d,
                                  void* ws, hipStream_t stream);

}  // namespace ts
