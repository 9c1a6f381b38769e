// Host-side interface of scoring with alternatives and of listed tokens
// (alternatives.hip), used by the entry points in api_losses.hip.  Every
// launcher assumes its arguments were validated there.
#pragma once

#include "losses.hpp"

namespace ts {

struct TopnOut {
  int n;                  // alternatives a row
  float* logprobs;        // null iff there are no tokens
  int32_t* ranks;         // may be null
  float* entropies;       // may be null
  int32_t* topn_ids;      // [rows, n], these two null iff n == 0
  float* topn_logprobs;
  float* row_stats;       // [rows, 2], may be null
  int32_t* row_status;    // may be null
};

// The tokens of TokenRows are [rows, n] here.
struct ListedOut {
  int n;
  float* logprobs;        // [rows, n]
  float* entropies;       // may be null
  float* row_stats;       // may be null
  int32_t* row_status;    // may be null
};

struct ListedGrad {
  int n;
  const float* row_stats;
  const float* logprobs;        // [rows, n]
  const float* grad_logprobs;   // [rows, n]
  const float* entropies;       // null iff grad_entropies is
  const float* grad_entropies;
};

size_t topn_workspace_size(int64_t rows, int64_t vocab);
size_t listed_workspace_size(int64_t rows, int64_t vocab);
hipError_t launch_token_logprobs_topn(const TokenRows& t, const TopnOut& o, void* ws,
                                      hipStream_t stream);
hipError_t launch_token_logprobs_listed(const TokenRows& t, const ListedOut& o, void* ws,
                                        hipStream_t stream);
hipError_t launch_token_logprobs_listed_backward(const TokenRows& t, const ListedGrad& g,
                                                 const GradRows& d, hipStream_t stream);

}  // namespace ts
