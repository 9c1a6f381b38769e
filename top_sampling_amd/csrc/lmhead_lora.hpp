// Host-side interface of the adapter projection (lmhead_lora.hip), used by
// the entry point in api_lora.hip.
#pragma once

#include "ts_internal.hpp"

namespace ts {

struct LoraArgs {
  const uint16_t* hidden;   // bf16 [rows, hidden_dim]
  int64_t ld_hidden;
  const uint16_t* lm_head;  // bf16 [vocab, hidden_dim]
  int64_t ld_lm_head;
  const uint16_t* a;        // bf16 [n_adapters][rank, hidden_dim]
  int64_t stride_a, ld_a;
  const uint16_t* b;        // bf16 [n_adapters][vocab, rank]
  int64_t stride_b, ld_b;
  const float* scales;      // [n_adapters] or null
  const int32_t* ids;       // [rows]
  float* logits;            // fp32 [rows, vocab]
  int64_t ld_logits;
  int rows, vocab, hidden_dim, n_adapters, rank;
};

// Whether a launch has room for these sizes' tiles.
bool lmhead_lora_fits(int64_t rows, int64_t vocab, int64_t hidden_dim);
size_t lmhead_lora_workspace_size(int64_t rows, int64_t rank);
hipError_t launch_lmhead_lora(const LoraArgs& p, void* ws, hipStream_t stream);

}  // namespace ts
