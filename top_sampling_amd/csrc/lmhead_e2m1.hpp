// Host-side interface of the 4-bit projection and quantization
// (lmhead_e2m1.hip), used by the entry points in api_e2m1.hip.  Every launcher
// assumes its arguments were validated there.
#pragma once

#include "ts_internal.hpp"

namespace ts {

constexpr int kE2m1Group = 32;  // entries of a row that share a scale

// A tile's hidden rows lie within 2^31 bytes of each other.
constexpr int64_t kE2m1MaxLdHidden = int64_t{1} << 21;

struct E2m1Rows {
  const uint8_t* codes;   // [rows, cols / 2], two codes a byte, the even column's in the low half
  int64_t ld;
  const uint8_t* scales;  // [rows, cols / 32], the exponent of the scale plus 127
  int64_t ld_scales;
};

hipError_t launch_quantize_groups_e2m1(const void* in, int bf16, int64_t ld_in, int rows, int cols,
                                       uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                                       int64_t ld_scales, hipStream_t stream);
hipError_t launch_dequantize_groups_e2m1(const E2m1Rows& in, int rows, int cols, void* out,
                                         int bf16, int64_t ld_out, hipStream_t stream);
// Whether a launch has room for these sizes' tiles.
bool lmhead_e2m1_fits(int64_t rows, int64_t vocab);
hipError_t launch_lmhead_e2m1(const uint16_t* hidden, int64_t ld_hidden, const E2m1Rows& lm_head,
                              float* logits, int64_t ld_logits, int rows, int vocab,
                              int hidden_dim, hipStream_t stream);

}  // namespace ts
