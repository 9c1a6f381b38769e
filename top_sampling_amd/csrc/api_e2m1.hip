// C ABI of the 4-bit quantization and projection (declared in
// include/top_sampling.h).  As in api.hip, every argument is validated on the
// host before anything is enqueued.
#include <stdarg.h>
#include <stdio.h>

#include "lmhead_e2m1.hpp"

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;

int fail(int code, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return ts::fail_message(code, msg);
}

int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return TS_OK;
  return fail(TS_EHIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Sizes of rows that are, or are to be, held in groups.
int group_sizes(int64_t rows, int64_t cols, int32_t type) {
  if (rows < 0 || cols < 0)
    return fail(TS_EINVAL, "negative size (rows=%lld cols=%lld)", (long long)rows,
                (long long)cols);
  if (type != TS_F32 && type != TS_BF16)
    return fail(TS_EINVAL, "type %d is neither TS_F32 nor TS_BF16", type);
  if (rows > kMaxDim || cols > kMaxDim) return fail(TS_EUNSUPPORTED, "size above 2^31-1");
  if (cols % ts::kE2m1Group)
    return fail(TS_EUNSUPPORTED, "cols %lld is no multiple of %d", (long long)cols,
                ts::kE2m1Group);
  return TS_OK;
}

// Leading dimensions and alignment of rows on both sides of a conversion.
int group_buffers(const void* values, int32_t type, int64_t ld_values, const void* codes,
                  int64_t ld_codes, const void* scales, int64_t ld_scales, int64_t cols) {
  if (!values || !codes || !scales) return fail(TS_EINVAL, "NULL pointer");
  if (ld_values < cols || ld_codes < cols / 2 || ld_scales < cols / ts::kE2m1Group)
    return fail(TS_EINVAL, "leading dimension below the row width (values %lld codes %lld "
                "scales %lld)", (long long)ld_values, (long long)ld_codes, (long long)ld_scales);
  if (!aligned(values, type == TS_BF16 ? 2 : 4) || !aligned(codes, 4) || ld_codes % 4)
    return fail(TS_EUNSUPPORTED, "values misaligned, or codes or their leading dimension no "
                "multiple of 4 bytes");
  return TS_OK;
}

}  // namespace

extern "C" {

int quantize_groups_e2m1(const void* in, int32_t in_type, int64_t rows, int64_t cols,
                         int64_t ld_in, void* codes, int64_t ld_codes, void* scales,
                         int64_t ld_scales, void* stream) {
  int st = group_sizes(rows, cols, in_type);
  if (st != TS_OK || rows == 0 || cols == 0) return st;
  st = group_buffers(in, in_type, ld_in, codes, ld_codes, scales, ld_scales, cols);
  if (st != TS_OK) return st;
  return hip_status(
      ts::launch_quantize_groups_e2m1(in, in_type == TS_BF16, ld_in, static_cast<int>(rows),
                                      static_cast<int>(cols), static_cast<uint8_t*>(codes),
                                      ld_codes, static_cast<uint8_t*>(scales), ld_scales,
                                      static_cast<hipStream_t>(stream)),
      "quantize_groups_e2m1 launch");
}

int dequantize_groups_e2m1(const void* codes, int64_t rows, int64_t cols, int64_t ld_codes,
                           const void* scales, int64_t ld_scales, void* out, int32_t out_type,
                           int64_t ld_out, void* stream) {
  int st = group_sizes(rows, cols, out_type);
  if (st != TS_OK || rows == 0 || cols == 0) return st;
  st = group_buffers(out, out_type, ld_out, codes, ld_codes, scales, ld_scales, cols);
  if (st != TS_OK) return st;
  const ts::E2m1Rows r{static_cast<const uint8_t*>(codes), ld_codes,
                       static_cast<const uint8_t*>(scales), ld_scales};
  return hip_status(
      ts::launch_dequantize_groups_e2m1(r, static_cast<int>(rows), static_cast<int>(cols), out,
                                        out_type == TS_BF16, ld_out,
                                        static_cast<hipStream_t>(stream)),
      "dequantize_groups_e2m1 launch");
}

int lmhead_logits_local_e2m1(const void* hidden, int64_t rows, int64_t hidden_dim,
                             int64_t ld_hidden, const void* lm_head, const void* lm_head_scales,
                             int64_t vocab_local, int64_t ld_lm_head, int64_t ld_scales,
                             float* logits, int64_t ld_logits, void* stream) {
  if (rows < 0 || vocab_local < 0 || hidden_dim < 0)
    return fail(TS_EINVAL, "negative size (rows=%lld vocab_local=%lld hidden_dim=%lld)",
                (long long)rows, (long long)vocab_local, (long long)hidden_dim);
  if (rows > kMaxDim || vocab_local > kMaxDim || hidden_dim > kMaxDim)
    return fail(TS_EUNSUPPORTED, "size above 2^31-1");
  if (rows == 0 || vocab_local == 0) return TS_OK;
  if (hidden_dim == 0) return fail(TS_EINVAL, "hidden_dim == 0 with a non-empty output");
  if (!hidden || !lm_head || !lm_head_scales || !logits) return fail(TS_EINVAL, "NULL pointer");
  if (ld_hidden < hidden_dim || ld_lm_head < hidden_dim / 2 ||
      ld_scales < hidden_dim / ts::kE2m1Group || ld_logits < vocab_local)
    return fail(TS_EINVAL, "leading dimension below the row width (ld_hidden=%lld ld_lm_head=%lld "
                "ld_scales=%lld ld_logits=%lld)", (long long)ld_hidden, (long long)ld_lm_head,
                (long long)ld_scales, (long long)ld_logits);
  if (hidden_dim % ts::kE2m1Group)
    return fail(TS_EUNSUPPORTED, "hidden_dim %lld is no multiple of %d", (long long)hidden_dim,
                ts::kE2m1Group);
  if (ld_hidden > ts::kE2m1MaxLdHidden)
    return fail(TS_EUNSUPPORTED, "ld_hidden %lld above %lld", (long long)ld_hidden,
                (long long)ts::kE2m1MaxLdHidden);
  if (ld_hidden % 8 || ld_lm_head % 16)
    return fail(TS_EUNSUPPORTED, "ld_hidden must be a multiple of 8 elements, ld_lm_head of 16 "
                "bytes");
  if (!aligned(hidden, 16) || !aligned(lm_head, 16) || !aligned(logits, 4))
    return fail(TS_EUNSUPPORTED, "hidden/lm_head must be 16-byte aligned, logits 4-byte aligned");
  if (!ts::lmhead_e2m1_fits(rows, vocab_local))
    return fail(TS_EUNSUPPORTED, "%lld x %lld logits are more than a launch has tiles for",
                (long long)rows, (long long)vocab_local);
  const ts::E2m1Rows w{static_cast<const uint8_t*>(lm_head), ld_lm_head,
                       static_cast<const uint8_t*>(lm_head_scales), ld_scales};
  return hip_status(
      ts::launch_lmhead_e2m1(static_cast<const uint16_t*>(hidden), ld_hidden, w, logits,
                             ld_logits, static_cast<int>(rows), static_cast<int>(vocab_local),
                             static_cast<int>(hidden_dim), static_cast<hipStream_t>(stream)),
      "lmhead_logits_local_e2m1 launch");
}

}  // extern "C"
