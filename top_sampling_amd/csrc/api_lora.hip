// C ABI of the adapter projection (declared in include/top_sampling.h).  As in
// api.hip, every argument is validated on the host before anything is
// enqueued.
#include <stdarg.h>
#include <stdio.h>

#include "lmhead_lora.hpp"

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

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" {

size_t lmhead_lora_workspace_bytes(int64_t rows, int64_t rank) {
  if (rows < 0 || rank < 0 || rows > TS_MAX_LORA_ROWS || rank > TS_MAX_LORA_RANK) return 0;
  return ts::lmhead_lora_workspace_size(rows, rank);
}

int lmhead_logits_local_lora(const void* hidden, int64_t rows, int64_t hidden_dim,
                             int64_t ld_hidden, const void* lm_head, int64_t vocab_local,
                             int64_t ld_lm_head, const void* lora_a, int64_t stride_a,
                             int64_t ld_a, const void* lora_b, int64_t stride_b, int64_t ld_b,
                             int64_t n_adapters, int64_t rank, const float* adapter_scales,
                             const int32_t* adapter_ids, float* logits, int64_t ld_logits,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (rows < 0 || vocab_local < 0 || hidden_dim < 0 || n_adapters < 0 || rank < 0)
    return fail(TS_EINVAL, "negative size (rows=%lld vocab_local=%lld hidden_dim=%lld "
                "n_adapters=%lld rank=%lld)", (long long)rows, (long long)vocab_local,
                (long long)hidden_dim, (long long)n_adapters, (long long)rank);
  if (n_adapters == 0 || rank == 0)
    return fail(TS_EINVAL, "no adapters, or adapters of rank 0: use lmhead_logits_local");
  if (rows > kMaxDim || vocab_local > kMaxDim || hidden_dim > kMaxDim || n_adapters > kMaxDim)
    return fail(TS_EUNSUPPORTED, "size above 2^31-1");
  if (rank > TS_MAX_LORA_RANK || rank % 8)
    return fail(TS_EUNSUPPORTED, "rank %lld is not a multiple of 8 up to %d (pad with zeros)",
                (long long)rank, TS_MAX_LORA_RANK);
  if (rows > TS_MAX_LORA_ROWS)
    return fail(TS_EUNSUPPORTED, "rows %lld above %d", (long long)rows, TS_MAX_LORA_ROWS);
  if (rows == 0 || vocab_local == 0) return TS_OK;
  if (hidden_dim == 0) return fail(TS_EINVAL, "hidden_dim == 0 with a non-empty output");
  if (!hidden || !lm_head || !lora_a || !lora_b || !adapter_ids || !logits)
    return fail(TS_EINVAL, "NULL pointer");
  if (ld_hidden < hidden_dim || ld_lm_head < hidden_dim || ld_a < hidden_dim || ld_b < rank ||
      ld_logits < vocab_local)
    return fail(TS_EINVAL, "leading dimension below the row width (ld_hidden=%lld "
                "ld_lm_head=%lld ld_a=%lld ld_b=%lld ld_logits=%lld)", (long long)ld_hidden,
                (long long)ld_lm_head, (long long)ld_a, (long long)ld_b, (long long)ld_logits);
  if (stride_a < 0 || stride_b < 0) return fail(TS_EINVAL, "negative adapter stride");
  if (hidden_dim % 8 || ld_hidden % 8 || ld_lm_head % 8 || ld_a % 8 || ld_b % 8 || stride_a % 8 ||
      stride_b % 8)
    return fail(TS_EUNSUPPORTED,
                "hidden_dim, leading dimensions and adapter strides must be multiples of 8");
  if (!aligned(hidden, 16) || !aligned(lm_head, 16) || !aligned(lora_a, 16) ||
      !aligned(lora_b, 16) || !aligned(logits, 4) || !aligned(adapter_ids, 4) ||
      !aligned(adapter_scales, 4))
    return fail(TS_EUNSUPPORTED, "hidden, lm_head, lora_a and lora_b must be 16-byte aligned, "
                "logits, adapter_ids and adapter_scales 4-byte aligned");
  if (!ts::lmhead_lora_fits(rows, vocab_local, hidden_dim))
    return fail(TS_EUNSUPPORTED, "more tiles of logits than a launch has workgroups for "
                "(rows=%lld vocab_local=%lld)", (long long)rows, (long long)vocab_local);
  const size_t need = ts::lmhead_lora_workspace_size(rows, rank);
  if (!workspace || workspace_bytes < need)
    return fail(TS_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned(workspace, 256)) return fail(TS_EUNSUPPORTED, "workspace not 256-byte aligned");
  ts::LoraArgs p{};
  p.hidden = static_cast<const uint16_t*>(hidden);
  p.ld_hidden = ld_hidden;
  p.lm_head = static_cast<const uint16_t*>(lm_head);
  p.ld_lm_head = ld_lm_head;
  p.a = static_cast<const uint16_t*>(lora_a);
  p.stride_a = stride_a;
  p.ld_a = ld_a;
  p.b = static_cast<const uint16_t*>(lora_b);
  p.stride_b = stride_b;
  p.ld_b = ld_b;
  p.scales = adapter_scales;
  p.ids = adapter_ids;
  p.logits = logits;
  p.ld_logits = ld_logits;
  p.rows = static_cast<int>(rows);
  p.vocab = static_cast<int>(vocab_local);
  p.hidden_dim = static_cast<int>(hidden_dim);
  p.n_adapters = static_cast<int>(n_adapters);
  p.rank = static_cast<int>(rank);
  const hipError_t e = ts::launch_lmhead_lora(p, workspace, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) return TS_OK;
  return fail(TS_EHIP, "lmhead_logits_local_lora launch: %s", hipGetErrorString(e));
}

}  // extern "C"
