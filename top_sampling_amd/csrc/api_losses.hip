// C ABI of token scoring and the losses (declared in include/top_sampling.h).
// As in api.hip, every argument is validated on the host before anything is
// enqueued, and valid calls only enqueue kernels on the caller's stream.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>

#include "alternatives.hpp"
#include "losses.hpp"

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

// The logits, tokens and temperature of a call into t.  rows == 0 passes
// without looking at the pointers.
int token_rows(ts::TokenRows& t, const void* logits, int32_t logits_type, int64_t rows,
               int64_t vocab, int64_t ld_logits, const int32_t* token_ids, double temperature,
               bool needs_tokens = true) {
  if (rows < 0 || vocab < 0)
    return fail(TS_EINVAL, "negative size (rows=%lld vocab=%lld)", (long long)rows,
                (long long)vocab);
  if (logits_type != TS_F32 && logits_type != TS_BF16)
    return fail(TS_EINVAL, "logits_type %d is neither TS_F32 nor TS_BF16", logits_type);
  if (rows > kMaxDim || vocab > kMaxDim) return fail(TS_EUNSUPPORTED, "size above 2^31-1");
  if (!(temperature >= static_cast<double>(TS_GREEDY_EPS)) || !(temperature < INFINITY))
    return fail(TS_EINVAL, "temperature %g is not a finite number of at least TS_GREEDY_EPS",
                temperature);
  t = ts::TokenRows{};
  t.rows = static_cast<int>(rows);
  t.vocab = static_cast<int>(vocab);
  t.bf16 = logits_type == TS_BF16;
  t.temperature = temperature;
  if (rows == 0) return TS_OK;
  if (vocab == 0) return fail(TS_EINVAL, "vocab == 0 with rows > 0");
  if (ld_logits < vocab)
    return fail(TS_EINVAL, "ld_logits %lld < vocab %lld", (long long)ld_logits, (long long)vocab);
  if (!logits || (needs_tokens && !token_ids)) return fail(TS_EINVAL, "NULL logits/token_ids");
  if (!aligned(logits, t.bf16 ? 2 : 4) || !aligned(token_ids, 4))
    return fail(TS_EUNSUPPORTED, "logits or token_ids misaligned");
  t.x = logits;
  t.ld = ld_logits;
  t.tokens = token_ids;
  return TS_OK;
}

// The gradient's rows into d; they are the logits' own (the gradient replaces
// them) or do not overlap them.
int grad_rows(ts::GradRows& d, const ts::TokenRows& t, void* grad_logits, int64_t ld_grad) {
  d.x = grad_logits;
  d.ld = ld_grad;
  if (t.rows == 0 || grad_logits == nullptr) return TS_OK;
  if (ld_grad < t.vocab)
    return fail(TS_EINVAL, "ld_grad %lld < vocab %d", (long long)ld_grad, t.vocab);
  const size_t size = t.bf16 ? 2 : 4;
  if (!aligned(grad_logits, size)) return fail(TS_EUNSUPPORTED, "grad_logits misaligned");
  if (grad_logits == t.x && (ld_grad == t.ld || t.rows == 1)) return TS_OK;
  const char* a = static_cast<const char*>(t.x);
  const char* b = static_cast<const char*>(grad_logits);
  const char* a_end = a + (static_cast<int64_t>(t.rows - 1) * t.ld + t.vocab) * size;
  const char* b_end = b + (static_cast<int64_t>(t.rows - 1) * ld_grad + t.vocab) * size;
  // Columns side by side in one buffer do not overlap either.
  if (t.rows > 1 && ld_grad == t.ld) {
    int64_t gap = (b - a) / static_cast<int64_t>(size) % ld_grad;
    if (gap < 0) gap += ld_grad;
    if (gap >= t.vocab && gap <= ld_grad - t.vocab) return TS_OK;
  }
  if (a < b_end && b < a_end)
    return fail(TS_EINVAL, "grad_logits overlaps logits without being the same rows");
  return TS_OK;
}

int workspace_ok(void* workspace, size_t given, size_t need) {
  if (!workspace || given < need)
    return fail(TS_EWORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                workspace ? given : (size_t)0);
  if (!aligned(workspace, 256)) return fail(TS_EUNSUPPORTED, "workspace not 256-byte aligned");
  return TS_OK;
}

bool all_aligned4(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 4)) return false;
  return true;
}

int listed_count(int32_t n) {
  if (n < 1) return fail(TS_EINVAL, "n_listed %d < 1", n);
  if (n > TS_MAX_LISTED) return fail(TS_EUNSUPPORTED, "n_listed %d above %d", n, TS_MAX_LISTED);
  return TS_OK;
}

// Finite and at least 0.
bool bound_ok(double v) { return v >= 0.0 && v < INFINITY; }

}  // namespace

extern "C" {

size_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab) {
  if (rows < 0 || vocab < 0 || rows > kMaxDim || vocab > kMaxDim) return 0;
  return ts::token_rows_workspace_size(rows, vocab, 0);
}

size_t preference_loss_workspace_bytes(int64_t rows, int64_t vocab, int64_t n_pairs) {
  if (rows < 0 || vocab < 0 || n_pairs < 0 || rows > kMaxDim || vocab > kMaxDim ||
      n_pairs > kMaxDim / 2)
    return 0;
  return ts::token_rows_workspace_size(rows, vocab, n_pairs);
}

int token_logprobs(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                   int64_t ld_logits, const int32_t* token_ids, double temperature,
                   float* logprobs, float* entropies, float* row_stats, int32_t* row_status,
                   void* workspace, size_t workspace_bytes, void* stream) {
  ts::TokenRows t;
  int st = token_rows(t, logits, logits_type, rows, vocab, ld_logits, token_ids, temperature);
  if (st != TS_OK || rows == 0) return st;
  if (!logprobs) return fail(TS_EINVAL, "NULL logprobs");
  if (!all_aligned4({logprobs, entropies, row_stats, row_status}))
    return fail(TS_EUNSUPPORTED, "misaligned output");
  st = workspace_ok(workspace, workspace_bytes, token_logprobs_workspace_bytes(rows, vocab));
  if (st != TS_OK) return st;
  const ts::ScoreOut o{logprobs, entropies, row_stats, row_status};
  return hip_status(ts::launch_token_logprobs(t, o, workspace, static_cast<hipStream_t>(stream)),
                    "token_logprobs launch");
}

int token_logprobs_backward(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                            int64_t ld_logits, const int32_t* token_ids, double temperature,
                            const float* row_stats, const float* grad_logprobs,
                            const float* entropies, const float* grad_entropies,
                            void* grad_logits, int64_t ld_grad, void* stream) {
  return token_logprobs_backward_ex(logits, logits_type, rows, vocab, ld_logits, token_ids,
                                    temperature, row_stats, nullptr, grad_logprobs, entropies,
                                    grad_entropies, grad_logits, ld_grad, stream);
}

int token_logprobs_backward_ex(const void* logits, int32_t logits_type, int64_t rows,
                               int64_t vocab, int64_t ld_logits, const int32_t* token_ids,
                               double temperature, const float* row_stats, const float* logprobs,
                               const float* grad_logprobs, const float* entropies,
                               const float* grad_entropies, void* grad_logits, int64_t ld_grad,
                               void* stream) {
  ts::TokenRows t;
  int st = token_rows(t, logits, logits_type, rows, vocab, ld_logits, token_ids, temperature);
  if (st != TS_OK || rows == 0) return st;
  if (!row_stats || !grad_logprobs || !grad_logits)
    return fail(TS_EINVAL, "NULL row_stats/grad_logprobs/grad_logits");
  if (grad_entropies && !entropies)
    return fail(TS_EINVAL, "grad_entropies without the forward pass's entropies");
  if (!all_aligned4({row_stats, logprobs, grad_logprobs, entropies, grad_entropies}))
    return fail(TS_EUNSUPPORTED, "misaligned input");
  ts::GradRows d;
  st = grad_rows(d, t, grad_logits, ld_grad);
  if (st != TS_OK) return st;
  const ts::ScoreGrad g{row_stats, logprobs, grad_logprobs, grad_entropies ? entropies : nullptr,
                        grad_entropies};
  return hip_status(
      ts::launch_token_logprobs_backward(t, g, d, static_cast<hipStream_t>(stream)),
      "token_logprobs_backward launch");
}

size_t token_logprobs_topn_workspace_bytes(int64_t rows, int64_t vocab) {
  if (rows < 0 || vocab < 0 || rows > kMaxDim || vocab > kMaxDim) return 0;
  return ts::topn_workspace_size(rows, vocab);
}

int token_logprobs_topn(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                        int64_t ld_logits, const int32_t* token_ids, double temperature,
                        int32_t max_logprobs, float* logprobs, int32_t* ranks, float* entropies,
                        int32_t* topn_ids, float* topn_logprobs, float* row_stats,
                        int32_t* row_status, void* workspace, size_t workspace_bytes,
                        void* stream) {
  ts::TokenRows t;
  int st = token_rows(t, logits, logits_type, rows, vocab, ld_logits, token_ids, temperature,
                      false);
  if (st != TS_OK) return st;
  if (max_logprobs < 0) return fail(TS_EINVAL, "max_logprobs %d < 0", max_logprobs);
  if (max_logprobs > TS_MAX_LOGPROBS)
    return fail(TS_EUNSUPPORTED, "max_logprobs %d above %d", max_logprobs, TS_MAX_LOGPROBS);
  if (rows == 0) return TS_OK;
  if (token_ids ? !logprobs : (logprobs || ranks))
    return fail(TS_EINVAL, "logprobs and ranks are those of token_ids: logprobs is needed with "
                "them, and neither is written without");
  if (max_logprobs > 0 && (!topn_ids || !topn_logprobs))
    return fail(TS_EINVAL, "NULL topn_ids/topn_logprobs");
  if (!all_aligned4({logprobs, ranks, entropies, topn_ids, topn_logprobs, row_stats, row_status}))
    return fail(TS_EUNSUPPORTED, "misaligned output");
  st = workspace_ok(workspace, workspace_bytes, token_logprobs_topn_workspace_bytes(rows, vocab));
  if (st != TS_OK) return st;
  const ts::TopnOut o{max_logprobs, logprobs,  ranks,     entropies,
                      topn_ids,     topn_logprobs, row_stats, row_status};
  return hip_status(
      ts::launch_token_logprobs_topn(t, o, workspace, static_cast<hipStream_t>(stream)),
      "token_logprobs_topn launch");
}

size_t token_logprobs_listed_workspace_bytes(int64_t rows, int64_t vocab) {
  if (rows < 0 || vocab < 0 || rows > kMaxDim || vocab > kMaxDim) return 0;
  return ts::listed_workspace_size(rows, vocab);
}

int token_logprobs_listed(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                          int64_t ld_logits, const int32_t* listed_ids, int32_t n_listed,
                          double temperature, float* logprobs, float* entropies, float* row_stats,
                          int32_t* row_status, void* workspace, size_t workspace_bytes,
                          void* stream) {
  ts::TokenRows t;
  int st = token_rows(t, logits, logits_type, rows, vocab, ld_logits, listed_ids, temperature);
  if (st != TS_OK) return st;
  st = listed_count(n_listed);
  if (st != TS_OK || rows == 0) return st;
  if (!logprobs) return fail(TS_EINVAL, "NULL logprobs");
  if (!all_aligned4({logprobs, entropies, row_stats, row_status}))
    return fail(TS_EUNSUPPORTED, "misaligned output");
  st = workspace_ok(workspace, workspace_bytes, token_logprobs_listed_workspace_bytes(rows, vocab));
  if (st != TS_OK) return st;
  const ts::ListedOut o{n_listed, logprobs, entropies, row_stats, row_status};
  return hip_status(
      ts::launch_token_logprobs_listed(t, o, workspace, static_cast<hipStream_t>(stream)),
      "token_logprobs_listed launch");
}

int token_logprobs_listed_backward(const void* logits, int32_t logits_type, int64_t rows,
                                   int64_t vocab, int64_t ld_logits, const int32_t* listed_ids,
                                   int32_t n_listed, double temperature, const float* row_stats,
                                   const float* logprobs, const float* grad_logprobs,
                                   const float* entropies, const float* grad_entropies,
                                   void* grad_logits, int64_t ld_grad, void* stream) {
  ts::TokenRows t;
  int st = token_rows(t, logits, logits_type, rows, vocab, ld_logits, listed_ids, temperature);
  if (st != TS_OK) return st;
  st = listed_count(n_listed);
  if (st != TS_OK || rows == 0) return st;
  if (!row_stats || !logprobs || !grad_logprobs || !grad_logits)
    return fail(TS_EINVAL, "NULL row_stats/logprobs/grad_logprobs/grad_logits");
  if (grad_entropies && !entropies)
    return fail(TS_EINVAL, "grad_entropies needs the forward pass's entropies");
  if (!all_aligned4({row_stats, logprobs, grad_logprobs, entropies, grad_entropies}))
    return fail(TS_EUNSUPPORTED, "misaligned input");
  ts::GradRows d;
  st = grad_rows(d, t, grad_logits, ld_grad);
  if (st != TS_OK) return st;
  const ts::ListedGrad g{n_listed, row_stats, logprobs, grad_logprobs, entropies, grad_entropies};
  return hip_status(
      ts::launch_token_logprobs_listed_backward(t, g, d, static_cast<hipStream_t>(stream)),
      "token_logprobs_listed_backward launch");
}

int policy_loss(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                int64_t ld_logits, const int32_t* token_ids, const ts_policy_params* params,
                const float* old_logprobs, const float* ref_logprobs, const float* advantages,
                const float* weights, const float* grad_loss, float* loss, float* logprobs,
                float* ratios, float* kl, int32_t* row_status, void* grad_logits, int64_t ld_grad,
                void* workspace, size_t workspace_bytes, void* stream) {
  if (!params) return fail(TS_EINVAL, "NULL params");
  ts::TokenRows t;
  int st = token_rows(t, logits, logits_type, rows, vocab, ld_logits, token_ids,
                      params->temperature);
  if (st != TS_OK) return st;
  if (!(params->clip_low >= 0.0) || !(params->clip_high >= 0.0))
    return fail(TS_EINVAL, "clip_low and clip_high must be at least 0 (inf: no clip)");
  if (!bound_ok(params->kl_coef))
    return fail(TS_EINVAL, "kl_coef %g is negative or not finite", params->kl_coef);
  if (!loss) return fail(TS_EINVAL, "NULL loss");
  if (!aligned(loss, 4)) return fail(TS_EUNSUPPORTED, "loss misaligned");
  if (rows > 0 && (!old_logprobs || !advantages))
    return fail(TS_EINVAL, "NULL old_logprobs/advantages");
  if (rows > 0 && params->kl_coef != 0.0 && !ref_logprobs)
    return fail(TS_EINVAL, "kl_coef without ref_logprobs");
  if (!all_aligned4({old_logprobs, ref_logprobs, advantages, weights, grad_loss, logprobs, ratios,
                     kl, row_status}))
    return fail(TS_EUNSUPPORTED, "misaligned pointer");
  ts::GradRows d;
  st = grad_rows(d, t, grad_logits, ld_grad);
  if (st != TS_OK) return st;
  if (rows > 0) {
    st = workspace_ok(workspace, workspace_bytes, token_logprobs_workspace_bytes(rows, vocab));
    if (st != TS_OK) return st;
  }
  t.weights = weights;
  const ts::PolicyArgs p{params->clip_low, params->clip_high, params->kl_coef, old_logprobs,
                         ref_logprobs,     advantages,        grad_loss,       loss,
                         logprobs,         ratios,            kl,              row_status};
  return hip_status(ts::launch_policy_loss(t, p, d, workspace, static_cast<hipStream_t>(stream)),
                    "policy_loss launch");
}

int preference_loss(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                    int64_t ld_logits, const int32_t* token_ids, const int32_t* seq_offsets,
                    int64_t n_pairs, const ts_preference_params* params,
                    const float* ref_logprobs, const float* pair_weights, const float* grad_loss,
                    float* loss, float* pair_losses, float* rewards, float* logprobs,
                    int32_t* row_status, void* grad_logits, int64_t ld_grad, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!params) return fail(TS_EINVAL, "NULL params");
  ts::TokenRows t;
  int st = token_rows(t, logits, logits_type, rows, vocab, ld_logits, token_ids,
                      params->temperature);
  if (st != TS_OK) return st;
  if (n_pairs < 0) return fail(TS_EINVAL, "n_pairs < 0");
  if (n_pairs > kMaxDim / 2) return fail(TS_EUNSUPPORTED, "n_pairs above 2^30-1");
  if (!(params->beta > 0.0) || !(params->beta < INFINITY))
    return fail(TS_EINVAL, "beta %g is not a finite number above 0", params->beta);
  if (!(params->label_smoothing >= 0.0) || !(params->label_smoothing <= 1.0))
    return fail(TS_EINVAL, "label_smoothing %g is not in [0, 1]",
                params->label_smoothing);
  if (!(fabs(params->margin) < INFINITY)) return fail(TS_EINVAL, "margin is not finite");
  if (params->flags & ~TS_PREFERENCE_MEAN)
    return fail(TS_EINVAL, "unknown flag bits 0x%x", params->flags);
  if (!loss) return fail(TS_EINVAL, "NULL loss");
  if (!aligned(loss, 4)) return fail(TS_EUNSUPPORTED, "loss misaligned");
  if (!seq_offsets && (rows > 0 || n_pairs > 0)) return fail(TS_EINVAL, "NULL seq_offsets");
  if (!all_aligned4({seq_offsets, ref_logprobs, pair_weights, grad_loss, pair_losses, rewards,
                     logprobs, row_status}))
    return fail(TS_EUNSUPPORTED, "misaligned pointer");
  ts::GradRows d;
  st = grad_rows(d, t, grad_logits, ld_grad);
  if (st != TS_OK) return st;
  if (rows > 0 || n_pairs > 0) {
    st = workspace_ok(workspace, workspace_bytes,
                      preference_loss_workspace_bytes(rows, vocab, n_pairs));
    if (st != TS_OK) return st;
  }
  const ts::PreferenceArgs p{params->beta,
                             params->label_smoothing,
                             params->margin,
                             params->flags & TS_PREFERENCE_MEAN,
                             static_cast<int>(n_pairs),
                             seq_offsets,
                             ref_logprobs,
                             pair_weights,
                             grad_loss,
                             loss,
                             pair_losses,
                             rewards,
                             logprobs,
                             row_status};
  return hip_status(
      ts::launch_preference_loss(t, p, d, workspace, static_cast<hipStream_t>(stream)),
      "preference_loss launch");
}

}  // extern "C"
