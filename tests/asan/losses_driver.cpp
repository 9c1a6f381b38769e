// Host-side driver of the argument checks of the adapter projection, token
// scoring and the losses, built with AddressSanitizer on the host code like
// abi_driver.cpp, which walks the other entry points: every call is rejected,
// or is a no-op, before any HIP call.  The overlap check of gradients and
// logits is walked over pointers on both sides, and the workspace queries over
// a range of sizes.  Exit status 0 means every return code was the expected
// one and the sanitizer found nothing.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/top_sampling.h"

static int failures = 0;

static void expect(int got, int want, const char* what) {
  if (got != want) {
    fprintf(stderr, "FAIL %s: got %d want %d (%s)\n", what, got, want, ts_last_error());
    ++failures;
  }
  if (got != TS_OK && strlen(ts_last_error()) == 0) {
    fprintf(stderr, "FAIL %s: empty ts_last_error\n", what);
    ++failures;
  }
}

// Aligned addresses, never dereferenced.
static char* const A = reinterpret_cast<char*>(0x10000000);
static float* const F = reinterpret_cast<float*>(0x10000000);
static int32_t* const I = reinterpret_cast<int32_t*>(0x10000000);

static int lora(int64_t rows, int64_t hidden, int64_t vocab, int64_t n, int64_t rank, int64_t ld_b,
                const void* b, float* out, void* ws, size_t bytes) {
  return lmhead_logits_local_lora(A, rows, hidden, hidden, A, vocab, hidden, A, hidden * rank,
                                  hidden, b, vocab * ld_b, ld_b, n, rank, nullptr, I, out, vocab, ws,
                                  bytes, nullptr);
}

static int score(int32_t type, int64_t rows, int64_t vocab, int64_t ld, const void* x,
                 double temperature, float* lp, void* ws, size_t bytes) {
  return token_logprobs(x, type, rows, vocab, ld, I, temperature, lp, nullptr, nullptr, nullptr, ws,
                        bytes, nullptr);
}

static int policy(int64_t rows, int64_t ld, void* grad, int64_t ld_grad, const ts_policy_params* p,
                  const float* ref, float* loss) {
  return policy_loss(A, TS_F32, rows, 100, ld, I, p, F, ref, F, nullptr, nullptr, loss, nullptr,
                     nullptr, nullptr, nullptr, grad, ld_grad, nullptr, 0, nullptr);
}

static int preference(int64_t rows, const int32_t* off, int64_t pairs,
                      const ts_preference_params* p, float* rewards) {
  return preference_loss(A, TS_BF16, rows, 100, 100, I, off, pairs, p, nullptr, nullptr, nullptr, F,
                         nullptr, rewards, nullptr, nullptr, nullptr, 0, nullptr, 0, nullptr);
}

int main() {
  char* const odd = A + 2;

  // adapter projection
  expect(lora(-1, 256, 64, 3, 16, 16, A, F, nullptr, 0), TS_EINVAL, "lora rows<0");
  expect(lora(4, 256, 64, 0, 16, 16, A, F, nullptr, 0), TS_EINVAL, "lora no adapters");
  expect(lora(4, 256, 64, 3, 0, 16, A, F, nullptr, 0), TS_EINVAL, "lora rank 0");
  expect(lora(4, 256, 64, 3, 12, 16, A, F, nullptr, 0), TS_EUNSUPPORTED, "lora rank%8");
  expect(lora(4, 256, 64, 3, TS_MAX_LORA_RANK + 8, 512, A, F, nullptr, 0), TS_EUNSUPPORTED,
         "lora rank");
  expect(lora(TS_MAX_LORA_ROWS + 1, 256, 64, 3, 16, 16, A, F, nullptr, 0), TS_EUNSUPPORTED,
         "lora rows");
  expect(lora(4, 0, 64, 3, 16, 16, A, F, nullptr, 0), TS_EINVAL, "lora hidden 0");
  expect(lora(4, 256, 64, 3, 16, 8, A, F, nullptr, 0), TS_EINVAL, "lora ld_b");
  expect(lora(4, 256, 64, 3, 16, 20, A, F, nullptr, 0), TS_EUNSUPPORTED, "lora ld_b%8");
  expect(lora(4, 256, 64, 3, 16, 16, nullptr, F, nullptr, 0), TS_EINVAL, "lora null b");
  expect(lora(4, 256, 64, 3, 16, 16, odd, F, nullptr, 0), TS_EUNSUPPORTED, "lora b align");
  expect(lora(4, 256, 64, 3, 16, 16, A, reinterpret_cast<float*>(odd), nullptr, 0),
         TS_EUNSUPPORTED, "lora logits align");
  expect(lora(4, 256, 64, 3, 16, 16, A, F, nullptr, 0), TS_EWORKSPACE, "lora no workspace");
  expect(lora(4, 256, 64, 3, 16, 16, A, F, A, 8), TS_EWORKSPACE, "lora small workspace");
  expect(lora(4, 256, 64, 3, 16, 16, A, F, A + 64, 1 << 30), TS_EUNSUPPORTED, "lora workspace align");
  expect(lora(64, 64, int64_t{1} << 30, 3, 8, 8, A, F, A, 1 << 30), TS_EUNSUPPORTED, "lora tiles");
  expect(lora(0, 256, 64, 3, 16, 16, nullptr, nullptr, nullptr, 0), TS_OK, "lora empty");
  expect(lora(4, 256, 0, 3, 16, 16, nullptr, nullptr, nullptr, 0), TS_OK, "lora no columns");
  if (lmhead_lora_workspace_bytes(-1, 8) != 0 ||
      lmhead_lora_workspace_bytes(4, TS_MAX_LORA_RANK + 1) != 0) {
    fprintf(stderr, "FAIL lora workspace of invalid sizes\n");
    ++failures;
  }
  size_t last = 0;
  for (int64_t rows : {1, 7, 640, 65536, TS_MAX_LORA_ROWS})
    for (int64_t rank : {8, 16, 24, TS_MAX_LORA_RANK}) {
      const size_t n = lmhead_lora_workspace_bytes(rows, rank);
      // three bf16 of every value of u, and the row's place and adapter
      if (n < static_cast<size_t>(rows * (6 * rank + 8)) || (rank > 8 && n < last)) {
        fprintf(stderr, "FAIL lora workspace %lld %lld: %zu\n", (long long)rows, (long long)rank, n);
        ++failures;
      }
      last = n;
    }

  // scoring
  expect(score(2, 4, 100, 100, A, 1.0, F, nullptr, 0), TS_EINVAL, "score type");
  expect(score(TS_F32, 4, 0, 100, A, 1.0, F, nullptr, 0), TS_EINVAL, "score vocab 0");
  expect(score(TS_F32, 4, 100, 99, A, 1.0, F, nullptr, 0), TS_EINVAL, "score ld");
  expect(score(TS_F32, int64_t{1} << 31, 100, 100, A, 1.0, F, nullptr, 0), TS_EUNSUPPORTED,
         "score rows");
  for (double t : {0.0, -1.0, static_cast<double>(INFINITY), static_cast<double>(NAN)})
    expect(score(TS_F32, 4, 100, 100, A, t, F, nullptr, 0), TS_EINVAL, "score temperature");
  expect(score(TS_F32, 4, 100, 100, odd, 1.0, F, nullptr, 0), TS_EUNSUPPORTED, "score align");
  expect(score(TS_BF16, 4, 100, 100, odd, 1.0, F, nullptr, 0), TS_EWORKSPACE, "score bf16 align");
  expect(score(TS_F32, 4, 100, 100, A, 1.0, nullptr, nullptr, 0), TS_EINVAL, "score null");
  expect(score(TS_F32, 4, 100, 100, A, 1.0, F, A, 8), TS_EWORKSPACE, "score small workspace");
  expect(score(TS_F32, 0, 100, 100, nullptr, 1.0, nullptr, nullptr, 0), TS_OK, "score empty");
  for (const void* lp : {static_cast<const void*>(nullptr), static_cast<const void*>(odd)}) {
    const float* kept = static_cast<const float*>(lp);
    expect(token_logprobs_backward_ex(A, TS_F32, 4, 100, 100, I, 1.0, F, kept, F, nullptr, nullptr,
                                      A + 400, 100, nullptr),
           kept ? TS_EUNSUPPORTED : TS_EINVAL, "backward overlap, logprobs align");
  }
  expect(token_logprobs_backward(A, TS_F32, 4, 100, 100, I, 1.0, F, F, nullptr, F, A, 100, nullptr),
         TS_EINVAL, "backward no entropies");
  expect(token_logprobs_backward(nullptr, TS_F32, 0, 100, 100, nullptr, 1.0, nullptr, nullptr,
                                 nullptr, nullptr, nullptr, 100, nullptr), TS_OK, "backward empty");

  // policy loss, and the gradient's place beside the logits' 4 rows of 100
  const ts_policy_params p{1.0, 0.2, 0.2, 0.0};
  for (const ts_policy_params& bad :
       {ts_policy_params{0.0, 0.2, 0.2, 0.0}, ts_policy_params{1.0, -0.1, 0.2, 0.0},
        ts_policy_params{1.0, 0.2, NAN, 0.0}, ts_policy_params{1.0, 0.2, 0.2, -1.0},
        ts_policy_params{1.0, 0.2, 0.2, 0.1}})
    expect(policy(4, 100, nullptr, 0, &bad, nullptr, F), TS_EINVAL, "policy params");
  expect(policy(4, 100, nullptr, 0, nullptr, nullptr, F), TS_EINVAL, "policy null params");
  expect(policy(4, 100, nullptr, 0, &p, nullptr, nullptr), TS_EINVAL, "policy null loss");
  for (int64_t at = -1000; at <= 1000; ++at) {
    // entries from the logits' first one; in its place, or with no entry shared
    const int64_t one = 100, four = 3 * 250 + 100;
    int64_t gap = at % 250;
    if (gap < 0) gap += 250;
    const bool apart = at >= four || at <= -four;
    expect(policy(4, 250, A + 4 * at, 250, &p, nullptr, F),
           at == 0 || apart || (gap >= 100 && gap <= 150) ? TS_EWORKSPACE : TS_EINVAL,
           "policy beside, same stride");
    expect(policy(4, 250, A + 4 * at, 249, &p, nullptr, F),
           at >= four || at <= -(3 * 249 + 100) ? TS_EWORKSPACE : TS_EINVAL,
           "policy beside, other stride");
    expect(policy(1, 250, A + 4 * at, 249, &p, nullptr, F),
           at == 0 || at >= one || at <= -one ? TS_EWORKSPACE : TS_EINVAL, "policy one row");
  }
  expect(policy(4, 100, A + 4000, 99, &p, nullptr, F), TS_EINVAL, "policy ld_grad");
  expect(policy(4, 100, A + 4002, 100, &p, nullptr, F), TS_EUNSUPPORTED, "policy grad align");

  // preference loss
  const ts_preference_params q{1.0, 0.1, 0.0, 0.0, 0};
  for (const ts_preference_params& bad :
       {ts_preference_params{0.0, 0.1, 0.0, 0.0, 0}, ts_preference_params{1.0, 0.0, 0.0, 0.0, 0},
        ts_preference_params{1.0, 0.1, 1.5, 0.0, 0}, ts_preference_params{1.0, 0.1, 0.0, NAN, 0},
        ts_preference_params{1.0, 0.1, 0.0, 0.0, 2}})
    expect(preference(4, I, 1, &bad, nullptr), TS_EINVAL, "preference params");
  expect(preference(4, I, 1, nullptr, nullptr), TS_EINVAL, "preference null params");
  expect(preference(4, nullptr, 1, &q, nullptr), TS_EINVAL, "preference null offsets");
  expect(preference(4, I, -1, &q, nullptr), TS_EINVAL, "preference pairs<0");
  expect(preference(4, I, int64_t{1} << 30, &q, nullptr), TS_EUNSUPPORTED, "preference pairs");
  expect(preference(4, I, 1, &q, reinterpret_cast<float*>(odd)), TS_EUNSUPPORTED,
         "preference align");
  expect(preference(4, I, 1, &q, nullptr), TS_EWORKSPACE, "preference no workspace");
  expect(preference(0, I, 1, &q, nullptr), TS_EWORKSPACE, "preference no rows, no workspace");

  // a record of 24, one of 16 and a term of 8 bytes a row at least
  for (int64_t rows : {int64_t{0}, int64_t{1}, int64_t{640}, int64_t{1} << 20, (int64_t{1} << 31) - 1})
    for (int64_t vocab : {int64_t{1}, int64_t{4097}, int64_t{151936}, (int64_t{1} << 31) - 1})
      for (int64_t pairs : {int64_t{0}, int64_t{3}, (int64_t{1} << 30) - 1})
        if (token_logprobs_workspace_bytes(rows, vocab) < static_cast<size_t>(rows) * 48 ||
            preference_loss_workspace_bytes(rows, vocab, pairs) <
                static_cast<size_t>(rows) * 48 + static_cast<size_t>(pairs) * 8) {
          fprintf(stderr, "FAIL workspace %lld %lld %lld\n", (long long)rows, (long long)vocab,
                  (long long)pairs);
          ++failures;
        }
  if (token_logprobs_workspace_bytes(-1, 10) != 0 ||
      preference_loss_workspace_bytes(4, 10, int64_t{1} << 30) != 0) {
    fprintf(stderr, "FAIL workspace of invalid sizes\n");
    ++failures;
  }

  printf("losses_driver: %d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
