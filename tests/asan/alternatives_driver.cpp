// Host-side driver of the argument checks of the 4-bit rows, scoring with
// alternatives and the listed tokens, built with AddressSanitizer on the host code
// like losses_driver.cpp: every call is rejected, or is a no-op, before any HIP call.
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

static int quantize(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ld,
                    void* codes, int64_t ldc, void* scales, int64_t lds) {
  const int a = quantize_groups_e2m1(x, type, rows, cols, ld, codes, ldc, scales, lds, nullptr);
  const int b = dequantize_groups_e2m1(codes, rows, cols, ldc, scales, lds, const_cast<void*>(x),
                                       type, ld, nullptr);
  return a == b ? a : -1000;  // both sides refuse the same
}

static int project(int64_t rows, int64_t hidden, int64_t ldh, const void* head, int64_t vocab,
                   int64_t ldw, int64_t lds, float* out, int64_t ldo) {
  return lmhead_logits_local_e2m1(A, rows, hidden, ldh, head, A, vocab, ldw, lds, out, ldo,
                                  nullptr);
}

static int topn(int64_t rows, int64_t vocab, int64_t ld, const int32_t* tokens, int32_t n,
                float* lp, int32_t* ranks, int32_t* ids, float* top, void* ws, size_t bytes) {
  return token_logprobs_topn(A, TS_F32, rows, vocab, ld, tokens, 1.0, n, lp, ranks, nullptr, ids,
                             top, nullptr, nullptr, ws, bytes, nullptr);
}

static int listed(int64_t rows, int64_t vocab, const int32_t* ids, int32_t n, double temperature,
                  float* lp, void* ws, size_t bytes) {
  return token_logprobs_listed(A, TS_BF16, rows, vocab, vocab, ids, n, temperature, lp, nullptr,
                               nullptr, nullptr, ws, bytes, nullptr);
}

static int listed_backward(int32_t n, const float* lp, const float* entropies,
                           const float* grad_entropies, void* grad, int64_t ld_grad) {
  return token_logprobs_listed_backward(A, TS_F32, 4, 100, 100, I, n, 1.0, F, lp, F, entropies,
                                        grad_entropies, grad, ld_grad, nullptr);
}

int main() {
  char* const odd = A + 2;
  float* const odd_f = reinterpret_cast<float*>(odd + 1);

  // rows in groups
  expect(quantize(A, TS_F32, -1, 64, 64, A, 32, A, 2), TS_EINVAL, "rows<0");
  expect(quantize(A, TS_F32, 4, -32, 64, A, 32, A, 2), TS_EINVAL, "cols<0");
  expect(quantize(A, 7, 4, 64, 64, A, 32, A, 2), TS_EINVAL, "type");
  expect(quantize(A, TS_F32, 4, 48, 64, A, 32, A, 2), TS_EUNSUPPORTED, "cols%32");
  expect(quantize(A, TS_F32, int64_t{1} << 31, 64, 64, A, 32, A, 2), TS_EUNSUPPORTED, "rows");
  expect(quantize(A, TS_F32, 4, 64, 63, A, 32, A, 2), TS_EINVAL, "ld");
  expect(quantize(A, TS_F32, 4, 64, 64, A, 28, A, 2), TS_EINVAL, "ld codes");
  expect(quantize(A, TS_F32, 4, 64, 64, A, 34, A, 2), TS_EUNSUPPORTED, "ld codes%4");
  expect(quantize(A, TS_F32, 4, 64, 64, A, 32, A, 1), TS_EINVAL, "ld scales");
  expect(quantize(nullptr, TS_F32, 4, 64, 64, A, 32, A, 2), TS_EINVAL, "null values");
  expect(quantize(A, TS_F32, 4, 64, 64, nullptr, 32, A, 2), TS_EINVAL, "null codes");
  expect(quantize(A, TS_F32, 4, 64, 64, A, 32, nullptr, 2), TS_EINVAL, "null scales");
  expect(quantize(odd, TS_F32, 4, 64, 64, A, 32, A, 2), TS_EUNSUPPORTED, "values align");
  expect(quantize(A, TS_BF16, 4, 64, 64, odd, 32, A, 2), TS_EUNSUPPORTED, "codes align");
  expect(quantize(nullptr, TS_F32, 0, 64, 64, nullptr, 32, nullptr, 2), TS_OK, "no rows");
  expect(quantize(nullptr, TS_BF16, 4, 0, 0, nullptr, 0, nullptr, 0), TS_OK, "no columns");

  // projection
  expect(project(-1, 64, 64, A, 10, 32, 2, F, 10), TS_EINVAL, "project rows<0");
  expect(project(4, 0, 64, A, 10, 32, 2, F, 10), TS_EINVAL, "project hidden 0");
  expect(project(4, 48, 64, A, 10, 32, 2, F, 10), TS_EUNSUPPORTED, "project hidden%32");
  expect(project(4, 64, 56, A, 10, 32, 2, F, 10), TS_EINVAL, "project ld_hidden");
  expect(project(4, 64, 68, A, 10, 32, 2, F, 10), TS_EUNSUPPORTED, "project ld_hidden%8");
  expect(project(4, 64, (int64_t{1} << 21) + 8, A, 10, 32, 2, F, 10), TS_EUNSUPPORTED,
         "project wide ld_hidden");
  expect(project(4, 64, 64, A, 10, 40, 2, F, 10), TS_EUNSUPPORTED, "project ld_lm_head%16");
  expect(project(4, 64, 64, A, 10, 32, 1, F, 10), TS_EINVAL, "project ld_scales");
  expect(project(4, 64, 64, A, 10, 32, 2, F, 9), TS_EINVAL, "project ld_logits");
  expect(project(4, 64, 64, odd, 10, 32, 2, F, 10), TS_EUNSUPPORTED, "project align");
  expect(project(4, 64, 64, A, 10, 32, 2, odd_f, 10), TS_EUNSUPPORTED, "project logits align");
  expect(project(4, 64, 64, nullptr, 10, 32, 2, F, 10), TS_EINVAL, "project null");
  expect(project(0x7fffffff, 64, 64, A, 0x7fffffff, 32, 2, F, 0x7fffffff), TS_EUNSUPPORTED,
         "project tiles");
  expect(project(0, 64, 64, nullptr, 10, 32, 2, nullptr, 10), TS_OK, "project no rows");
  expect(project(4, 64, 64, nullptr, 0, 32, 2, nullptr, 0), TS_OK, "project no columns");

  // alternatives
  expect(topn(4, 0, 100, I, 5, F, I, I, F, nullptr, 0), TS_EINVAL, "topn vocab 0");
  expect(topn(4, 100, 99, I, 5, F, I, I, F, nullptr, 0), TS_EINVAL, "topn ld");
  expect(topn(4, 100, 100, I, -1, F, I, I, F, nullptr, 0), TS_EINVAL, "topn n<0");
  expect(topn(4, 100, 100, I, TS_MAX_LOGPROBS + 1, F, I, I, F, nullptr, 0), TS_EUNSUPPORTED,
         "topn n");
  expect(topn(4, 100, 100, I, 5, nullptr, I, I, F, nullptr, 0), TS_EINVAL, "topn no logprobs");
  expect(topn(4, 100, 100, nullptr, 5, F, nullptr, I, F, nullptr, 0), TS_EINVAL,
         "topn logprobs of no token");
  expect(topn(4, 100, 100, nullptr, 5, nullptr, I, I, F, nullptr, 0), TS_EINVAL,
         "topn ranks of no token");
  expect(topn(4, 100, 100, I, 5, F, I, nullptr, F, nullptr, 0), TS_EINVAL, "topn no ids");
  expect(topn(4, 100, 100, I, 5, F, I, I, odd_f, nullptr, 0), TS_EUNSUPPORTED, "topn align");
  expect(topn(4, 100, 100, I, 5, F, I, I, F, nullptr, 0), TS_EWORKSPACE, "topn no workspace");
  expect(topn(4, 100, 100, nullptr, 0, nullptr, nullptr, nullptr, nullptr, A, 8), TS_EWORKSPACE,
         "topn small workspace");
  expect(topn(0, 100, 100, I, 5, nullptr, nullptr, nullptr, nullptr, nullptr, 0), TS_OK,
         "topn no rows");

  // listed tokens
  expect(listed(4, 100, I, 0, 1.0, F, nullptr, 0), TS_EINVAL, "listed 0");
  expect(listed(4, 100, I, TS_MAX_LISTED + 1, 1.0, F, nullptr, 0), TS_EUNSUPPORTED, "listed n");
  expect(listed(4, 100, nullptr, 3, 1.0, F, nullptr, 0), TS_EINVAL, "listed null ids");
  expect(listed(4, 100, I, 3, 0.0, F, nullptr, 0), TS_EINVAL, "listed temperature");
  expect(listed(4, 100, I, 3, NAN, F, nullptr, 0), TS_EINVAL, "listed NaN temperature");
  expect(listed(4, 100, I, 3, 1.0, nullptr, nullptr, 0), TS_EINVAL, "listed null logprobs");
  expect(listed(4, 100, I, 3, 1.0, odd_f, nullptr, 0), TS_EUNSUPPORTED, "listed align");
  expect(listed(4, 100, I, 3, 1.0, F, A, 8), TS_EWORKSPACE, "listed small workspace");
  expect(listed(0, 100, nullptr, 3, 1.0, nullptr, nullptr, 0), TS_OK, "listed no rows");
  expect(listed_backward(0, F, nullptr, nullptr, A, 100), TS_EINVAL, "backward 0");
  expect(listed_backward(3, nullptr, nullptr, nullptr, A, 100), TS_EINVAL,
         "backward null logprobs");
  expect(listed_backward(3, F, nullptr, F, A, 100), TS_EINVAL, "backward no entropies");
  expect(listed_backward(3, F, nullptr, nullptr, nullptr, 100), TS_EINVAL, "backward null grad");
  expect(listed_backward(3, F, nullptr, nullptr, A, 99), TS_EINVAL, "backward ld_grad");
  expect(listed_backward(3, F, nullptr, nullptr, A + 400, 100), TS_EINVAL, "backward overlap");
  expect(listed_backward(3, odd_f, nullptr, nullptr, A, 100), TS_EUNSUPPORTED, "backward align");

  // a record of 24 and a count of 4 bytes a row, and an entry of its groups
  for (int64_t rows :
       {int64_t{0}, int64_t{1}, int64_t{640}, int64_t{1} << 20, (int64_t{1} << 31) - 1})
    for (int64_t vocab : {int64_t{1}, int64_t{4097}, int64_t{151936}, (int64_t{1} << 31) - 1}) {
      const size_t least = static_cast<size_t>(rows) * (28 + 4 * (vocab / 32));
      if (token_logprobs_topn_workspace_bytes(rows, vocab) < least ||
          token_logprobs_listed_workspace_bytes(rows, vocab) < static_cast<size_t>(rows) * 24) {
        fprintf(stderr, "FAIL workspace %lld %lld\n", (long long)rows, (long long)vocab);
        ++failures;
      }
    }
  if (token_logprobs_topn_workspace_bytes(-1, 10) != 0 ||
      token_logprobs_listed_workspace_bytes(4, int64_t{1} << 31) != 0) {
    fprintf(stderr, "FAIL workspace of invalid sizes\n");
    ++failures;
  }

  printf("alternatives_driver: %d failures\n", failures);
  return failures == 0 ? 0 : 1;
}
