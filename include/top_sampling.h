/*
 * top_sampling.h -- C ABI of the MI355X (gfx950) batch-sharded sampling path.
 *
 * One tensor-parallel rank's share of batch-sharded sampling, as described on
 * the page "Qwen4Exp batch-sharded sampling: inside vLLM PR #61018"
 * (orcarouter.ai blog, ja/nl/fr editions):
 *
 *   1. lmhead_logits_local       -- the rank's own vocabulary slice of the
 *      projection, with no gather (sections "What batch-sharded sampling is,
 *      in one paragraph" and "Why three lines were the whole job": the
 *      model's local-logits hook hands back only the rank's vocabulary shard);
 *   2. sampler_assemble_vocab_slices -- the receive side of the all-to-all:
 *      vocabulary slices from every rank stitched into full-vocabulary rows
 *      for the rank's slice of requests (section "What batch-sharded sampling
 *      is, in one paragraph");
 *   3. sampler_sample            -- the per-row sampler over
 *      batch x (speculative tokens + 1) rows: temperature, top-k, top-p,
 *      log-probabilities and seeded sampling (same section; the page names
 *      top-k, top-p and a non-negative max_logprobs, not their arithmetic);
 *   2+3. sampler_assemble_and_sample -- both in one call that reads the
 *      received logits once.
 *
 * Conventions shared by every call
 *   - All pointers to bulk data are DEVICE pointers unless stated otherwise.
 *     The caller owns every buffer; the library never allocates device
 *     memory, never synchronises the host and never prints.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Work is enqueued asynchronously on it.
 *   - A nonzero return value means argument validation failed and NOTHING was
 *     enqueued: invalid configurations are rejected up front rather than
 *     degraded silently.  This follows the fail-fast convention of the
 *     sequence-parallel patch described on the page "Qwen 4 leak: SGLang
 *     shards the Qwen4Exp prefill" (orcarouter.ai blog, ja edition), section
 *     "The cost to you: constraints": unsupported configurations fail during
 *     argument validation.  ts_last_error() then describes the failure for
 *     the calling thread.  TS_EHIP reports a failed kernel launch.
 *   - The preconditions batch-sharded sampling states (page "Qwen4Exp
 *     batch-sharded sampling: inside vLLM PR #61018", section "What
 *     batch-sharded sampling is, in one paragraph") include a non-negative
 *     max_logprobs: max_logprobs < 0 is TS_EINVAL in every sampler call.
 *   - Measurement and check aids that are not steps of the path (clock
 *     probe, noise readout) are declared in top_sampling_measure.h.
 *   - Sizes of zero are valid no-ops.
 *   - Matrices are row-major with an explicit leading dimension (elements).
 */
#ifndef TOP_SAMPLING_H_
#define TOP_SAMPLING_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
enum {
  TS_OK = 0,
  TS_EINVAL = -1,        /* bad sizes, leading dimensions or NULL pointers     */
  TS_EUNSUPPORTED = -2,  /* valid but outside what the kernels take (alignment,
                            limits such as TS_MAX_LOGPROBS)                    */
  TS_EWORKSPACE = -3,    /* workspace NULL or smaller than required            */
  TS_EHIP = -4           /* the HIP runtime rejected a launch                  */
};

/* Per-row status written by sampler_sample. */
enum {
  TS_ROW_OK = 0,
  TS_ROW_BAD_PARAMS = 1,  /* temperature < 0 or not finite; top_k < 0;
                             top_p not in (0, 1]; n_logprobs not in
                             [0, max_logprobs]                               */
  TS_ROW_BAD_LOGITS = 2   /* a NaN or +inf logit, or no finite logit          */
};

/* Element types of logits and of rows to be quantized. */
enum { TS_F32 = 0, TS_BF16 = 1 };

#define TS_MAX_LOGPROBS 1024   /* largest accepted max_logprobs              */
#define TS_MAX_SLICES 64       /* largest accepted n_slices                  */
#define TS_GREEDY_EPS 1e-6f    /* temperatures below this sample greedily    */
/* sampler_sample_ex flags */
#define TS_LOGPROBS_PROCESSED 1 /* log-probabilities of the sampled distribution */

/*
 * Sampling parameters of one row (24 bytes, 8-byte aligned; an array of
 * `rows` of them lives in device memory).
 *   temperature  0 (or < TS_GREEDY_EPS): greedy argmax of the raw logits.
 *   top_k        0 or >= vocab: no top-k filter; 1: greedy.  Every token
 *                tied with the k-th largest logit is kept.
 *   top_p        1: no top-p filter.  Otherwise the smallest set of most
 *                likely tokens (of the temperature-scaled distribution
 *                renormalised over the top-k set) whose mass reaches top_p;
 *                the crossing token and its ties are kept.
 *   n_logprobs   how many of the row's largest logits to report (<= the
 *                call's max_logprobs).
 *   seed         RNG key of the row.  Sampling is Gumbel-max:
 *                token = argmax over kept v of (l_v - max l) / T + g_v,
 *                g_v = -ln(-ln u_v), u_v = ((x >> 9) + 1/2) * 2^-23 where x
 *                is word (v & 3) of Philox4x32-10 with key (seed lo32,
 *                seed hi32) and counter (v >> 2, row lo32, row hi32, 0),
 *                row = row_offset + local row (Salmon et al., "Parallel
 *                Random Numbers: As Easy as 1, 2, 3", SC'11).  Lowest id
 *                wins exact ties.
 */
typedef struct ts_row_params {
  float temperature;
  int32_t top_k;
  float top_p;
  int32_t n_logprobs;
  uint64_t seed;
} ts_row_params;

/*
 * lmhead_logits_local: logits[r, v] = sum_h hidden[r, h] * lm_head[v, h].
 *
 * The rank's local vocabulary projection: only the slice of the vocabulary
 * this rank holds (vocab_local rows of lm_head), never gathered.
 *   hidden     bf16 [rows, hidden_dim], leading dimension ld_hidden
 *   lm_head    bf16 [vocab_local, hidden_dim], leading dimension ld_lm_head
 *              (both K-contiguous)
 *   logits     fp32 [rows, vocab_local] written with leading dimension
 *              ld_logits >= vocab_local, so a slice can be written straight
 *              into a wider buffer.
 * Products of bf16 are exact in fp32; accumulation is fp32 (MFMA).
 * Requirements (else TS_EUNSUPPORTED): hidden_dim % 8 == 0, ld_hidden and
 * ld_lm_head multiples of 8, hidden and lm_head 16-byte aligned, logits
 * 4-byte aligned.  rows, vocab_local < 2^31.
 */
int lmhead_logits_local(const void* hidden, int64_t rows, int64_t hidden_dim,
                        int64_t ld_hidden, const void* lm_head, int64_t vocab_local,
                        int64_t ld_lm_head, float* logits, int64_t ld_logits,
                        void* stream);

/*
 * lmhead_logits_local_lora: lmhead_logits_local for rows that each have their
 * own low-rank adapter:
 *   logits[r, v] = sum_h hidden[r, h] lm_head[v, h]
 *                + adapter_scales[a] sum_k lora_b[a][v, k]
 *                                    (sum_h hidden[r, h] lora_a[a][k, h]),
 *   a = adapter_ids[r].
 * One call serves the requests of a batch whatever adapters they have; rows
 * need no order.  A row of adapter -1 has none and gets exactly what
 * lmhead_logits_local gives.  A row whose id is below -1 or >= n_adapters gets
 * a row of NaN, which the sampler reports as TS_ROW_BAD_LOGITS.  A row only
 * depends on its own adapter: infinities or NaN in another one's weights do
 * not reach it.
 *   lora_a   bf16 [n_adapters][rank, hidden_dim]: adapter a at lora_a +
 *            a * stride_a, leading dimension ld_a
 *   lora_b   bf16 [n_adapters][vocab_local, rank]: this rank's vocabulary
 *            slice of every adapter, adapter a at lora_b + a * stride_b,
 *            leading dimension ld_b
 *   adapter_scales  fp32 [n_adapters], or NULL for 1
 *   adapter_ids     int32 [rows]
 *   workspace       as for sampler_sample; lmhead_lora_workspace_bytes
 * Adapters of several ranks are padded with zeros to the largest.  Products
 * and sums are fp32; the inner sums are not rounded to bf16.
 * Requirements (else TS_EUNSUPPORTED): those of lmhead_logits_local, rank a
 * multiple of 8 up to TS_MAX_LORA_RANK, rows up to TS_MAX_LORA_ROWS, ld_a, ld_b
 * and the strides multiples of 8, lora_a and lora_b 16-byte aligned, no more
 * logits than one launch has tiles for (hidden_dim % 64 == 0: 2^30 - 1024
 * columns for up to 64 rows, and 2^23 - 8 tiles of 128 x 128 for more; other
 * sizes: 2^24 - 8 tiles of up to 256 x 256, and 2^31 - 257 columns).
 * n_adapters == 0 or rank == 0 is TS_EINVAL.
 */
#define TS_MAX_LORA_RANK 256       /* largest accepted adapter rank          */
#define TS_MAX_LORA_ROWS 1048576   /* largest accepted row count (the rows
                                      are put in order by comparison)        */
size_t lmhead_lora_workspace_bytes(int64_t rows, int64_t rank);
int lmhead_logits_local_lora(const void* hidden, int64_t rows, int64_t hidden_dim,
                             int64_t ld_hidden, const void* lm_head, int64_t vocab_local,
                             int64_t ld_lm_head, const void* lora_a, int64_t stride_a,
                             int64_t ld_a, const void* lora_b, int64_t stride_b, int64_t ld_b,
                             int64_t n_adapters, int64_t rank, const float* adapter_scales,
                             const int32_t* adapter_ids, float* logits, int64_t ld_logits,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * FP8 projection.  The pages' measured deployment is an FP8 checkpoint and
 * their patch cluster unpacks e4m3 bytes (sections "The 1.5% estimate, and
 * the measurement next to it" and "The patch cluster"); they state no
 * scaling scheme.  Reading: W8A8 with one fp32 scale per row on both
 * operands.  A row x is held as OCP E4M3 codes q (one byte each; no
 * infinities, largest magnitude 448, 0x7F/0xFF NaN) with x ~ s * dec(q),
 * s = max|x| / 448.
 *
 * quantize_rows_e4m3: per-row dynamic quantization of bf16 data:
 *   scales[r] = max_c |in[r, c]| / 448 in fp32 (NaN ignored; 1 for a row
 *   of zeros); out[r, c] = the E4M3 code nearest in[r, c] / scales[r]
 *   (quotient in fp32), ties to the even code, saturating at +-448, NaN ->
 *   0x7F.
 *   in      bf16 [rows, cols], leading dimension ld_in (elements)
 *   out     codes [rows, cols], leading dimension ld_out (bytes)
 *   scales  fp32 [rows]
 * Caller-owned device buffers; in 2-byte and scales 4-byte aligned.
 *
 * lmhead_logits_local_e4m3: logits[r, v] = hidden_scales[r] *
 *   lm_head_scales[v] * sum_h dec(hidden[r, h]) * dec(lm_head[v, h]),
 *   fp32 accumulation (every product of two E4M3 values is exact in fp32),
 *   over the rank's own vocabulary slice, never gathered.
 *   hidden          codes [rows, hidden_dim], leading dimension ld_hidden
 *   hidden_scales   fp32 [rows]
 *   lm_head         codes [vocab_local, hidden_dim], leading dimension ld_lm_head
 *   lm_head_scales  fp32 [vocab_local]
 *   logits          fp32 [rows, vocab_local], leading dimension ld_logits
 * Requirements (else TS_EUNSUPPORTED): hidden_dim a multiple of 128,
 * ld_hidden and ld_lm_head multiples of 16, codes 16-byte aligned, logits
 * and scales 4-byte aligned.  Other errors and the empty cases as for
 * lmhead_logits_local.
 */
int quantize_rows_e4m3(const void* in, int64_t rows, int64_t cols, int64_t ld_in, void* out,
                       int64_t ld_out, float* scales, void* stream);
int lmhead_logits_local_e4m3(const void* hidden, const float* hidden_scales, int64_t rows,
                             int64_t hidden_dim, int64_t ld_hidden, const void* lm_head,
                             const float* lm_head_scales, int64_t vocab_local, int64_t ld_lm_head,
                             float* logits, int64_t ld_logits, void* stream);

/*
 * 4-bit projection.  Rows are held as OCP MX FP4 (Open Compute Project
 * Microscaling Formats 1.0): every 32 consecutive entries of a row are a group
 * with one scale s = 2^e, held as the byte e + 127 (E8M0; 255 is NaN), and every
 * entry is an E2M1 code (bit 3 the sign; 0, 0.5, 1, 1.5, 2, 3, 4, 6), two codes
 * a byte with the even column's in the low half: 4.25 bits an entry.  The entry
 * stands for s times its code's value.  type TS_F32 or TS_BF16.
 *
 * quantize_groups_e2m1: for each group
 *   e = the least integer >= -127 with max|x| <= 7 * 2^e (values above 6 s, the
 *   largest, lose at most the half step below it), 0 for a group of zeros, and
 *   125 at most, so that a finite x stands as a finite value;
 *   code = the value nearest x / s, ties to the even code, the sign x's.  A group
 *   with a NaN or an infinity gets the scale byte 255 and codes 0.
 *   in      [rows, cols] of in_type, leading dimension ld_in (elements)
 *   codes   [rows, cols / 2] bytes, leading dimension ld_codes (bytes)
 *   scales  [rows, cols / 32] bytes, leading dimension ld_scales (bytes)
 * dequantize_groups_e2m1: the values the codes stand for, in out_type; both types
 *   hold them exactly, but for those past the largest number, which are infinite.
 *   A group of scale byte 255 gives NaN.
 * Requirements of both (else TS_EUNSUPPORTED): cols a multiple of 32, codes
 * 4-byte aligned and ld_codes a multiple of 4, values aligned to their type.
 * codes and scales must not overlap the values.
 *
 * lmhead_logits_local_e2m1: lmhead_logits_local with such an lm_head,
 *   logits[r, v] = sum_h hidden[r, h] * 2^e[v, h / 32] * q[v, h],
 *   over the rank's own vocabulary slice, never gathered.  hidden stays bf16;
 *   every product is exact in fp32 and sums are fp32.
 *   The entries 2^e q are those that dequantize_groups_e2m1 gives: past the largest
 *   number (scale bytes 253 and 254, which quantize_groups_e2m1 does not write) they
 *   are infinite, and 0 times them is NaN.
 *   hidden          bf16 [rows, hidden_dim], leading dimension ld_hidden
 *   lm_head         codes [vocab_local, hidden_dim / 2], leading dimension
 *                   ld_lm_head (bytes)
 *   lm_head_scales  [vocab_local, hidden_dim / 32], leading dimension ld_scales
 *                   (bytes), any alignment
 *   logits          fp32 [rows, vocab_local], leading dimension ld_logits
 * Requirements (else TS_EUNSUPPORTED): hidden_dim a multiple of 32, ld_hidden of
 * 8 and up to 2^21, ld_lm_head of 16, hidden and lm_head 16-byte aligned, logits 4-byte aligned,
 * vocab_local up to 2^31 - 1024, and no more than 2^22 - 1 tiles of 64 x 256
 * logits.  Other errors and the empty cases as for lmhead_logits_local.
 */
int quantize_groups_e2m1(const void* in, int32_t in_type, int64_t rows, int64_t cols,
                         int64_t ld_in, void* codes, int64_t ld_codes, void* scales,
                         int64_t ld_scales, void* stream);
int dequantize_groups_e2m1(const void* codes, int64_t rows, int64_t cols, int64_t ld_codes,
                           const void* scales, int64_t ld_scales, void* out, int32_t out_type,
                           int64_t ld_out, void* stream);
int lmhead_logits_local_e2m1(const void* hidden, int64_t rows, int64_t hidden_dim,
                             int64_t ld_hidden, const void* lm_head, const void* lm_head_scales,
                             int64_t vocab_local, int64_t ld_lm_head, int64_t ld_scales,
                             float* logits, int64_t ld_logits, void* stream);

/*
 * sampler_workspace_bytes: device workspace sampler_sample needs for these
 * sizes (host-only computation; callable without a GPU).  The caller owns
 * the workspace, as every other buffer: serving replays fixed graph buckets
 * (page "Qwen 4 leak: SGLang shards the Qwen4Exp prefill", section "The
 * layout bug they had to fix first": fixed physical CUDA-graph buckets), so
 * the library allocates nothing per call and the caller sizes each bucket's
 * workspace once from this query.  Returns 0 for negative sizes or
 * max_logprobs < 0 (the non-negative max_logprobs precondition of page
 * "Qwen4Exp batch-sharded sampling: inside vLLM PR #61018", section "What
 * batch-sharded sampling is, in one paragraph").
 */
size_t sampler_workspace_bytes(int64_t rows, int64_t vocab, int32_t max_logprobs);

/*
 * sampler_sample: sample one token per row and report log-probabilities.
 *   logits          fp32 [rows, vocab], leading dimension ld_logits; read only.
 *   params          device array of `rows` ts_row_params.
 *   row_offset      global index of local row 0 (keys the RNG, so a rank's
 *                   share of rows draws exactly what the unsharded call would).
 *   max_logprobs    0..TS_MAX_LOGPROBS: width of the top-N outputs.
 *   token_ids       int32 [rows]: sampled token, -1 for a row whose status != 0.
 *   token_logprobs  fp32 [rows] or NULL: raw log_softmax of the sampled token
 *                   (NaN for a bad row).
 *   topn_ids        int32 [rows, max_logprobs] (may be NULL iff max_logprobs
 *                   == 0): the row's n_logprobs largest logits, largest first,
 *                   lower id first on ties; unused slots -1.
 *   topn_logprobs   fp32 [rows, max_logprobs]: their raw log-probabilities;
 *                   unused slots -inf; NaN for a bad row.
 *   row_status      int32 [rows] or NULL: TS_ROW_* per row.
 *   workspace       device scratch of at least sampler_workspace_bytes(...)
 *                   bytes, 256-byte aligned; contents need no initialisation
 *                   and are clobbered.
 * Log-probabilities describe the raw distribution log_softmax(logits)
 * (unscaled, unfiltered).  Calls that share a workspace must be ordered on
 * one stream.  vocab < 2^31.
 */
int sampler_sample(const float* logits, int64_t rows, int64_t vocab, int64_t ld_logits,
                   const ts_row_params* params, int64_t row_offset, int32_t max_logprobs,
                   int32_t* token_ids, float* token_logprobs, int32_t* topn_ids,
                   float* topn_logprobs, int32_t* row_status, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * sampler_sample_noalloc: sampler_sample for callers that cannot allocate --
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, outputs and results as sampler_sample, without
 * the workspace: the library keeps a file-scope device array of
 * TS_NOALLOC_SCRATCH_BYTES per GPU (placed when the runtime loads the
 * library on that GPU, held until the process ends) and uses it as the
 * workspace.  The call allocates and frees nothing.
 *   - TS_EUNSUPPORTED if sampler_workspace_bytes(rows, vocab, max_logprobs)
 *     exceeds TS_NOALLOC_SCRATCH_BYTES (e.g. 640 x 151,936 x 20 needs about
 *     43 MB and fits; use sampler_sample with a caller workspace beyond it).
 *   - Every call on a GPU shares that GPU's array: calls that overlap on one
 *     GPU (different streams, or different host threads) race and must be
 *     serialised by the caller.  The array needs no clearing between calls.
 *   - TS_EHIP if no HIP device is current or the array's device address
 *     cannot be obtained.
 */
#define TS_NOALLOC_SCRATCH_BYTES (96ull << 20)
int sampler_sample_noalloc(const float* logits, int64_t rows, int64_t vocab, int64_t ld_logits,
                           const ts_row_params* params, int64_t row_offset, int32_t max_logprobs,
                           int32_t* token_ids, float* token_logprobs, int32_t* topn_ids,
                           float* topn_logprobs, int32_t* row_status, void* stream);

/*
 * sampler_workspace_bytes_slices: device workspace sampler_sample_slices
 * needs (host-only computation).  slice_cols is a HOST array of n_slices
 * entries.
 */
size_t sampler_workspace_bytes_slices(int64_t rows, const int64_t* slice_cols, int32_t n_slices,
                                      int32_t max_logprobs);

/*
 * sampler_sample_slices: sampler_sample over a rank's batch slice that is
 * still held as the vocabulary slices the exchange delivered, without
 * stitching them into one buffer first (the step after the all-to-all on
 * the page "Qwen4Exp batch-sharded sampling: inside vLLM PR #61018", section
 * "What batch-sharded sampling is, in one paragraph": each rank receives the
 * vocabulary slices of its requests).  Global column off_s + c of row r is
 * slices[s][r * slice_ld[s] + c], off_s = slice_cols[0] + ... +
 * slice_cols[s-1]; vocab = the sum of slice_cols.
 *   slices      HOST array of n_slices DEVICE pointers (fp32, read only)
 *   slice_cols, slice_ld   HOST arrays of n_slices entries
 * Every other argument, output and the results are those of sampler_sample
 * on the stitched [rows, vocab] buffer; the workspace is sized by
 * sampler_workspace_bytes_slices.  1 <= n_slices <= TS_MAX_SLICES.  Slices
 * that start at a column not a multiple of 4 take the exact per-row kernel
 * (same results, slower).
 */
int sampler_sample_slices(const float* const* slices, const int64_t* slice_cols,
                          const int64_t* slice_ld, int32_t n_slices, int64_t rows,
                          const ts_row_params* params, int64_t row_offset, int32_t max_logprobs,
                          int32_t* token_ids, float* token_logprobs, int32_t* topn_ids,
                          float* topn_logprobs, int32_t* row_status, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * sampler_sample_ex: sampler_sample_slices with a flags word (0 gives
 * sampler_sample_slices exactly; sampler_sample is the one-slice case).
 *   TS_LOGPROBS_PROCESSED  token_logprobs and topn_logprobs describe the
 *       distribution the token is drawn from instead of the raw
 *       log_softmax(logits): (l - m)/T - ln(sum over the kept set of
 *       exp((l - m)/T)) for tokens the filters keep, -inf for the others; a
 *       greedy row is a point mass (0 for the chosen token, -inf for the
 *       rest).  top-N lists the same ids as the raw mode (the N largest
 *       logits).  The pages ask only for a non-negative max_logprobs
 *       (section "What batch-sharded sampling is, in one paragraph"); this
 *       is the processed variant of the same output.  Top-p-only rows whose
 *       nucleus reaches below the listed candidates take the exact per-row
 *       kernel in this mode.
 * Other flag bits: TS_EINVAL.  Workspace: sampler_workspace_bytes_slices.
 */
int sampler_sample_ex(const float* const* slices, const int64_t* slice_cols,
                      const int64_t* slice_ld, int32_t n_slices, int64_t rows,
                      const ts_row_params* params, int64_t row_offset, int32_t max_logprobs,
                      int32_t flags, int32_t* token_ids, float* token_logprobs, int32_t* topn_ids,
                      float* topn_logprobs, int32_t* row_status, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * sampler_assemble_vocab_slices: out[r, off_s + c] = slice_s[r, c] with
 * off_s = slice_cols[0] + ... + slice_cols[s-1].
 *   slices      HOST array of n_slices DEVICE pointers, slice s fp32
 *               [rows, slice_cols[s]] with leading dimension slice_ld[s]
 *   slice_cols, slice_ld   HOST arrays of n_slices entries
 *   out         fp32 [rows, sum slice_cols], leading dimension ld_out
 * A bit-exact copy.  1 <= n_slices <= TS_MAX_SLICES.  Slices must not
 * overlap `out`.
 */
int sampler_assemble_vocab_slices(const float* const* slices, const int64_t* slice_cols,
                                  const int64_t* slice_ld, int32_t n_slices, int64_t rows,
                                  float* out, int64_t ld_out, void* stream);

/*
 * sampler_assemble_and_sample: sampler_assemble_vocab_slices followed by
 * sampler_sample_ex on the same received slices, with one read of the
 * logits instead of two.  The rank's step after the exchange on the page
 * "Qwen4Exp batch-sharded sampling: inside vLLM PR #61018", section "What
 * batch-sharded sampling is, in one paragraph", stitches the received
 * vocabulary slices into its batch rows and samples them.  Here the
 * sampler's first pass reads every logit of every row from the slices once,
 * for its row statistics and candidates, and in the same pass writes it to
 * `out`.
 *   out, ld_out   as in sampler_assemble_vocab_slices: fp32
 *                 [rows, sum slice_cols], written in full and bit-exact;
 *                 the slices must not overlap it.
 *   Every other argument and output, and the workspace
 *   (sampler_workspace_bytes_slices), are as in sampler_sample_ex.
 * `out` is exactly what sampler_assemble_vocab_slices writes.  The sampling
 * outputs follow the same definitions as sampler_sample_ex; the call may cut
 * the rows into narrower chunks (8 instead of 16 float4 per thread when
 * that keeps at most 24 chunks per row, which overlaps the extra copy
 * traffic better), so fp32 sums and the log-probabilities may differ from
 * sampler_sample_ex's in the last bits.
 * Shapes whose rows all take the exact per-row kernel (slices that start at
 * a column not a multiple of 4) run the assembly kernel first instead.
 * Arguments of both calls are validated before anything is enqueued.
 */
int sampler_assemble_and_sample(const float* const* slices, const int64_t* slice_cols,
                                const int64_t* slice_ld, int32_t n_slices, int64_t rows,
                                float* out, int64_t ld_out, const ts_row_params* params,
                                int64_t row_offset, int32_t max_logprobs, int32_t flags,
                                int32_t* token_ids, float* token_logprobs, int32_t* topn_ids,
                                float* topn_logprobs, int32_t* row_status, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * Scoring, losses and adapters: what a serving or training step does next to
 * the sampling path.  The pages only name the sampled tokens'
 * log-probabilities; the calls below take GIVEN tokens, and the definitions
 * are written out here.
 *
 * Shared by token_logprobs, token_logprobs_backward, token_logprobs_topn,
 * token_logprobs_listed(_backward), policy_loss and preference_loss:
 *   logits       [rows, vocab], leading dimension ld_logits, of logits_type
 *                TS_F32 or TS_BF16; any alignment of the rows.  -inf marks a
 *                token that is not allowed (probability 0).
 *   token_ids    int32 [rows]: the token of each row.  A negative id leaves
 *                the row out: its logits are not read, its log-probability
 *                is 0 and its gradient row is 0, whatever the row holds.
 *   temperature  finite, >= TS_GREEDY_EPS (else TS_EINVAL).  Log-probabilities
 *                are those of logits / temperature; 1 gives the sampler's raw
 *                log_softmax.  A logit further below the row's largest than fp32
 *                reaches has probability 0 at any temperature.
 *   row_status   int32 [rows] or NULL: TS_ROW_BAD_PARAMS for a token id >=
 *                vocab, TS_ROW_BAD_LOGITS for a row with a NaN or +inf logit
 *                or no finite one.  Such a row's outputs and gradient row are
 *                NaN, and so is a loss it takes part in.
 *   grad_logits  [rows, vocab] in the logits' type, leading dimension
 *                ld_grad >= vocab.  It may be the logits themselves (same
 *                pointer and, with more than one row, leading dimension: the
 *                gradient replaces them);
 *                any other overlap is TS_EINVAL (columns of one buffer beside
 *                the logits' columns, with the same leading dimension, are
 *                none).  Columns past vocab are not written.
 *   workspace    as for sampler_sample: 256-byte aligned scratch, no
 *                initialisation, ordered on one stream by whoever shares it.
 * Sums over the vocabulary are fp32 per thread and double from there on;
 * per-row arithmetic is double, outputs are rounded once.  Results do not
 * depend on the order in which workgroups run; the order of a row's sum goes by
 * the call's sizes and by where in a cache line its row starts.  rows == 0 writes nothing but
 * a loss of 0.  rows, vocab < 2^31.
 */
/*
 * token_logprobs: lp[r] = z_t - ln sum_j exp(z_j), z = logits[r] / temperature,
 * t = token_ids[r], and optionally the entropy H[r] = -sum_j p_j ln p_j of
 * p = softmax(z).
 *   logprobs   fp32 [rows]
 *   entropies  fp32 [rows] or NULL
 *   row_stats  fp32 [rows, 2] or NULL: max_j logits[r, j] and
 *              sum_j exp((logits[r, j] - max) / temperature), for
 *              token_logprobs_backward
 *
 * token_logprobs_backward: the gradient of the logits of any function of the
 * two, from grad_logprobs = dL/dlp (fp32 [rows]) and, with the forward pass's
 * entropies, grad_entropies = dL/dH (fp32 [rows] or NULL):
 *   dL/dlogits[r, j] = (dL/dlp (1[j = t] - p_j)
 *                       - dL/dH p_j (ln p_j + H)) / temperature.
 * token_ids, temperature and the logits are the forward call's.  A row whose
 * gradients are both 0 gives a row of zeros without reading its logits.  No
 * workspace.
 *
 * token_logprobs_backward_ex: the same with the forward pass's logprobs (fp32
 * [rows] or NULL).  The token's own entry holds 1 - p_t, and the sum in
 * row_stats, rounded to fp32, has no digits of that below 2^-24; with logprobs
 * the entry is right relative to 1 - p_t.
 */
size_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab);
int token_logprobs(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                   int64_t ld_logits, const int32_t* token_ids, double temperature,
                   float* logprobs, float* entropies, float* row_stats, int32_t* row_status,
                   void* workspace, size_t workspace_bytes, void* stream);
int token_logprobs_backward(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                            int64_t ld_logits, const int32_t* token_ids, double temperature,
                            const float* row_stats, const float* grad_logprobs,
                            const float* entropies, const float* grad_entropies,
                            void* grad_logits, int64_t ld_grad, void* stream);
int token_logprobs_backward_ex(const void* logits, int32_t logits_type, int64_t rows,
                               int64_t vocab, int64_t ld_logits, const int32_t* token_ids,
                               double temperature, const float* row_stats, const float* logprobs,
                               const float* grad_logprobs, const float* entropies,
                               const float* grad_entropies, void* grad_logits, int64_t ld_grad,
                               void* stream);

/*
 * token_logprobs_topn: token_logprobs with each token's rank and the row's most
 * likely alternatives, in the same read of the logits.  Tokens are in the order of
 * (logit descending, id ascending), -inf last.
 *   ranks          int32 [rows] or NULL: the token's place in that order, from 1
 *                  (topn_ids[r, ranks[r] - 1] is the token where that is listed)
 *   topn_ids       int32 [rows, max_logprobs]: the first max_logprobs tokens of
 *                  the order; -1 past the vocabulary's size
 *   topn_logprobs  fp32 [rows, max_logprobs]: their log-probabilities, at the
 *                  call's temperature; -inf in unused places
 * max_logprobs 0..TS_MAX_LOGPROBS; with 0 topn_ids and topn_logprobs may be NULL.
 * token_ids may be NULL: no token is asked for (logprobs and ranks NULL) and every
 * row takes part.  A left-out row has rank 0 and lists nothing; a bad row has rank
 * 0, ids -1 and NaN.  entropies, row_stats and row_status as in token_logprobs;
 * row_stats serve token_logprobs_backward and token_logprobs_listed_backward.
 * Some rows may be read again, once or several times (same results, slower): those
 * with few entries for each alternative, below about 512 in fp32 and 1,024 in bf16 for
 * up to 48 alternatives, 128 and 256 for up to 128, 32 and 64 beyond; and those where
 * more than 2,048 entries reach the bound that the largest of groups of neighbouring
 * entries give, as with very many equal logits or the likely tokens side by side.
 */
size_t token_logprobs_topn_workspace_bytes(int64_t rows, int64_t vocab);
int token_logprobs_topn(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                        int64_t ld_logits, const int32_t* token_ids, double temperature,
                        int32_t max_logprobs, float* logprobs, int32_t* ranks, float* entropies,
                        int32_t* topn_ids, float* topn_logprobs, float* row_stats,
                        int32_t* row_status, void* workspace, size_t workspace_bytes,
                        void* stream);

/*
 * token_logprobs_listed: log-probabilities of n_listed tokens a row, such as
 * another model's alternatives.
 *   listed_ids  int32 [rows, n_listed], 1 <= n_listed <= TS_MAX_LISTED.  A negative
 *               id is an unused place (log-probability 0, its gradient is not
 *               read); a row of which all are negative is left out.  An id may be
 *               listed several times.  An id >= vocab makes the row
 *               TS_ROW_BAD_PARAMS.
 *   logprobs    fp32 [rows, n_listed]
 *   entropies, row_stats, row_status  as in token_logprobs
 *
 * token_logprobs_listed_backward: the gradient of the logits of any function of
 * these, from grad_logprobs = dL/dlp (fp32 [rows, n_listed]) and, with the forward
 * pass's entropies, grad_entropies = dL/dH (fp32 [rows] or NULL):
 *   dL/dlogits[r, j] = (sum_{i: id_i = j} dL/dlp_i - p_j sum_i dL/dlp_i
 *                       - dL/dH p_j (ln p_j + H)) / temperature.
 * listed_ids, temperature and the logits are the forward call's, and row_stats
 * and logprobs its outputs.  A row whose gradients are all 0 gives a row of zeros,
 * whatever its logits hold.  No workspace.
 */
#define TS_MAX_LISTED 1024   /* largest accepted n_listed */
size_t token_logprobs_listed_workspace_bytes(int64_t rows, int64_t vocab);
int token_logprobs_listed(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                          int64_t ld_logits, const int32_t* listed_ids, int32_t n_listed,
                          double temperature, float* logprobs, float* entropies, float* row_stats,
                          int32_t* row_status, void* workspace, size_t workspace_bytes,
                          void* stream);
int token_logprobs_listed_backward(const void* logits, int32_t logits_type, int64_t rows,
                                   int64_t vocab, int64_t ld_logits, const int32_t* listed_ids,
                                   int32_t n_listed, double temperature, const float* row_stats,
                                   const float* logprobs, const float* grad_logprobs,
                                   const float* entropies, const float* grad_entropies,
                                   void* grad_logits, int64_t ld_grad, void* stream);

/*
 * policy_loss: the clipped policy loss with a KL term,
 *   r   = exp(lp - old_logprobs)
 *   s   = min(r A, clip(r, 1 - clip_low, 1 + clip_high) A),  A = advantages
 *   kl  = exp(ref_logprobs - lp) - (ref_logprobs - lp) - 1
 *   loss = sum over rows of weights (-s + kl_coef kl),
 * and, with grad_logits, grad_loss times its gradient:
 *   dloss/dlp = weights (-A r [s = r A] + kl_coef (1 - exp(ref - lp))).
 * The weights hold the average the caller wants (1 / tokens, 1 / (sequences x
 * length), ...).  A row of weight 0, like one of a negative token id, is left
 * out.  A = 0 gives s = 0 at any ratio.
 * A token of probability 0 (lp = -inf) with a finite ref has r = 0 and kl =
 * inf; with kl_coef > 0 the loss is inf then and, as the row's dloss/dlp is,
 * no entry of its gradient row is finite.
 *   params         HOST struct; clip_low and clip_high >= 0, inf for no clip
 *   old_logprobs   fp32 [rows]: log-probabilities when the tokens were drawn
 *   ref_logprobs   fp32 [rows], or NULL if kl_coef == 0
 *   advantages     fp32 [rows]
 *   weights        fp32 [rows], or NULL for 1
 *   grad_loss      fp32 [1] (device), or NULL for 1
 *   loss           fp32 [1]
 *   logprobs, ratios, kl   fp32 [rows] or NULL: lp, r and kl (0, 1 and 0 for
 *                  a row that is left out; kl is 0 without ref_logprobs)
 *   grad_logits    or NULL for the loss alone
 * Workspace: token_logprobs_workspace_bytes.
 */
typedef struct ts_policy_params {
  double temperature;
  double clip_low;
  double clip_high;
  double kl_coef;
} ts_policy_params;
int policy_loss(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                int64_t ld_logits, const int32_t* token_ids, const ts_policy_params* params,
                const float* old_logprobs, const float* ref_logprobs, const float* advantages,
                const float* weights, const float* grad_loss, float* loss, float* logprobs,
                float* ratios, float* kl, int32_t* row_status, void* grad_logits, int64_t ld_grad,
                void* workspace, size_t workspace_bytes, void* stream);

/*
 * preference_loss: the loss of paired log ratios.  Sequence i is rows
 * [seq_offsets[i], seq_offsets[i + 1]); sequences 0 .. n_pairs - 1 are the
 * chosen answers and n_pairs + i is the rejected one of pair i.
 *   rho_i  = sum over the sequence's rows that are not left out of
 *            (lp - ref_logprobs), divided by their number (if any) with
 *            TS_PREFERENCE_MEAN
 *   z      = beta (rho_chosen - rho_rejected) - margin
 *   l      = -(1 - label_smoothing) ln sigmoid(z)
 *            - label_smoothing ln sigmoid(-z)
 *   loss   = sum over pairs of pair_weights l,
 * and, with grad_logits, grad_loss times its gradient.  An empty sequence
 * has rho = 0.  A term of factor 0 is 0 at any z: a token of probability 0 in
 * the rejected answer alone (z = inf) adds no loss and no gradient at
 * label_smoothing 0.  Rows before the first and after the last sequence take no
 * part (log-probability and gradient row 0).  A pair of weight 0 adds
 * nothing to the loss and the gradient.
 *   seq_offsets    int32 [2 n_pairs + 1], non-decreasing (the rows' gradient
 *                  is unspecified where sequences overlap); used clamped to
 *                  [0, rows]
 *   params         HOST struct; beta > 0, label_smoothing in [0, 1]
 *   ref_logprobs   fp32 [rows], or NULL for 0 (no reference)
 *   pair_weights   fp32 [n_pairs], or NULL for 1 / n_pairs
 *   grad_loss      fp32 [1] (device), or NULL for 1
 *   loss           fp32 [1]
 *   pair_losses    fp32 [n_pairs] or NULL: l
 *   rewards        fp32 [2 n_pairs] or NULL: beta rho
 *   logprobs       fp32 [rows] or NULL
 *   grad_logits    or NULL for the loss alone
 * Workspace: preference_loss_workspace_bytes.  n_pairs < 2^30.
 */
#define TS_PREFERENCE_MEAN 1
typedef struct ts_preference_params {
  double temperature;
  double beta;
  double label_smoothing;
  double margin;
  int32_t flags;
} ts_preference_params;
size_t preference_loss_workspace_bytes(int64_t rows, int64_t vocab, int64_t n_pairs);
int preference_loss(const void* logits, int32_t logits_type, int64_t rows, int64_t vocab,
                    int64_t ld_logits, const int32_t* token_ids, const int32_t* seq_offsets,
                    int64_t n_pairs, const ts_preference_params* params,
                    const float* ref_logprobs, const float* pair_weights, const float* grad_loss,
                    float* loss, float* pair_losses, float* rewards, float* logprobs,
                    int32_t* row_status, void* grad_logits, int64_t ld_grad, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * ts_status_string: name of a TS_* return code (a static string; unknown
 * codes give "TS_UNKNOWN").  ts_last_error: a description of the calling
 * thread's last nonzero return (a per-thread static buffer, overwritten by
 * that thread's next failure).  Both serve the fail-fast convention above:
 * a rejected configuration says why it was rejected (page "Qwen 4 leak:
 * SGLang shards the Qwen4Exp prefill", section "The cost to you:
 * constraints").  Host-only; callable without a GPU.
 */
const char* ts_status_string(int status);
const char* ts_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* TOP_SAMPLING_H_ */
