// Log-probabilities of given tokens, the two losses built on them, and the
// gradients of the logits, on gfx950.
//
// For a row x of logits, a token t and a temperature T:
//   m = max_j x_j,  e_j = exp((x_j - m) / T),  S = sum_j e_j,  p_j = e_j / S
//   lp = (x_t - m) / T - ln S                              (log-probability)
//   H  = ln S - (1 / S) sum_j e_j ln e_j                   (entropy)
// A scalar that depends on the row through g = dL/dlp and h = dL/dH has
//   dL/dx_j = [g (1[j = t] - p_j) - h p_j (lp_j + H)] / T
//           = e_j (a + b log2 e_j) + 1[j = t] g / T,
//   a = -(g + h (H - ln S)) / (S T),   b = -h ln 2 / (S T),
// and the entry of the token itself is written as a value of its own, from
// 1 - p_t = -expm1(lp), which keeps its digits when p_t is near 1 as lp does (see
// TokenBatch; a backward pass has it from the forward pass's log-probabilities).
//
// All of it is bound by the logits' bytes: about ten instructions an element
// (the exponential counts for four) against four or two bytes read.
//   stats  one pass over the logits with a running maximum and sum per
//          thread; a row is cut into chunks so that a few rows fill the card
//          too; one record per (row, chunk)
//   rows   joins a row's records and does the per-row arithmetic in double
//          (a ratio next to a clip border decides a whole gradient row)
//   grad   reads the logits again and writes the gradient
//   whole  short or many rows: stats and rows in one, a row per workgroup
//   pairs  the preference loss's sums over its sequences
//   policy_row_at_once  the policy loss with its gradient in one read
// Measured alone: stats reads 640 x 151,936 fp32 in 63 us (6.2 TB/s), grad
// reads and writes 256 x 248,320 bf16 in 40 us (6.3 TB/s).
// exp(x / T) is taken as exp2((x - m) c) with c = log2(e) / T held as two
// floats, so a temperature's rounding does not tilt the whole sum.  The entropy
// goes by that exponent and not by x - m, whose sums pass fp32's range, and 1 /
// T^2 its least number, where logits and temperature are large.
#include "token_rows.hpp"

namespace ts {
namespace {

// What the gradient pass needs of a row: entry j is e_j (a + b log2 e_j),
// the token's entry is `own`.  All zero: the row's gradient is zero.
struct RowGrad {
  float m, a, b, own;
};

// Which rows of a call take part; the others are not read.
struct RowsIn {
  const int32_t* tokens;   // a negative one leaves its row out,
  const float* weights;    // as a weight of 0 does,
  const int32_t* offsets;  // and a place outside [offsets[0], offsets[n_seqs])
  int n_seqs;

  __device__ __forceinline__ bool left_out(int row) const {
    return tokens[row] < 0 || (weights != nullptr && weights[row] == 0.0f) ||
           (offsets != nullptr && (row < offsets[0] || row >= offsets[n_seqs]));
  }
};

template <typename T, bool ENT>
__global__ __launch_bounds__(kThreads) void stats_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, RowsIn in, Scale sc, Cut cut,
    Part* __restrict__ parts) {
  __shared__ Part wave_part[kThreads / 64];
  const int tid = threadIdx.x;
  const int64_t total = static_cast<int64_t>(rows) * cut.chunks;
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
    const int row = static_cast<int>(b / cut.chunks), chunk = static_cast<int>(b % cut.chunks);
    if (in.left_out(row)) continue;
    float m = -INFINITY;
    double s = 0.0, u = 0.0;
    row_stats<T, ENT, kThreads>(x + static_cast<int64_t>(row) * ld, vocab, chunk * cut.len,
                                (chunk + 1) * cut.len, chunk == cut.chunks - 1, sc, m, s, u);
    join_group<ENT, kThreads>(m, s, u, sc, wave_part);
    if (tid == 0) parts[b] = Part{s, u, m, 0.0f};
    __syncthreads();
  }
}

// -------------------------------------------------------------------- rows
constexpr int kRowLanes = 8;                          // lanes that join one row's records
constexpr int kRowsPerGroup = kThreads / kRowLanes;

// A row's records joined by kRowLanes lanes; the row is not left out.
template <bool ENT, typename T>
__device__ __forceinline__ RowStats join_row(const T* x, int64_t ld, int vocab, int token, int row,
                                             const Part* parts, const Cut& cut, const Scale& sc) {
  const int lane = threadIdx.x % kRowLanes;
  const T* rx = x + static_cast<int64_t>(row) * ld;
  const float xt = static_cast<float>(rx[min(token, vocab - 1)]);
  TokenBatch<T, kBatch> batch;
  batch.load(rx, stats_shape(rx, vocab), cut.len, kThreads, token);
  RowStats r;
  r.m = -INFINITY;
  r.s = r.u = 0.0;
  for (int i = lane; i < cut.chunks; i += kRowLanes) {
    const Part p = parts[static_cast<int64_t>(row) * cut.chunks + i];
    const float top = max_nan(r.m, p.m);
    const float ref = top == -INFINITY ? 0.0f : top;
    const float d0 = fmaxf(r.m - ref, sc.floor), d1 = fmaxf(p.m - ref, sc.floor);
    const double f0 = exp_t(d0, sc), f1 = exp_t(d1, sc);
    if (ENT)
      r.u = f0 * (r.u + log2_t(d0, sc) * r.s) + f1 * (p.u + log2_t(d1, sc) * p.s);
    r.s = f0 * r.s + f1 * p.s;
    r.m = top;
  }
  join_lanes<ENT>(r.m, r.s, r.u, kRowLanes, sc);
  if (next_to_one(r.m, r.s, token, vocab, xt)) r.s += batch.lost(r.m, sc);
  finish_row(r, token, vocab, xt, sc);
  return r;
}

// The gradient record of dL/dlp = g (no entropy term).
__device__ __forceinline__ RowGrad row_grad(const RowStats& r, double g, const Scale& sc) {
  if (r.status != TS_ROW_OK) return RowGrad{0.0f, NAN, 0.0f, NAN};
  if (g == 0.0) return RowGrad{0.0f, 0.0f, 0.0f, 0.0f};
  return RowGrad{r.m, static_cast<float>(-g * sc.inv_t / r.s), 0.0f,
                 static_cast<float>(g * sc.inv_t * -expm1(r.lp))};
}

// What a row of token_logprobs writes, left out and not; by one thread.
__device__ __forceinline__ void score_left_out(const ScoreOut& o, int64_t r) {
  o.logprobs[r] = 0.0f;
  if (o.entropies) o.entropies[r] = 0.0f;
  if (o.row_stats) o.row_stats[2 * r] = o.row_stats[2 * r + 1] = 0.0f;
  if (o.row_status) o.row_status[r] = TS_ROW_OK;
}

__device__ __forceinline__ void score_row(const ScoreOut& o, const RowStats& st, int64_t r) {
  const bool ok = st.status == TS_ROW_OK;
  o.logprobs[r] = static_cast<float>(st.lp);
  if (o.entropies)
    o.entropies[r] = ok ? static_cast<float>(log(st.s) - st.u * M_LN2 / st.s) : NAN;
  if (o.row_stats) {
    o.row_stats[2 * r] = ok ? st.m : NAN;
    o.row_stats[2 * r + 1] = ok ? static_cast<float>(st.s) : NAN;
  }
  if (o.row_status) o.row_status[r] = st.status;
}

template <bool ENT, typename T>
__global__ __launch_bounds__(kThreads) void score_rows_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ tokens,
    Scale sc, const Part* __restrict__ parts, Cut cut, ScoreOut o) {
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerGroup + threadIdx.x / kRowLanes;
       row < rows; row += static_cast<int64_t>(gridDim.x) * kRowsPerGroup) {
    const int r = static_cast<int>(row);
    const bool writes = threadIdx.x % kRowLanes == 0;
    if (tokens[r] < 0) {
      if (writes) score_left_out(o, row);
      continue;
    }
    const RowStats st = join_row<ENT>(x, ld, vocab, tokens[r], r, parts, cut, sc);
    if (writes) score_row(o, st, row);
  }
}

// A workgroup takes a row as a whole, in one launch instead of two.
template <bool ENT, typename T>
__global__ __launch_bounds__(kThreads) void score_whole_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ tokens,
    Scale sc, ScoreOut o) {
  __shared__ Part wave_part[kThreads / 64];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int token = tokens[r];
    if (token < 0) {
      if (threadIdx.x == 0) score_left_out(o, r);
      continue;
    }
    const T* rx = x + r * ld;
    const float xt = static_cast<float>(rx[min(token, vocab - 1)]);
    RowStats st;
    st.m = -INFINITY;
    st.s = st.u = 0.0;
    row_stats<T, ENT, kThreads>(rx, vocab, 0, vocab / Vec<T>::n, true, sc, st.m, st.s, st.u);
    join_group<ENT, kThreads>(st.m, st.s, st.u, sc, wave_part);
    regain_digits(rx, vocab, token, xt, sc, st);
    if (threadIdx.x == 0) {
      finish_row(st, token, vocab, xt, sc);
      score_row(o, st, r);
    }
    __syncthreads();
  }
}

// Sum of n doubles by one workgroup, in a fixed order; thread 0 gets it.
__device__ __forceinline__ double group_sum(const double* v, int64_t n) {
  __shared__ double wave_sum[kThreads / 64];
  double s = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < n; i += kThreads) s += v[i];
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d, 64);
  if ((threadIdx.x & 63) == 0) wave_sum[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < kThreads / 64; ++w) s += wave_sum[w];
  return s;
}

__global__ __launch_bounds__(kThreads) void sum_kernel(const double* __restrict__ v, int64_t n,
                                                       float* __restrict__ out) {
  const double s = group_sum(v, n);
  if (threadIdx.x == 0) *out = static_cast<float>(s);
}

// What a left-out row of the policy loss writes, and one that takes part; both
// by one thread.  The latter returns the row's gradient record.
__device__ __forceinline__ void policy_left_out(const PolicyArgs& p, int r, double* losses) {
  losses[r] = 0.0;
  if (p.logprobs) p.logprobs[r] = 0.0f;
  if (p.ratios) p.ratios[r] = 1.0f;
  if (p.kl) p.kl[r] = 0.0f;
  if (p.row_status) p.row_status[r] = TS_ROW_OK;
}

// The row's own inputs, read ahead of the statistics.
struct PolicyRow {
  float weight, advantage, old_lp, ref_lp, grad_loss;
};

__device__ __forceinline__ PolicyRow policy_row_inputs(const PolicyArgs& p, const float* weights,
                                                       int r) {
  return PolicyRow{weights ? weights[r] : 1.0f, p.advantages[r], p.old_logprobs[r],
                   p.ref_logprobs ? p.ref_logprobs[r] : 0.0f, p.grad_loss ? *p.grad_loss : 1.0f};
}

__device__ __forceinline__ RowGrad policy_row(const PolicyArgs& p, const PolicyRow& in,
                                              const RowStats& st, const Scale& sc, int r,
                                              double* losses) {
  const double w = in.weight, adv = in.advantage;
  const double ratio = exp(st.lp - static_cast<double>(in.old_lp));
  const double low = 1.0 - p.clip_low, high = 1.0 + p.clip_high;
  // min(r A, clip(r) A): the bound that holds against the advantage's sign is
  // the only one that can bind.  A = 0 gives 0 at any ratio.
  const bool inside = adv >= 0.0 ? !(ratio > high) : !(ratio < low);
  double gain = 0.0, g = 0.0;
  if (adv != 0.0) {
    gain = (inside ? ratio : (adv >= 0.0 ? high : low)) * adv;
    g = inside ? -adv * ratio : 0.0;
  }
  double kl = 0.0;
  if (p.ref_logprobs != nullptr) {
    const double gap = static_cast<double>(in.ref_lp) - st.lp;
    const double em = expm1(gap);
    // A token of probability 0 (gap = inf) has the limit, not inf - inf.
    kl = gap == INFINITY ? gap : em - gap;
    if (p.kl_coef != 0.0) g -= p.kl_coef * em;
  }
  double loss = -gain;
  if (p.kl_coef != 0.0) loss += p.kl_coef * kl;
  losses[r] = st.status == TS_ROW_OK ? w * loss : NAN;
  if (p.logprobs) p.logprobs[r] = static_cast<float>(st.lp);
  if (p.ratios) p.ratios[r] = static_cast<float>(ratio);
  if (p.kl) p.kl[r] = static_cast<float>(kl);
  if (p.row_status) p.row_status[r] = st.status;
  return row_grad(st, static_cast<double>(in.grad_loss) * w * g, sc);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void policy_rows_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, RowsIn rows_in, Scale sc,
    const Part* __restrict__ parts, Cut cut, PolicyArgs p, RowGrad* __restrict__ grads,
    double* losses, int sum_here) {
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerGroup + threadIdx.x / kRowLanes;
       row < rows; row += static_cast<int64_t>(gridDim.x) * kRowsPerGroup) {
    const int r = static_cast<int>(row);
    const bool writes = threadIdx.x % kRowLanes == 0;
    if (rows_in.left_out(r)) {
      if (writes) {
        policy_left_out(p, r, losses);
        if (grads) grads[r] = RowGrad{0.0f, 0.0f, 0.0f, 0.0f};
      }
      continue;
    }
    const PolicyRow in = policy_row_inputs(p, rows_in.weights, r);
    const RowStats st = join_row<false>(x, ld, vocab, rows_in.tokens[r], r, parts, cut, sc);
    if (!writes) continue;
    const RowGrad g = policy_row(p, in, st, sc, r, losses);
    if (grads) grads[r] = g;
  }
  if (sum_here) {
    __syncthreads();
    const double s = group_sum(losses, rows);
    if (threadIdx.x == 0) *p.loss = static_cast<float>(s);
  }
}

// The loss alone, a row per workgroup.
template <typename T>
__global__ __launch_bounds__(kThreads) void policy_whole_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, RowsIn rows_in, Scale sc,
    PolicyArgs p, double* losses) {
  __shared__ Part wave_part[kThreads / 64];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int r = static_cast<int>(row);
    const int token = rows_in.tokens[r];
    if (rows_in.left_out(r)) {
      if (threadIdx.x == 0) policy_left_out(p, r, losses);
      continue;
    }
    const PolicyRow in = policy_row_inputs(p, rows_in.weights, r);
    const T* rx = x + row * ld;
    const float xt = static_cast<float>(rx[min(token, vocab - 1)]);
    RowStats st;
    st.m = -INFINITY;
    st.s = st.u = 0.0;
    row_stats<T, false, kThreads>(rx, vocab, 0, vocab / Vec<T>::n, true, sc, st.m, st.s, st.u);
    join_group<false, kThreads>(st.m, st.s, st.u, sc, wave_part);
    regain_digits(rx, vocab, token, xt, sc, st);
    if (threadIdx.x == 0) {
      finish_row(st, token, vocab, xt, sc);
      policy_row(p, in, st, sc, r, losses);
    }
    __syncthreads();
  }
}

// What a row of the preference loss writes, left out and not; by one thread.
// The gradient records are for dL/dlp = 1; the pair kernel scales them.
__device__ __forceinline__ void preference_left_out(const PreferenceArgs& p, int r, double* ratios,
                                                    RowGrad* grads) {
  ratios[r] = 0.0;
  if (p.logprobs) p.logprobs[r] = 0.0f;
  if (p.row_status) p.row_status[r] = TS_ROW_OK;
  if (grads) grads[r] = RowGrad{0.0f, 0.0f, 0.0f, 0.0f};
}

__device__ __forceinline__ void preference_row(const PreferenceArgs& p, const RowStats& st,
                                               const Scale& sc, int r, double* ratios,
                                               RowGrad* grads) {
  ratios[r] = st.lp - (p.ref_logprobs ? static_cast<double>(p.ref_logprobs[r]) : 0.0);
  if (p.logprobs) p.logprobs[r] = static_cast<float>(st.lp);
  if (p.row_status) p.row_status[r] = st.status;
  if (grads) grads[r] = row_grad(st, 1.0, sc);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void preference_rows_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, RowsIn rows_in, Scale sc,
    const Part* __restrict__ parts, Cut cut, PreferenceArgs p, RowGrad* __restrict__ grads,
    double* __restrict__ ratios) {
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerGroup + threadIdx.x / kRowLanes;
       row < rows; row += static_cast<int64_t>(gridDim.x) * kRowsPerGroup) {
    const int r = static_cast<int>(row);
    const bool writes = threadIdx.x % kRowLanes == 0;
    if (rows_in.left_out(r)) {
      if (writes) preference_left_out(p, r, ratios, grads);
      continue;
    }
    const RowStats st = join_row<false>(x, ld, vocab, rows_in.tokens[r], r, parts, cut, sc);
    if (writes) preference_row(p, st, sc, r, ratios, grads);
  }
}

// A row per workgroup, in one launch instead of two.
template <typename T>
__global__ __launch_bounds__(kThreads) void preference_whole_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, RowsIn rows_in, Scale sc,
    PreferenceArgs p, RowGrad* __restrict__ grads, double* __restrict__ ratios) {
  __shared__ Part wave_part[kThreads / 64];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int r = static_cast<int>(row);
    if (rows_in.left_out(r)) {
      if (threadIdx.x == 0) preference_left_out(p, r, ratios, grads);
      continue;
    }
    const int token = rows_in.tokens[r];
    const T* rx = x + row * ld;
    const float xt = static_cast<float>(rx[min(token, vocab - 1)]);
    RowStats st;
    st.m = -INFINITY;
    st.s = st.u = 0.0;
    row_stats<T, false, kThreads>(rx, vocab, 0, vocab / Vec<T>::n, true, sc, st.m, st.s, st.u);
    join_group<false, kThreads>(st.m, st.s, st.u, sc, wave_part);
    regain_digits(rx, vocab, token, xt, sc, st);
    if (threadIdx.x == 0) {
      finish_row(st, token, vocab, xt, sc);
      preference_row(p, st, sc, r, ratios, grads);
    }
    __syncthreads();
  }
}

// One workgroup per pair, half of it for each answer: the log-ratio sums of its
// two sequences, the pair's loss, and the factors of its rows' gradient
// records.  The rows' records are joined before, over the whole card: done here,
// one pair of 1,000-row answers over 32,000 entries took 178 us in all, not 133,
// and 8 pairs of 64-row answers over 151,936 entries (bf16) 164, not 156.
__device__ __forceinline__ void seq_bounds(const int32_t* offsets, int seq, int rows, int& from,
                                           int& to) {
  from = min(max(offsets[seq], 0), rows);
  to = min(max(offsets[seq + 1], from), rows);
}

constexpr int kPairThreads = 512;

__global__ __launch_bounds__(kPairThreads) void preference_pairs_kernel(
    int rows, const int32_t* __restrict__ tokens, PreferenceArgs p,
    const double* __restrict__ ratios, RowGrad* __restrict__ grads, double* __restrict__ losses) {
  constexpr int kWaves = kPairThreads / 64;
  constexpr int kSide = kPairThreads / 2;  // threads of each answer
  __shared__ double wave_sum[kWaves];
  __shared__ int wave_n[kWaves];
  __shared__ double coef[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int side = tid / kSide;
  for (int pair = blockIdx.x; pair < p.n_pairs; pair += gridDim.x) {
    int from, to;
    seq_bounds(p.seq_offsets, pair + side * p.n_pairs, rows, from, to);
    double sum = 0.0;
    int n = 0;
    for (int64_t row = int64_t{from} + tid % kSide; row < to; row += kSide) {
      if (tokens[row] < 0) continue;
      sum += ratios[row];
      ++n;
    }
    for (int d = 32; d > 0; d >>= 1) {
      sum += __shfl_xor(sum, d, 64);
      n += __shfl_xor(n, d, 64);
    }
    if (lane == 0) {
      wave_sum[wave] = sum;
      wave_n[wave] = n;
    }
    __syncthreads();
    if (tid == 0) {
      double rho[2], per[2];
      for (int q = 0; q < 2; ++q) {
        double s = 0.0;
        int count = 0;
        for (int w = q * kWaves / 2; w < (q + 1) * kWaves / 2; ++w) {
          s += wave_sum[w];
          count += wave_n[w];
        }
        per[q] = p.mean && count > 0 ? 1.0 / count : 1.0;
        rho[q] = s * per[q];
      }
      const double beta = p.beta, eps = p.label_smoothing;
      const double z = beta * (rho[0] - rho[1]) - p.margin;
      const double soft = log1p(exp(-fabs(z)));  // -ln sigmoid(|z|)
      // A term of factor 0 is left out: at an infinite z (a token of probability
      // 0 in one answer) it would be 0 x inf.
      const double loss = (eps != 1.0 ? (1.0 - eps) * (soft + fmax(-z, 0.0)) : 0.0) +
                          (eps != 0.0 ? eps * (soft + fmax(z, 0.0)) : 0.0);
      const double weight = p.pair_weights ? static_cast<double>(p.pair_weights[pair])
                                           : 1.0 / p.n_pairs;
      // dl/dz = -(1 - eps) sigmoid(-z) + eps sigmoid(z)
      const double small = exp(-fabs(z)) / (1.0 + exp(-fabs(z))), large = 1.0 - small;
      const double up = z >= 0.0 ? large : small, down = z >= 0.0 ? small : large;
      const double dz = z != z ? z : eps * up - (1.0 - eps) * down;
      const double gl = p.grad_loss ? static_cast<double>(*p.grad_loss) : 1.0;
      // A pair of weight 0 is out of the sum, whatever its rows hold.
      losses[pair] = weight == 0.0 ? 0.0 : weight * (z != z ? z : loss);
      coef[0] = weight == 0.0 ? 0.0 : gl * weight * dz * beta * per[0];
      coef[1] = weight == 0.0 ? 0.0 : -gl * weight * dz * beta * per[1];
      if (p.pair_losses) p.pair_losses[pair] = static_cast<float>(z != z ? z : loss);
      if (p.rewards) {
        p.rewards[pair] = static_cast<float>(beta * rho[0]);
        p.rewards[pair + p.n_pairs] = static_cast<float>(beta * rho[1]);
      }
    }
    __syncthreads();
    if (grads != nullptr) {
      const double k = coef[side];
      for (int64_t row = int64_t{from} + tid % kSide; row < to; row += kSide) {
        if (tokens[row] < 0) continue;
        RowGrad r = grads[row];
        if (k == 0.0) {
          r = RowGrad{0.0f, 0.0f, 0.0f, 0.0f};
        } else {
          r.a = static_cast<float>(r.a * k);
          r.own = static_cast<float>(r.own * k);
        }
        grads[row] = r;
      }
    }
    __syncthreads();
  }
}

// -------------------------------------------------------------------- grad
// A row's record from the forward pass's statistics and the caller's
// gradients of the log-probability and the entropy.  The token's entry is only
// worked out by the workgroup that writes it (`mine`), from its logit xt.
__device__ __forceinline__ RowGrad score_row_grad(const ScoreGrad& g, int row, bool skip,
                                                  bool mine, float xt, const Scale& sc) {
  const double dg = g.grad_logprobs[row];
  const double dh = g.grad_entropies ? static_cast<double>(g.grad_entropies[row]) : 0.0;
  if (skip || (dg == 0.0 && dh == 0.0)) return RowGrad{0.0f, 0.0f, 0.0f, 0.0f};
  const float m = g.row_stats[2 * static_cast<int64_t>(row)];
  const double s = g.row_stats[2 * static_cast<int64_t>(row) + 1];
  const double ln_s = log(s);
  const double h = g.entropies && dh != 0.0 ? static_cast<double>(g.entropies[row]) : 0.0;
  double own = 0.0;
  if (mine) {
    double lp = (static_cast<double>(xt) - m) * sc.inv_t - ln_s;
    // Next to 1, S in fp32 has lost the digits of 1 - p, which the forward pass's
    // log-probability has.  The two differ by the roundings of S and of that one,
    // 2^-24 and 2^-28; one that is further off was changed since and is not used.
    const double kept = g.logprobs ? g.logprobs[row] : NAN;
    if (lp > -1.0 / 16 && fabs(kept - lp) < 0x1p-23) lp = kept;
    own = dg * -expm1(lp);
    if (dh != 0.0 && lp > -1e30) own -= dh * exp(lp) * (lp + h);
  }
  return RowGrad{m, static_cast<float>(-(dg + (dh != 0.0 ? dh * (h - ln_s) : 0.0)) * sc.inv_t / s),
                 static_cast<float>(-dh * M_LN2 * sc.inv_t / s),
                 static_cast<float>(own * sc.inv_t)};
}

// The gradient of vectors [v0, v1) of a row (and with `edge` of the entries at
// its ends), slab by slab from the last to the first: the end of what the
// statistics pass read is still in the caches.  The stores go past them.
template <typename T, bool ENT, int THREADS>
__device__ __forceinline__ void row_grad_pass(const T* row, T* out, int vocab, int v0, int v1,
                                              bool edge, int token, const RowGrad& g,
                                              const Scale& sc) {
  constexpr int VN = Vec<T>::n;
  const Shape f = row_shape(out, vocab);
  constexpr int SLAB = THREADS * kBatch;
  using V = typename Vec<T>::Type;
  const int tid = threadIdx.x;
  const int end = min(v1, f.whole);
  const bool zero = g.a == 0.0f && g.b == 0.0f && g.own == 0.0f;
  auto entry = [&](float x, bool is_token) {
    const float k = log2_t(x - g.m, sc);
    const float ex = __builtin_amdgcn_exp2f(k);
    return is_token ? g.own : (ENT ? ex * fmaf(g.b, fmaxf(k, kLeastLog2), g.a) : ex * g.a);
  };
  if (edge && tid < f.edge) {
    const int at = f.template at<T>(tid);
    out[at] = static_cast<T>(zero ? 0.0f : entry(static_cast<float>(row[at]), at == token));
  }
  if (v0 >= end) return;
  row += f.head;
  out += f.head;
  // The token's vector, and its place in there, if it is one of these.
  const bool in_body = token >= f.head;
  const int token_vec = in_body ? (token - f.head) / VN : -1;
  const int token_e = in_body ? (token - f.head) % VN : 0;
  int v = v0 + (end - 1 - v0) / SLAB * SLAB;
  Slab<T, THREADS> next;
  if (!zero) next.load(row, v, end);
  for (; v >= v0; v -= SLAB) {
    float w[kBatch][VN];
    if (zero) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int e = 0; e < VN; ++e) w[j][e] = 0.0f;
    } else {
      next.unpack(w);
      if (v > v0) next.load(row, v - SLAB, end);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
#pragma unroll
        for (int e = 0; e < VN; ++e) w[j][e] = entry(w[j][e], false);
        if (v + j * THREADS + tid == token_vec) {
#pragma unroll
          for (int e = 0; e < VN; ++e) w[j][e] = e == token_e ? g.own : w[j][e];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = v + j * THREADS + tid;
      V o;
#pragma unroll
      for (int e = 0; e < VN; ++e) o[e] = static_cast<T>(w[j][e]);
      if (i < end)
        __builtin_nontemporal_store(o, reinterpret_cast<V*>(out + static_cast<int64_t>(i) * VN));
    }
  }
}

// ENT: the records have an entropy term (b).  With SCORE the records are made
// here from the caller's gradients; otherwise they come from the row kernels,
// and workgroup 0 also sums the loss terms that those left.
template <typename T, bool SCORE, bool ENT>
__global__ __launch_bounds__(kThreads) void grad_kernel(
    const T* x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ tokens, Scale sc,
    Cut cut, const RowGrad* __restrict__ grads, ScoreGrad sg, T* d, int64_t ldd,
    const double* __restrict__ losses, int64_t n_losses, float* __restrict__ loss) {
  constexpr int VN = Vec<T>::n;
  const int64_t total = static_cast<int64_t>(rows) * cut.chunks;
  if (!SCORE && blockIdx.x == 0) {
    const double s = group_sum(losses, n_losses);
    if (threadIdx.x == 0) *loss = static_cast<float>(s);
  }
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
    // Last row first, as the end of the logits is what the caches still hold.
    const int row = rows - 1 - static_cast<int>(b / cut.chunks);
    const int chunk = cut.chunks - 1 - static_cast<int>(b % cut.chunks);
    const T* rx = x + static_cast<int64_t>(row) * ld;
    T* rd = d + static_cast<int64_t>(row) * ldd;
    const int token = tokens[row];
    RowGrad g;
    if (SCORE) {
      const bool skip = token < 0;
      // The gradient may replace the logits, so the token's own logit is only
      // read by the workgroup that also writes it.
      const Shape f = row_shape(rd, vocab);
      const int vec = (token - f.head) / VN;
      const int owner = token < f.head || vec >= f.whole ? cut.chunks - 1 : vec / cut.len;
      const bool mine = token >= 0 && token < vocab && owner == chunk;
      const float xt = mine ? static_cast<float>(rx[token]) : 0.0f;
      g = score_row_grad(sg, row, skip, mine, xt, sc);
      __syncthreads();
    } else {
      g = grads[row];
    }
    row_grad_pass<T, ENT, kThreads>(rx, rd, vocab, chunk * cut.len, (chunk + 1) * cut.len,
                                    chunk == cut.chunks - 1, token, g, sc);
  }
}

// -------------------------------------------------- policy loss in one read
// One workgroup per row, which holds the row between the statistics and the
// gradient: every exponential goes into a register (REGS batches) or into LDS
// (LDS batches), relative to the thread's maximum at that point, and the
// gradient pass only scales it.
//   Long rows have a CU to themselves: 144 registers and 64 LDS words a thread
// hold 106,496 entries; what a longer row has beyond them is read a second
// time.  In two passes the second read costs as much as the first, out of the
// Infinity Cache too: reads and writes together pass at 6.5-6.8 TB/s.  Loss and
// gradient of 640 x 151,936 fp32 in two passes and in one: 192 and 157 us (one
// read and one write take 120 at that rate, the three tenths that are read
// again 18); 1,024 x 151,936 bf16: 155 and 127.  Loads one batch ahead are best
// (1,024 x 151,936: two ahead 142 us, all at once 150; the batches' exponentials
// then run after the loads and not under them), as are nine register batches
// (with ten, which spill two registers in bf16, 1,021 x 100,277 takes 91 us, not
// 87).  Holding the logits and not the exponentials, twice as many in bf16 and
// so two workgroups a CU, is no faster (129 us), and slower for short rows.
//   Short rows have two (up to 32,768 entries) or four (16,384) workgroups on a
// CU, so that one's reads run under another's writes and row arithmetic.  With a
// CU to themselves and without, us: 1,000 x 32,000 fp32 48 and 43, bf16 33 and
// 25; 1,000 x 4,096 fp32 19 and 10; 8,192 x 16,384 bf16 165 and 82; 8 x 32,000
// 10.1 and 10.0.  Half of their batches in LDS leave the registers that four
// workgroups can have (all in registers: 1,000 x 32,000 bf16 41 us).
constexpr int kTinyRow = 16384;
constexpr int kOneVals = 16;  // entries of a thread's batch

template <typename T, int THREADS, int REGS, int LDS, int WAVES>
__global__ __launch_bounds__(THREADS, WAVES) void policy_row_at_once_kernel(
    const T* x, int64_t ld, int rows, int vocab, RowsIn rows_in, Scale sc, PolicyArgs p, T* d,
    int64_t ldd, double* __restrict__ losses) {
  constexpr int VN = Vec<T>::n;
  constexpr int NV = kOneVals / VN;  // vectors of a thread's batch
  using V = typename Vec<T>::Type;
  __shared__ f32x4 held_lds[LDS * kOneVals / 4][THREADS];
  __shared__ Part wave_part[THREADS / 64];
  __shared__ RowGrad row_record;
  const Shape f = row_shape(d + static_cast<int64_t>(blockIdx.x) * ldd, vocab);
  const int whole = f.whole;
  const int batches = (whole + NV * THREADS - 1) / (NV * THREADS);

  // No loop over rows: with one the compiler keeps the batches' registers
  // across rows, and 700 of them spill.
  const int r = blockIdx.x;
  const int64_t row = r;
  // The thread's number, unknown to the compiler as such: it would work out
  // the places of all batches ahead and keep them in registers.
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const T* rx = x + row * ld;
  T* rd = d + row * ldd;
  const int token = rows_in.tokens[r];
  if (rows_in.left_out(r)) {
    if (tid == 0) policy_left_out(p, r, losses);
    row_grad_pass<T, false, THREADS>(rx, rd, vocab, 0, whole, true, token,
                                         RowGrad{0.0f, 0.0f, 0.0f, 0.0f}, sc);
    return;
  }
  const PolicyRow in = policy_row_inputs(p, rows_in.weights, r);
  const float xt = static_cast<float>(rx[min(token, vocab - 1)]);

  TokenBatch<T, NV> batch;
  if (threadIdx.x < 64) batch.load(rx, f, max(whole, 1), THREADS, token);
  const char* body = reinterpret_cast<const char*>(rx + f.head);
  float m = -INFINITY;
  double s = 0.0, u = 0.0;
  auto load = [&](int b, V (&raw)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = min((b * NV + j) * THREADS + tid, whole - 1);
      raw[j] = *reinterpret_cast<const V*>(body + static_cast<uint32_t>(i) * 16u);
    }
  };
  // Batch b's exponentials, relative to the maximum it leaves in m, and the
  // next batch's loads.
  V raw[NV];
  auto add = [&](int b, float (&e)[kOneVals]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in_row = (b * NV + j) * THREADS + tid < whole;
#pragma unroll
      for (int k = 0; k < VN; ++k)
        e[j * VN + k] = in_row ? static_cast<float>(raw[j][k]) : -INFINITY;
    }
    if (b + 1 < batches) load(b + 1, raw);
    float top = m;
#pragma unroll
    for (int k = 0; k < kOneVals; k += 2) top = max_nan(max_nan(top, e[k]), e[k + 1]);
    const float ref = top == -INFINITY ? 0.0f : top;
    s *= static_cast<double>(exp_t(fmaxf(m - ref, sc.floor), sc));
    m = top;
#pragma unroll
    for (int k = 0; k < kOneVals; ++k) e[k] = exp_t(e[k] - ref, sc);
    float sum[kOneVals / 2];
#pragma unroll
    for (int k = 0; k < kOneVals / 2; ++k) sum[k] = e[k] + e[k + kOneVals / 2];
#pragma unroll
    for (int n = kOneVals / 4; n > 0; n >>= 1)
#pragma unroll
      for (int k = 0; k < n; ++k) sum[k] += sum[k + n];
    s += sum[0];
  };

  constexpr int kKept = REGS + LDS;
  float held[REGS][kOneVals], top_at[kKept];
  if (batches > 0) load(0, raw);
#pragma unroll
  for (int b = 0; b < REGS; ++b) {
    if (b < batches) {
      add(b, held[b]);
      top_at[b] = m;
    }
  }
#pragma unroll
  for (int q = 0; q < LDS; ++q) {
    const int b = REGS + q;
    if (b < batches) {
      float e[kOneVals];
      add(b, e);
      top_at[b] = m;
#pragma unroll
      for (int k = 0; k < kOneVals / 4; ++k)
        held_lds[q * (kOneVals / 4) + k][tid] = f32x4{e[4 * k], e[4 * k + 1], e[4 * k + 2],
                                                      e[4 * k + 3]};
    }
  }
  for (int b = kKept; b < batches; ++b) {
    float e[kOneVals];
    add(b, e);
  }
  const bool in_edge = tid < f.edge;
  const int edge_at = in_edge ? f.template at<T>(tid) : 0;
  float edge_x = -INFINITY;
  if (in_edge) {
    edge_x = static_cast<float>(rx[edge_at]);
    const float top = max_nan(m, edge_x), ref = top == -INFINITY ? 0.0f : top;
    s = s * exp_t(fmaxf(m - ref, sc.floor), sc) + exp_t(edge_x - ref, sc);
    m = top;
  }
  join_group<false, THREADS>(m, s, u, sc, wave_part);
  if (threadIdx.x < THREADS / 64 && next_to_one(m, s, token, vocab, xt))
    s += batch.lost(m, sc);
  if (tid == 0) {
    RowStats st;
    st.m = m;
    st.s = s;
    finish_row(st, token, vocab, xt, sc);
    row_record = policy_row(p, in, st, sc, r, losses);
  }
  __syncthreads();
  const RowGrad g = row_record;

  // The gradient, the read-again batches first: their end is in the L2.
  asm volatile("" : "+v"(tid));
  const bool in_body = token >= f.head;
  const int token_vec = in_body ? (token - f.head) / VN : -1;
  const int token_e = in_body ? (token - f.head) % VN : 0;
  char* out = reinterpret_cast<char*>(rd + f.head);
  const bool zero = g.a == 0.0f && g.own == 0.0f;
  auto store = [&](int b, const float (&e)[kOneVals], float top) {
    const float scale = zero ? 0.0f : exp_t(fmaxf(top - g.m, sc.floor), sc) * g.a;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = (b * NV + j) * THREADS + tid;
      V o;
#pragma unroll
      for (int k = 0; k < VN; ++k) o[k] = static_cast<T>(e[j * VN + k] * scale);
      if (i == token_vec) {
#pragma unroll
        for (int k = 0; k < VN; ++k) o[k] = k == token_e ? static_cast<T>(g.own) : o[k];
      }
      if (i < whole)
        __builtin_nontemporal_store(o, reinterpret_cast<V*>(out + static_cast<uint32_t>(i) * 16u));
    }
  };
  if (batches > kKept)
    row_grad_pass<T, false, THREADS>(rx, rd, vocab, kKept * NV * THREADS, whole, false,
                                         token, g, sc);
  if (in_edge)
    rd[edge_at] = static_cast<T>(zero ? 0.0f
                                      : edge_at == token ? g.own : exp_t(edge_x - g.m, sc) * g.a);
#pragma unroll
  for (int q = LDS - 1; q >= 0; --q) {
    const int b = REGS + q;
    if (b < batches) {
      float e[kOneVals];
#pragma unroll
      for (int k = 0; k < kOneVals / 4; ++k) {
        const f32x4 v = held_lds[q * (kOneVals / 4) + k][tid];
#pragma unroll
        for (int t = 0; t < 4; ++t) e[4 * k + t] = v[t];
      }
      store(b, e, top_at[b]);
    }
  }
#pragma unroll
  for (int b = REGS - 1; b >= 0; --b) {
    if (b < batches) store(b, held[b], top_at[b]);
  }
}

// -------------------------------------------------------------- workspace

struct Workspace {
  Part* parts;
  RowGrad* grads;
  double* terms;   // of the rows: loss terms, or log ratios
  double* losses;  // of the pairs
  size_t bytes;
};

Workspace lay_out(void* base, int64_t rows, int64_t vocab, int64_t n_pairs) {
  const int chunks = std::max(cut_rows(rows, vocab, Vec<float>::n).chunks,
                              cut_rows(rows, vocab, Vec<__bf16>::n).chunks);
  char* p = static_cast<char*>(base);
  size_t at = 0;
  Workspace w;
  w.parts = reinterpret_cast<Part*>(p + at);
  at += round256(sizeof(Part) * static_cast<size_t>(rows) * chunks);
  w.grads = reinterpret_cast<RowGrad*>(p + at);
  at += round256(sizeof(RowGrad) * static_cast<size_t>(rows));
  w.terms = reinterpret_cast<double*>(p + at);
  at += round256(sizeof(double) * static_cast<size_t>(rows));
  w.losses = reinterpret_cast<double*>(p + at);
  at += round256(sizeof(double) * static_cast<size_t>(n_pairs));
  w.bytes = at;
  return w;
}


template <typename T, bool ENT>
hipError_t launch_stats(const TokenRows& t, const Scale& sc, const Cut& cut, const Workspace& w,
                        const RowsIn& in, hipStream_t stream) {
  hipLaunchKernelGGL((stats_kernel<T, ENT>), dim3(grid_of(int64_t{t.rows} * cut.chunks)),
                     dim3(kThreads), 0, stream, static_cast<const T*>(t.x), t.ld, t.rows, t.vocab,
                     in, sc, cut, w.parts);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_grad(const TokenRows& t, const Scale& sc, const Cut& cut, const Workspace& w,
                       const GradRows& d, const double* losses, int64_t n_losses, float* loss,
                       hipStream_t stream) {
  hipLaunchKernelGGL((grad_kernel<T, false, false>), dim3(grid_of(int64_t{t.rows} * cut.chunks)),
                     dim3(kThreads), 0, stream, static_cast<const T*>(t.x), t.ld, t.rows, t.vocab,
                     t.tokens, sc, cut, w.grads, ScoreGrad{}, static_cast<T*>(d.x), d.ld, losses,
                     n_losses, loss);
  return hipGetLastError();
}

hipError_t launch_sum(const double* v, int64_t n, float* out, hipStream_t stream) {
  hipLaunchKernelGGL(sum_kernel, dim3(1), dim3(kThreads), 0, stream, v, n, out);
  return hipGetLastError();
}

template <typename T>
hipError_t token_logprobs_t(const TokenRows& t, const ScoreOut& o, void* ws, hipStream_t stream) {
  const Scale sc = make_scale(t.temperature);
  const Cut cut = cut_rows(t.rows, t.vocab, Vec<T>::n);
  const Workspace w = lay_out(ws, t.rows, t.vocab, 0);
  const RowsIn in{t.tokens, nullptr, nullptr, 0};
  if (whole_rows(t.rows, t.vocab, Vec<T>::n)) {
    const dim3 grid(grid_of(t.rows));
    if (o.entropies != nullptr)
      hipLaunchKernelGGL((score_whole_kernel<true, T>), grid, dim3(kThreads), 0, stream,
                         static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, t.tokens, sc, o);
    else
      hipLaunchKernelGGL((score_whole_kernel<false, T>), grid, dim3(kThreads), 0, stream,
                         static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, t.tokens, sc, o);
    return hipGetLastError();
  }
  const dim3 grid(grid_of((t.rows + int64_t{kRowsPerGroup} - 1) / kRowsPerGroup));
  if (o.entropies != nullptr) {
    const hipError_t e = launch_stats<T, true>(t, sc, cut, w, in, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((score_rows_kernel<true, T>), grid, dim3(kThreads), 0, stream,
                       static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, t.tokens, sc, w.parts,
                       cut, o);
  } else {
    const hipError_t e = launch_stats<T, false>(t, sc, cut, w, in, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((score_rows_kernel<false, T>), grid, dim3(kThreads), 0, stream,
                       static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, t.tokens, sc, w.parts,
                       cut, o);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t token_logprobs_backward_t(const TokenRows& t, const ScoreGrad& g, const GradRows& d,
                                     hipStream_t stream) {
  const Scale sc = make_scale(t.temperature);
  const Cut cut = cut_rows(t.rows, t.vocab, Vec<T>::n);
  const dim3 grid(grid_of(int64_t{t.rows} * cut.chunks));
  if (g.grad_entropies != nullptr)
    hipLaunchKernelGGL((grad_kernel<T, true, true>), grid, dim3(kThreads), 0, stream,
                       static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, t.tokens, sc, cut,
                       nullptr, g, static_cast<T*>(d.x), d.ld, nullptr, 0, nullptr);
  else
    hipLaunchKernelGGL((grad_kernel<T, true, false>), grid, dim3(kThreads), 0, stream,
                       static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, t.tokens, sc, cut,
                       nullptr, g, static_cast<T*>(d.x), d.ld, nullptr, 0, nullptr);
  return hipGetLastError();
}

template <typename T>
hipError_t policy_loss_t(const TokenRows& t, const PolicyArgs& p, const GradRows& d, void* ws,
                         hipStream_t stream) {
  const Scale sc = make_scale(t.temperature);
  const Cut cut = cut_rows(t.rows, t.vocab, Vec<T>::n);
  const Workspace w = lay_out(ws, t.rows, t.vocab, 0);
  const RowsIn in{t.tokens, t.weights, nullptr, 0};
  const bool back = d.x != nullptr;
  // A row per workgroup keeps a CU busy for 5 us and 0.15 ns an entry, whatever
  // the number of rows; in two passes the rows are cut up over the card.  With
  // gradient, two passes and one, us: 8 rows of 32,000 10.5 and 10.0, of 151,936
  // 13.8 and 26.6; fp32, 64 rows of 151,936 26 and 28, 96 35 and 29; bf16, 96
  // rows of 151,936 23 and 26, 128 27.6 and 26.4.
  if (back && t.rows <= (1 << 22) && t.vocab <= (1 << 29) &&
      (t.vocab <= kShortRow || t.rows >= (t.bf16 ? 128 : 96))) {
    auto launch = [&](auto kernel, int threads) {
      hipLaunchKernelGGL(kernel, dim3(t.rows), dim3(threads), 0, stream,
                         static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, in, sc, p,
                         static_cast<T*>(d.x), d.ld, w.terms);
      return hipGetLastError();
    };
    const hipError_t one =
        t.vocab <= kTinyRow    ? launch(policy_row_at_once_kernel<T, 256, 2, 2, 4>, 256)
        : t.vocab <= kShortRow ? launch(policy_row_at_once_kernel<T, 512, 2, 2, 4>, 512)
                               : launch(policy_row_at_once_kernel<T, 512, 9, 4, 2>, 512);
    return one != hipSuccess ? one : launch_sum(w.terms, t.rows, p.loss, stream);
  }
  if (!back && whole_rows(t.rows, t.vocab, Vec<T>::n)) {
    hipLaunchKernelGGL((policy_whole_kernel<T>), dim3(grid_of(t.rows)), dim3(kThreads), 0, stream,
                       static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, in, sc, p, w.terms);
    const hipError_t one = hipGetLastError();
    return one != hipSuccess ? one : launch_sum(w.terms, t.rows, p.loss, stream);
  }
  hipError_t e = launch_stats<T, false>(t, sc, cut, w, in, stream);
  if (e != hipSuccess) return e;
  // Without a gradient and with one workgroup of rows, that one adds up the
  // loss; with a gradient the last pass does, otherwise a kernel of its own.
  const bool sum_here = !back && t.rows <= kRowsPerGroup;
  hipLaunchKernelGGL((policy_rows_kernel<T>),
                     dim3(grid_of((t.rows + int64_t{kRowsPerGroup} - 1) / kRowsPerGroup)),
                     dim3(kThreads), 0, stream, static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, in, sc, w.parts,
                     cut, p, back ? w.grads : nullptr, w.terms, sum_here);
  e = hipGetLastError();
  if (e != hipSuccess || sum_here) return e;
  return back ? launch_grad<T>(t, sc, cut, w, d, w.terms, t.rows, p.loss, stream)
              : launch_sum(w.terms, t.rows, p.loss, stream);
}

template <typename T>
hipError_t preference_loss_t(const TokenRows& t, const PreferenceArgs& p, const GradRows& d,
                             void* ws, hipStream_t stream) {
  const Scale sc = make_scale(t.temperature);
  const Cut cut = cut_rows(t.rows, t.vocab, Vec<T>::n);
  const Workspace w = lay_out(ws, t.rows, t.vocab, p.n_pairs);
  const RowsIn in{t.tokens, nullptr, p.seq_offsets, 2 * p.n_pairs};
  const bool back = d.x != nullptr && t.rows > 0;
  RowGrad* grads = back ? w.grads : nullptr;
  hipError_t e = hipSuccess;
  if (t.rows > 0 && whole_rows(t.rows, t.vocab, Vec<T>::n)) {
    hipLaunchKernelGGL((preference_whole_kernel<T>), dim3(grid_of(t.rows)), dim3(kThreads), 0,
                       stream, static_cast<const T*>(t.x), t.ld, t.rows, t.vocab, in, sc, p, grads,
                       w.terms);
    e = hipGetLastError();
  } else if (t.rows > 0) {
    e = launch_stats<T, false>(t, sc, cut, w, in, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((preference_rows_kernel<T>),
                       dim3(grid_of((t.rows + int64_t{kRowsPerGroup} - 1) / kRowsPerGroup)),
                       dim3(kThreads), 0, stream, static_cast<const T*>(t.x), t.ld, t.rows,
                       t.vocab, in, sc, w.parts, cut, p, grads, w.terms);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  if (p.n_pairs > 0) {
    hipLaunchKernelGGL(preference_pairs_kernel, dim3(grid_of(p.n_pairs, kPairThreads)),
                       dim3(kPairThreads), 0, stream, t.rows, t.tokens, p, w.terms, grads,
                       w.losses);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return back ? launch_grad<T>(t, sc, cut, w, d, w.losses, p.n_pairs, p.loss, stream)
              : launch_sum(w.losses, p.n_pairs, p.loss, stream);
}

}  // namespace

size_t token_rows_workspace_size(int64_t rows, int64_t vocab, int64_t n_pairs) {
  return lay_out(nullptr, rows, vocab, n_pairs).bytes;
}

hipError_t launch_token_logprobs(const TokenRows& t, const ScoreOut& o, void* ws,
                                 hipStream_t stream) {
  return t.bf16 ? token_logprobs_t<__bf16>(t, o, ws, stream)
                : token_logprobs_t<float>(t, o, ws, stream);
}

hipError_t launch_token_logprobs_backward(const TokenRows& t, const ScoreGrad& g,
                                          const GradRows& d, hipStream_t stream) {
  return t.bf16 ? token_logprobs_backward_t<__bf16>(t, g, d, stream)
                : token_logprobs_backward_t<float>(t, g, d, stream);
}

hipError_t launch_policy_loss(const TokenRows& t, const PolicyArgs& p, const GradRows& d, void* ws,
                              hipStream_t stream) {
  if (t.rows == 0) return launch_sum(nullptr, 0, p.loss, stream);
  return t.bf16 ? policy_loss_t<__bf16>(t, p, d, ws, stream)
                : policy_loss_t<float>(t, p, d, ws, stream);
}

hipError_t launch_preference_loss(const TokenRows& t, const PreferenceArgs& p, const GradRows& d,
                                  void* ws, hipStream_t stream) {
  return t.bf16 ? preference_loss_t<__bf16>(t, p, d, ws, stream)
                : preference_loss_t<float>(t, p, d, ws, stream);
}

}  // namespace ts
