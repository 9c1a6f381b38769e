// Device code shared by the kernels that read logits rows once (losses.hip,
// alternatives.hip): a row's statistics and what is worked out from them.
//
// For a row x of logits, a token t and a temperature T:
//   m = max_j x_j,  e_j = exp((x_j - m) / T),  S = sum_j e_j,  p_j = e_j / S
//   lp = (x_t - m) / T - ln S                              (log-probability)
//   H  = ln S - (1 / S) sum_j e_j ln e_j                   (entropy)
#pragma once

#include <float.h>
#include <math.h>

#include <algorithm>

#include "losses.hpp"

namespace ts {

constexpr int kThreads = 256;
constexpr int kBatch = 4;                       // 16-byte vectors a thread has in flight
constexpr int kSlab = kThreads * kBatch;        // vectors a workgroup takes at a time
constexpr int kMaxChunkSlabs = 2;               // longest chunk, in slabs
constexpr int kTargetGroups = 1024;             // workgroups wanted for few rows
constexpr int64_t kMaxThreads = int64_t{1} << 31;  // of one launch (grid-stride beyond): HIP
                                                   // counts a dimension's threads in 32 bits
constexpr int kShortRow = 32768;                // entries: see whole_rows()

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// Rows start wherever the caller's leading dimension puts them; the 16-byte
// accesses only assume the element's own alignment.
typedef f32x4 f32x4u __attribute__((aligned(4)));
typedef bf16x8 bf16x8u __attribute__((aligned(2)));

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  using Type = f32x4u;
};
template <>
struct Vec<__bf16> {
  static constexpr int n = 8;
  using Type = bf16x8u;
};

// The temperature, as the kernels use it.
struct Scale {
  float c_hi, c_lo;  // log2(e) / T in two floats, both above 0
  float floor;       // x - m below this gives exp2 = 0
  double inv_t;
};

inline Scale make_scale(double temperature) {
  Scale s;
  const double c = M_LOG2E / temperature;
  s.c_hi = static_cast<float>(c);
  if (s.c_hi >= c) s.c_hi = nextafterf(s.c_hi, 0.0f);
  // Beyond temperatures of 1e30 these leave the normal numbers.  They stay above
  // 0, at least 2^-149, which is 2^-21 in the exponent of the largest logits.
  constexpr float kLeast = 0x1p-149f;
  s.c_hi = std::max(s.c_hi, kLeast);
  s.c_lo = std::max(static_cast<float>(c - static_cast<double>(s.c_hi)), kLeast);
  s.inv_t = 1.0 / temperature;
  s.floor = static_cast<float>(std::max(-200.0 / c, -static_cast<double>(FLT_MAX)));
  return s;
}

// exp((x - m) / T) of t = x - m.  Both products of t = -inf are -inf, so a
// token that is not allowed gives exp2(-inf) = 0 without a test.
__device__ __forceinline__ float log2_t(float t, const Scale& s) {
  return fmaf(t, s.c_hi, t * s.c_lo);
}

__device__ __forceinline__ float exp_t(float t, const Scale& s) {
  return __builtin_amdgcn_exp2f(log2_t(t, s));
}

// A log2 e_j below this is taken as this: e_j is 0, and 0 x -inf is not.
constexpr float kLeastLog2 = -200.0f;

// The running maximum keeps a NaN (and +inf), so a bad logit shows in it.
__device__ __forceinline__ float max_nan(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}

// One chunk's share of a row.
struct Part {
  double s, u;  // sum of e, sum of e log2 e
  float m, pad;
};

struct Cut {
  int len;     // vectors per chunk
  int chunks;  // chunks per row
};

// A chunk is at most kMaxChunkSlabs slabs.  With few rows the chunks get
// shorter until there are about kTargetGroups of them, down to one vector a
// thread.
inline Cut cut_rows(int64_t rows, int64_t vocab, int vec) {
  const int64_t nvec = vocab >= vec ? vocab / vec : 1;  // whole vectors
  int64_t want = (nvec + kSlab * kMaxChunkSlabs - 1) / (kSlab * kMaxChunkSlabs);
  const int64_t fill = rows > 0 ? (kTargetGroups + rows - 1) / rows : 1;
  const int64_t most = (nvec + kThreads - 1) / kThreads;
  if (fill > want) want = fill < most ? fill : most;
  if (want < 1) want = 1;
  int64_t len = (nvec + want - 1) / want;
  const int64_t unit = len > kSlab ? kSlab : kThreads;
  len = (len + unit - 1) / unit * unit;
  Cut c;
  c.len = static_cast<int>(len);
  c.chunks = static_cast<int>((nvec + len - 1) / len);
  return c;
}

// Whether the statistics take a row per workgroup instead of a chunk.  Short
// rows do at any number, as that saves the records and a launch (2,000
// entries: 4 against 6 us, 32,000 and 500 rows 13 against 17).  Long ones take a
// CU too long unless there are enough of them: bf16, 128 rows of 151,936 17
// against 15 us, 256 18 against 22, 1,024 62 against 70; fp32, 512 rows of
// 60,000 25 against 27, 640 of 151,936 73 both ways, 800 97 against 89.
inline bool whole_rows(int64_t rows, int64_t vocab, int vec) {
  return vocab <= kShortRow || (rows >= 192 && (vec > 4 || vocab <= 2 * kShortRow));
}

// Joins (m, s, u) of a group of `width` lanes (a power of two); every lane
// gets the result.  An empty part has m = -inf and s = u = 0.
template <bool ENT>
__device__ __forceinline__ void join_lanes(float& m, double& s, double& u, int width,
                                           const Scale& sc) {
  float top = m;
  for (int d = width >> 1; d > 0; d >>= 1) top = max_nan(top, __shfl_xor(top, d, width));
  const float shift = fmaxf(m - (top == -INFINITY ? 0.0f : top), sc.floor);
  const double f = exp_t(shift, sc);
  if (ENT) u = f * (u + log2_t(shift, sc) * s);
  s *= f;
  for (int d = width >> 1; d > 0; d >>= 1) {
    s += __shfl_xor(s, d, width);
    if (ENT) u += __shfl_xor(u, d, width);
  }
  m = top;
}

// The sum of a thread's batch, added up pair by pair (in place).
template <int VN>
__device__ __forceinline__ float tree_sum(float (&w)[kBatch][VN]) {
  float* v = &w[0][0];
#pragma unroll
  for (int n = kBatch * VN / 2; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] += v[i + n];
  return v[0];
}

// A row as vectors: `edge` entries at its two ends, and between them `whole`
// vectors from entry `head` on, which starts a cache line of `lines`, the
// gradient's row.  With vectors from entry 0 on a row of odd length has every
// store across a line's border.  From 0 and from a line on, 1,021 x 100,277:
// loss and gradient, bf16 104 and 87 us (87 too where the rows are whole lines
// apart), fp32 180 and 164; backward pass of the log-probabilities, bf16 84
// and 74, fp32 152 and 142.  From a 16-byte border on: bf16 98 and 75, fp32 179
// and 150.
// Loads alone only mind bf16's 2-byte borders (log-probabilities, bf16 47 and
// 42 us, fp32 74 both ways), so the statistics of fp32 rows, whose last digits
// depend on how a row is cut, are taken from entry 0 on.
struct Shape {
  int head, whole, edge;

  // The place of edge entry i.
  template <typename T>
  __device__ __forceinline__ int at(int i) const {
    return i < head ? i : i + whole * Vec<T>::n;
  }
};

constexpr int kLine = 128;

template <typename T>
__device__ __forceinline__ Shape row_shape(const T* lines, int vocab) {
  constexpr int PER = kLine / sizeof(T);
  const int past = static_cast<int>(reinterpret_cast<uintptr_t>(lines) / sizeof(T) % PER);
  Shape f;
  f.head = min((PER - past) % PER, vocab);
  f.whole = (vocab - f.head) / Vec<T>::n;
  f.edge = vocab - f.whole * Vec<T>::n;
  return f;
}

// The cut of the statistics.
template <typename T>
__device__ __forceinline__ Shape stats_shape(const T* row, int vocab) {
  return sizeof(T) < 4 ? row_shape(row, vocab)
                       : Shape{0, vocab / Vec<T>::n, vocab % Vec<T>::n};
}

// ------------------------------------------------------------------- stats
// A slab of a row's whole vectors, THREADS x kBatch of them from v on; past
// `end` the loads repeat the last vector and are not used.
template <typename T, int THREADS>
struct Slab {
  typename Vec<T>::Type raw[kBatch];

  __device__ __forceinline__ void load(const T* row, int v, int end) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = min(v + j * THREADS + static_cast<int>(threadIdx.x), end - 1);
      raw[j] = *reinterpret_cast<const typename Vec<T>::Type*>(row + static_cast<int64_t>(i) *
                                                                         Vec<T>::n);
    }
  }
  __device__ __forceinline__ void unpack(float (&w)[kBatch][Vec<T>::n]) const {
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
#pragma unroll
      for (int e = 0; e < Vec<T>::n; ++e) w[j][e] = static_cast<float>(raw[j][e]);
  }
};

// A thread's share of vectors [v0, v1) of a row joined into m, s, u; `edge`:
// also the entries at the row's ends.  The next slab's loads are in flight
// while a slab is added up.
// `visit` sees every slab's entries (-inf past the row's end) and every edge entry.
struct NoVisit {
  static constexpr bool kOn = false;
};

template <typename T, bool ENT, int THREADS, typename Visit = NoVisit>
__device__ __forceinline__ void row_stats(const T* row, int vocab, int v0, int v1, bool edge,
                                          const Scale& sc, float& m, double& s, double& u,
                                          Visit* visit = nullptr) {
  constexpr int VN = Vec<T>::n;
  const int tid = threadIdx.x;
  const Shape f = stats_shape(row, vocab);
  const T* body = row + f.head;
  const int end = min(v1, f.whole);
  Slab<T, THREADS> next;
  if (v0 < end) next.load(body, v0, end);
  for (int v = v0; v < end; v += THREADS * kBatch) {
    float w[kBatch][VN], ut[kBatch][VN];
    next.unpack(w);
    if (v + THREADS * kBatch < end) {
      next.load(body, v + THREADS * kBatch, end);
    }
    if (v + THREADS * kBatch > end) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int e = 0; e < VN; ++e)
          w[j][e] = v + j * THREADS + tid < end ? w[j][e] : -INFINITY;
    }
    float top = Visit::kOn ? -INFINITY : m;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
#pragma unroll
      for (int e = 0; e < VN; e += 2) top = max_nan(max_nan(top, w[j][e]), w[j][e + 1]);
    if constexpr (Visit::kOn) {
      visit->slab(v, end, w, top);
      top = max_nan(m, top);
    }
    const float ref = top == -INFINITY ? 0.0f : top;
    const float shift = fmaxf(m - ref, sc.floor);
    const double keep = exp_t(shift, sc);
    if (ENT) u = keep * (u + log2_t(shift, sc) * s);
    s *= keep;
    m = top;
    // A batch is added up as a tree, and the batches in double: behind a term
    // near 1, terms below half an fp32 step would all be lost one by one, and
    // every row with one likely token came out 1e-7 too likely.
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
#pragma unroll
      for (int e = 0; e < VN; ++e) {
        const float k = log2_t(w[j][e] - ref, sc);
        const float ex = __builtin_amdgcn_exp2f(k);
        w[j][e] = ex;
        if (ENT) ut[j][e] = ex * fmaxf(k, kLeastLog2);
      }
    s += tree_sum(w);
    if (ENT) u += tree_sum(ut);
  }
  if (edge && tid < f.edge) {
    const float x = static_cast<float>(row[f.template at<T>(tid)]);
    if constexpr (Visit::kOn) visit->edge(f.template at<T>(tid), x);
    const float top = max_nan(m, x), ref = top == -INFINITY ? 0.0f : top;
    const float shift = fmaxf(m - ref, sc.floor), k = log2_t(x - ref, sc);
    const double keep = exp_t(shift, sc), ex = __builtin_amdgcn_exp2f(k);
    if (ENT) u = keep * (u + log2_t(shift, sc) * s) + ex * fmaxf(k, kLeastLog2);
    s = keep * s + ex;
    m = top;
  }
}

// The workgroup's (m, s, u) joined; the first threads have the result.
template <bool ENT, int THREADS>
__device__ __forceinline__ void join_group(float& m, double& s, double& u, const Scale& sc,
                                           Part* wave_part) {
  constexpr int WAVES = THREADS / 64;
  const int tid = threadIdx.x;
  join_lanes<ENT>(m, s, u, 64, sc);
  if ((tid & 63) == 0) wave_part[tid >> 6] = Part{s, u, m, 0.0f};
  __syncthreads();
  if (tid < WAVES) {
    const Part p = wave_part[tid];
    m = p.m;
    s = p.s;
    u = p.u;
    join_lanes<ENT>(m, s, u, WAVES, sc);
  }
}

struct RowStats {
  float m;
  double s, u;
  double lp;   // log-probability of the token (NaN for a bad row)
  int status;
};

// The batch that holds the token, of NV vectors that a thread among `threads` took
// at a time from a multiple of `len` on, and what its fp32 sum lost of the terms
// beside the token's own 1.  A token with p near 1 has S = 1 + d and lp = -ln S =
// -d, and whatever shares its batch is rounded to 2^-24 there: 1 - p of 1e-8 came
// out 0.  Taken again by the lanes of a group of NV, a vector of the batch each:
// the same tree, and the sum in double.  Loaded ahead where a row's end would wait
// for it (640 x 151,936 fp32 with entropy: 69.2 us if not, 68.7 so, 68.4 without
// any of this; 1,021 x 100,277 bf16 loss and gradient 89.4 and without 88.8).
template <typename T, int NV>
struct TokenBatch {
  typename Vec<T>::Type raw;
  bool in_body, in_row;  // the token is in a batch; this lane's vector is too

  __device__ __forceinline__ void load(const T* row, const Shape& f, int len, int threads,
                                       int token) {
    const int vec = (token - f.head) / Vec<T>::n;
    in_body = token >= f.head && vec < f.whole;  // the row's ends are added in double
    if (!in_body) return;
    const int v0 = vec / len * len, end = min(v0 + len, f.whole);
    const int v = v0 + (vec - v0) / (NV * threads) * (NV * threads) + (vec - v0) % threads +
                  static_cast<int>(threadIdx.x % NV) * threads;
    in_row = v < end;
    raw = *reinterpret_cast<const typename Vec<T>::Type*>(
        row + f.head + static_cast<int64_t>(min(v, end - 1)) * Vec<T>::n);
  }

  // With m the token's logit.
  __device__ __forceinline__ double lost(float m, const Scale& sc) const {
    constexpr int VN = Vec<T>::n;
    if (!in_body) return 0.0;
    float e[VN];
    double exact = 0.0;
#pragma unroll
    for (int k = 0; k < VN; ++k) {
      e[k] = exp_t((in_row ? static_cast<float>(raw[k]) : -INFINITY) - m, sc);
      exact += e[k];
    }
#pragma unroll
    for (int d = NV / 2; d > 0; d >>= 1) {
      exact += __shfl_xor(exact, d, NV);
#pragma unroll
      for (int k = 0; k < VN; ++k) e[k] += __shfl_xor(e[k], d, NV);
    }
#pragma unroll
    for (int n = VN / 2; n > 0; n >>= 1)
#pragma unroll
      for (int k = 0; k < n; ++k) e[k] += e[k + n];
    return exact - e[0];
  }
};

// Whether a row's S needs that: a larger 1 - p has its digits in fp32 (2^-24 of
// S is 2^-20 of it at most, and a tree has five levels).
__device__ __forceinline__ bool next_to_one(float m, double s, int token, int vocab, float xt) {
  return xt == m && s < 1.0 + 1.0 / 16 && token < vocab;
}

// Status and log-probability from the joined statistics and the token's logit.
__device__ __forceinline__ void finish_row(RowStats& r, int token, int vocab, float xt,
                                           const Scale& sc) {
  r.status = token >= vocab ? TS_ROW_BAD_PARAMS
                            : (fabsf(r.m) < INFINITY ? TS_ROW_OK : TS_ROW_BAD_LOGITS);
  r.lp = r.status == TS_ROW_OK ? (static_cast<double>(xt) - r.m) * sc.inv_t - log(r.s) : NAN;
}

// A row that one workgroup of kThreads took as a whole, by the lanes that hold
// the joined statistics.
template <typename T>
__device__ __forceinline__ void regain_digits(const T* row, int vocab, int token, float xt,
                                              const Scale& sc, RowStats& r) {
  if (threadIdx.x < kThreads / 64 && next_to_one(r.m, r.s, token, vocab, xt)) {
    const Shape f = stats_shape(row, vocab);
    TokenBatch<T, kBatch> batch;
    batch.load(row, f, max(f.whole, 1), kThreads, token);
    r.s += batch.lost(r.m, sc);
  }
}

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

inline int grid_of(int64_t groups, int threads = kThreads) {
  return static_cast<int>(std::clamp<int64_t>(groups, 1, kMaxThreads / threads));
}

}  // namespace ts
