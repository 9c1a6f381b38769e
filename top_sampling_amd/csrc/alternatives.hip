// Log-probabilities of given tokens with their rank and the row's most likely
// alternatives, and of several listed tokens a row with the gradient of the
// logits, on gfx950.
//
// With m, S, p_j and H of a row as in token_rows.hpp:
//   rank    1 + the number of tokens before t in the order of (logit descending,
//           id ascending); the alternatives are that order's first n tokens
//   listed  lp_i = (x[id_i] - m) / T - ln S for the row's ids id_0 .. id_(n-1)
//   dL/dx_j = [sum_{i: id_i = j} g_i - G p_j - h p_j (ln p_j + H)] / T,
//           g_i = dL/dlp_i, G = sum_i g_i, h = dL/dH
//           = e_j (a + b log2 e_j) + 1/T sum_{i: id_i = j} g_i,
//           a = -(G + h (H - ln S)) / (S T),  b = -h ln 2 / (S T);
//           a listed token's entry is written as a value of its own, from
//           1 - p = -expm1(lp), as in the single-token gradient.
// Bound by the logits' bytes: one read forwards, a read and a write backwards.
//
// The alternatives cost no second read: while the statistics pass has the
// logits in registers it also writes the largest of every group of entries, the 16
// (fp32) or 32 of a thread or, for smaller n, of 8 neighbouring threads.  A lower
// bound of the n-th largest logit follows from those alone, and only the groups that
// reach it, little more than n, are looked into again.
#include "alternatives.hpp"

#include <type_traits>

#include "token_rows.hpp"

namespace ts {
namespace {

constexpr int kGroupBits = 3;         // 8 threads share a group
constexpr int kListedGroups = 1280;   // groups looked into, at most
constexpr int kCandidates = 2048;     // entries put in order, at most
constexpr int kHeldGroups = 5;        // of a thread in registers
constexpr int kQuadMost = 48;         // see bound_of_quads
// Beyond this many alternatives every thread has its own groups (shared and own: 640 x
// 151,936 fp32, n = 100 105 and 143 us, 150 121 and 136, 200 137 and 140; 1,021 x
// 100,277 bf16 118 and 123, 143 and 121, 173 and 122).
constexpr int kSharedMost = 128;
static_assert(kSharedMost <= kThreads, "bound_of_threads takes no more");

// How the statistics pass leaves the largest entries of groups, each of 2^bits
// neighbouring threads: group g of slab s of a row's chunk c is number
// (c slabs + s) per_slab + g.
struct Groups {
  int chunk_len, slabs, bits, per_row;

  __host__ __device__ __forceinline__ int per_slab() const { return kThreads >> bits; }
};

Groups make_groups(const Cut& cut, int n) {
  Groups g;
  g.chunk_len = cut.len;
  g.slabs = (cut.len + kSlab - 1) / kSlab;
  g.bits = n > kSharedMost ? 0 : kGroupBits;
  g.per_row = cut.chunks * g.slabs * g.per_slab();
  return g;
}

// A row as one chunk.
Cut whole_cut(int64_t vocab, int vec) {
  return Cut{static_cast<int>(std::max<int64_t>(vocab / vec, 1)), 1};
}

// The largest of a value over 8 neighbouring lanes; all of them get it.
__device__ __forceinline__ float max_of_8(float x) {
  auto step = [](float v, auto ctrl) {
    return max_nan(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                                    0, __builtin_bit_cast(int, v),
                                                    decltype(ctrl)::value, 0xF, 0xF, true)));
  };
  x = step(x, std::integral_constant<int, 0xB1>{});   // quad_perm [1, 0, 3, 2]
  x = step(x, std::integral_constant<int, 0x4E>{});   // quad_perm [2, 3, 0, 1]
  return step(x, std::integral_constant<int, 0x141>{});  // row_half_mirror
}

// The largest fp32 number below a finite x.
__device__ __forceinline__ float next_below(float x) {
  const uint32_t b = __float_as_uint(x);
  return x == 0.0f ? __uint_as_float(0x80000001u) : __uint_as_float(x > 0.0f ? b - 1 : b + 1);
}

// What the statistics pass does beside adding up: groups, and the entries
// before the token in the order.  Those are the ones above the token's logit xt and,
// in front of it, the ones that equal it; a slab that does not reach xt is passed
// over.
template <typename T>
struct TopVisit {
  static constexpr bool kOn = true;
  float* groups;   // of the row's chunk, or null
  bool shared;     // by 8 threads each
  int v0;          // the chunk's first vector
  float xt, below; // the token's logit, +inf if there is none
  int token, token_vec, token_e;
  int better;      // this lane's
  int wave_better; // the wave's

  __device__ __forceinline__ void slab(int v, int end, const float (&w)[kBatch][Vec<T>::n],
                                       float high) {
    if (groups != nullptr) {
      const int first = (v - v0) / kSlab * kThreads + static_cast<int>(threadIdx.x);
      if (shared) {
        const float top = max_of_8(high);
        if (threadIdx.x % (1 << kGroupBits) == 0) groups[first >> kGroupBits] = top;
      } else {
        groups[first] = high;
      }
    }
    if (!__any(high >= xt)) return;
    if (xt == -INFINITY) {  // nothing is below: among the masked ones the ids decide
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = v + j * kThreads + static_cast<int>(threadIdx.x);
#pragma unroll
        for (int e = 0; e < Vec<T>::n; ++e)
          better += (w[j][e] > xt || (i < min(token_vec, end))) ? 1 : 0;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = v + j * kThreads + static_cast<int>(threadIdx.x);
        const float least = i < token_vec ? below : xt;
#pragma unroll
        for (int e = 0; e < Vec<T>::n; ++e) wave_better += __popcll(__ballot(w[j][e] > least));
      }
    }
    if (v <= token_vec && token_vec < min(v + kSlab, end)) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (v + j * kThreads + static_cast<int>(threadIdx.x) == token_vec) {
#pragma unroll
          for (int e = 0; e < Vec<T>::n; ++e) better += (e < token_e && w[j][e] == xt) ? 1 : 0;
        }
    }
  }
  __device__ __forceinline__ void edge(int at, float x) {
    better += (x > xt || (x == xt && at < token)) ? 1 : 0;
  }
  // A lane's share of the row's count.
  __device__ __forceinline__ int count() const {
    return better + ((threadIdx.x & 63) == 0 ? wave_better : 0);
  }
};

template <typename T>
__device__ __forceinline__ TopVisit<T> make_visit(const Shape& f, float* groups, int bits, int v0,
                                                  float xt, int token) {
  TopVisit<T> v;
  v.groups = groups;
  v.shared = bits != 0;
  v.v0 = v0;
  v.xt = xt;
  v.below = next_below(xt);
  v.token = token;
  const bool in_body = token >= f.head;
  v.token_vec = in_body ? (token - f.head) / Vec<T>::n : -1;
  v.token_e = in_body ? (token - f.head) % Vec<T>::n : 0;
  v.better = v.wave_better = 0;
  return v;
}

// Sum of an int over the workgroup; every thread gets it.
__device__ __forceinline__ int group_count(int n, int* wave_n) {
  for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d, 64);
  if ((threadIdx.x & 63) == 0) wave_n[threadIdx.x >> 6] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) n += wave_n[w];
  return n;
}

// float -> uint32 in the order of the numbers, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  uint32_t b = __float_as_uint(x);
  b = b == 0x80000000u ? 0u : b;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float number_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// An entry's place in the order of alternatives: larger is earlier.
__device__ __forceinline__ uint64_t entry_key(float x, int id) {
  return static_cast<uint64_t>(order_of(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(id));
}

struct TopShared {
  uint64_t cand[kCandidates];
  int group[kListedGroups];
  alignas(16) uint32_t most[kThreads];
  int hist[256];
  int n_groups, n_cand, wave_n[kThreads / 64];
  uint32_t bound;
  uint32_t low[kThreads / 64];
  int need, above, step, first_id, done;
  Part wave_part[kThreads / 64];
  double s, ln_s;
};

// A bound of the n-th largest of the keys from `low` to `high`, of which there are n or
// more: in 256 steps of a power of two, and again in the step that holds it, until at
// most `most` keys reach the bound or it is that key.  each(use) gives every thread
// its keys; those outside are passed over.
template <typename Key, typename Each>
__device__ __forceinline__ Key bound_by_steps(Key low, Key high, int n, int most, TopShared& sh,
                                              Each each) {
  int shift = max(64 - __clzll(static_cast<long long>(high - low)) - 8, 0);
  if (threadIdx.x == 0) {
    sh.need = n;
    sh.above = 0;
  }
  for (;;) {
    sh.hist[threadIdx.x] = 0;
    __syncthreads();
    each([&](Key key) {
      const Key step = (key - low) >> shift;  // far out below `low`
      if (key >= low && step < 256) atomicAdd(&sh.hist[static_cast<int>(step)], 1);
    });
    __syncthreads();
    // The step that holds the key: its own keys and those above reach `need`.
    int over = 0;
    for (int d = threadIdx.x + 1; d < 256; ++d) over += sh.hist[d];
    const int mine = sh.hist[threadIdx.x];
    const int need = sh.need, above = sh.above;
    __syncthreads();
    if (over < need && over + mine >= need) {
      sh.step = threadIdx.x;
      sh.need = need - over;
      sh.above = above + over;
      sh.done = above + over + mine <= most;
    }
    __syncthreads();
    low += static_cast<Key>(sh.step) << shift;
    if (sh.done || shift == 0) return low;
    shift = max(shift - 8, 0);
  }
}

// A bound that n of the threads' numbers reach (n <= kThreads): the n-th largest.
// 0 if fewer of them are above 0.
__device__ __forceinline__ uint32_t bound_of_threads(uint32_t most, int n, TopShared& sh) {
  const int tid = threadIdx.x;
  sh.most[tid] = most;
  __syncthreads();
  int place = 0;
  const uint4* m4 = reinterpret_cast<const uint4*>(sh.most);
#pragma unroll 4
  for (int k = 0; k < kThreads / 4; ++k) {
    const uint4 v = m4[k];
    place += (v.x > most || (v.x == most && 4 * k < tid)) ? 1 : 0;
    place += (v.y > most || (v.y == most && 4 * k + 1 < tid)) ? 1 : 0;
    place += (v.z > most || (v.z == most && 4 * k + 2 < tid)) ? 1 : 0;
    place += (v.w > most || (v.w == most && 4 * k + 3 < tid)) ? 1 : 0;
  }
  if (place == n - 1) sh.bound = most;
  __syncthreads();
  return sh.bound;
}

// The same from the largest of every four threads (n <= kThreads / 4), by every wave
// for itself: a quarter of the numbers, a sixteenth of the comparisons, and a bound
// that hardly more groups reach as long as n is small beside them (at n = 20 some 24
// of 1,187).  Below -inf's number if fewer than n of the quads have a group.
__device__ __forceinline__ uint32_t bound_of_quads(uint32_t most, int n, TopShared& sh) {
  const int tid = threadIdx.x, lane = tid & 63;
  auto step = [](uint32_t v, auto ctrl) {
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
                      0, static_cast<int>(v), decltype(ctrl)::value, 0xF, 0xF, true)));
  };
  most = step(most, std::integral_constant<int, 0xB1>{});  // quad_perm [1, 0, 3, 2]
  most = step(most, std::integral_constant<int, 0x4E>{});  // quad_perm [2, 3, 0, 1]
  if ((tid & 3) == 0) sh.most[tid >> 2] = most;
  __syncthreads();
  const uint32_t mine = sh.most[lane];
  int above = 0;  // strictly
  const uint4* m4 = reinterpret_cast<const uint4*>(sh.most);
#pragma unroll 4
  for (int k = 0; k < 16; ++k) {
    const uint4 v = m4[k];
    above += (v.x > mine ? 1 : 0) + (v.y > mine ? 1 : 0) + (v.z > mine ? 1 : 0) +
             (v.w > mine ? 1 : 0);
  }
  // The n-th largest is the least of those with fewer than n above them.
  uint32_t least = above < n ? mine : 0xffffffffu;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1)
    least = min(least, static_cast<uint32_t>(__shfl_xor(static_cast<int>(least), d, 64)));
  return least;
}

// The least of all threads' k-th largest of the numbers they hold (k <= kHeldGroups).
__device__ __forceinline__ uint32_t low_of_held(const uint32_t (&held)[kHeldGroups], int k,
                                                TopShared& sh) {
  uint32_t low = 0;
#pragma unroll
  for (int i = 0; i < kHeldGroups; ++i) {
    int above = 0;  // strictly
#pragma unroll
    for (int j = 0; j < kHeldGroups; ++j) above += held[j] > held[i] ? 1 : 0;
    int reach = 0;
#pragma unroll
    for (int j = 0; j < kHeldGroups; ++j) reach += held[j] >= held[i] ? 1 : 0;
    if (above < k && reach >= k) low = held[i];
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1)
    low = min(low, static_cast<uint32_t>(__shfl_xor(static_cast<int>(low), d, 64)));
  if ((threadIdx.x & 63) == 0) sh.low[threadIdx.x >> 6] = low;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) low = min(low, sh.low[w]);
  return low;
}

// Adds the first n - n_cand entries by id that equal a number, of which there are
// as many, to sh.cand.  Masks leave rows that end in the order of ids soon: the first
// step finds all unless most of the first ids are allowed.
template <typename T>
__device__ __forceinline__ void add_equal(const T* row, int vocab, uint32_t number, int n,
                                          TopShared& sh) {
  constexpr int kRun = 8;
  const int tid = threadIdx.x, lane = tid & 63;
  int at = sh.n_cand;
  __syncthreads();
  for (int64_t base = 0; base < vocab && at < n; base += kThreads * kRun) {
    const int64_t id = base + tid * kRun;
    uint32_t hits = 0;
#pragma unroll
    for (int u = 0; u < kRun; ++u)
      if (id + u < vocab && order_of(static_cast<float>(row[id + u])) == number) hits |= 1u << u;
    const int mine = __popc(hits);
    int before = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(before, d, 64);
      before += lane >= d ? up : 0;
    }
    if (lane == 63) sh.wave_n[tid >> 6] = before;
    before -= mine;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      before += w < tid >> 6 ? sh.wave_n[w] : 0;
      total += sh.wave_n[w];
    }
    for (int place = at + before; hits != 0 && place < n; ++place, hits &= hits - 1)
      sh.cand[place] = static_cast<uint64_t>(number) << 32 |
                       (0xffffffffu - static_cast<uint32_t>(id + __ffs(hits) - 1));
    at += total;
    __syncthreads();
  }
  if (tid == 0) sh.n_cand = n;
  __syncthreads();
}

// Entries of a row into sh.cand, the n first ones (n <= vocab) among them and none
// that comes before one that is missing; n_cand in no order.  By the whole workgroup.
template <typename T>
__device__ __forceinline__ void find_candidates(const T* row, int vocab, const Groups& gs,
                                                const float* groups, float st_m, int n,
                                                TopShared& sh) {
  constexpr int VN = Vec<T>::n;
  const int tid = threadIdx.x;
  const Shape f = stats_shape(row, vocab);
  // The slabs that the row reaches come first.
  const int full = f.whole / gs.chunk_len;
  const int slabs = full * gs.slabs + (f.whole - full * gs.chunk_len + kSlab - 1) / kSlab;
  const int live = slabs * gs.per_slab();
  // A thread's groups, the first ones' largest entries in registers.
  uint32_t held[kHeldGroups];
  const int held_end = kHeldGroups * kThreads;
  auto each_group = [&](auto use) {
#pragma unroll
    for (int k = 0; k < kHeldGroups; ++k)
      if (tid + k * kThreads < live) use(tid + k * kThreads, held[k]);
#pragma unroll 8
    for (int g = held_end + tid; g < live; g += kThreads) use(g, order_of(groups[g]));
  };
  // All entries that reach a bound, unless there are too many.
  auto collect = [&](uint32_t bound) {
    if (tid == 0) sh.n_groups = sh.n_cand = 0;
    __syncthreads();
    each_group([&](int g, uint32_t top) {
      if (top < bound) return;
      const int at = atomicAdd(&sh.n_groups, 1);
      if (at < kListedGroups) sh.group[at] = g;
    });
    __syncthreads();
    const int count = sh.n_groups;
    if (count > kListedGroups) return false;
    auto add = [&](float x, int id) {
      if (order_of(x) < bound) return;
      const int at = atomicAdd(&sh.n_cand, 1);
      if (at < kCandidates) sh.cand[at] = entry_key(x, id);
    };
    if (tid < f.edge) {
      const int at = f.template at<T>(tid);
      add(static_cast<float>(row[at]), at);
    }
    // A vector of a group; several groups' loads on their way.
    constexpr int kAtOnce = 4;
    const int lanes = 1 << gs.bits, vecs = lanes * kBatch, step = kThreads / vecs;
    const int vec = ((tid & (vecs - 1)) >> gs.bits) * kThreads + (tid & (lanes - 1));
    for (int k0 = tid / vecs; k0 < count; k0 += kAtOnce * step) {
      typename Vec<T>::Type w[kAtOnce];
      int at[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int k = k0 + u * step;
        at[u] = -1;
        if (k >= count) continue;
        const int g = sh.group[k], slab = g / gs.per_slab(), c = slab / gs.slabs;
        const int64_t first = static_cast<int64_t>(c) * gs.chunk_len;
        const int64_t v = first + (slab - c * gs.slabs) * kSlab +
                          (g & (gs.per_slab() - 1)) * lanes + vec;
        if (v >= min(first + gs.chunk_len, static_cast<int64_t>(f.whole))) continue;
        at[u] = f.head + static_cast<int>(v) * VN;
        w[u] = *reinterpret_cast<const typename Vec<T>::Type*>(row + at[u]);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (at[u] < 0) continue;
#pragma unroll
        for (int e = 0; e < VN; ++e) add(static_cast<float>(w[u][e]), at[u] + e);
      }
    }
    __syncthreads();
    return sh.n_cand <= kCandidates;
  };

  // A thread's own groups: twice as many as a bound needs, or it lets too many entries
  // through.  Shared ones are not counted: where fewer than n quads (8 a slab) or, above
  // kQuadMost, groups (32 a slab) have entries, the bound is -inf's number or less, every
  // entry reaches it, and a row of more than kCandidates is gone through twice in vain
  // before the steps below.  640 rows, us (20 alternatives from 8,580 fp32 and 17,160 bf16
  // entries on, and 40 from 17,284 and 34,568 on, have a bound): fp32 4,096, n = 5 17, 20
  // 47; 8,192, 20 73; 9,000, 20 25, 40 85; 16,384, 40 140; bf16 32,000, n = 20 33, 40 222.
  if (gs.bits != 0 || live >= 2 * n) {
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < kHeldGroups; ++k) {
      const int g = tid + k * kThreads;
      held[k] = g < live ? order_of(groups[g]) : 0u;
    }
    uint32_t bound;
    if (gs.bits != 0) {
      each_group([&](int, uint32_t top) { most = max(most, top); });
      bound = n <= kQuadMost ? bound_of_quads(most, n, sh) : bound_of_threads(most, n, sh);
    } else {
      const uint32_t low = low_of_held(held, (n + kThreads - 1) / kThreads, sh);
      bound = bound_by_steps(low, order_of(st_m), n, n + n / 8, sh, [&](auto use) {
        each_group([&](int, uint32_t top) { use(top); });
      });
    }
    // Too many: equal entries, masked ones most often.  Then those above, and of the
    // equal ones the first.  Still too many: the steps below, as where likely tokens lie
    // side by side (640 x 151,936 fp32, logits that rise with the ids, n = 20: 1,140 us
    // where 88 are usual).
    for (int above = 0; above < 2; ++above) {
      if (collect(bound + above)) {
        if (sh.n_cand < n) add_equal(row, vocab, bound, n, sh);
        return;
      }
      __syncthreads();
    }
  }
  // No bound, or one that lets too many through: few groups beside n (rows shorter than
  // 32 n fp32 or 64 n bf16 entries for a thread's own groups, 128 n and 256 n for shared
  // ones, 512 n and 1,024 n up to kQuadMost).  The row is gone through again, at least
  // twice (1,000 x 4,000 fp32, n = 300 78 us).
  auto each_entry = [&](auto use) {
    for (int64_t i = tid; i < vocab; i += kThreads)
      use(entry_key(static_cast<float>(row[i]), static_cast<int>(i)));
  };
  const uint64_t bound =
      bound_by_steps(uint64_t{0}, ~uint64_t{0}, n, kCandidates, sh, each_entry);
  if (tid == 0) sh.n_cand = 0;
  __syncthreads();
  each_entry([&](uint64_t key) {
    if (key >= bound) sh.cand[atomicAdd(&sh.n_cand, 1)] = key;
  });
  __syncthreads();
}

// Puts sh.cand in falling order (bitonic sort).  More than kThreads of them: a place
// counted for each takes as many comparisons as the square.
__device__ __forceinline__ void sort_candidates(int count, TopShared& sh) {
  int size = kThreads;
  while (size < count) size *= 2;
  for (int i = count + static_cast<int>(threadIdx.x); i < size; i += kThreads) sh.cand[i] = 0;
  __syncthreads();
  for (int run = 2; run <= size; run *= 2) {
    for (int apart = run / 2; apart > 0; apart /= 2) {
      for (int p = threadIdx.x; p < size / 2; p += kThreads) {
        const int i = (p & ~(apart - 1)) * 2 + (p & (apart - 1)), j = i + apart;
        const uint64_t a = sh.cand[i], b = sh.cand[j];
        if (((i & run) == 0) == (a < b)) {
          sh.cand[i] = b;
          sh.cand[j] = a;
        }
      }
      __syncthreads();
    }
  }
}

// A row that is left out, and one with a bad status.
__device__ __forceinline__ void topn_no_row(const TopnOut& o, int64_t r, int status) {
  const bool bad = status != TS_ROW_OK;
  if (threadIdx.x == 0) {
    if (o.logprobs) {
      o.logprobs[r] = bad ? NAN : 0.0f;
      if (o.ranks) o.ranks[r] = 0;
    }
    if (o.entropies) o.entropies[r] = bad ? NAN : 0.0f;
    if (o.row_stats) o.row_stats[2 * r] = o.row_stats[2 * r + 1] = bad ? NAN : 0.0f;
    if (o.row_status) o.row_status[r] = status;
  }
  for (int i = threadIdx.x; i < o.n; i += kThreads) {
    o.topn_ids[r * o.n + i] = -1;
    o.topn_logprobs[r * o.n + i] = bad ? NAN : -INFINITY;
  }
}

// A row's outputs from its joined statistics (held by the first threads), the
// number of entries before its token, and its groups.  By the whole workgroup.
template <typename T>
__device__ __forceinline__ void finish_topn(const T* row, int64_t r, int vocab, int token,
                                            bool has_token, float xt, RowStats& st, int better,
                                            const Groups& gs, const float* groups, const Cut& cut,
                                            const Scale& sc, const TopnOut& o, TopShared& sh) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    sh.wave_part[0] = Part{st.s, st.u, st.m, 0.0f};
    sh.first_id = has_token ? token : 0;
  }
  const int before = group_count(better, sh.wave_n);  // waits for the others too
  st.m = sh.wave_part[0].m;
  st.s = sh.wave_part[0].s;
  st.u = sh.wave_part[0].u;
  const int status = has_token && token >= vocab ? TS_ROW_BAD_PARAMS
                     : fabsf(st.m) < INFINITY    ? TS_ROW_OK
                                                 : TS_ROW_BAD_LOGITS;
  if (status != TS_ROW_OK) {
    topn_no_row(o, r, status);
    return;
  }
  const int n = min(o.n, vocab);
  uint64_t key = 0;
  int place = n;
  bool sorted = false;
  if (n > 0) {
    find_candidates(row, vocab, gs, groups, st.m, n, sh);
    const int count = sh.n_cand;
    sorted = count > kThreads;
    if (sorted) {
      sort_candidates(count, sh);
      if (tid == 0) sh.first_id = static_cast<int>(0xffffffffu - static_cast<uint32_t>(sh.cand[0]));
    } else if (tid < count) {
      key = sh.cand[tid];
      place = 0;
      for (int k = 0; k < count; ++k) place += sh.cand[k] > key ? 1 : 0;
      if (place == 0) sh.first_id = static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
    }
    __syncthreads();
  }
  // The digits of 1 - p of the one token that may have p next to 1.
  if (tid < 64) {
    const int first = sh.first_id;
    const float x1 = n > 0 ? st.m : has_token ? xt : -INFINITY;
    if (tid < kBatch && next_to_one(st.m, st.s, first, vocab, x1)) {
      const Shape f = stats_shape(row, vocab);
      TokenBatch<T, kBatch> batch;
      batch.load(row, f, cut.chunks == 1 ? max(f.whole, 1) : cut.len, kThreads, first);
      st.s += batch.lost(st.m, sc);
    }
    if (tid == 0) {
      sh.s = st.s;
      sh.ln_s = log(st.s);
    }
  }
  __syncthreads();
  const double ln_s = sh.ln_s;
  if (tid == 0) {
    if (o.logprobs) {
      o.logprobs[r] = static_cast<float>((static_cast<double>(xt) - st.m) * sc.inv_t - ln_s);
      if (o.ranks) o.ranks[r] = before + 1;
    }
    if (o.entropies) o.entropies[r] = static_cast<float>(ln_s - st.u * M_LN2 / sh.s);
    if (o.row_stats) {
      o.row_stats[2 * r] = st.m;
      o.row_stats[2 * r + 1] = static_cast<float>(sh.s);
    }
    if (o.row_status) o.row_status[r] = TS_ROW_OK;
  }
  auto put = [&](int at, uint64_t k) {
    const float x = number_of(static_cast<uint32_t>(k >> 32));
    o.topn_ids[r * o.n + at] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
    o.topn_logprobs[r * o.n + at] =
        static_cast<float>((static_cast<double>(x) - st.m) * sc.inv_t - ln_s);
  };
  if (sorted) {
    for (int i = tid; i < n; i += kThreads) put(i, sh.cand[i]);
  } else if (place < n) {
    put(place, key);
  }
  for (int i = n + tid; i < o.n; i += kThreads) {
    o.topn_ids[r * o.n + i] = -1;
    o.topn_logprobs[r * o.n + i] = -INFINITY;
  }
}

// Statistics and outputs in one launch want 157 to 178 registers.  Four workgroups a CU,
// 128 registers and some spilled (6 to 35), are the better half of the time.  us with four
// and three: 20 alternatives, 640 x 32,000 fp32 29 and 27, bf16 33 and 27; 4,000 x 32,000
// 143 and 134, 123 and 111; 100 of them, fp32 192 and 207; 5, 4,000 x 4,096 fp32 46 and
// 54, 4,000 x 8,192 bf16 67 and 60.  Two: 27, 36, 135, 144, 208, 54 and 82.
template <bool ENT, typename T>
__global__ __launch_bounds__(kThreads, 4) void topn_whole_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ tokens,
    Scale sc, Cut cut, Groups gs, float* groups, TopnOut o) {
  __shared__ TopShared sh;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const bool has_token = tokens != nullptr;
    const int token = has_token ? tokens[r] : -1;
    if (has_token && token < 0) {
      topn_no_row(o, r, TS_ROW_OK);
      continue;
    }
    const T* rx = x + r * ld;
    const float xt = has_token ? static_cast<float>(rx[min(token, vocab - 1)]) : INFINITY;
    float* gr = groups + r * gs.per_row;
    TopVisit<T> visit = make_visit<T>(stats_shape(rx, vocab), o.n > 0 ? gr : nullptr, gs.bits, 0,
                                      xt, token);
    RowStats st;
    st.m = -INFINITY;
    st.s = st.u = 0.0;
    row_stats<T, ENT, kThreads>(rx, vocab, 0, vocab / Vec<T>::n, true, sc, st.m, st.s, st.u,
                                &visit);
    join_group<ENT, kThreads>(st.m, st.s, st.u, sc, sh.wave_part);
    __syncthreads();
    finish_topn(rx, r, vocab, token, has_token, xt, st, visit.count(), gs, gr, cut, sc, o, sh);
    __syncthreads();
  }
}

template <bool ENT, typename T>
__global__ __launch_bounds__(kThreads) void topn_stats_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ tokens,
    Scale sc, Cut cut, Groups gs, float* __restrict__ groups, Part* __restrict__ parts,
    int* __restrict__ betters, int want_groups) {
  __shared__ Part wave_part[kThreads / 64];
  __shared__ int wave_n[kThreads / 64];
  const int tid = threadIdx.x;
  const int64_t total = static_cast<int64_t>(rows) * cut.chunks;
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
    const int row = static_cast<int>(b / cut.chunks), chunk = static_cast<int>(b % cut.chunks);
    const int token = tokens ? tokens[row] : -1;
    if (tokens && token < 0) continue;
    const T* rx = x + static_cast<int64_t>(row) * ld;
    const float xt = tokens ? static_cast<float>(rx[min(token, vocab - 1)]) : INFINITY;
    float* gr = groups + static_cast<int64_t>(row) * gs.per_row + chunk * gs.slabs * gs.per_slab();
    TopVisit<T> visit = make_visit<T>(stats_shape(rx, vocab), want_groups ? gr : nullptr,
                                      gs.bits, chunk * cut.len, xt, token);
    float m = -INFINITY;
    double s = 0.0, u = 0.0;
    row_stats<T, ENT, kThreads>(rx, vocab, chunk * cut.len, (chunk + 1) * cut.len,
                                chunk == cut.chunks - 1, sc, m, s, u, &visit);
    join_group<ENT, kThreads>(m, s, u, sc, wave_part);
    const int n = group_count(visit.count(), wave_n);
    if (tid == 0) {
      parts[b] = Part{s, u, m, 0.0f};
      betters[b] = n;
    }
    __syncthreads();
  }
}

// A row's latency from records to outputs, 9 us, is what bounds it, so the number of
// rows on a CU counts: four with 128 registers (three with 152: 1,021 x 100,277 bf16
// 75 us and 64, 4,000 x 40,000 118 and 108; five with 96 spill: 68 and 119).  A wave
// a row, four rows a workgroup, takes longer yet (640 x 151,936 fp32, 20 alternatives
// 117 us and 85).
template <bool ENT, typename T>
__global__ __launch_bounds__(kThreads, 4) void topn_rows_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ tokens,
    Scale sc, Cut cut, Groups gs, const float* __restrict__ groups,
    const Part* __restrict__ parts, const int* __restrict__ betters, TopnOut o) {
  __shared__ TopShared sh;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const bool has_token = tokens != nullptr;
    const int token = has_token ? tokens[r] : -1;
    if (has_token && token < 0) {
      topn_no_row(o, r, TS_ROW_OK);
      continue;
    }
    const T* rx = x + r * ld;
    const float xt = has_token ? static_cast<float>(rx[min(token, vocab - 1)]) : INFINITY;
    RowStats st;
    st.m = -INFINITY;
    st.s = st.u = 0.0;
    int better = 0;
    for (int i = threadIdx.x; i < cut.chunks; i += kThreads) {
      const Part p = parts[r * cut.chunks + i];
      const float top = max_nan(st.m, p.m), ref = top == -INFINITY ? 0.0f : top;
      const float d0 = fmaxf(st.m - ref, sc.floor), d1 = fmaxf(p.m - ref, sc.floor);
      const double f0 = exp_t(d0, sc), f1 = exp_t(d1, sc);
      if (ENT) st.u = f0 * (st.u + log2_t(d0, sc) * st.s) + f1 * (p.u + log2_t(d1, sc) * p.s);
      st.s = f0 * st.s + f1 * p.s;
      st.m = top;
      better += betters[r * cut.chunks + i];
    }
    join_group<ENT, kThreads>(st.m, st.s, st.u, sc, sh.wave_part);
    __syncthreads();
    finish_topn(rx, r, vocab, token, has_token, xt, st, better, gs,
                groups + r * gs.per_row, cut, sc, o, sh);
    __syncthreads();
  }
}

// ------------------------------------------------------------------ listed
// Whether none of a row's ids is used; by the whole workgroup.
__device__ __forceinline__ bool none_listed(const int32_t* ids, int n) {
  bool any = false;
  for (int i = threadIdx.x; i < n; i += kThreads) any |= ids[i] >= 0;
  return __syncthreads_or(any) == 0;
}

// What a row that is left out writes, or one with a bad status; by a wave.
__device__ __forceinline__ void listed_no_row(const ListedOut& o, const int32_t* ids, int64_t r,
                                              int status, int lane) {
  const float v = status == TS_ROW_OK ? 0.0f : NAN;
  for (int i = lane; i < o.n; i += 64) o.logprobs[r * o.n + i] = ids[i] < 0 ? 0.0f : v;
  if (lane != 0) return;
  if (o.entropies) o.entropies[r] = v;
  if (o.row_stats) o.row_stats[2 * r] = o.row_stats[2 * r + 1] = v;
  if (o.row_status) o.row_status[r] = status;
}

// A row's outputs from its joined statistics, which every lane of the wave has.
// `len`: how the row was cut.
template <typename T>
__device__ __forceinline__ void finish_listed(const T* row, int64_t r, int vocab,
                                              const int32_t* ids, RowStats& st, int len,
                                              const Scale& sc, const ListedOut& o, int lane) {
  bool past = false;
  int first = -1;
  for (int i = lane; i < o.n; i += 64) {
    const int id = ids[i];
    past |= id >= vocab;
    if (id >= 0 && id < vocab && static_cast<float>(row[id]) == st.m) first = id;
  }
  const int status = __any(past) ? TS_ROW_BAD_PARAMS
                     : fabsf(st.m) < INFINITY ? TS_ROW_OK : TS_ROW_BAD_LOGITS;
  if (status != TS_ROW_OK) {
    listed_no_row(o, ids, r, status, lane);
    return;
  }
  // At most one id has p next to 1; the digits of its 1 - p.
  const uint64_t holds = __ballot(first >= 0);
  if (holds != 0) {
    first = __shfl(first, __ffsll(static_cast<unsigned long long>(holds)) - 1, 64);
    if (next_to_one(st.m, st.s, first, vocab, st.m)) {
      double more = 0.0;
      if (lane < kBatch) {
        TokenBatch<T, kBatch> batch;
        batch.load(row, stats_shape(row, vocab), len, kThreads, first);
        more = batch.lost(st.m, sc);
      }
      st.s += __shfl(more, 0, 64);
    }
  }
  const double ln_s = log(st.s);
  for (int i = lane; i < o.n; i += 64) {
    const int id = ids[i];
    o.logprobs[r * o.n + i] =
        id < 0 ? 0.0f
               : static_cast<float>((static_cast<double>(static_cast<float>(row[id])) - st.m) *
                                        sc.inv_t - ln_s);
  }
  if (lane != 0) return;
  if (o.entropies) o.entropies[r] = static_cast<float>(ln_s - st.u * M_LN2 / st.s);
  if (o.row_stats) {
    o.row_stats[2 * r] = st.m;
    o.row_stats[2 * r + 1] = static_cast<float>(st.s);
  }
  if (o.row_status) o.row_status[r] = TS_ROW_OK;
}

template <bool ENT, typename T>
__global__ __launch_bounds__(kThreads) void listed_whole_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ ids,
    Scale sc, ListedOut o) {
  __shared__ Part wave_part[kThreads / 64];
  const int tid = threadIdx.x;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int32_t* row_ids = ids + r * o.n;
    if (none_listed(row_ids, o.n)) {
      if (tid < 64) listed_no_row(o, row_ids, r, TS_ROW_OK, tid);
      continue;
    }
    const T* rx = x + r * ld;
    RowStats st;
    st.m = -INFINITY;
    st.s = st.u = 0.0;
    row_stats<T, ENT, kThreads>(rx, vocab, 0, vocab / Vec<T>::n, true, sc, st.m, st.s, st.u);
    join_group<ENT, kThreads>(st.m, st.s, st.u, sc, wave_part);
    if (tid < 64) {
      st.m = __shfl(st.m, 0, 64);
      st.s = __shfl(st.s, 0, 64);
      st.u = __shfl(st.u, 0, 64);
      finish_listed(rx, r, vocab, row_ids, st, max(stats_shape(rx, vocab).whole, 1), sc, o, tid);
    }
    __syncthreads();
  }
}

template <bool ENT, typename T>
__global__ __launch_bounds__(kThreads) void listed_stats_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ ids,
    int n, Scale sc, Cut cut, Part* __restrict__ parts) {
  __shared__ Part wave_part[kThreads / 64];
  const int64_t total = static_cast<int64_t>(rows) * cut.chunks;
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
    const int row = static_cast<int>(b / cut.chunks), chunk = static_cast<int>(b % cut.chunks);
    if (none_listed(ids + static_cast<int64_t>(row) * n, n)) continue;
    float m = -INFINITY;
    double s = 0.0, u = 0.0;
    row_stats<T, ENT, kThreads>(x + static_cast<int64_t>(row) * ld, vocab, chunk * cut.len,
                                (chunk + 1) * cut.len, chunk == cut.chunks - 1, sc, m, s, u);
    join_group<ENT, kThreads>(m, s, u, sc, wave_part);
    if (threadIdx.x == 0) parts[b] = Part{s, u, m, 0.0f};
    __syncthreads();
  }
}

// A wave a row.
template <bool ENT, typename T>
__global__ __launch_bounds__(kThreads) void listed_rows_kernel(
    const T* __restrict__ x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ ids,
    Scale sc, Cut cut, const Part* __restrict__ parts, ListedOut o) {
  const int lane = threadIdx.x & 63;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
       r < rows; r += static_cast<int64_t>(gridDim.x) * (kThreads / 64)) {
    const int32_t* row_ids = ids + r * o.n;
    bool any = false;
    for (int i = lane; i < o.n; i += 64) any |= row_ids[i] >= 0;
    if (!__any(any)) {
      listed_no_row(o, row_ids, r, TS_ROW_OK, lane);
      continue;
    }
    RowStats st;
    st.m = -INFINITY;
    st.s = st.u = 0.0;
    for (int i = lane; i < cut.chunks; i += 64) {
      const Part p = parts[r * cut.chunks + i];
      const float top = max_nan(st.m, p.m), ref = top == -INFINITY ? 0.0f : top;
      const float d0 = fmaxf(st.m - ref, sc.floor), d1 = fmaxf(p.m - ref, sc.floor);
      const double f0 = exp_t(d0, sc), f1 = exp_t(d1, sc);
      if (ENT) st.u = f0 * (st.u + log2_t(d0, sc) * st.s) + f1 * (p.u + log2_t(d1, sc) * p.s);
      st.s = f0 * st.s + f1 * p.s;
      st.m = top;
    }
    join_lanes<ENT>(st.m, st.s, st.u, 64, sc);
    finish_listed(x + r * ld, r, vocab, row_ids, st, cut.len, sc, o, lane);
  }
}

// A row's dense entries: entry j is e_j (a + b log2 e_j).
struct DenseGrad {
  float m, a, b;

  template <bool ENT>
  __device__ __forceinline__ float entry(float x, const Scale& sc) const {
    const float k = log2_t(x - m, sc);
    const float ex = __builtin_amdgcn_exp2f(k);
    return ENT ? ex * fmaf(b, fmaxf(k, kLeastLog2), a) : ex * a;
  }
};

// A workgroup writes a chunk of a row's dense part, from the last slab to the first,
// then the listed entries in it.  Their values need no logit, only the forward
// pass's log-probabilities, so the gradient may replace the logits.  An id that is
// listed several times is written once, by its first place, from the sum of its
// gradients.  The first slab's loads are on their way while the row's coefficients
// are worked out (1,021 x 100,277 bf16, 64 listed tokens and the entropy: 127 us
// without that, 85 so).  640 x 151,936 fp32 takes 125 us (6.2 TB/s); with a row
// a workgroup 167 where this took 135, with five workgroups a CU 146.
template <typename T, bool ENT>
__global__ __launch_bounds__(kThreads, 4) void listed_grad_kernel(
    const T* x, int64_t ld, int rows, int vocab, const int32_t* __restrict__ ids, Scale sc,
    Cut cut, ListedGrad g, T* d, int64_t ldd) {
  constexpr int VN = Vec<T>::n;
  using V = typename Vec<T>::Type;
  __shared__ double wave_sum[kThreads / 64];
  __shared__ int4 s_ids[TS_MAX_LISTED / 4];
  __shared__ float s_g[TS_MAX_LISTED];
  const int tid = threadIdx.x;
  const int quads = (g.n + 3) / 4;
  const int64_t total = static_cast<int64_t>(rows) * cut.chunks;
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
    // Last row first, as the end of the logits is what the caches still hold.
    const int row = rows - 1 - static_cast<int>(b / cut.chunks);
    const int chunk = cut.chunks - 1 - static_cast<int>(b % cut.chunks);
    const int64_t at = static_cast<int64_t>(row) * g.n;
    const T* rx = x + static_cast<int64_t>(row) * ld;
    T* rd = d + static_cast<int64_t>(row) * ldd;
    const Shape f = row_shape(rd, vocab);
    const int v0 = chunk * cut.len, end = min(v0 + cut.len, f.whole);
    const bool last = chunk == cut.chunks - 1;
    const T* body = rx + f.head;
    T* out = rd + f.head;
    int v = v0 + (end - 1 - v0) / kSlab * kSlab;
    Slab<T, kThreads> next;
    if (v0 < end) next.load(body, v, end);

    const double dh_row = ENT ? static_cast<double>(g.grad_entropies[row]) : 0.0;
    const float m = g.row_stats[2 * static_cast<int64_t>(row)];
    const double s = g.row_stats[2 * static_cast<int64_t>(row) + 1];
    const double h_row = ENT ? static_cast<double>(g.entropies[row]) : 0.0;
    double sum = 0.0;
    bool any = false;
    for (int i = tid; i < 4 * quads; i += kThreads) {
      const int id = i < g.n ? ids[at + i] : -1;
      const float gi = id < 0 ? 0.0f : g.grad_logprobs[at + i];
      reinterpret_cast<int*>(s_ids)[i] = id;
      s_g[i] = gi;
      sum += gi;
      any |= id >= 0 && (gi != 0.0f || dh_row != 0.0);
    }
    for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k, 64);
    if ((tid & 63) == 0) wave_sum[tid >> 6] = sum;
    const bool live = __syncthreads_or(any) != 0;
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) sum += wave_sum[w];
    const double dh = live ? dh_row : 0.0;
    const double h = dh != 0.0 ? h_row : 0.0;
    DenseGrad dense{0.0f, 0.0f, 0.0f};
    if (live) {
      dense.m = m;
      dense.a = static_cast<float>(-(sum + (dh != 0.0 ? dh * (h - log(s)) : 0.0)) * sc.inv_t / s);
      dense.b = static_cast<float>(-dh * M_LN2 * sc.inv_t / s);
    }
    const bool zero = dense.a == 0.0f && dense.b == 0.0f;
    if (last && tid < f.edge) {
      const int place = f.template at<T>(tid);
      rd[place] = static_cast<T>(
          zero ? 0.0f : dense.template entry<ENT>(static_cast<float>(rx[place]), sc));
    }
    for (; v >= v0 && v0 < end; v -= kSlab) {
      float w[kBatch][VN];
      next.unpack(w);
      if (v > v0) next.load(body, v - kSlab, end);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = v + j * kThreads + tid;
        V o;
#pragma unroll
        for (int e = 0; e < VN; ++e)
          o[e] = static_cast<T>(zero ? 0.0f : dense.template entry<ENT>(w[j][e], sc));
        if (i < end)
          __builtin_nontemporal_store(o, reinterpret_cast<V*>(out + static_cast<int64_t>(i) * VN));
      }
    }
    __syncthreads();  // before entries of the same places
    for (int i = tid; live && i < g.n; i += kThreads) {
      const int id = reinterpret_cast<const int*>(s_ids)[i];
      if (id < 0 || id >= vocab) continue;
      const int vec = (id - f.head) / VN;
      const bool in_body = id >= f.head && vec < f.whole;
      if (in_body ? vec < v0 || vec >= end : !last) continue;
      bool is_first = true;
      double mine = 0.0;
#pragma unroll 4
      for (int k = 0; k < quads; ++k) {
        const int4 q = s_ids[k];
        if (q.x != id && q.y != id && q.z != id && q.w != id) continue;
        const int four[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (four[e] != id) continue;
          is_first = is_first && 4 * k + e >= i;
          mine += s_g[4 * k + e];
        }
      }
      if (!is_first) continue;
      // g (1 - p) of its own share, -p of the others'.
      const double lp = g.logprobs[at + i], p = exp(lp);
      double value = mine * -expm1(lp) - (sum - mine) * p;
      if (ENT && dh != 0.0 && !(lp < -1e30)) value -= dh * p * (lp + h);
      rd[id] = static_cast<T>(static_cast<float>(value * sc.inv_t));
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------- workspace
struct TopnSpace {
  Part* parts;
  int* betters;
  float* groups;
  size_t bytes;
};

TopnSpace lay_out_topn(void* base, int64_t rows, int64_t vocab) {
  size_t chunks = 0, groups = 0;
  for (const int vec : {Vec<float>::n, Vec<__bf16>::n}) {
    for (const Cut& cut : {cut_rows(rows, vocab, vec), whole_cut(vocab, vec)}) {
      chunks = std::max(chunks, static_cast<size_t>(cut.chunks));
      groups = std::max(groups, static_cast<size_t>(make_groups(cut, kSharedMost + 1).per_row));
    }
  }
  char* p = static_cast<char*>(base);
  size_t at = 0;
  TopnSpace w;
  w.parts = reinterpret_cast<Part*>(p + at);
  at += round256(sizeof(Part) * static_cast<size_t>(rows) * chunks);
  w.betters = reinterpret_cast<int*>(p + at);
  at += round256(sizeof(int) * static_cast<size_t>(rows) * chunks);
  w.groups = reinterpret_cast<float*>(p + at);
  at += round256(sizeof(float) * static_cast<size_t>(rows) * groups);
  w.bytes = at;
  return w;
}

template <typename T, bool ENT>
hipError_t topn_t(const TokenRows& t, const TopnOut& o, void* ws, hipStream_t stream) {
  const Scale sc = make_scale(t.temperature);
  const TopnSpace w = lay_out_topn(ws, t.rows, t.vocab);
  const T* x = static_cast<const T*>(t.x);
  // Short rows take a workgroup each in one launch (4 x 4,096 16 us, 1,000 x 32,000
  // fp32 40 and cut up 46).  Longer ones have their outputs in a second launch, whatever
  // their number: those need 128 registers where the statistics need 80, and hold the
  // reads up (640 x 151,936 fp32, 20 alternatives 100 us in one launch, 89 in two).
  if (t.vocab <= kShortRow) {
    const Cut cut = whole_cut(t.vocab, Vec<T>::n);
    hipLaunchKernelGGL((topn_whole_kernel<ENT, T>), dim3(grid_of(t.rows)), dim3(kThreads), 0,
                       stream, x, t.ld, t.rows, t.vocab, t.tokens, sc, cut, make_groups(cut, o.n),
                       w.groups, o);
    return hipGetLastError();
  }
  // The statistics take whole bf16 rows where there are many (512 x 151,936 62 us, cut
  // up 68; 1,021 x 100,277 75 and 85; 400 x 100,000 40 and 38); fp32 ones never (1,000 x
  // 60,000 71 and 67).
  const Cut cut = Vec<T>::n > 4 && t.rows >= 512 ? whole_cut(t.vocab, Vec<T>::n)
                                                 : cut_rows(t.rows, t.vocab, Vec<T>::n);
  const Groups gs = make_groups(cut, o.n);
  hipLaunchKernelGGL((topn_stats_kernel<ENT, T>), dim3(grid_of(int64_t{t.rows} * cut.chunks)),
                     dim3(kThreads), 0, stream, x, t.ld, t.rows, t.vocab, t.tokens, sc, cut, gs,
                     w.groups, w.parts, w.betters, o.n > 0);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((topn_rows_kernel<ENT, T>), dim3(grid_of(t.rows)), dim3(kThreads), 0, stream,
                     x, t.ld, t.rows, t.vocab, t.tokens, sc, cut, gs, w.groups, w.parts, w.betters,
                     o);
  return hipGetLastError();
}

template <typename T, bool ENT>
hipError_t listed_t(const TokenRows& t, const ListedOut& o, void* ws, hipStream_t stream) {
  const Scale sc = make_scale(t.temperature);
  const T* x = static_cast<const T*>(t.x);
  if (whole_rows(t.rows, t.vocab, Vec<T>::n)) {
    hipLaunchKernelGGL((listed_whole_kernel<ENT, T>), dim3(grid_of(t.rows)), dim3(kThreads), 0,
                       stream, x, t.ld, t.rows, t.vocab, t.tokens, sc, o);
    return hipGetLastError();
  }
  const Cut cut = cut_rows(t.rows, t.vocab, Vec<T>::n);
  Part* parts = static_cast<Part*>(ws);
  hipLaunchKernelGGL((listed_stats_kernel<ENT, T>), dim3(grid_of(int64_t{t.rows} * cut.chunks)),
                     dim3(kThreads), 0, stream, x, t.ld, t.rows, t.vocab, t.tokens, o.n, sc, cut,
                     parts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((listed_rows_kernel<ENT, T>),
                     dim3(grid_of((t.rows + int64_t{kThreads / 64} - 1) / (kThreads / 64))),
                     dim3(kThreads), 0, stream, x, t.ld, t.rows, t.vocab, t.tokens, sc, cut, parts,
                     o);
  return hipGetLastError();
}

template <typename T, bool ENT>
hipError_t listed_backward_t(const TokenRows& t, const ListedGrad& g, const GradRows& d,
                             hipStream_t stream) {
  const Scale sc = make_scale(t.temperature);
  const Cut cut = cut_rows(t.rows, t.vocab, Vec<T>::n);
  hipLaunchKernelGGL((listed_grad_kernel<T, ENT>), dim3(grid_of(int64_t{t.rows} * cut.chunks)),
                     dim3(kThreads), 0, stream, static_cast<const T*>(t.x), t.ld, t.rows, t.vocab,
                     t.tokens, sc, cut, g, static_cast<T*>(d.x), d.ld);
  return hipGetLastError();
}

}  // namespace

size_t topn_workspace_size(int64_t rows, int64_t vocab) {
  return lay_out_topn(nullptr, rows, vocab).bytes;
}

size_t listed_workspace_size(int64_t rows, int64_t vocab) {
  const int chunks = std::max(cut_rows(rows, vocab, Vec<float>::n).chunks,
                              cut_rows(rows, vocab, Vec<__bf16>::n).chunks);
  return round256(sizeof(Part) * static_cast<size_t>(rows) * chunks);
}

hipError_t launch_token_logprobs_topn(const TokenRows& t, const TopnOut& o, void* ws,
                                      hipStream_t stream) {
  if (t.bf16)
    return o.entropies ? topn_t<__bf16, true>(t, o, ws, stream)
                       : topn_t<__bf16, false>(t, o, ws, stream);
  return o.entropies ? topn_t<float, true>(t, o, ws, stream)
                     : topn_t<float, false>(t, o, ws, stream);
}

hipError_t launch_token_logprobs_listed(const TokenRows& t, const ListedOut& o, void* ws,
                                        hipStream_t stream) {
  if (t.bf16)
    return o.entropies ? listed_t<__bf16, true>(t, o, ws, stream)
                       : listed_t<__bf16, false>(t, o, ws, stream);
  return o.entropies ? listed_t<float, true>(t, o, ws, stream)
                     : listed_t<float, false>(t, o, ws, stream);
}

hipError_t launch_token_logprobs_listed_backward(const TokenRows& t, const ListedGrad& g,
                                                 const GradRows& d, hipStream_t stream) {
  if (t.bf16)
    return g.grad_entropies ? listed_backward_t<__bf16, true>(t, g, d, stream)
                            : listed_backward_t<__bf16, false>(t, g, d, stream);
  return g.grad_entropies ? listed_backward_t<float, true>(t, g, d, stream)
                          : listed_backward_t<float, false>(t, g, d, stream);
}

}  // namespace ts
