// Logits of rows that each have their own low-rank adapter beside the shared
// lm_head, on gfx950:
//   logits[r, v] = sum_h x[r, h] W[v, h] + s_a sum_k B_a[v, k] u[r, k],
//   u[r, k] = sum_h x[r, h] A_a[k, h],   a = the row's adapter.
//
// Two steps.  The down step computes s_a u for every row, and each row's
// place in the order of (adapter, row).  The up step adds B_a (s_a u).
//
// u is held as three bf16 numbers whose sum is its fp32 value, so that the
// matrix cores' products with B lose nothing: rounding u to bf16 once would
// leave 2^-9 of the adapter's share in the fp32 logits.
#include <algorithm>

#include "lmhead_lora.hpp"

namespace ts {
namespace {

constexpr int kNoAdapter = -1, kBadAdapter = -2;
constexpr int kParts = 3;  // bf16 numbers that hold one fp32 value of u
constexpr int kWindow = 16;  // ranks that are worked on at a time
constexpr int kDownThreads = 256;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__host__ __device__ constexpr int padded_rank(int rank) {
  return (rank + kWindow - 1) / kWindow * kWindow;
}

// What the down step leaves, rows in the order of (adapter, row).
struct DownRows {
  __bf16* u;     // [rows][padded rank / 16][kParts][16], zeros past the rank
  int32_t* row;  // the row at this place
  int32_t* id;   // its adapter, kNoAdapter or kBadAdapter
};

// Value k of a row of u.
__device__ __forceinline__ float whole_u(const __bf16* u, int k) {
  const __bf16* part = u + k / kWindow * (kParts * kWindow) + k % kWindow;
  float sum = 0.0f;
#pragma unroll
  for (int q = kParts - 1; q >= 0; --q) sum += static_cast<float>(part[q * kWindow]);
  return sum;
}

__device__ __forceinline__ int adapter_of(int id, int n_adapters) {
  if (id >= 0 && id < n_adapters) return id;
  return id == kNoAdapter ? kNoAdapter : kBadAdapter;
}

// One workgroup per row and kWindow ranks, four ranks a wave; kDownStep
// 512-wide pieces of the row and of A are in flight at a time.  Bound by the
// L2's delivery of A, read once per row, and by HBM's where the projection has
// run since A was read: 640 rows of 4,096 at rank 32 take 16 us in that order, 64
// at rank 16 take 12.  With A in the caches they take 12 and 5; four rows a
// workgroup sharing what they have of one adapter 16 and 14 then, and four and
// eight pieces in flight 13 and 16 us at 640 rows.
constexpr int kDownStep = 2;

__global__ __launch_bounds__(kDownThreads) void lora_down_kernel(LoraArgs p, DownRows out) {
  constexpr int kWaves = kDownThreads / 64;
  constexpr int kPerWave = kWindow / kWaves;
  __shared__ int before_wave[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rp = padded_rank(p.rank);
  const int k0 = blockIdx.y * kWindow + wave * kPerWave;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const int id = adapter_of(p.ids[r], p.n_adapters);
    int before = 0;
    for (int i = tid; i < p.rows; i += kDownThreads) {
      const int other = adapter_of(p.ids[i], p.n_adapters);
      before += other < id || (other == id && i < r);
    }
    float sum[kPerWave] = {};
    if (id >= 0 && k0 < p.rank) {  // the rank is a multiple of 8, so of kPerWave
      const uint16_t* x = p.hidden + static_cast<int64_t>(r) * p.ld_hidden;
      const uint16_t* a = p.a + static_cast<int64_t>(id) * p.stride_a +
                          static_cast<int64_t>(k0) * p.ld_a;
      const unsigned hidden = p.hidden_dim;  // h0 may pass 2^31
      for (unsigned h0 = lane * 8; h0 < hidden; h0 += kDownStep * 512) {
        bf16x8 xv[kDownStep], av[kDownStep][kPerWave];
#pragma unroll
        for (int q = 0; q < kDownStep; ++q) {
          const unsigned h = min(h0 + q * 512, hidden - 8);
          xv[q] = *reinterpret_cast<const bf16x8*>(x + h);
#pragma unroll
          for (int k = 0; k < kPerWave; ++k)
            av[q][k] = *reinterpret_cast<const bf16x8*>(a + k * p.ld_a + h);
        }
#pragma unroll
        for (int q = 0; q < kDownStep; ++q) {
          if (h0 + q * 512 >= hidden) continue;
#pragma unroll
          for (int k = 0; k < kPerWave; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              sum[k] = fmaf(static_cast<float>(xv[q][e]), static_cast<float>(av[q][k][e]), sum[k]);
        }
      }
    }
    for (int d = 32; d > 0; d >>= 1) {
      before += __shfl_xor(before, d, 64);
#pragma unroll
      for (int k = 0; k < kPerWave; ++k) sum[k] += __shfl_xor(sum[k], d, 64);
    }
    if (lane == 0) before_wave[wave] = before;
    __syncthreads();
    int place = 0;
    for (int w = 0; w < kWaves; ++w) place += before_wave[w];
    if (tid == 0 && blockIdx.y == 0) {
      out.row[place] = r;
      out.id[place] = id;
    }
    const float scale = id >= 0 && p.scales ? p.scales[id] : 1.0f;
    __bf16* u = out.u + (static_cast<int64_t>(place) * rp + blockIdx.y * kWindow) * kParts +
                wave * kPerWave;
#pragma unroll
    for (int k = 0; k < kPerWave; ++k) {
      float rest = sum[k] * scale;
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        const __bf16 part = static_cast<__bf16>(rest);
        if (lane == k) u[q * kWindow + k] = part;
        // Of an infinity nothing is left (the difference would be NaN).
        rest = fabsf(static_cast<float>(part)) < INFINITY ? rest - static_cast<float>(part) : 0.0f;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The projection with the up step inside (hidden size a multiple of 64).
//
// The main loop is lmhead_logits_local's: v_mfma_f32_32x32x16_bf16, 64-wide K
// steps through LDS stages filled by direct loads (two, or more where a CU has
// few waves), the XOR swizzle of the 16-byte chunks, row tiles of an lm_head
// strip back to back on one XCD.  Rows
// are taken in the order of their adapters, through a row list for the loads
// and the stores, so a tile holds few adapters and each in one run of rows.
//
// After the last K step the same stages carry on with "panels" of B: the
// strip's BN rows of the B of four of the tile's adapters, in windows of 16
// ranks, in the stage's lm_head part.  u of those adapters' rows for the same
// 16 ranks lies in the hidden part.  Both come ahead of their use, the first
// ones under the last K steps: read from global memory where it is used, u cost
// a latency per block and slice (6 us a panel), and panels that were loaded
// after the K steps, two stages at a time, cost 64 rows with 64 adapters of
// rank 64 over 18,992 columns 122 us, not 115, with 32 of rank 16 over 151,936
// columns 259, not 253.  The windows of one panel follow each other, as they
// share B's cache lines (the other order took 64 rows with 64 adapters of rank
// 64 from 0.5 to 0.7 ms).  A 32-row block takes the adapters that its rows have,
// with u of the other rows set to 0 in the A fragment.
//
// 0 x inf is not 0, so infinities and NaN in B are set to 0 as well, and a tile
// that met one adds their products to the rows of that adapter alone after its
// logits are stored.  An infinite u would make NaN of those zeros, so where B
// has such entries u's own are set to 0 too, and their products come later with
// B's (a product that the matrix cores had already is infinite or NaN, and the
// same added again changes nothing).  A row never sees another adapter's weights,
// and what it gets does not depend on the rows beside it.  (Adding every product through a
// selection of the adapter's rows instead cost 18 us a tile of 320 x 256 with
// nine adapters of rank 32, where the main loop takes 150.)
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4u __attribute__((aligned(4)));

constexpr int kBK = 64;  // K per LDS stage
constexpr int kXcds = 8;
constexpr int kStoreStride = 36;  // floats of a row of the store scratch
constexpr int kStoreFloats = 32 * kStoreStride;

template <int LOADS, int FIRST, int NW, int AUX>
__device__ __forceinline__ void load_stage(const uint16_t* const* src, uint8_t* stage, int wave,
                                           int k0) {
#pragma unroll
  for (int q = 0; q < FIRST; ++q)
    __builtin_amdgcn_global_load_lds(src[q] + k0, stage + (wave + NW * q) * 1024, 16, 0, 0);
#pragma unroll
  for (int q = FIRST; q < LOADS; ++q)
    __builtin_amdgcn_global_load_lds(src[q] + k0, stage + (wave + NW * q) * 1024, 16, 0, AUX);
}

// The adapters of a tile's rows.  A run is the rows of one adapter.
template <int BM, int NW>
struct TileRuns {
  int row[BM];        // the row at each place, ~row for a bad adapter
  int id[BM];         // its adapter
  int adapter[BM];    // of each run
  int start[BM + 1];  // the runs' first places, and the end of the last
  int wave_runs[NW];
  int met_non_finite;
};

// Panel `pn` of window `w`: BN rows of the B of four runs, side by side, into
// the lm_head part of a stage.  Past the last run or the rank any valid
// address: those values are not used.
template <int BM, int LOADS, int A_LOADS, int NW>
__device__ __forceinline__ void lora_panel(const LoraArgs& p, const TileRuns<BM, NW>& tr, int runs,
                                           int w, int pn, int n0, int wave, int lane,
                                           uint8_t* stage) {
#pragma unroll 1
  for (int q = A_LOADS; q < LOADS; ++q) {
    const int r = 8 * (wave + NW * q) + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    const int run = min(pn * (kBK / kWindow) + (c >> 1), runs - 1);
    const int k = w * kWindow + (c & 1) * 8;
    const uint16_t* src = p.b + static_cast<int64_t>(tr.adapter[run]) * p.stride_b +
                          static_cast<int64_t>(n0 + min(r - BM, p.vocab - 1 - n0)) * p.ld_b +
                          (k < p.rank ? k : 0);
    __builtin_amdgcn_global_load_lds(src, stage + (wave + NW * q) * 1024, 16, 0, 0);
  }
}

// Window `w` of u of the tile's rows into the hidden part of a stage, kUChunks
// 16-byte chunks a row, of which the last is padding that spreads a fragment's
// 32 rows over the banks.  Blocks [from, to) of 64 chunks each.
constexpr int kUChunks = kParts * kWindow / 8 + 1;

template <int BM, int NW>
__device__ __forceinline__ void lora_rows(const DownRows& d, int rp, int w, int m0, int from,
                                          int to, int M, int wave, int lane, uint8_t* stage) {
  static_assert((BM * kUChunks + 63) / 64 <= BM / 8, "u of the rows fits");
#pragma unroll 1
  for (int q = from + wave; q < to; q += NW) {
    const int i = q * 64 + lane;
    const int place = min(m0 + i / kUChunks, M - 1);
    const int c = min(i % kUChunks, kUChunks - 2);
    const __bf16* src =
        d.u + (static_cast<int64_t>(place) * rp + w * kWindow) * kParts + c * 8;
    __builtin_amdgcn_global_load_lds(src, stage + q * 1024, 16, 0, 0);
  }
}

constexpr uint16_t kExponent = 0x7f80;  // of a bf16; all ones: infinity or NaN

__device__ __forceinline__ bf16x8 finite_part(const bf16x8& v) {
  typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
  u16x8 b = __builtin_bit_cast(u16x8, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] = (b[e] & kExponent) == kExponent ? uint16_t{0} : b[e];
  return __builtin_bit_cast(bf16x8, b);
}

// Whether one of eight bf16 is an infinity or a NaN.
__device__ __forceinline__ bool not_finite(const bf16x8& v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 b = __builtin_bit_cast(u32x4, v);
  // Adding 1 to an exponent of all ones carries into the sign's place.
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= (b[i] & 0x7f807f80u) + 0x00800080u;
  return (any & 0x80008000u) != 0;
}

// Waits until at most N of the wave's loads are on their way and its LDS reads
// are done, then for the other waves.  Neither a fence nor __syncthreads(), which
// would wait for the direct loads of the later stages as well.
template <int N>
__device__ __forceinline__ void wait_stage() {
  static_assert(N < 64, "vmcnt has six bits");
  // vmcnt in bits 3:0 and 15:14, lgkmcnt 0, expcnt left at its maximum.
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
  asm volatile("s_barrier" ::: "memory");
}

// STAGES: LDS stages, of which all but one are loaded ahead.
// WAVES: waves that a SIMD is to hold, which bounds the registers.
template <int BM, int BN, int WAVES_M, int WAVES_N, int AUX, int STAGES, int WAVES>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, WAVES) void lora_gemm_kernel(
    LoraArgs p, DownRows d, int tiles_m, int tiles_total, int tiles_per_xcd) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  constexpr int TM = WM / 32, TN = WN / 32;
  constexpr int ROWS = BM + BN;
  constexpr int STAGE = ROWS * 128;
  constexpr int LOADS = ROWS / 8 / NW;
  constexpr int A_LOADS = BM / 8 / NW;
  static_assert(ROWS / 8 % NW == 0 && BM / 8 % NW == 0, "blocks split evenly over the waves");
  static_assert(WM % 32 == 0 && WN % 32 == 0, "wave tile of whole 32x32 blocks");
  static_assert(NW * kStoreFloats * 4 <= STAGES * STAGE, "store scratch fits the stages");
  static_assert(BM <= 64 * NW, "a thread for every row of the tile");

  // One array: with several, the compiler makes every fragment read wait for
  // the direct loads of the next stage.
  using Runs = TileRuns<BM, NW>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * STAGE + sizeof(Runs)];
  Runs& tr = *reinterpret_cast<Runs*>(lds + STAGES * STAGE);

  const int bid = blockIdx.x;
  const int tile = (bid % kXcds) * tiles_per_xcd + bid / kXcds;
  if (tile >= tiles_total) return;
  const int m0 = tile % tiles_m * BM, n0 = tile / tiles_m * BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm0 = (wave / WAVES_N) * WM, wn0 = (wave % WAVES_N) * WN;
  const int M = p.rows, N = p.vocab;

  // Source of this lane's 16 bytes in each of the wave's blocks: chunk c of
  // LDS row r sits at c ^ ((r >> 1) & 7).
  const int chunk_row = lane >> 3;
  const uint16_t* src[LOADS];
#pragma unroll
  for (int q = 0; q < LOADS; ++q) {
    const int r = 8 * (wave + NW * q) + chunk_row;
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    if (q < A_LOADS)
      src[q] = p.hidden + static_cast<int64_t>(d.row[min(m0 + r, M - 1)]) * p.ld_hidden + c * 8;
    else
      src[q] = p.lm_head + static_cast<int64_t>(n0 + min(r - BM, N - 1 - n0)) * p.ld_lm_head +
               c * 8;
  }
  const bool in = tid < BM && m0 + tid < M;
  const int my_id = in ? d.id[m0 + tid] : kNoAdapter;
  const int my_row = in ? d.row[m0 + tid] : 0;
  if (tid < BM) {
    tr.id[tid] = my_id;
    tr.row[tid] = my_id == kBadAdapter ? ~my_row : my_row;
  }
  if (tid == 0) tr.met_non_finite = 0;
  const int ksteps = p.hidden_dim / kBK;
#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st)
    if (st < ksteps) load_stage<LOADS, A_LOADS, NW, AUX>(src, lds + st * STAGE, wave, st * kBK);

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const int frow = lane & 31, fhalf = lane >> 5;
  int aoff[TM], boff[TN], aswz[TM], bswz[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = wm0 + i * 32 + frow;
    aoff[i] = r * 128;
    aswz[i] = (r >> 1) & 7;
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int r = BM + wn0 + j * 32 + frow;
    boff[j] = r * 128;
    bswz[j] = (r >> 1) & 7;
  }
  auto frags = [&](int buf, int kk, bf16x8 (&af)[TM], bf16x8 (&bfr)[TN]) {
    const int chunk = kk * 2 + fhalf;
    const uint8_t* base = lds + buf * STAGE;
#pragma unroll
    for (int i = 0; i < TM; ++i)
      af[i] = *reinterpret_cast<const bf16x8*>(base + aoff[i] + ((chunk ^ aswz[i]) << 4));
#pragma unroll
    for (int j = 0; j < TN; ++j)
      bfr[j] = *reinterpret_cast<const bf16x8*>(base + boff[j] + ((chunk ^ bswz[j]) << 4));
  };

  // Waits until the step's loads have landed in LDS for every wave; the stage of
  // the step before is free then.  A wave's loads land in order, LOADS of them a
  // step; `full`: the later STAGES - 2 steps are all on their way.
  auto wait_step = [&](bool full) {
    if constexpr (STAGES == 2) {
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    } else {
      if (full)
        wait_stage<LOADS * (STAGES - 2)>();
      else
        wait_stage<0>();
    }
  };

  // MFMAs between two fragment reads, or reads after each MFMA where those are
  // fewer.
  constexpr int kMfmas = TM * TN, kReads = TM + TN;
  constexpr bool kMoreReads = kMfmas < kReads;
  constexpr int kGroupMfmas = kMoreReads ? 1 : kMfmas / kReads;
  constexpr int kGroupReads = kMoreReads ? (kReads + kMfmas - 1) / kMfmas : 1;
  constexpr int kGroups = kMoreReads ? kMfmas : kReads;
  auto k_step = [&](int cur) __attribute__((always_inline)) {
    bf16x8 af[2][TM], bfr[2][TN];
    frags(cur, 0, af[0], bfr[0]);
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk) {
      if (kk + 1 < kBK / 16) frags(cur, kk + 1, af[(kk + 1) & 1], bfr[(kk + 1) & 1]);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[kk & 1][i], bfr[kk & 1][j],
                                                               acc[i][j], 0, 0, 0);
    }
    // This step's first fragments, then per 16-wide slice its MFMAs with the
    // next slice's fragment reads spread between them.
    __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk) {
      if (kk + 1 < kBK / 16) {
#pragma unroll
        for (int t = 0; t < kGroups; ++t) {
          __builtin_amdgcn_sched_group_barrier(0x008, kGroupMfmas, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, kGroupReads, 0);
        }
        if (kMfmas > kGroupMfmas * kGroups)
          __builtin_amdgcn_sched_group_barrier(0x008, kMfmas - kGroupMfmas * kGroups, 0);
      } else {
        __builtin_amdgcn_sched_group_barrier(0x008, kMfmas, 0);
      }
    }
  };
  int step = 0, cur = 0;  // the step worked on, and its stage
  auto after = [](int stage) { return stage + 1 == STAGES ? 0 : stage + 1; };
  for (; step < ksteps - (STAGES - 1); ++step, cur = after(cur)) {
    wait_step(true);
    load_stage<LOADS, A_LOADS, NW, AUX>(src, lds + (cur == 0 ? STAGES - 1 : cur - 1) * STAGE, wave,
                                        (step + STAGES - 1) * kBK);
    k_step(cur);
  }

  // ---- the adapters
  // The tile's runs.  Its barriers leave the loads on their way.
  int runs = 0;
  {
    wait_stage<63>();
    const int id = tid < BM ? tr.id[tid] : kNoAdapter;
    const bool starts = id >= 0 && (tid == 0 || id != tr.id[tid - 1]);
    const uint64_t mask = __ballot(starts);
    if (lane == 0) tr.wave_runs[wave] = __popcll(mask);
    wait_stage<63>();
    int before = 0;
    for (int w = 0; w < NW; ++w) {
      before += w < wave ? tr.wave_runs[w] : 0;
      runs += tr.wave_runs[w];
    }
    if (starts) {
      const int run = before + __popcll(mask & ((1ull << lane) - 1));
      tr.adapter[run] = id;
      tr.start[run] = tid;
    }
    if (tid == 0) tr.start[runs] = min(BM, M - m0);
    wait_stage<63>();
  }
  // The steps after the K steps: a window of a panel each, its first ones loaded
  // under the last K steps.
  constexpr int kRuns = kBK / kWindow;  // of a panel
  const int rp = padded_rank(p.rank);
  const int windows = rp / kWindow;
  const int total = ksteps + (runs + kRuns - 1) / kRuns * windows;
  int issued = ksteps;
  auto issue = [&](uint8_t* to) {
    const int q = issued - ksteps;
    const int pn = q / windows, w = q - pn * windows;
    lora_panel<BM, LOADS, A_LOADS, NW>(p, tr, runs, w, pn, n0, wave, lane, to);
    // With more stages the waits count on LOADS loads a step; otherwise only
    // the rows that have the panel's adapters.
    const int from = STAGES > 2 ? 0 : tr.start[pn * kRuns] * kUChunks / 64;
    const int end = STAGES > 2 ? BM / 8
                               : (tr.start[min(pn * kRuns + kRuns, runs)] * kUChunks + 63) / 64;
    lora_rows<BM, NW>(d, rp, w, m0, from, end, M, wave, lane, to);
    ++issued;
  };
  while (issued < min(total, STAGES - 1)) issue(lds + issued * STAGE);
  auto next_step = [&]() {
    wait_step(issued - step == STAGES - 1);
    if (issued < total) issue(lds + (cur == 0 ? STAGES - 1 : cur - 1) * STAGE);
  };
#pragma unroll 1
  for (; step < ksteps; ++step, cur = after(cur)) {
    next_step();
    k_step(cur);
  }
#pragma unroll 1
  for (; step < total; ++step, cur = after(cur)) {
    next_step();
    const int q = step - ksteps;
    const int pn = q / windows, w = q - pn * windows;
    const uint8_t* stage = lds + cur * STAGE;
    const uint8_t* ub = stage + (wm0 + frow) * (kUChunks * 16) + fhalf * 16;
    // Where the panel's runs start and end within the wave's rows.
    const int starts = tr.start[min(pn * kRuns + min(lane, kRuns), runs)] - wm0;
    bf16x8 bfr[kRuns][TN];
    bool odd = false;
#pragma unroll
    for (int kk = 0; kk < kRuns; ++kk)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        bfr[kk][j] = *reinterpret_cast<const bf16x8*>(stage + boff[j] +
                                                      (((kk * 2 + fhalf) ^ bswz[j]) << 4));
        if (w * kWindow + fhalf * 8 >= p.rank) bfr[kk][j] = bf16x8{};
        odd = odd || not_finite(bfr[kk][j]);
      }
    const bool any_odd = __ballot(odd) != 0;
    if (any_odd) {
#pragma unroll
      for (int kk = 0; kk < kRuns; ++kk)
#pragma unroll
        for (int j = 0; j < TN; ++j) bfr[kk][j] = finite_part(bfr[kk][j]);
      if (lane == 0) tr.met_non_finite = 1;
    }
#pragma unroll
    for (int kk = 0; kk < kRuns; ++kk) {
      const int from = __builtin_amdgcn_readlane(starts, kk);
      const int to = __builtin_amdgcn_readlane(starts, kk + 1);
      if (to <= 0 || from >= WM || from == to) continue;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (to <= i * 32 || from >= i * 32 + 32) continue;
        const bool mine = i * 32 + frow >= from && i * 32 + frow < to;
        bf16x8 uf[kParts];
#pragma unroll
        for (int t = 0; t < kParts; ++t) {
          uf[t] = *reinterpret_cast<const bf16x8*>(ub + i * 32 * kUChunks * 16 + t * kWindow * 2);
          if (!mine) uf[t] = bf16x8{};
        }
        if (any_odd) {
#pragma unroll
          for (int t = 0; t < kParts; ++t) uf[t] = finite_part(uf[t]);
        }
#pragma unroll
        for (int t = kParts - 1; t >= 0; --t)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] =
                __builtin_amdgcn_mfma_f32_32x32x16_bf16(uf[t], bfr[kk][j], acc[i][j], 0, 0, 0);
      }
    }
  }

  // ---- the logits, a row segment at a time through a scratch of the wave's
  __syncthreads();  // every wave is done reading the stages
  float* scr = reinterpret_cast<float*>(lds) + wave * kStoreFloats;
  const int c0 = (lane & 7) * 4;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        scr[(8 * (e >> 2) + 4 * fhalf + (e & 3)) * kStoreStride + frow] = acc[i][j][e];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      const int col = wn0 + j * 32 + c0, left = N - n0;  // from n0 on
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int rr = (lane >> 3) + 8 * q;
        const int at = wm0 + i * 32 + rr;
        f32x4 v = *reinterpret_cast<const f32x4*>(scr + rr * kStoreStride + c0);
        if (m0 + at >= M || col >= left) continue;
        int row = tr.row[at];
        if (row < 0) {
          row = ~row;
#pragma unroll
          for (int t = 0; t < 4; ++t) v[t] = NAN;
        }
        float* dst = p.logits + static_cast<int64_t>(row) * p.ld_logits + n0 + col;
        if (col + 3 < left) {
          *reinterpret_cast<f32x4u*>(dst) = v;
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (col + t < left) dst[t] = v[t];
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  }

  // ---- what infinities and NaN in B and in u add to their adapters' rows
  __syncthreads();
  if (tr.met_non_finite == 0) return;
  for (int at = tid; at < BM * BN; at += 64 * NW) {
    const int place = at / BN;
    if (m0 + place >= M || at % BN >= N - n0 || tr.id[place] < 0) continue;
    const int v = n0 + at % BN;
    const __bf16* u = d.u + static_cast<int64_t>(m0 + place) * rp * kParts;
    const uint16_t* b = p.b + static_cast<int64_t>(tr.id[place]) * p.stride_b +
                        static_cast<int64_t>(v) * p.ld_b;
    float sum = 0.0f;
    for (int k = 0; k < p.rank; ++k) {
      const float uk = whole_u(u, k);
      if ((b[k] & kExponent) == kExponent || !(fabsf(uk) < INFINITY))
        sum = fmaf(uk, __uint_as_float(static_cast<uint32_t>(b[k]) << 16), sum);
    }
    p.logits[static_cast<int64_t>(tr.row[place]) * p.ld_logits + v] += sum;
  }
}

template <int BM, int BN, int WAVES_M, int WAVES_N, int AUX, int STAGES, int WAVES>
hipError_t launch_tile(const LoraArgs& p, const DownRows& d, hipStream_t stream) {
  const int tiles_m = (p.rows + BM - 1) / BM;
  const int tiles_n = (p.vocab - 1) / BN + 1;
  const int total = tiles_m * tiles_n;
  const int per_xcd = (total + kXcds - 1) / kXcds;
  hipLaunchKernelGGL((lora_gemm_kernel<BM, BN, WAVES_M, WAVES_N, AUX, STAGES, WAVES>),
                     dim3(per_xcd * kXcds), dim3(64 * WAVES_M * WAVES_N), 0, stream, p, d, tiles_m,
                     total, per_xcd);
  return hipGetLastError();
}

// One row tile reads the lm_head once, past the caches (AUX 2), as the weights
// of a model's layers come between two calls: 4 x 18,992 (H = 4,096) 42 us
// instead of 48, 64 x 16,384 43 instead of 49, 128 x 31,040 74 and 80, 160 x
// 60,000 132 and 149, 256 x 151,936 397 and 414.  With several row tiles those
// after the first find it in the L2.
template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES, int WAVES>
hipError_t launch_fused(const LoraArgs& p, const DownRows& d, hipStream_t stream) {
  return p.rows <= BM ? launch_tile<BM, BN, WAVES_M, WAVES_N, 2, STAGES, WAVES>(p, d, stream)
                      : launch_tile<BM, BN, WAVES_M, WAVES_N, 0, STAGES, WAVES>(p, d, stream);
}

// ------------------------------------------- other hidden sizes: a second pass
constexpr int kUpCols = 256;

// logits += B_a u, one workgroup per row and kUpCols columns.
__global__ __launch_bounds__(kUpCols) void lora_add_kernel(LoraArgs p, DownRows d) {
  const int rp = padded_rank(p.rank);
  const int64_t v = static_cast<int64_t>(blockIdx.x) * kUpCols + threadIdx.x;
  for (int place = blockIdx.y; place < p.rows; place += gridDim.y) {
    const int id = d.id[place];
    if (id == kNoAdapter || v >= p.vocab) continue;
    float* out = p.logits + static_cast<int64_t>(d.row[place]) * p.ld_logits + v;
    if (id == kBadAdapter) {
      *out = NAN;
      continue;
    }
    const __bf16* u = d.u + static_cast<int64_t>(place) * rp * kParts;
    const uint16_t* b = p.b + static_cast<int64_t>(id) * p.stride_b + v * p.ld_b;
    float sum = 0.0f;
    for (int k = 0; k < p.rank; k += 8) {
      const bf16x8 bv = *reinterpret_cast<const bf16x8*>(b + k);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum = fmaf(whole_u(u, k + e), static_cast<float>(bv[e]), sum);
      }
    }
    *out += sum;
  }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

DownRows lay_out(void* base, int64_t rows, int64_t rank, size_t* bytes) {
  char* p = static_cast<char*>(base);
  size_t at = 0;
  DownRows d;
  d.u = reinterpret_cast<__bf16*>(p + at);
  at += round256(sizeof(__bf16) * kParts * static_cast<size_t>(rows) *
                 static_cast<size_t>(padded_rank(static_cast<int>(rank))));
  d.row = reinterpret_cast<int32_t*>(p + at);
  at += round256(sizeof(int32_t) * static_cast<size_t>(rows));
  d.id = reinterpret_cast<int32_t*>(p + at);
  at += round256(sizeof(int32_t) * static_cast<size_t>(rows));
  *bytes = at;
  return d;
}

}  // namespace

size_t lmhead_lora_workspace_size(int64_t rows, int64_t rank) {
  size_t bytes;
  lay_out(nullptr, rows, rank, &bytes);
  return bytes;
}

// HIP counts a launch's threads in 32 bits.  The smallest tiles that many
// columns can get are 64 x 128 and 128 x 128 with eight waves, those of the
// second pass's projection 64, 128 and 256 x 256 with four, which also adds a
// tile to the columns in an int.
bool lmhead_lora_fits(int64_t rows, int64_t vocab, int64_t hidden_dim) {
  const bool fused = hidden_dim % kBK == 0;
  const int64_t bm = rows <= 64 ? 64 : (fused || rows <= 128 ? 128 : 256), bn = fused ? 128 : 256;
  const int64_t tiles = (rows + bm - 1) / bm * ((vocab + bn - 1) / bn);
  return (tiles + kXcds - 1) / kXcds * kXcds * (fused ? 512 : 256) < int64_t{1} << 32 &&
         (fused || vocab <= 0x7fffffff - bn);
}

hipError_t launch_lmhead_lora(const LoraArgs& p, void* ws, hipStream_t stream) {
  size_t bytes;
  const DownRows d = lay_out(ws, p.rows, p.rank, &bytes);
  hipLaunchKernelGGL(lora_down_kernel,
                     dim3(p.rows < (1 << 18) ? p.rows : (1 << 18), padded_rank(p.rank) / kWindow),
                     dim3(kDownThreads), 0, stream, p, d);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.hidden_dim % kBK == 0) {
    auto tiles = [&](int64_t bm, int64_t bn) {
      return (p.rows + bm - 1) / bm * ((p.vocab + bn - 1) / bn);
    };
    // Few tiles: the smallest that makes no more than one a CU, with as many
    // stages as help.  H = 4,096, weights not in the caches, us:
    //   rows x columns    32 x 32  64 x 64  64 x 128  128 x 128  next below
    //     4 x  4,748         28       30        37         45
    //    32 x  9,496         35       34        42         49
    //    64 x 16,384         73       43        50         53
    //   128 x 16,384         94       70        54         65         66
    //    64 x 18,992         77       67        52         55         82
    //   128 x 25,000        125      106        83         69         72
    //   320 x  9,496        111       79        75         56         64
    if (tiles(32, 32) <= 256) return launch_fused<32, 32, 1, 1, 6, 1>(p, d, stream);
    if (tiles(64, 64) <= 256) return launch_fused<64, 64, 2, 2, 6, 1>(p, d, stream);
    if (tiles(64, 128) <= 256) return launch_fused<64, 128, 2, 4, 5, 2>(p, d, stream);
    if (tiles(128, 128) <= 256) return launch_fused<128, 128, 2, 4, 4, 2>(p, d, stream);
    // One row tile and many columns: several workgroups a CU.  x 151,936, three
    // stages and two, us: 8 rows 209 and 228, 32 rows 226 and 266, 48 rows 234
    // and 253, 64 rows 243 and 234.
    if (p.rows <= 48) return launch_tile<64, 128, 2, 4, 2, 3, 4>(p, d, stream);
    if (p.rows <= 64) return launch_tile<64, 128, 1, 4, 2, 2, 3>(p, d, stream);
    if (p.rows <= 128) return launch_tile<128, 128, 2, 4, 2, 2, 4>(p, d, stream);
    // More rows: the tile whose rounds over the card take least, by what a round
    // of it takes in 10 ns a K step (us, H = 4,096, but 2,560 of 133 and 256
    // rows; 192n is 192 x 128):
    //   rows x columns     128   192n   192   256   320
    //   133 x  31,040       79     67    95    97   104
    //   256 x  31,040       76     91    82    88    92
    //   300 x  18,992       92    125   101   114   133
    //   512 x  18,992      150    130   110   121   136
    //   640 x  18,992      171    219   225   154   168
    //   192 x  40,000      153    136   121   126   137
    //   640 x  31,040      230    262   218   245   175
    //   160 x 151,936      441    366   371   390   433
    //   384 x 151,936      608    649   553   645   760
    auto rounds = [&](int64_t bm, int64_t bn, int64_t at_once, int64_t cost) {
      return (tiles(bm, bn) + at_once - 1) / at_once * cost;
    };
    const int64_t t128 = rounds(128, 128, 512, 140), t192n = rounds(192, 128, 256, 120);
    const int64_t t192 = rounds(192, 256, 256, 180), t256 = rounds(256, 256, 256, 205);
    const int64_t t320 = rounds(320, 256, 256, 245);
    const int64_t least = std::min({t128, t192n, t192, t256, t320});
    if (t320 == least) return launch_fused<320, 256, 2, 4, 2, 2>(p, d, stream);
    if (t256 == least) return launch_fused<256, 256, 2, 4, 2, 2>(p, d, stream);
    if (t192 == least) return launch_fused<192, 256, 2, 4, 2, 2>(p, d, stream);
    if (t192n == least) return launch_fused<192, 128, 2, 4, 3, 2>(p, d, stream);
    return launch_tile<128, 128, 2, 4, 0, 2, 4>(p, d, stream);
  }
  e = launch_lmhead_gemm(p.hidden, p.ld_hidden, p.lm_head, p.ld_lm_head, p.logits, p.ld_logits,
                         p.rows, p.vocab, p.hidden_dim, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(lora_add_kernel,
                     dim3((p.vocab + int64_t{kUpCols} - 1) / kUpCols,
                          p.rows < 65535 ? p.rows : 65535),
                     dim3(kUpCols), 0, stream, p, d);
  return hipGetLastError();
}

}  // namespace ts
