// 4-bit rows with a scale per group, and the local vocabulary projection from
// them, on gfx950.
//
// A row is held as OCP MX FP4: groups of 32 consecutive entries share a scale
// s = 2^e (E8M0: one byte, e + 127, 255 NaN), and each entry is a code of E2M1
// (sign, two bits of exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6),
// two to a byte, the even column in the low half.  4.25 bits an entry.
//   quantize   e = least integer >= -127 with max|x| <= 7 * 2^e: what lies
//              above 6 s then loses at most the half step of E2M1's last
//              binade (and e <= 125, so that no finite entry becomes infinite);
//              code = the value nearest x / s, ties to the even code
//   project    logits[r, v] = sum_h hidden[r, h] * 2^e[v, h / 32] * q[v, h]
// A power of two times an E2M1 value has two significant bits, so it is a bf16
// number and its products with bf16 are exact in fp32: the lm_head becomes
// matrix-core fragments in registers (v_cvt_scalef32_pk_bf16_fp4: two entries
// and their scale in one instruction), nothing is rounded, and only the fp32
// sums differ from the definition.
#include <stdlib.h>

#include <algorithm>

#include "lmhead_e2m1.hpp"
#include "tile_store.hpp"

namespace ts {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kXcds = 8;
constexpr int kCus = 256;

// The scale of a byte, as the conversions take it: they read the exponent
// alone, so 0 is 2^-127 and 255 NaN.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// ------------------------------------------------------------ quantization
constexpr int QT = 256;
constexpr int kUnit = 8;                         // entries a thread takes at a time
constexpr int kUnitsPerGroup = kE2m1Group / kUnit;

// Where a thread is in the rows, cut into units; steps of the whole grid.
struct Units {
  int64_t row;
  int at, per_row, step_rows, step_at;

  __device__ __forceinline__ Units(int cols, int64_t first, int64_t step) {
    per_row = cols / kUnit;
    row = first / per_row;
    at = static_cast<int>(first % per_row);
    step_rows = static_cast<int>(step / per_row);
    step_at = static_cast<int>(step % per_row);
  }
  __device__ __forceinline__ void next() {
    row += step_rows;
    at += step_at;
    if (at >= per_row) {
      at -= per_row;
      ++row;
    }
  }
};

// Units whose loads a thread has on their way, a grid apart.  The grid has just these
// for bf16 (151,936 x 4,096: 290 us to codes, 284 back, 5.5 TB/s; one unit at a time
// in 8,192 workgroups 328 and 392) and one a thread for fp32 (60,000 x 4,096: 190 and
// 225 us, four 202 and 277).  Stores of whole 16 bytes go past the caches (3%); fp32's
// pairs of them must not (392 us and 225).
constexpr int kAtOnce = 4;

// A unit as it lies in memory.
template <bool BF16>
struct Raw;
template <>
struct Raw<true> {
  u16x8 v;
  __device__ __forceinline__ void load(const void* in, int64_t at) {
    v = *reinterpret_cast<const u16x8u*>(static_cast<const uint16_t*>(in) + at);
  }
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(static_cast<uint32_t>(v[i]) << 16);
  }
};
template <>
struct Raw<false> {
  f32x4 lo, hi;
  __device__ __forceinline__ void load(const void* in, int64_t at) {
    const f32x4u* p = reinterpret_cast<const f32x4u*>(static_cast<const float*>(in) + at);
    lo = p[0];
    hi = p[1];
  }
  __device__ __forceinline__ float operator[](int i) const { return i < 4 ? lo[i] : hi[i - 4]; }
};

// Four neighbouring lanes hold a group.  The scale's byte comes from the bits
// of the group's largest magnitude 1.m * 2^(E - 127): E - 2 where 1.m <= 1.75,
// else E - 1.  As integers magnitudes are in order, with infinity and NaN last.
template <bool BF16>
__global__ __launch_bounds__(QT) void quantize_groups_kernel(
    const void* __restrict__ in, int64_t ld_in, int rows, int cols, uint8_t* __restrict__ codes,
    int64_t ld_codes, uint8_t* __restrict__ scales, int64_t ld_scales) {
  Units u(cols, static_cast<int64_t>(blockIdx.x) * QT + threadIdx.x,
          static_cast<int64_t>(gridDim.x) * QT);
  while (u.row < rows) {
    Raw<BF16> x[kAtOnce];
    int64_t row[kAtOnce];
    int at[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      row[k] = u.row;
      at[k] = u.at;
      if (u.row < rows) x[k].load(in, u.row * ld_in + u.at * kUnit);
      u.next();
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (row[k] >= rows) break;
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) top = max(top, __float_as_uint(x[k][i]) & 0x7fffffffu);
      top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1, 4)));
      top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2, 4)));
      int byte =
          max(static_cast<int>(top >> 23) - 2 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
      byte = min(byte, 252);  // 6 * 2^125 is finite
      if (top == 0) byte = 127;
      if (top >= 0x7f800000u) byte = 255;
      uint32_t w = 0;
      // Past the last finite byte nothing is written but zeros beside the NaN.
      if (byte != 255) {
        const float s = scale_of(byte);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[k][0], x[k][1], s, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[k][2], x[k][3], s, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[k][4], x[k][5], s, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[k][6], x[k][7], s, 3);
      }
      __builtin_nontemporal_store(
          w, reinterpret_cast<uint32_t*>(codes + row[k] * ld_codes + at[k] * (kUnit / 2)));
      if (at[k] % kUnitsPerGroup == 0)
        scales[row[k] * ld_scales + at[k] / kUnitsPerGroup] = static_cast<uint8_t>(byte);
    }
  }
}

template <bool BF16>
__global__ __launch_bounds__(QT) void dequantize_groups_kernel(E2m1Rows in, int rows, int cols,
                                                               void* __restrict__ out,
                                                               int64_t ld_out) {
  Units u(cols, static_cast<int64_t>(blockIdx.x) * QT + threadIdx.x,
          static_cast<int64_t>(gridDim.x) * QT);
  while (u.row < rows) {
    uint32_t code[kAtOnce], byte[kAtOnce];
    int64_t place[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      place[k] = -1;
      if (u.row < rows) {
        code[k] =
            *reinterpret_cast<const uint32_t*>(in.codes + u.row * in.ld + u.at * (kUnit / 2));
        byte[k] = in.scales[u.row * in.ld_scales + u.at / kUnitsPerGroup];
        place[k] = u.row * ld_out + u.at * kUnit;
      }
      u.next();
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (place[k] < 0) break;
      const uint32_t w = code[k];
      const float s = scale_of(byte[k]);
      if (BF16) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
        const u16x8u v = __builtin_bit_cast(
            u16x8u, bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]});
        __builtin_nontemporal_store(
            v, reinterpret_cast<u16x8u*>(static_cast<uint16_t*>(out) + place[k]));
      } else {
        f32x4u* p = reinterpret_cast<f32x4u*>(static_cast<float*>(out) + place[k]);
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
        const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
        const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
        p[0] = f32x4u{a[0], a[1], b[0], b[1]};
        p[1] = f32x4u{c[0], c[1], d[0], d[1]};
      }
    }
  }
}

// ---------------------------------------------------------------- fragments
// Eight entries as matrix-core operands.
__device__ __forceinline__ bf16x8 frag_of(uint32_t w, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// --------------------------------------------------------------- few rows
// Up to 16 NT rows: bound by the lm_head's bytes, so nothing else may hold their
// loads up.  A wave keeps its share of every hidden row in registers (NS steps of
// 128 entries) and the workgroup's waves have the row's shares side by side; then
// the workgroup goes through the lm_head, 16 VT rows (a tile) at a time, with the
// loads of AHEAD tiles on their way.  A lane's 16 bytes of codes are one group: lane
// l has row l % 16, groups 4 s + l / 16, and a load has 64 bytes of each of 16 rows.
// In v_mfma_f32_16x16x32_bf16 lane l holds entries 8 (l / 16) .. + 7 of a slice of
// 32; any order of the sum's entries will do as long as both operands share it,
// so slice i takes the i-th eight entries of each lane's group.  The shares are
// added up through LDS, in a fixed order, by one wave while the others go on.
// Where the waves' shares are not the whole row, the lm_head is gone through again
// for each further part of it, and the sums so far come back from the logits.
// Bound by the lm_head's loads: 1 x 4,096 x 151,936 takes 57 us (5.8 TB/s), 16 rows
// 70, 32 rows 78.  Reading the same bytes in this pattern and nothing else takes 53;
// the scales' loads 3 to 9 of it, the waves' meeting for a tile about 10.  Measured and
// dropped: one tile's loads on their way only (82 us), scales byte by byte (+8), loads
// past the caches (+10: a row's line is asked for twice), every wave at every sum
// (+2), the hidden rows in LDS and whole rows a wave (73 us, 16 rows 76).  The widest
// shapes spill: shares of 1,024 that are not all whole 9 registers, in several parts 21
// (5 where whole), and 32 rows in several parts 4 where they are not whole.
constexpr int kStep = 128;  // entries of a row in one step
constexpr int kFewWaves = 8;

// Waits for the wave's LDS writes and then for the other waves, but not for loads
// on their way, as __syncthreads() would.
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt 0; vmcnt and expcnt at their maxima
  asm volatile("s_barrier" ::: "memory");
}

// Register i of lane row k (lanes 16 k .. 16 k + 15) and register k of lane row i
// change places.
__device__ __forceinline__ void turn_4x4(u32x4 (&c)[4]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    auto swap32 = [&](int a, int b) {
      const auto v = __builtin_amdgcn_permlane32_swap(c[a][d], c[b][d], false, false);
      c[a][d] = v[0];
      c[b][d] = v[1];
    };
    auto swap16 = [&](int a, int b) {
      const auto v = __builtin_amdgcn_permlane16_swap(c[a][d], c[b][d], false, false);
      c[a][d] = v[0];
      c[b][d] = v[1];
    };
    swap32(0, 2);
    swap32(1, 3);
    swap16(0, 1);
    swap16(2, 3);
  }
}

// WHOLE: the waves' shares of the row's parts are all whole.  PARTS: there is more
// than one.
template <int NT, int NS, int VT, int AHEAD, bool WHOLE, bool PARTS>
__global__ __launch_bounds__(64 * kFewWaves, 2) void lmhead_e2m1_few_kernel(
    const uint16_t* __restrict__ X, int64_t ldx, E2m1Rows w, float* C, int64_t ldc, int M, int N,
    int K, int tiles, int parts, int vec_out) {
  constexpr int BV = 16 * VT, BV4 = BV / 4;
  constexpr int GROUPS = 4 * NS;  // of a wave's share
  extern __shared__ float shares[];  // [2][waves][16 NT][BV]
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int groups = K / kE2m1Group;
  typedef uint32_t Words __attribute__((ext_vector_type(NS)));
  typedef uint32_t WordsU __attribute__((ext_vector_type(NS), aligned(1)));

  // A tile's codes and the scales of the wave's groups: where the row has all of
  // them (WHOLE) a row's, otherwise those of the lane's own groups, byte by byte
  // (past the row's end another's, which meet zeros, and must not be NaN).  And the
  // lane's sums of the parts before.
  struct Tile {
    u32x4 code[VT][NS];
    Words scale[VT];
    f32x4 before;
  };
  const int step = gridDim.x;
  const int first = blockIdx.x, last = first + (tiles - 1 - first) / step * step;
  float* mine = shares + wave * (16 * NT * BV);
  const int half = waves * 16 * NT * BV;
  int buf = 0;

  for (int part = 0; part < parts; ++part) {
    const int g0 = (part * waves + wave) * GROUPS;  // the wave's first group
    // Hidden rows r16 + 16 n, the entries of this lane's groups.  Loaded as a group
    // a load, its four chunks in the four lanes of a row, and turned: with a lane's
    // own group in four loads each of them has 64 pieces of 16 bytes.
    bf16x8 x[NT][NS][4];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = r16 + 16 * n;
        const uint16_t* p = X + static_cast<int64_t>(min(r, M - 1)) * ldx + 8 * q;
        u32x4 c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c[i] = *reinterpret_cast<const u32x4*>(p + min(g0 + 4 * s + i, groups - 1) * 32);
        turn_4x4(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[n][s][i] = __builtin_bit_cast(bf16x8, c[i]);
          if (r >= M || g0 + 4 * s + q >= groups) x[n][s][i] = bf16x8{};
        }
      }
    }

    // Entry i of a tile's M x BV4 quadruples of logits is added up by this lane.
    auto place = [&](int turn) {
      const int w_at = wave - turn;
      return (w_at < 0 ? w_at + waves : w_at) * 64 + lane;
    };
    auto load = [&](int tile, int turn, Tile& to) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < VT; ++t) {
        const int64_t v = min(tile * BV + t * 16 + r16, N - 1);
        const uint8_t* pc = w.codes + v * w.ld;
        const uint8_t* ps = w.scales + v * w.ld_scales;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const int g = min(g0 + 4 * s + q, groups - 1);
          to.code[t][s] = *reinterpret_cast<const u32x4*>(pc + g * 16);
          if (!WHOLE) to.scale[t][s] = ps[g];
        }
        if (WHOLE) to.scale[t] = *reinterpret_cast<const WordsU*>(ps + g0);
      }
      if (PARTS) {
        const int i = place(turn), r = i / BV4;
        const int64_t col = static_cast<int64_t>(tile) * BV + i % BV4 * 4;
        to.before = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (part > 0 && r < M) {
          const float* from = C + static_cast<int64_t>(r) * ldc + col;
          if (vec_out && col + 3 < N) {
            to.before = *reinterpret_cast<const f32x4*>(from);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (col + e < N) to.before[e] = from[e];
          }
        }
      }
    };
    auto scale_at = [&](const Tile& from, int t, int s) {
      if (WHOLE) return scale_of(from.scale[t][s] >> (8 * q) & 255u);
      return g0 + 4 * s + q < groups ? scale_of(from.scale[t][s]) : 1.0f;
    };
    auto take = [&](int tile, int turn, const Tile& from) __attribute__((always_inline)) {
      f32x4 acc[VT][NT];
#pragma unroll
      for (int t = 0; t < VT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[t][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < VT; ++t)
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const float sc = scale_at(from, t, s);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bf16x8 a = frag_of(from.code[t][s][i], sc);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              acc[t][n] =
                  __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, x[n][s][i], acc[t][n], 0, 0, 0);
          }
        }
      // Lane l holds lm_head rows 4 q .. 4 q + 3 of hidden row l % 16.
#pragma unroll
      for (int t = 0; t < VT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (r16 + 16 * n < M)
            *reinterpret_cast<f32x4*>(mine + buf * half + (r16 + 16 * n) * BV + t * 16 + 4 * q) =
                acc[t][n];
      wait_lds();
      for (int i = place(turn); i < M * BV4; i += 64 * waves) {
        const int r = i / BV4, c = i % BV4 * 4;
        const float* p = shares + buf * half + r * BV + c;
        f32x4 sum = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
        for (int k = 1; k < kFewWaves; ++k)
          if (k < waves) sum += *reinterpret_cast<const f32x4*>(p + k * (16 * NT * BV));
        if (PARTS) sum += from.before;
        const int64_t col = static_cast<int64_t>(tile) * BV + c;
        float* to = C + static_cast<int64_t>(r) * ldc + col;
        if (vec_out && col + 3 < N) {
          *reinterpret_cast<f32x4*>(to) = sum;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < N) to[e] = sum[e];
        }
      }
      buf ^= 1;
    };

    // Past the last tile its loads are made again, so that the waits can count on
    // them.
    Tile ring[AHEAD + 1];
    int tile = first, turn = 0;
    auto wrap = [&](int t) { return t >= waves ? t % waves : t; };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load(min(tile + u * step, last), wrap(u), ring[u]);
    for (bool more = true; more;) {
#pragma unroll
      for (int u = 0; u <= AHEAD; ++u) {
        load(min(tile + AHEAD * step, last), wrap(turn + AHEAD), ring[(u + AHEAD) % (AHEAD + 1)]);
        take(tile, turn, ring[u]);
        tile += step;
        turn = wrap(turn + 1);
        more = tile < tiles;
        if (!more) break;
      }
    }
    // The next part reads these logits back, in other waves.
    if (PARTS && part + 1 < parts) {
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    }
  }
}

// ------------------------------------------------------- tiles of rows
constexpr int kBK = 64;

// The hidden rows' direct loads are buffer loads: behind global ones, which the
// compiler counts as flat, it would wait for every register load at once.  (A
// plain function: the host pass does not emit the kernel stub when the builtin
// sits in a lambda.)
__device__ __forceinline__ void hidden_to_lds(__amdgpu_buffer_rsrc_t rows, uint8_t* to, int at) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rows, to, 16, at, 0, 0, 0);
}

template <int LOADS, int NW>
__device__ __forceinline__ void issue_hidden(__amdgpu_buffer_rsrc_t rows, const int* at,
                                             const int* back, uint8_t* stage, int wave, int k0,
                                             bool half) {
#pragma unroll
  for (int q = 0; q < LOADS; ++q)
    hidden_to_lds(rows, stage + (wave + NW * q) * 1024,
                  (half ? at[q] - back[q] : at[q]) + 2 * k0);
}

// Waits until at most N of the wave's loads are on their way and its LDS reads
// are done, then for the other waves; a fence would wait for the later steps'
// loads as well.
template <int N>
__device__ __forceinline__ void wait_stage() {
  static_assert(N < 64, "vmcnt has six bits");
  asm volatile("" ::: "memory");
  // vmcnt in bits 3:0 and 15:14, lgkmcnt 0, expcnt left at its maximum.
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
  asm volatile("s_barrier" ::: "memory");
}

// A wave's accumulator blocks to C; `lds` is free.
template <int TM, int TN>
__device__ __forceinline__ void store_output(const f32x16 (&acc)[TM][TN], uint8_t* lds, int wave,
                                             int lane, float* __restrict__ C, int64_t ldc,
                                             int row0, int col0, int M, int N, int vec_out) {
  if (vec_out) {
    store_tile_rows<false>(acc, reinterpret_cast<float*>(lds), wave, lane, C, ldc, row0, col0, M,
                           N, nullptr, nullptr);
    return;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int col = col0 + j * 32 + (lane & 31);
      if (col >= N) continue;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int row = row0 + i * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        if (row < M) C[static_cast<int64_t>(row) * ldc + col] = acc[i][j][e];
      }
    }
  }
}

// -------------------------------------------------------------- many rows
// BM x BN tiles, K in steps of 64.  The hidden rows go through a ring of AHEAD + 1
// LDS stages (rows of 128 bytes, 16-byte chunks swizzled by the row pair); the
// lm_head goes straight into registers, AHEAD steps ahead too, 16 bytes a lane,
// which is one group: lane l has row l % 32 and the step's group l / 32.  Slice i
// of a step takes the i-th eight entries of each lane's group, so its hidden
// fragment is chunk 4 (l / 32) + i.  A wave has all of the tile's hidden rows, so the
// conversions (four instructions a fragment, two to five products) are made once.
// Bound by the matrix cores: 640 x 4,096 x 151,936 takes 628 to 682 us with the clock of
// the run (1.17 PFLOP/s and more; the bf16 projection 720); 6 of the 160-row tile's
// registers spill.  Few row tiles are bound by what a step waits for (64
// rows past the caches 262 us, through them 164, 122 to 126 since the scales come
// several at a time).  Without gain there: the codes of two steps in pieces of 64 bytes,
// those of four at once, tiles that begin at different steps.
// Scales come several groups at a time, 16 for 64 rows and 8 for more, where 16 take
// registers that are not there (rows of that many groups; us in one run with 16, 8 and,
// as a shorter row has them, a byte a step: 640 x 4,096 x 151,936 748, 671 and 705; 256
// rows 310, 309 and 337; 64 x 2,560 x 100,000 59, 65 and 70.  Other runs are up to a tenth
// faster throughout: 650, 283 and 53 as it is).
template <int BM>
constexpr int kScales = BM <= 64 ? 16 : 8;

template <int WORDS>
using Words = uint32_t __attribute__((ext_vector_type(WORDS)));

// Scales from byte `bytes` (less than 4 WORDS) on, or from the one after it.
template <int WORDS>
__device__ __forceinline__ Words<WORDS> scales_from(Words<WORDS> w, int bytes, int one) {
  auto word = [&](int i) { return i < WORDS ? w[i] : 0u; };
  for (; bytes >= 4; bytes -= 4) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = word(i + 1);
  }
  const int by = 8 * (bytes + one);  // up to 32
  Words<WORDS> to;
#pragma unroll
  for (int i = 0; i < WORDS; ++i)
    to[i] = static_cast<uint32_t>((static_cast<uint64_t>(word(i + 1)) << 32 | w[i]) >> by);
  return to;
}

// WIDE: the row has kScales<BM> groups or more.
template <int BM, int BN, int NW, int AHEAD, bool WIDE>
__global__ __launch_bounds__(64 * NW, 2) void lmhead_e2m1_tiles_kernel(
    const uint16_t* __restrict__ X, int64_t ldx, E2m1Rows w, float* __restrict__ C, int64_t ldc,
    int M, int N, int K, int tiles_m, int tiles_total, int tiles_per_xcd, int vec_out) {
  constexpr int WN = BN / NW;
  constexpr int TM = BM / 32, TN = WN / 32;
  constexpr int RING = AHEAD + 1;
  constexpr int STAGE = BM * 128;
  constexpr int A_LOADS = BM / 8 / NW;
  constexpr int W_LOADS = WIDE ? TN : 2 * TN;  // codes, and scales if each step has its own
  constexpr int SCRATCH = NW * kTileStoreFloats * 4;
  static_assert(BM / 8 % NW == 0, "blocks must split evenly over the waves");
  static_assert(BM % 32 == 0 && WN % 32 == 0, "wave tile of whole 32x32 blocks");
  __shared__ __attribute__((
      aligned(1024))) uint8_t lds[RING * STAGE > SCRATCH ? RING * STAGE : SCRATCH];

  const int bid = blockIdx.x;
  const int tile = (bid % kXcds) * tiles_per_xcd + bid / kXcds;
  if (tile >= tiles_total) return;
  const int m0 = tile % tiles_m * BM, n0 = tile / tiles_m * BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn0 = wave * WN;
  const int frow = lane & 31, fhalf = lane >> 5;

  const int steps = (K + kBK - 1) / kBK, full_steps = K / kBK;
  // A last step of one group: the other half of each LDS row repeats it and
  // meets zeros.
  const __amdgpu_buffer_rsrc_t hidden = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(X + static_cast<int64_t>(m0) * ldx), 0, -1, 0x00020000);
  int at[A_LOADS], back[A_LOADS];  // bytes
#pragma unroll
  for (int q = 0; q < A_LOADS; ++q) {
    const int row = 8 * (wave + NW * q) + (lane >> 3);
    const int c = (lane & 7) ^ ((row >> 1) & 7);
    at[q] = static_cast<int>(min(row, M - 1 - m0) * static_cast<int>(ldx)) * 2 + c * 16;
    back[q] = c >= 4 ? 64 : 0;
  }
  const uint8_t* wp[TN];
  const uint8_t* sp[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int64_t v = min(n0 + wn0 + j * 32 + frow, N - 1);
    wp[j] = w.codes + v * w.ld;
    sp[j] = w.scales + v * w.ld_scales;
  }
  const int groups = K / kE2m1Group;

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  int aoff[TM], aswz[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = i * 32 + frow;
    aoff[i] = r * 128;
    aswz[i] = (r >> 1) & 7;
  }

  u32x4 code[RING][TN];
  uint32_t scale[RING][TN];  // of a step; WIDE: of several steps
  constexpr int SCALES = kScales<BM>, SWORDS = SCALES / 4;
  typedef Words<SWORDS> ScalesU __attribute__((aligned(1)));
  Words<SWORDS> scales[TN], next_scales[TN];
  auto load_scales = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      next_scales[j] = *reinterpret_cast<const ScalesU*>(sp[j] + min(2 * ks, groups - SCALES));
  };
  // Before step ks: its scales are the first two bytes, this lane's the first.
  auto turn_scales = [&](int ks) __attribute__((always_inline)) {
    if (ks % (SCALES / 2) == 0) {
      const int back = 2 * ks - min(2 * ks, groups - SCALES);
#pragma unroll
      for (int j = 0; j < TN; ++j) scales[j] = scales_from<SWORDS>(next_scales[j], back, fhalf);
      load_scales(ks + SCALES / 2);
    } else {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int i = 0; i < SWORDS; ++i)
          scales[j][i] = __builtin_amdgcn_alignbit(i + 1 < SWORDS ? scales[j][i + 1] : 0u,
                                                   scales[j][i], 16);
      }
    }
  };
  // The loads of a step, in an order that the waits count on: the hidden rows
  // first, then codes and scales, and none across the ends.
  auto load_step = [&](int ks, int slot) __attribute__((always_inline)) {
    ks = min(ks, steps - 1);
    __builtin_amdgcn_sched_barrier(0);
    issue_hidden<A_LOADS, NW>(hidden, at, back, lds + slot * STAGE, wave, ks * kBK,
                              ks >= full_steps);
    __builtin_amdgcn_sched_barrier(0);
    const int g = min(2 * ks + fhalf, groups - 1);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      code[slot][j] = *reinterpret_cast<const u32x4*>(wp[j] + g * 16);
      if (!WIDE) scale[slot][j] = sp[j][g];
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](int slot, bool half) __attribute__((always_inline)) {
    const uint8_t* base = lds + slot * STAGE;
    u32x4 now[TN];
    float sc[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      now[j] = code[slot][j];
      sc[j] = scale_of(WIDE ? scales[j][0] & 255u : scale[slot][j]);
      if (half && fhalf) {
        now[j] = u32x4{0, 0, 0, 0};
        sc[j] = 1.0f;
      }
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int chunk = 4 * fhalf + kk;
      bf16x8 af[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        af[i] = *reinterpret_cast<const bf16x8*>(base + aoff[i] + ((chunk ^ aswz[i]) << 4));
        if (half && fhalf) af[i] = bf16x8{};  // 0 x inf is not 0
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const bf16x8 b = frag_of(now[j][kk], sc[j]);
#pragma unroll
        for (int i = 0; i < TM; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[i], b, acc[i][j], 0, 0, 0);
      }
    }
  };

  if (WIDE) load_scales(0);
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) load_step(u, u);
  int ks = 0;
  for (; ks + RING <= full_steps; ks += RING) {
#pragma unroll
    for (int u = 0; u < RING; ++u) {
      // Behind the step's hidden rows: its codes and scales, and AHEAD - 1 steps (a load
      // of several scales among them makes the wait longer than it need be).
      wait_stage<W_LOADS + (AHEAD - 1) * (A_LOADS + W_LOADS)>();
      if (WIDE) turn_scales(ks + u);
      load_step(ks + u + AHEAD, (u + AHEAD) % RING);
      multiply(u, false);
    }
  }
  const int rest = steps - ks;  // at most RING: their loads are on their way but for the last's
#pragma unroll
  for (int u = 0; u < RING; ++u) {
    if (u < rest) {
      wait_stage<0>();
      if (WIDE) turn_scales(ks + u);
      if (u == 0) load_step(ks + AHEAD, AHEAD % RING);
      multiply(u, ks + u >= full_steps);
    }
  }

  // The loads past the last step have landed too, and every wave is done reading.
  wait_stage<0>();
  store_output<TM, TN>(acc, lds, wave, lane, C, ldc, m0, n0 + wn0, M, N, vec_out);
}

int unit_grid(int rows, int cols, bool bf16) {
  const int64_t units = static_cast<int64_t>(rows) * (cols / kUnit);
  const int64_t groups = (units - 1) / (bf16 ? QT * kAtOnce : QT) + 1;
  return static_cast<int>(std::min<int64_t>(groups, (int64_t{1} << 31) / QT - 1));
}

struct Projection {
  const uint16_t* hidden;
  int64_t ld_hidden;
  E2m1Rows w;
  float* logits;
  int64_t ld_logits;
  int rows, vocab, hidden_dim;
};

// ONE: the row is one part.
template <int NT, int NS, int VT, int AHEAD, bool ONE>
hipError_t launch_few(const Projection& p, hipStream_t stream) {
  const int shares = (p.hidden_dim - 1) / (NS * kStep) + 1;
  const int parts = (shares - 1) / kFewWaves + 1, waves = (shares - 1) / parts + 1;
  const int tiles = (p.vocab - 1) / (16 * VT) + 1;
  const int lds = 2 * waves * 16 * NT * 16 * VT * 4;
  const bool whole = p.hidden_dim == parts * waves * NS * kStep;
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(std::min(tiles, kCus)), dim3(64 * waves), lds, stream, p.hidden,
                       p.ld_hidden, p.w, p.logits, p.ld_logits, p.rows, p.vocab, p.hidden_dim,
                       tiles, parts, rows_take_vector_stores(p.logits, p.ld_logits));
    return hipGetLastError();
  };
  if constexpr (!ONE) {
    if (parts > 1)
      return whole ? launch(lmhead_e2m1_few_kernel<NT, NS, VT, AHEAD, true, true>)
                   : launch(lmhead_e2m1_few_kernel<NT, NS, VT, AHEAD, false, true>);
  }
  return whole ? launch(lmhead_e2m1_few_kernel<NT, NS, VT, AHEAD, true, false>)
               : launch(lmhead_e2m1_few_kernel<NT, NS, VT, AHEAD, false, false>);
}

template <int BM, int BN, int NW, int AHEAD>
hipError_t launch_tiles(const Projection& p, hipStream_t stream) {
  const int tiles_m = (p.rows - 1) / BM + 1, tiles_n = (p.vocab - 1) / BN + 1;
  const int total = tiles_m * tiles_n;
  const int per_xcd = (total + kXcds - 1) / kXcds;
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(per_xcd * kXcds), dim3(64 * NW), 0, stream, p.hidden,
                       p.ld_hidden, p.w, p.logits, p.ld_logits, p.rows, p.vocab, p.hidden_dim,
                       tiles_m, total, per_xcd, rows_take_vector_stores(p.logits, p.ld_logits));
    return hipGetLastError();
  };
  return p.hidden_dim >= kScales<BM> * kE2m1Group
             ? launch(lmhead_e2m1_tiles_kernel<BM, BN, NW, AHEAD, true>)
             : launch(lmhead_e2m1_tiles_kernel<BM, BN, NW, AHEAD, false>);
}

constexpr int kFewRows = 32;

// Shares of 512 entries a wave, of 256 where the row is short or the hidden rows
// many, of 1,024 where a row would take two parts.  Two tiles of rows at once where
// the row has few shares: 5 x 2,560 x 31,037 10.9 us, one 12.4; 1 x 2,560 x 248,320
// 58 and 64; 1 x 4,096 x 151,936 61 and 57.  Four of short rows: 4 x 256 x 100,000
// 9.5, shares of 512 14.6; 16 x 1,024 x 100,000 16.8 and 17.2; 32 x 256 x 100,000 17
// and 22.  Rows of 8,192, 4 x 100,000: 84 us at once, 103 in two parts.
hipError_t launch_few_rows(const Projection& p, hipStream_t stream) {
  const int k = p.hidden_dim;
  if (p.rows <= 16) {
    if (k <= 1024) return launch_few<1, 2, 4, 1, true>(p, stream);
    if (k <= 7 * 512) return launch_few<1, 4, 2, 1, true>(p, stream);
    return k <= 8 * 512 ? launch_few<1, 4, 1, 2, true>(p, stream)
                        : launch_few<1, 8, 1, 1, false>(p, stream);
  }
  return k <= 1024 ? launch_few<2, 2, 2, 2, true>(p, stream)
                   : launch_few<2, 4, 1, 2, false>(p, stream);
}

// The kernel for few rows up to 32 of them, unless the row is short, us, it and 64-row
// tiles: 32 x 4,096 x 151,936 78 and 114; 32 x 1,024 x 100,000 23 and 21, 32 x 512 19 and
// 14, 16 x 512 13.5 and 13, 16 x 256 13.5 and 10.
// From 33 rows on the tiles take 116 us, at 64 124.
// Up to 64, 64 x 256 tiles, or 64 x 128 where those would leave a quarter of the CUs
// without one (64 x 4,096 x 31,000: 34 and 25; 48 x 6,144 x 60,000 70 and 71).  Beyond,
// 128 or 160 rows a tile, whichever takes less: a tile of 160 rows takes 1.2 times one of
// 128 (4,096 x 151,936, 160 and 128 rows a tile: 160 rows 204 and 272, 256 332 and 283,
// 320 338 and 392, 640 650 and 658; 1,024 x 100,000 707 and 687), and 64 again where
// they are too few (128 x 4,096 x 31,000 38 and 53; 128 x 60,000 76 and 65).
int choose(const Projection& p) {
  if (p.rows <= kFewRows && p.hidden_dim > 32 * p.rows) return 1;
  const int64_t wide = (p.vocab - 1) / 256 + 1;
  auto fill = [&](int64_t rows) { return (p.rows + rows - 1) / rows * wide >= kCus * 3 / 4; };
  if (p.rows > 64) {
    const int64_t by128 = (p.rows + int64_t{127}) / 128, by160 = (p.rows + int64_t{159}) / 160;
    const bool tall = by160 * 6 < by128 * 5;
    if (fill(tall ? 160 : 128)) return tall ? 5 : 4;
  }
  return fill(64) ? 3 : 2;
}

}  // namespace

hipError_t launch_quantize_groups_e2m1(const void* in, int bf16, int64_t ld_in, int rows, int cols,
                                       uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                                       int64_t ld_scales, hipStream_t stream) {
  const dim3 grid(unit_grid(rows, cols, bf16));
  if (bf16)
    hipLaunchKernelGGL((quantize_groups_kernel<true>), grid, dim3(QT), 0, stream, in, ld_in, rows,
                       cols, codes, ld_codes, scales, ld_scales);
  else
    hipLaunchKernelGGL((quantize_groups_kernel<false>), grid, dim3(QT), 0, stream, in, ld_in, rows,
                       cols, codes, ld_codes, scales, ld_scales);
  return hipGetLastError();
}

hipError_t launch_dequantize_groups_e2m1(const E2m1Rows& in, int rows, int cols, void* out,
                                         int bf16, int64_t ld_out, hipStream_t stream) {
  const dim3 grid(unit_grid(rows, cols, bf16));
  if (bf16)
    hipLaunchKernelGGL((dequantize_groups_kernel<true>), grid, dim3(QT), 0, stream, in, rows, cols,
                       out, ld_out);
  else
    hipLaunchKernelGGL((dequantize_groups_kernel<false>), grid, dim3(QT), 0, stream, in, rows,
                       cols, out, ld_out);
  return hipGetLastError();
}

// HIP counts a launch's threads in 32 bits (512 a tile at most), and column
// numbers past the last tile must stay below 2^31.
bool lmhead_e2m1_fits(int64_t rows, int64_t vocab) {
  if (vocab > 0x7fffffff - 1023) return false;
  const int64_t tiles_n = (vocab + 255) / 256;
  return (rows + 63) / 64 <= ((int64_t{1} << 22) - 1) / tiles_n;
}

// TS_GEMM_TILE=1..5 forces a shape (the tests run every one).
hipError_t launch_lmhead_e2m1(const uint16_t* hidden, int64_t ld_hidden, const E2m1Rows& lm_head,
                              float* logits, int64_t ld_logits, int rows, int vocab,
                              int hidden_dim, hipStream_t stream) {
  const Projection p{hidden, ld_hidden, lm_head, logits, ld_logits, rows, vocab, hidden_dim};
  const char* env = getenv("TS_GEMM_TILE");
  int sel = env ? atoi(env) : 0;
  if (sel < 1 || sel > 5 || (sel == 1 && rows > kFewRows)) sel = choose(p);
  switch (sel) {
    case 1: return launch_few_rows(p, stream);
    case 2: return launch_tiles<64, 128, 4, 3>(p, stream);
    case 3: return launch_tiles<64, 256, 4, 3>(p, stream);
    case 4: return launch_tiles<128, 256, 4, 2>(p, stream);
    default: return launch_tiles<160, 256, 4, 2>(p, stream);
  }
}

}  // namespace ts
