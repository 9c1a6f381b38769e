// 4-bit rows with a scale per group, and the local vocabulary projection from
// them, on gfx950.
//
// A row is held as OCP MX FP4: groups of 32 consecutive entries share a scale
// s = 2^e (E8M0: one byte, e + 127, 255 NaN), and each entry is a code of E2M1
// (sign, two bits of exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6),
// two to a byte, the even column in the low half.  4.25 bits an entry.
//   quantize   e = least integer >= -127 with max|x| <= 7 * 2^e: what lies
//              above 6 s then loses at most the half step of E2M1's last
//              binade (and e <= 125, so that no finite entry becomes infinite); code = the value nearest x / s, ties to the even code
//   project    logits[r, v] = sum_h hidden[r, h] * 2^e[v, h / 32] * q[v, h]
// A power of two times an E2M1 value has two significant bits, so it is a bf16
// number and its products with bf16 are exact in fp32: the lm_head becomes
// matrix-core fragments in registers (v_cvt_scalef32_pk_bf16_fp4: two entries
// and their scale in one instruction), nothing is rounded, and only the fp32
// sums differ from the definition.
#include <stdlib.h>

#include "lmhead_e2m1.hpp"
#include "tile_store.hpp"

namespace ts {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kXcds = 8;

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

template <bool BF16>
__device__ __forceinline__ void load_unit(const void* in, int64_t at, float (&x)[kUnit]) {
  if (BF16) {
    const u16x8u v = *reinterpret_cast<const u16x8u*>(static_cast<const uint16_t*>(in) + at);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(v[i]) << 16);
  } else {
    const float* p = static_cast<const float*>(in) + at;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4u v = *reinterpret_cast<const f32x4u*>(p + 4 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * h + i] = v[i];
    }
  }
}

// Four neighbouring lanes hold a group.  The scale's byte comes from the bits
// of the group's largest magnitude 1.m * 2^(E - 127): E - 2 where 1.m <= 1.75,
// else E - 1.  As integers magnitudes are in order, with infinity and NaN last.
template <bool BF16>
__global__ __launch_bounds__(QT) void quantize_groups_kernel(
    const void* __restrict__ in, int64_t ld_in, int rows, int cols, uint8_t* __restrict__ codes,
    int64_t ld_codes, uint8_t* __restrict__ scales, int64_t ld_scales) {
  Units u(cols, static_cast<int64_t>(blockIdx.x) * QT + threadIdx.x,
          static_cast<int64_t>(gridDim.x) * QT);
  for (; u.row < rows; u.next()) {
    float x[kUnit];
    load_unit<BF16>(in, u.row * ld_in + u.at * kUnit, x);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1, 4)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2, 4)));
    int byte = max(static_cast<int>(top >> 23) - 2 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
    byte = min(byte, 252);  // 6 * 2^125 is finite
    if (top == 0) byte = 127;
    if (top >= 0x7f800000u) byte = 255;
    uint32_t w = 0;
    // Past the last finite byte nothing is written but zeros beside the NaN.
    if (byte != 255) {
      const float s = scale_of(byte);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
    }
    *reinterpret_cast<uint32_t*>(codes + u.row * ld_codes + u.at * (kUnit / 2)) = w;
    if (u.at % kUnitsPerGroup == 0)
      scales[u.row * ld_scales + u.at / kUnitsPerGroup] = static_cast<uint8_t>(byte);
  }
}

template <bool BF16>
__global__ __launch_bounds__(QT) void dequantize_groups_kernel(E2m1Rows in, int rows, int cols,
                                                               void* __restrict__ out,
                                                               int64_t ld_out) {
  Units u(cols, static_cast<int64_t>(blockIdx.x) * QT + threadIdx.x,
          static_cast<int64_t>(gridDim.x) * QT);
  for (; u.row < rows; u.next()) {
    const uint32_t w =
        *reinterpret_cast<const uint32_t*>(in.codes + u.row * in.ld + u.at * (kUnit / 2));
    const float s = scale_of(in.scales[u.row * in.ld_scales + u.at / kUnitsPerGroup]);
    const int64_t at = u.row * ld_out + u.at * kUnit;
    if (BF16) {
      u16x8u v;
      auto put = [&](int i, bf16x2 q) {
        const uint32_t b = __builtin_bit_cast(uint32_t, q);
        v[2 * i] = static_cast<uint16_t>(b);
        v[2 * i + 1] = static_cast<uint16_t>(b >> 16);
      };
      put(0, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
      put(1, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
      put(2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
      put(3, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
      *reinterpret_cast<u16x8u*>(static_cast<uint16_t*>(out) + at) = v;
    } else {
      float* p = static_cast<float*>(out) + at;
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
      const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
      const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
      *reinterpret_cast<f32x4u*>(p) = f32x4u{a[0], a[1], b[0], b[1]};
      *reinterpret_cast<f32x4u*>(p + 4) = f32x4u{c[0], c[1], d[0], d[1]};
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
// Up to 16 NT rows: bound by the lm_head's bytes, each read once.  A wave keeps
// its share of every hidden row in registers (NS steps of 128 entries) and the
// workgroup's waves take the row's shares side by side; then the workgroup goes
// through the lm_head, 16 VT rows at a time.  A lane loads 16 bytes of codes,
// which is one group: lane l has row l % 16, groups 4 s + l / 16.  In
// v_mfma_f32_16x16x32_bf16 lane l holds entries 8 (l / 16) .. + 7 of a slice of
// 32; any order of the sum's entries will do as long as both operands share it,
// so slice i takes the i-th eight entries of each lane's group.  The shares are
// added up through LDS, in a fixed order.
constexpr int kStep = 128;  // entries of a row in one step
constexpr int kMaxWaves = 16;

template <int NT, int NS, int VT, int MAX_WAVES>
__global__ __launch_bounds__(64 * MAX_WAVES) void lmhead_e2m1_few_kernel(
    const uint16_t* __restrict__ X, int64_t ldx, E2m1Rows w, float* __restrict__ C, int64_t ldc,
    int M, int N, int K, int tiles) {
  constexpr int BV = 16 * VT;
  extern __shared__ float part[];  // [2][waves][16 NT][BV]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int groups = K / kE2m1Group;

  // Hidden rows r16 + 16 n, the entries of this lane's groups.
  bf16x8 x[NT][NS][4];
  bool live[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int g = (wave * NS + s) * 4 + q;
    live[s] = g < groups;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = r16 + 16 * n;
      const uint16_t* p = X + static_cast<int64_t>(min(r, M - 1)) * ldx + min(g, groups - 1) * 32;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[n][s][i] = *reinterpret_cast<const bf16x8*>(p + 8 * i);
        if (r >= M || g >= groups) x[n][s][i] = bf16x8{};
      }
    }
  }

  u32x4 code[VT][NS];
  uint32_t scale[VT][NS];
  auto load = [&](int tile) {
#pragma unroll
    for (int t = 0; t < VT; ++t) {
      const int64_t v = min(tile * BV + t * 16 + r16, N - 1);
      const uint8_t* pc = w.codes + v * w.ld;
      const uint8_t* ps = w.scales + v * w.ld_scales;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int g = min((wave * NS + s) * 4 + q, groups - 1);
        code[t][s] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(pc + g * 16));
        scale[t][s] = ps[g];
      }
    }
  };

  int tile = blockIdx.x;
  if (tile < tiles) load(tile);
  float* mine = part + wave * (16 * NT * BV);
  const int half = waves * 16 * NT * BV;
  int buf = 0;
  for (; tile < tiles; tile += gridDim.x) {
    f32x4 acc[VT][NT];
#pragma unroll
    for (int t = 0; t < VT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[t][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int t = 0; t < VT; ++t)
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        // A group past the row has zeros on the other side, and must not be NaN.
        const float sc = live[s] ? scale_of(scale[t][s]) : 1.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 a = frag_of(code[t][s][i], sc);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            acc[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, x[n][s][i], acc[t][n], 0, 0, 0);
        }
      }
    if (tile + static_cast<int>(gridDim.x) < tiles) load(tile + gridDim.x);
    // Lane l holds lm_head rows 4 q .. 4 q + 3 of hidden row l % 16.
#pragma unroll
    for (int t = 0; t < VT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (r16 + 16 * n < M)
          *reinterpret_cast<f32x4*>(mine + buf * half + (r16 + 16 * n) * BV + t * 16 + 4 * q) =
              acc[t][n];
    __syncthreads();
    for (int i = tid; i < M * BV; i += blockDim.x) {
      const int r = i / BV, c = i % BV;
      const float* p = part + buf * half + i;
      float sum = p[0];
      for (int k = 1; k < waves; ++k) sum += p[k * (16 * NT * BV)];
      if (tile * BV + c < N) C[static_cast<int64_t>(r) * ldc + tile * BV + c] = sum;
    }
    buf ^= 1;
  }
}

// -------------------------------------------------------------- many rows
// BM x BN tiles, K in steps of 64.  The hidden rows go through double-buffered
// LDS as in the bf16 kernel (rows of 128 bytes, 16-byte chunks swizzled by the
// row pair); the lm_head goes straight into registers, 16 bytes a lane, which is
// one group: lane l has row l % 32 and the step's group l / 32.  Slice i of a
// step takes the i-th eight entries of each lane's group, so its hidden
// fragment is chunk 4 (l / 32) + i.
constexpr int kBK = 64;

template <int LOADS, int NW>
__device__ __forceinline__ void issue_hidden(const uint16_t* const* src, uint8_t* stage, int wave,
                                             int k0) {
#pragma unroll
  for (int q = 0; q < LOADS; ++q)
    __builtin_amdgcn_global_load_lds(src[q] + k0, stage + (wave + NW * q) * 1024, 16, 0, 0);
}

template <int BM, int BN, int WAVES_M, int WAVES_N>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, 1) void lmhead_e2m1_kernel(
    const uint16_t* __restrict__ X, int64_t ldx, E2m1Rows w, float* __restrict__ C, int64_t ldc,
    int M, int N, int K, int tiles_m, int tiles_total, int tiles_per_xcd, int vec_out) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  constexpr int TM = WM / 32, TN = WN / 32;
  constexpr int STAGE = BM * 128;
  constexpr int LOADS = BM / 8 / NW;
  constexpr int SCRATCH = NW * kTileStoreFloats * 4;
  static_assert(BM / 8 % NW == 0, "blocks must split evenly over the waves");
  static_assert(WM % 32 == 0 && WN % 32 == 0, "wave tile of whole 32x32 blocks");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE > SCRATCH ? 2 * STAGE : SCRATCH];

  const int bid = blockIdx.x;
  const int tile = (bid % kXcds) * tiles_per_xcd + bid / kXcds;
  if (tile >= tiles_total) return;
  const int m0 = tile % tiles_m * BM, n0 = tile / tiles_m * BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm0 = (wave / WAVES_N) * WM, wn0 = (wave % WAVES_N) * WN;
  const int frow = lane & 31, fhalf = lane >> 5;

  const int steps = (K + kBK - 1) / kBK;
  // A last step of one group only: the other half of each LDS row repeats it
  // and meets zeros.
  const bool half_step = K % kBK != 0;
  const uint16_t* src[LOADS];
  const uint16_t* src_half[LOADS];
#pragma unroll
  for (int q = 0; q < LOADS; ++q) {
    const int row = 8 * (wave + NW * q) + (lane >> 3);
    const int c = (lane & 7) ^ ((row >> 1) & 7);
    const uint16_t* p = X + static_cast<int64_t>(min(m0 + row, M - 1)) * ldx;
    src[q] = p + c * 8;
    src_half[q] = p + (c & 3) * 8;
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
    const int r = wm0 + i * 32 + frow;
    aoff[i] = r * 128;
    aswz[i] = (r >> 1) & 7;
  }

  u32x4 code[TN];
  uint32_t scale[TN];
  auto load_w = [&](int ks) {
    const int g = min(2 * ks + fhalf, groups - 1);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      code[j] = *reinterpret_cast<const u32x4*>(wp[j] + g * 16);
      scale[j] = sp[j][g];
    }
  };

  issue_hidden<LOADS, NW>(steps == 1 && half_step ? src_half : src, lds, wave, 0);
  load_w(0);
  for (int ks = 0; ks < steps; ++ks) {
    const int cur = ks & 1;
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    u32x4 now[TN];
    float sc[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      now[j] = code[j];
      sc[j] = scale_of(scale[j]);
    }
    const bool last_half = half_step && ks == steps - 1;
    if (last_half && fhalf) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        now[j] = u32x4{0, 0, 0, 0};
        sc[j] = 1.0f;
      }
    }
    if (ks + 1 < steps) {
      issue_hidden<LOADS, NW>(half_step && ks + 2 == steps ? src_half : src,
                              lds + (cur ^ 1) * STAGE, wave, (ks + 1) * kBK);
      load_w(ks + 1);
    }
    const uint8_t* base = lds + cur * STAGE;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int chunk = 4 * fhalf + kk;
      bf16x8 af[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        af[i] = *reinterpret_cast<const bf16x8*>(base + aoff[i] + ((chunk ^ aswz[i]) << 4));
        // 0 x inf is not 0.
        if (last_half && fhalf) af[i] = bf16x8{};
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const bf16x8 b = frag_of(now[j][kk], sc[j]);
#pragma unroll
        for (int i = 0; i < TM; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[i], b, acc[i][j], 0, 0, 0);
      }
    }
  }

  __syncthreads();  // every wave is done reading the stages
  if (vec_out) {
    store_tile_rows<false>(acc, reinterpret_cast<float*>(lds), wave, lane, C, ldc, m0 + wm0,
                           n0 + wn0, M, N, nullptr, nullptr);
    return;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int col = n0 + wn0 + j * 32 + frow;
      if (col >= N) continue;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int row = m0 + wm0 + i * 32 + 8 * (e >> 2) + 4 * fhalf + (e & 3);
        if (row < M) C[static_cast<int64_t>(row) * ldc + col] = acc[i][j][e];
      }
    }
  }
}

int unit_grid(int rows, int cols) {
  const int64_t groups = (static_cast<int64_t>(rows) * (cols / kUnit) + QT - 1) / QT;
  return static_cast<int>(groups < 8192 ? groups : 8192);
}

struct Projection {
  const uint16_t* hidden;
  int64_t ld_hidden;
  E2m1Rows w;
  float* logits;
  int64_t ld_logits;
  int rows, vocab, hidden_dim;
};

template <int NT, int NS, int VT, int MAX_WAVES>
hipError_t launch_few(const Projection& p, int waves, hipStream_t stream) {
  const int tiles = (p.vocab - 1) / (16 * VT) + 1;
  const int lds = 2 * waves * 16 * NT * 16 * VT * 4;
  const int grid = tiles < 512 ? tiles : 512;
  hipLaunchKernelGGL((lmhead_e2m1_few_kernel<NT, NS, VT, MAX_WAVES>), dim3(grid), dim3(64 * waves), lds,
                     stream, p.hidden, p.ld_hidden, p.w, p.logits, p.ld_logits, p.rows, p.vocab,
                     p.hidden_dim, tiles);
  return hipGetLastError();
}

template <int BM, int BN, int WAVES_M, int WAVES_N>
hipError_t launch_tiles(const Projection& p, hipStream_t stream) {
  const int tiles_m = (p.rows - 1) / BM + 1, tiles_n = (p.vocab - 1) / BN + 1;
  const int total = tiles_m * tiles_n;
  const int per_xcd = (total + kXcds - 1) / kXcds;
  hipLaunchKernelGGL((lmhead_e2m1_kernel<BM, BN, WAVES_M, WAVES_N>), dim3(per_xcd * kXcds),
                     dim3(64 * WAVES_M * WAVES_N), 0, stream, p.hidden, p.ld_hidden, p.w, p.logits,
                     p.ld_logits, p.rows, p.vocab, p.hidden_dim, tiles_m, total, per_xcd,
                     rows_take_vector_stores(p.logits, p.ld_logits));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_groups_e2m1(const void* in, int bf16, int64_t ld_in, int rows, int cols,
                                       uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                                       int64_t ld_scales, hipStream_t stream) {
  const dim3 grid(unit_grid(rows, cols));
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
  const dim3 grid(unit_grid(rows, cols));
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

// TS_GEMM_TILE=1..5 forces a shape (the tests run every one): 1: the kernel for
// few rows, where it can take the sizes; 2: 64 x 256; 3: 128 x 256; 4: 256 x
// 256; 5: 320 x 256.
hipError_t launch_lmhead_e2m1(const uint16_t* hidden, int64_t ld_hidden, const E2m1Rows& lm_head,
                              float* logits, int64_t ld_logits, int rows, int vocab,
                              int hidden_dim, hipStream_t stream) {
  const Projection p{hidden, ld_hidden, lm_head, logits, ld_logits, rows, vocab, hidden_dim};
  const char* env = getenv("TS_GEMM_TILE");
  int sel = env ? atoi(env) : 0;
  const int steps = (hidden_dim - 1) / kStep + 1;
  const bool few = rows <= 32 && steps <= 4 * kMaxWaves;
  if (sel < 1 || sel > 5 || (sel == 1 && !few)) {
    const int64_t pad256 = (rows + int64_t{255}) / 256 * 256, pad320 = (rows + int64_t{319}) / 320 * 320;
    sel = few ? 1 : rows <= 64 ? 2 : rows <= 128 ? 3 : pad320 < pad256 ? 5 : 4;
  }
  switch (sel) {
    case 1: {
      const int waves = (steps + 3) / 4;
      if (waves > 8)
        return rows <= 16 ? launch_few<1, 4, 1, kMaxWaves>(p, waves, stream)
                          : launch_few<2, 4, 1, kMaxWaves>(p, waves, stream);
      return rows <= 16 ? launch_few<1, 4, 2, 8>(p, waves, stream)
                        : launch_few<2, 4, 2, 8>(p, waves, stream);
    }
    case 2: return launch_tiles<64, 256, 1, 4>(p, stream);
    case 3: return launch_tiles<128, 256, 2, 4>(p, stream);
    case 4: return launch_tiles<256, 256, 2, 4>(p, stream);
    default: return launch_tiles<320, 256, 2, 4>(p, stream);
  }
}

}  // namespace ts
