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
#include "lmhead_lora.hpp"

namespace ts {
namespace {

constexpr int kNoAdapter = -1, kBadAdapter = -2;
constexpr int kParts = 3;  // bf16 numbers that hold one fp32 u
constexpr int kDownThreads = 256;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__host__ __device__ constexpr int padded_rank(int rank) { return (rank + 15) / 16 * 16; }

// What the down step leaves, rows in the order of (adapter, row).
struct DownRows {
  __bf16* u;     // [rows][kParts][padded rank], zeros past the rank
  int32_t* row;  // the row at this place
  int32_t* id;   // its adapter, kNoAdapter or kBadAdapter
};

__device__ __forceinline__ int adapter_of(int id, int n_adapters) {
  if (id >= 0 && id < n_adapters) return id;
  return id == kNoAdapter ? kNoAdapter : kBadAdapter;
}

// One workgroup per row.
__global__ __launch_bounds__(kDownThreads) void lora_down_kernel(LoraArgs p, DownRows out) {
  __shared__ int before_wave[kDownThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const int id = adapter_of(p.ids[r], p.n_adapters);
    int before = 0;
    for (int i = tid; i < p.rows; i += kDownThreads) {
      const int other = adapter_of(p.ids[i], p.n_adapters);
      before += other < id || (other == id && i < r);
    }
    for (int d = 32; d > 0; d >>= 1) before += __shfl_xor(before, d, 64);
    if (lane == 0) before_wave[wave] = before;
    __syncthreads();
    int place = 0;
    for (int w = 0; w < kDownThreads / 64; ++w) place += before_wave[w];
    if (tid == 0) {
      out.row[place] = r;
      out.id[place] = id;
    }
    const int rp = padded_rank(p.rank);
    __bf16* u = out.u + static_cast<int64_t>(place) * kParts * rp;
    const uint16_t* x = p.hidden + static_cast<int64_t>(r) * p.ld_hidden;
    for (int k = wave; k < rp; k += kDownThreads / 64) {
      float sum = 0.0f;
      if (id >= 0 && k < p.rank) {
        const uint16_t* a = p.a + static_cast<int64_t>(id) * p.stride_a + static_cast<int64_t>(k) * p.ld_a;
        for (int h = lane * 8; h < p.hidden_dim; h += 64 * 8) {
          const bf16x8 xv = *reinterpret_cast<const bf16x8*>(x + h);
          const bf16x8 av = *reinterpret_cast<const bf16x8*>(a + h);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sum = fmaf(static_cast<float>(xv[e]), static_cast<float>(av[e]), sum);
        }
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
        if (p.scales) sum *= p.scales[id];
      }
      if (lane == 0) {
        float rest = sum;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          const __bf16 part = static_cast<__bf16>(rest);
          u[q * rp + k] = part;
          rest -= static_cast<float>(part);
        }
      }
    }
    __syncthreads();
  }
}

constexpr int kUpCols = 256;

// logits += B_a u, one workgroup per row and kUpCols columns.
__global__ __launch_bounds__(kUpCols) void lora_add_kernel(LoraArgs p, DownRows d) {
  const int rp = padded_rank(p.rank);
  const int v = blockIdx.x * kUpCols + threadIdx.x;
  for (int place = blockIdx.y; place < p.rows; place += gridDim.y) {
    const int id = d.id[place];
    if (id == kNoAdapter || v >= p.vocab) continue;
    float* out = p.logits + static_cast<int64_t>(d.row[place]) * p.ld_logits + v;
    if (id == kBadAdapter) {
      *out = NAN;
      continue;
    }
    const __bf16* u = d.u + static_cast<int64_t>(place) * kParts * rp;
    const uint16_t* b = p.b + static_cast<int64_t>(id) * p.stride_b + static_cast<int64_t>(v) * p.ld_b;
    float sum = 0.0f;
    for (int k = 0; k < p.rank; k += 8) {
      const bf16x8 bv = *reinterpret_cast<const bf16x8*>(b + k);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float uk = static_cast<float>(u[k + e]) + static_cast<float>(u[rp + k + e]) +
                         static_cast<float>(u[2 * rp + k + e]);
        sum = fmaf(uk, static_cast<float>(bv[e]), sum);
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
  at += round256(sizeof(__bf16) * kParts * static_cast<size_t>(padded_rank(static_cast<int>(rank))) *
                 static_cast<size_t>(rows));
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

hipError_t launch_lmhead_lora(const LoraArgs& p, void* ws, hipStream_t stream) {
  size_t bytes;
  const DownRows d = lay_out(ws, p.rows, p.rank, &bytes);
  hipLaunchKernelGGL(lora_down_kernel, dim3(p.rows < (1 << 20) ? p.rows : (1 << 20)),
                     dim3(kDownThreads), 0, stream, p, d);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = launch_lmhead_gemm(p.hidden, p.ld_hidden, p.lm_head, p.ld_lm_head, p.logits, p.ld_logits,
                         p.rows, p.vocab, p.hidden_dim, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(lora_add_kernel,
                     dim3((p.vocab + kUpCols - 1) / kUpCols, p.rows < 65535 ? p.rows : 65535),
                     dim3(kUpCols), 0, stream, p, d);
  return hipGetLastError();
}

}  // namespace ts
