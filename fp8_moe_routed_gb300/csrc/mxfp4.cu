// mxfp4.cu -- microscaled 4-bit (MXFP4) quantisation of activations and expert
// weights, and the way back.
//
// Layouts: codes two a byte along K (the even k in the low half). Scale bytes by
// 32-bit words of four consecutive blocks: word [K / 128][row], so that the words
// of consecutive rows, which the product's scale loads take by the warp, are
// contiguous. A last word's bytes past K / 32 mean nothing and are never used.
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fp8moe_status.cuh"
#include "groups.cuh"
#include "kernels.h"
#include "mxfp4.cuh"
#include "pdl.cuh"
#include "vec16.cuh"

namespace fp8moe {
namespace mx {

// The larger magnitudes' bf16 bits, in both halves.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  return __vmaxu2(a, b & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t max_bits2(const uint4& v) {
  return max_abs2(max_abs2(max_abs2(v.x & 0x7FFF7FFFu, v.y), v.z), v.w);
}

// Eight values times inv as codes; the codes of a NaN block (whatever the conversion
// made of it) are zeros.
__device__ __forceinline__ uint32_t quantize8(const uint4& v, uint32_t byte, float inv) {
  float2 f[4];
  Vec<__nv_bfloat16>::unpack(v, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], both(inv));
  const uint32_t q = f32x8_to_e2m1x8(f);
  return byte == kMxNan ? 0u : q;
}

// ------------------------------------------------------------ activation rows
// Bound by HBM: 2 bytes read, 17/32 written per value. Four lanes hold a block
// (8 values, one 16-byte load each), so a warp's loads and code stores are
// contiguous; two shuffles give the block's largest magnitude, and the 16 lanes of
// a scale word join their four bytes. A warp takes 1024 values of one row: four
// loads in flight per lane. (32768 x 7168: 98 us = 6.1 TB/s; two loads in flight 126 us,
// eight 103 us.)
constexpr int kRowsThreads = 256;
constexpr int kRowsUnroll = 4;

__global__ void __launch_bounds__(kRowsThreads)
mx_quantize_rows_kernel(const uint4* __restrict__ x, int64_t M, int K,
                        const int32_t* __restrict__ gs, int E, uint32_t* __restrict__ codes,
                        uint32_t* __restrict__ scales, int64_t scale_stride, int report) {
  __shared__ int32_t s_lo, s_hi;
  pdl_launch_dependents();
  group_row_range_warp0(gs, E, M, 0, E, &s_lo, &s_hi, report && blockIdx.x == 0);
  __syncthreads();
  const int64_t T = s_hi;
  const int nvec = K / 8;                       // 16-byte vectors (and code words) of a row
  const int chunks = (nvec + 32 * kRowsUnroll - 1) / (32 * kRowsUnroll);
  const int lane = threadIdx.x & 31;
  const int64_t items = T * chunks;
  const int64_t step = (int64_t)gridDim.x * (kRowsThreads / 32);
  for (int64_t it = (int64_t)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5); it < items;
       it += step) {
    const int64_t row = it / chunks;
    const int v0 = (int)(it - row * chunks) * (32 * kRowsUnroll) + lane;
    uint4 v[kRowsUnroll];
#pragma unroll
    for (int i = 0; i < kRowsUnroll; ++i)
      v[i] = v0 + 32 * i < nvec ? __ldg(x + row * nvec + v0 + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kRowsUnroll; ++i) {
      uint32_t m = max_bits2(v[i]);
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t byte = mx_scale_byte(max(m & 0xFFFFu, m >> 16));
      const int vi = v0 + 32 * i;
      if (vi < nvec) codes[row * nvec + vi] = quantize8(v[i], byte, mx_inv_scale(byte));
      uint32_t word = byte << (8 * ((lane >> 2) & 3));
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      if ((lane & 15) == 0 && vi < nvec) scales[(vi / 16) * scale_stride + row] = word;
    }
  }
}

// ------------------------------------------------------------- expert weights
// w [E, K, N] -> codes [E, N, K/2]: blocks run along K, which is not the contiguous
// axis of the framework's weights, so a tile is turned through shared memory. A
// CTA takes 256 k x 64 columns; a warp takes one block row of 32 k, each lane two
// columns: 32 loads of 128 contiguous bytes per warp, all in flight. The codes of a
// column's 256 k leave as 128 contiguous bytes. (8 x 7168 x 4096: 97 us = 6.1 TB/s.)
constexpr int kWtThreads = 256;
constexpr int kWtK = 256, kWtN = 64;

__global__ void __launch_bounds__(kWtThreads)
mx_quantize_weights_kernel(const uint32_t* __restrict__ w, int K, int N, int k_tiles, int n_tiles,
                           uint8_t* __restrict__ codes, uint32_t* __restrict__ scales) {
  // 36-word rows: 16-byte aligned, and eight consecutive rows fall into different banks
  __shared__ uint4 s_code[kWtN][kWtK / 32 + 1];
  __shared__ uint32_t s_scale[kWtK / kMxWord][kWtN];    // written by bytes, read by words
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tile = blockIdx.x;
  const int kt = (int)(tile % k_tiles);
  const int nt = (int)((tile / k_tiles) % n_tiles);
  const int64_t e = tile / ((int64_t)k_tiles * n_tiles);
  const int k0 = kt * kWtK + warp * kMxBlock, n0 = nt * kWtN;
  const int n = n0 + 2 * lane;
  uint32_t v[kMxBlock];
  const bool in = k0 < K && n < N;      // K % 32 == 0: a block is whole or absent
  const uint32_t* src = w + ((e * K + k0) * (int64_t)N + n) / 2;
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i) v[i] = in ? __ldg(src + (int64_t)i * (N / 2)) : 0u;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i) m = max_abs2(m, v[i]);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t byte = mx_scale_byte(c ? m >> 16 : m & 0xFFFFu);
    const float inv = mx_inv_scale(byte);
    uint32_t q[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      // this column's eight values of the group, two a word
      uint4 x;
      uint32_t* const p = &x.x;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = __byte_perm(v[8 * g + 2 * i], v[8 * g + 2 * i + 1], c ? 0x7632 : 0x5410);
      q[g] = quantize8(x, byte, inv);
    }
    s_code[2 * lane + c][warp] = make_uint4(q[0], q[1], q[2], q[3]);
    reinterpret_cast<uint8_t*>(&s_scale[warp >> 2][2 * lane + c])[warp & 3] = (uint8_t)byte;
  }
  __syncthreads();
  const int64_t row_bytes = K / 2;
#pragma unroll
  for (int i = threadIdx.x; i < kWtN * (kWtK / 32); i += kWtThreads) {
    const int r = i / (kWtK / 32), b = i % (kWtK / 32);
    const int kb = kt * kWtK + b * kMxBlock;
    if (n0 + r < N && kb < K)
      *reinterpret_cast<uint4*>(codes + (e * N + n0 + r) * row_bytes + kb / 2) = s_code[r][b];
  }
  const int words = (K + kMxWord - 1) / kMxWord;
  if (threadIdx.x < kWtN * (kWtK / kMxWord)) {
    const int g = threadIdx.x / kWtN, r = threadIdx.x % kWtN;
    const int word = kt * (kWtK / kMxWord) + g;
    if (word < words && n0 + r < N)
      scales[(e * words + word) * N + n0 + r] = s_scale[g][r];
  }
}

// ----------------------------------------------------------------- dequantise
// codes [E, N, K/2] -> bf16 [E, N, K], exact (an e2m1 value times a power of two;
// below bf16's subnormals it rounds to nearest even). Bound by HBM: 2 bytes written,
// 17/32 read per value. A lane turns 8 codes (one word) into 16 bytes, so a warp
// stores 512 contiguous bytes; four words in flight per lane. (8 x 7168 x 4096: 89 us =
// 6.7 TB/s.)
constexpr int kDqUnroll = 4;

__global__ void __launch_bounds__(kRowsThreads)
mx_dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                     int64_t rows, int N, int K, uint4* __restrict__ out) {
  const int nvec = K / 8;
  const int words = (K + kMxWord - 1) / kMxWord;
  const int chunks = (nvec + 32 * kDqUnroll - 1) / (32 * kDqUnroll);
  const int lane = threadIdx.x & 31;
  const int64_t items = rows * chunks;
  const int64_t step = (int64_t)gridDim.x * (kRowsThreads / 32);
  for (int64_t it = (int64_t)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5); it < items;
       it += step) {
    const int64_t row = it / chunks;             // expert * N + n
    const int64_t e = row / N;
    const int n = (int)(row - e * N);
    const int v0 = (int)(it - row * chunks) * (32 * kDqUnroll) + lane;
    uint32_t c[kDqUnroll], b[kDqUnroll];
#pragma unroll
    for (int i = 0; i < kDqUnroll; ++i) {
      const int vi = v0 + 32 * i;
      if (vi >= nvec) continue;
      c[i] = __ldg(codes + row * nvec + vi);
      b[i] = __ldg(scales + ((e * words + vi / 16) * N + n) * 4 + ((vi >> 2) & 3));
    }
#pragma unroll
    for (int i = 0; i < kDqUnroll; ++i) {
      const int vi = v0 + 32 * i;
      if (vi >= nvec) continue;
      const float s = mx_scale(b[i]);
      uint32_t h[4];
      e2m1x8_to_f16x2x4(c[i], h);
      float2 f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        half2_to_f32(h[k], f[k].x, f[k].y);
        f[k] = mul2(f[k], both(s));
      }
      out[row * nvec + vi] = Vec<__nv_bfloat16>::pack(f);
    }
  }
}

int grid_for(int64_t items, int num_sms, int ctas_per_sm) {
  const int64_t want = (items + kRowsThreads / 32 - 1) / (kRowsThreads / 32);
  const int64_t most = (int64_t)num_sms * ctas_per_sm;
  return (int)(want < most ? want : most);
}

}  // namespace mx
}  // namespace fp8moe

FP8MOE_DEFINE_STATUS_TAKE(fp8moe_status_take_mxfp4)

cudaError_t fp8moe_launch_mxfp4_quantize_rows(const void* x, int64_t M, int K, const int32_t* gs,
                                              int E, uint8_t* codes, uint8_t* scales,
                                              int64_t scale_stride, int num_sms, int report,
                                              cudaStream_t s) {
  using namespace fp8moe::mx;
  const int chunks = (K / 8 + 32 * kRowsUnroll - 1) / (32 * kRowsUnroll);
  // the resident CTAs (45 registers a thread): every one reads the group sizes once
  mx_quantize_rows_kernel<<<grid_for(M * chunks, num_sms, 5), kRowsThreads, 0, s>>>(
      static_cast<const uint4*>(x), M, K, gs, E, reinterpret_cast<uint32_t*>(codes),
      reinterpret_cast<uint32_t*>(scales), scale_stride, report);
  return cudaGetLastError();
}

cudaError_t fp8moe_launch_mxfp4_quantize_weights(const void* w, int E, int K, int N, uint8_t* codes,
                                                 uint8_t* scales, cudaStream_t s) {
  using namespace fp8moe::mx;
  const int k_tiles = (K + kWtK - 1) / kWtK, n_tiles = (N + kWtN - 1) / kWtN;
  const int64_t tiles = (int64_t)E * k_tiles * n_tiles;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  mx_quantize_weights_kernel<<<(unsigned)tiles, kWtThreads, 0, s>>>(
      static_cast<const uint32_t*>(w), K, N, k_tiles, n_tiles, codes,
      reinterpret_cast<uint32_t*>(scales));
  return cudaGetLastError();
}

cudaError_t fp8moe_launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int E,
                                           int N, int K, void* out, int num_sms, cudaStream_t s) {
  using namespace fp8moe::mx;
  const int64_t rows = (int64_t)E * N;
  const int chunks = (K / 8 + 32 * kDqUnroll - 1) / (32 * kDqUnroll);
  // many short CTAs: an even end (7168 x 4096 x 8: 90 us against 106 with 8 per SM)
  mx_dequantize_kernel<<<grid_for(rows * chunks, num_sms, 64), kRowsThreads, 0, s>>>(
      reinterpret_cast<const uint32_t*>(codes), scales, rows, N, K, static_cast<uint4*>(out));
  return cudaGetLastError();
}
