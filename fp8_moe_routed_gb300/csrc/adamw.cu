// adamw.cu -- one AdamW step over many tensors, with the moments in 32 bits or in 8, and what
// the next forward takes: a bf16 copy, or the experts' 8-bit codes with their channel scales.
//
//   m = b1 m + (1 - b1) g        v = b2 v + (1 - b2) g g
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every product, sum, root and quotient is rounded by itself to f32 (no contraction), so that a
// step has one right answer, however the tensors are cut into units. Moments in 8 bits: e4m3
// codes of m and of sqrt(v), with an f32 scale for 128 values, rounded up or down by chance in
// proportion to what is lost: rounded to nearest, a moment whose change in a step is below half
// a code's spacing (6 %; b2 = 0.999 changes v by 0.1 %) would never move.
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fp8moe_status.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "quantize.cuh"

namespace fp8moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSteps = 4;                        // quads of values that a lane has in flight
constexpr int kUnit = kWarps * kSteps * 128;     // values of a unit (a CTA's share)
constexpr int kTileRows = 128, kTileCols = 128;  // a unit of a tensor with codes
constexpr uint32_t kAll = 0xffffffffu;

// 32 bits for the value at `i` of a tensor, from a key of the seed, the step and the tensor:
// products with the odd numbers next to 2^32 times the fractions of the golden ratio and of the
// roots of 5, 3 and 2, and shifts between them. (Means, correlations between neighbours, steps
// and halves within the noise of 2^20 draws.)
__device__ __forceinline__ uint32_t random_bits(uint64_t i, uint32_t key) {
  uint32_t x = (uint32_t)i * 0x9E3779B9u + (uint32_t)(i >> 32) * 0x3C6EF373u + key;
  x = (x ^ (x >> 16)) * 0xBB67AE85u;
  x = (x ^ (x >> 15)) * 0x6A09E667u;
  return x ^ (x >> 16);
}

// Four values of a lane.
struct Quad {
  float p[4], g[4], m[4], v[4];
  uint32_t mc, vc;               // 8-bit moments: codes
  float ms, vs;                  // and their scales
};

struct Rates {
  float keep, rate, root, b1, c1, b2, c2, eps, grad;
  bool scaled;
  uint32_t key;
};

// VEC: the four values follow each other, on the boundary of four; else they are 32 apart.
template <bool VEC>
__device__ __forceinline__ int64_t place(int64_t i0, int lane, int j) {
  return VEC ? i0 + lane * 4 + j : i0 + j * 32 + lane;
}

__device__ __forceinline__ void load4(const float* a, float (&x)[4]) {
  const float4 v = __ldcs(reinterpret_cast<const float4*>(a));
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void store4(float* a, const float (&x)[4]) {
  __stcs(reinterpret_cast<float4*>(a), make_float4(x[0], x[1], x[2], x[3]));
}

template <int BITS, bool GB, bool VEC>
__device__ __forceinline__ void load_quad(const AdamwEntry& d, int64_t i0, int lane, bool ok,
                                          Quad& q) {
  if constexpr (VEC) {
    if (!ok) {
      q = Quad{};
      return;
    }
    const int64_t i = i0 + lane * 4;
    load4(d.p + i, q.p);
    if constexpr (GB) {
      const uint2 w = __ldcs(reinterpret_cast<const uint2*>(
          static_cast<const __nv_bfloat16*>(d.g) + i));
      q.g[0] = bf16lo_to_f32(w.x), q.g[1] = bf16hi_to_f32(w.x);
      q.g[2] = bf16lo_to_f32(w.y), q.g[3] = bf16hi_to_f32(w.y);
    } else {
      load4(static_cast<const float*>(d.g) + i, q.g);
    }
    if constexpr (BITS == 32) {
      load4(static_cast<const float*>(d.m) + i, q.m);
      load4(static_cast<const float*>(d.v) + i, q.v);
    } else {
      q.mc = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(d.m) + i));
      q.vc = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(d.v) + i));
    }
  } else {
    q.mc = q.vc = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = place<VEC>(i0, lane, j);
      const bool in = ok && i < d.n;
      q.p[j] = in ? d.p[i] : 0.0f;
      if constexpr (GB)
        q.g[j] = in ? __bfloat162float(static_cast<const __nv_bfloat16*>(d.g)[i]) : 0.0f;
      else
        q.g[j] = in ? static_cast<const float*>(d.g)[i] : 0.0f;
      if constexpr (BITS == 32) {
        q.m[j] = in ? static_cast<const float*>(d.m)[i] : 0.0f;
        q.v[j] = in ? static_cast<const float*>(d.v)[i] : 0.0f;
      } else if (in) {
        q.mc |= (uint32_t)static_cast<const uint8_t*>(d.m)[i] << (8 * j);
        q.vc |= (uint32_t)static_cast<const uint8_t*>(d.v)[i] << (8 * j);
      }
    }
  }
  if constexpr (BITS == 8) {
    q.ms = ok ? d.m_scale[i0 >> 7] : 0.0f;
    q.vs = ok ? d.v_scale[i0 >> 7] : 0.0f;
  }
}

__device__ __forceinline__ void decode4(uint32_t codes, float scale, float (&x)[4]) {
  const uint32_t lo = e4m3x2_to_f16x2((uint16_t)codes), hi = e4m3x2_to_f16x2((uint16_t)(codes >> 16));
  half2_to_f32(lo, x[0], x[1]);
  half2_to_f32(hi, x[2], x[3]);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(x[j], scale);
}

// A block's scale from the bits of its largest magnitude: max / 448, or 0 where that is not a
// normal number (its inverse would not be one). NaN and infinity stay and spoil the block.
__device__ __forceinline__ float block_scale(uint32_t most) {
  const float s = __fmul_rn(__uint_as_float(most), 1.0f / 448);
  return s < 0x1p-126f ? 0.0f : s;
}

// |x| as an e4m3 code by chance: |x| / scale * 2^-120 has the code's bits on top of its own
// (both formats' subnormals included), and 16 random bits decide about the 20 below. The largest
// of a block has the code 0x7E (448) exactly; 0x7F would be the code of a NaN.
__device__ __forceinline__ uint32_t encode(float x, float inverse, uint32_t random16) {
  const float y = __fmul_rn(__fmul_rn(fabsf(x), inverse), 0x1p-120f);
  return min((__float_as_uint(y) + (random16 << 4) + 8u) >> 20, 0x7Eu);
}

template <int BITS, bool VEC>
__device__ __forceinline__ void step_quad(const AdamwEntry& d, const Rates& r, int64_t i0, int lane,
                                          bool ok, Quad& q) {
  float root[4];
  if constexpr (BITS == 8) {
    decode4(q.mc, q.ms, q.m);
    decode4(q.vc, q.vs, q.v);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float g = r.scaled ? __fmul_rn(q.g[j], r.grad) : q.g[j];
    const float v = BITS == 8 ? __fmul_rn(q.v[j], q.v[j]) : q.v[j];
    q.m[j] = __fadd_rn(__fmul_rn(q.m[j], r.b1), __fmul_rn(g, r.c1));
    q.v[j] = __fadd_rn(__fmul_rn(v, r.b2), __fmul_rn(__fmul_rn(g, r.c2), g));
    root[j] = __fsqrt_rn(q.v[j]);
    const float step = __fdiv_rn(q.m[j], __fadd_rn(__fmul_rn(root[j], r.root), r.eps));
    q.p[j] = __fsub_rn(__fmul_rn(q.p[j], r.keep), __fmul_rn(step, r.rate));
  }
  if constexpr (BITS == 8) {
    uint32_t mm = 0, vm = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = ok && (VEC || place<VEC>(i0, lane, j) < d.n);
      mm = max(mm, in ? __float_as_uint(q.m[j]) & 0x7fffffffu : 0u);
      vm = max(vm, in ? __float_as_uint(root[j]) & 0x7fffffffu : 0u);
    }
    q.ms = block_scale(__reduce_max_sync(kAll, mm));
    q.vs = block_scale(__reduce_max_sync(kAll, vm));
    const float mi = q.ms != 0.0f ? __frcp_rn(q.ms) : 0.0f;
    const float vi = q.vs != 0.0f ? __frcp_rn(q.vs) : 0.0f;
    q.mc = q.vc = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t bits = random_bits((uint64_t)place<VEC>(i0, lane, j), r.key);
      const uint32_t mc = encode(q.m[j], mi, bits & 0xffffu) |
                          (__float_as_uint(q.m[j]) >> 31) << 7;
      // a second moment that is not zero never becomes zero: m / eps would follow
      uint32_t vc = encode(root[j], vi, bits >> 16);
      if (vc == 0u && root[j] > 0.0f && q.vs > 0.0f) vc = 1u;
      q.mc |= mc << (8 * j);
      q.vc |= vc << (8 * j);
    }
  }
}

template <int BITS, bool VEC>
__device__ __forceinline__ void store_quad(const AdamwEntry& d, int64_t i0, int lane, bool ok,
                                           const Quad& q) {
  if (!ok) return;
  if constexpr (VEC) {
    const int64_t i = i0 + lane * 4;
    store4(d.p + i, q.p);
    if constexpr (BITS == 32) {
      store4(static_cast<float*>(d.m) + i, q.m);
      store4(static_cast<float*>(d.v) + i, q.v);
    } else {
      __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d.m) + i), q.mc);
      __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d.v) + i), q.vc);
    }
    if (d.copy)
      __stcs(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(d.copy) + i),
             make_uint2(f32x2_to_bf16x2(q.p[0], q.p[1]), f32x2_to_bf16x2(q.p[2], q.p[3])));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = place<VEC>(i0, lane, j);
      if (i >= d.n) continue;
      d.p[i] = q.p[j];
      if constexpr (BITS == 32) {
        static_cast<float*>(d.m)[i] = q.m[j];
        static_cast<float*>(d.v)[i] = q.v[j];
      } else {
        static_cast<uint8_t*>(d.m)[i] = (uint8_t)(q.mc >> (8 * j));
        static_cast<uint8_t*>(d.v)[i] = (uint8_t)(q.vc >> (8 * j));
      }
      if (d.copy) static_cast<__nv_bfloat16*>(d.copy)[i] = __float2bfloat16_rn(q.p[j]);
    }
  }
  if constexpr (BITS == 8) {
    if (lane == 0) {
      d.m_scale[i0 >> 7] = q.ms;
      d.v_scale[i0 >> 7] = q.vs;
    }
  }
}

// kUnit values in order.
template <int BITS, bool GB, bool VEC>
__device__ __forceinline__ void linear_unit(const AdamwEntry& d, const Rates& r, int64_t base) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Quad q[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t i0 = base + (s * kWarps + warp) * 128;
    load_quad<BITS, GB, VEC>(d, i0, lane, i0 < d.n, q[s]);
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t i0 = base + (s * kWarps + warp) * 128;
    const bool ok = i0 < d.n;
    step_quad<BITS, VEC>(d, r, i0, lane, ok, q[s]);
    store_quad<BITS, VEC>(d, i0, lane, ok, q[s]);
  }
}

// kTileRows x kTileCols weights of an expert [K, N]: also the largest magnitude of each column.
template <int BITS, bool GB>
__device__ __forceinline__ void tile_unit(const AdamwEntry& d, const Rates& r, uint32_t unit,
                                          uint32_t* s_most) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tiles_n = (d.N + kTileCols - 1) / kTileCols;
  const uint32_t tiles_k = (d.K + kTileRows - 1) / kTileRows;
  const uint32_t tile_n = unit % tiles_n, rest = unit / tiles_n;
  const uint32_t tile_k = rest % tiles_k, e = rest / tiles_k;
  const int col = tile_n * kTileCols;
  const bool ok_col = col + lane * 4 < d.N;      // N is a multiple of 16
  const int64_t expert = (int64_t)e * d.K * d.N;
  uint32_t most[4] = {0, 0, 0, 0};
  for (int k0 = tile_k * kTileRows; k0 < d.K && k0 < (int)(tile_k + 1) * kTileRows;
       k0 += kWarps * kSteps) {
    Quad q[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int k = k0 + s * kWarps + warp;
      load_quad<BITS, GB, true>(d, expert + (int64_t)k * d.N + col, lane, k < d.K && ok_col, q[s]);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int k = k0 + s * kWarps + warp;
      const int64_t i0 = expert + (int64_t)k * d.N + col;
      const bool ok = k < d.K && ok_col;
      step_quad<BITS, true>(d, r, i0, lane, ok, q[s]);
      store_quad<BITS, true>(d, i0, lane, ok, q[s]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ok) most[j] = max(most[j], __float_as_uint(q[s].p[j]) & 0x7fffffffu);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s_most[warp * kTileCols + lane * 4 + j] = most[j];
  __syncthreads();
  for (int c = threadIdx.x; c < kTileCols && col + c < d.N; c += kThreads) {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = max(m, s_most[w * kTileCols + c]);
    atomicMax(d.most + (int64_t)e * d.N + col + c, m);
  }
}

template <int kCapacity>
struct AdamwTable {
  AdamwCommon c;
  AdamwEntry at[kCapacity];
};

template <int kCapacity>
__global__ void __launch_bounds__(kThreads, 2) adamw_kernel(
    const __grid_constant__ AdamwTable<kCapacity> table) {
  __shared__ uint32_t s_most[kWarps * kTileCols];
  const AdamwCommon& c = table.c;
  int lo = 0, hi = c.count - 1;                  // the last entry whose units begin at or before
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table.at[mid].first_unit <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamwEntry& d = table.at[lo];
  const uint32_t unit = blockIdx.x - d.first_unit;
  Rates r;
  r.b1 = c.b1, r.c1 = c.c1, r.b2 = c.b2, r.c2 = c.c2, r.eps = c.eps;
  r.scaled = c.grad_scale != nullptr;
  r.grad = r.scaled ? *c.grad_scale : 1.0f;
  if (c.rates != nullptr) {                      // step or rate on the device
    r.keep = (float)(1.0 - c.rates->lr * d.weight_decay);
    r.rate = c.rates->rate, r.root = c.rates->root;
    r.key = c.rates->key;
  } else {
    r.keep = d.keep, r.rate = c.rate, r.root = c.root;
    r.key = c.key;
  }
  r.key += 0xBB67AE85u * d.which;
  const int64_t base = (int64_t)unit * kUnit;
  const bool gb = d.g_bf16;
  if (d.tiles) {
    if (d.bits == 32) gb ? tile_unit<32, true>(d, r, unit, s_most) : tile_unit<32, false>(d, r, unit, s_most);
    else gb ? tile_unit<8, true>(d, r, unit, s_most) : tile_unit<8, false>(d, r, unit, s_most);
  } else if (d.vec && base + kUnit <= d.n) {
    if (d.bits == 32) gb ? linear_unit<32, true, true>(d, r, base) : linear_unit<32, false, true>(d, r, base);
    else gb ? linear_unit<8, true, true>(d, r, base) : linear_unit<8, false, true>(d, r, base);
  } else {
    if (d.bits == 32) gb ? linear_unit<32, true, false>(d, r, base) : linear_unit<32, false, false>(d, r, base);
    else gb ? linear_unit<8, true, false>(d, r, base) : linear_unit<8, false, false>(d, r, base);
  }
}

// What a step or rate on the device makes of the constants, in 64 bits as the host does; and
// zeros for the columns' largest magnitudes.
__global__ void adamw_prepare_kernel(AdamwRates* rates, const int64_t* step, int64_t host_step,
                                     const float* lr, double host_lr, double beta1, double beta2,
                                     uint32_t seed, uint32_t* most, int64_t count) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (rates != nullptr && i == 0) {
    const int64_t t = step != nullptr ? *step : host_step;
    const double rate = lr != nullptr ? (double)*lr : host_lr;
    rates->lr = rate;
    rates->rate = (float)(rate / (1.0 - pow(beta1, (double)t)));
    rates->root = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)t)));
    rates->key = seed + 0x6A09E667u * (uint32_t)t;
  }
  for (int64_t j = i; j < count; j += (int64_t)gridDim.x * blockDim.x) most[j] = 0u;
}

// The columns' largest magnitudes of weights [E, K, N], where the step's units are not tiles.
__global__ void __launch_bounds__(kThreads) column_max_kernel(const float* p, int K, int N,
                                                              uint32_t* most) {
  __shared__ uint32_t s_most[kWarps * kTileCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * kTileCols, k0 = blockIdx.y * kTileRows;
  const int64_t expert = (int64_t)blockIdx.z * K * N;
  uint32_t m[4] = {0, 0, 0, 0};
  for (int k = k0 + warp; k < K && k < k0 + kTileRows; k += kWarps) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = col + j * 32 + lane;
      if (c < N) m[j] = max(m[j], __float_as_uint(p[expert + (int64_t)k * N + c]) & 0x7fffffffu);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s_most[warp * kTileCols + j * 32 + lane] = m[j];
  __syncthreads();
  for (int c = threadIdx.x; c < kTileCols && col + c < N; c += kThreads) {
    uint32_t v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = max(v, s_most[w * kTileCols + c]);
    atomicMax(most + (int64_t)blockIdx.z * N + col + c, v);
  }
}

// codes = e4m3(p / scale), scale = max(column's largest, 1e-12) / 448, both as the library's
// other quantisers have them (quantize.cuh).
template <bool VEC>
__global__ void __launch_bounds__(kThreads) weight_codes_kernel(const float* p, int K, int N,
                                                                const uint32_t* most,
                                                                uint8_t* codes, float* scale) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * kTileCols, k0 = blockIdx.y * kTileRows;
  const int64_t e = blockIdx.z;
  float s[4], rl[4], rh[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = col + (VEC ? lane * 4 + j : j * 32 + lane);
    float a = c < N ? __uint_as_float(most[e * N + c]) : 1.0f;
    a = a < kEps ? kEps : a;                     // a NaN stays
    s[j] = __fdiv_rn(a, kE4m3Max);
    bracket(s[j], rl[j], rh[j]);
    if (blockIdx.y == 0 && warp == 0 && c < N) scale[e * N + c] = s[j];
  }
  const int64_t expert = e * K * N;
  for (int k = k0 + warp; k < K && k < k0 + kTileRows; k += kWarps) {
    const int64_t i0 = expert + (int64_t)k * N + col;
    float x[4];
    if constexpr (VEC) {
      if (col + lane * 4 >= N) continue;
      load4(p + i0 + lane * 4, x);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = col + j * 32 + lane < N ? p[i0 + j * 32 + lane] : 0.0f;
    }
    const uint16_t lo = quotient_x2<false>(x[0], x[1], s[0], s[1], rl[0], rl[1], rh[0], rh[1]);
    const uint16_t hi = quotient_x2<false>(x[2], x[3], s[2], s[3], rl[2], rl[3], rh[2], rh[3]);
    const uint32_t w = (uint32_t)lo | (uint32_t)hi << 16;
    if constexpr (VEC) {
      *reinterpret_cast<uint32_t*>(codes + i0 + lane * 4) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j * 32 + lane < N) codes[i0 + j * 32 + lane] = (uint8_t)(w >> (8 * j));
    }
  }
}

template <int kCapacity>
cudaError_t launch_table(const AdamwCommon& c, const AdamwEntry* at, int count, uint32_t units,
                         cudaStream_t s) {
  static thread_local AdamwTable<kCapacity> t;   // up to 27 KB: not on the stack
  t.c = c;
  t.c.count = count;
  for (int i = 0; i < count; ++i) t.at[i] = at[i];
  adamw_kernel<kCapacity><<<units, kThreads, 0, s>>>(t);
  return cudaGetLastError();
}

}  // namespace
}  // namespace fp8moe

using namespace fp8moe;

uint64_t fp8moe_adamw_units(const AdamwEntry& d) {
  if (!d.tiles) return (uint64_t)(d.n + kUnit - 1) / kUnit;
  const uint64_t E = (uint64_t)d.n / ((uint64_t)d.K * d.N);
  return E * ((d.K + kTileRows - 1) / kTileRows) * ((d.N + kTileCols - 1) / kTileCols);
}

cudaError_t fp8moe_launch_adamw(const AdamwCommon& common, AdamwEntry* at, int count,
                                cudaStream_t s) {
  uint64_t units = 0;
  for (int i = 0; i < count; ++i) {
    at[i].first_unit = (uint32_t)units;
    units += fp8moe_adamw_units(at[i]);
  }
  // a table of 16 entries is a launch's usual few KB of parameters, one of 256 nearly all of them
  return count <= 16 ? launch_table<16>(common, at, count, (uint32_t)units, s)
                     : launch_table<kAdamwEntries>(common, at, count, (uint32_t)units, s);
}

cudaError_t fp8moe_launch_adamw_prepare(AdamwRates* rates, const int64_t* step, int64_t host_step,
                                        const float* lr, double host_lr, double beta1,
                                        double beta2, uint32_t seed, uint32_t* most, int64_t count,
                                        cudaStream_t s) {
  const int64_t want = (count + 1023) / 1024;
  adamw_prepare_kernel<<<(unsigned)(want < 1 ? 1 : want > 304 ? 304 : want), 256, 0, s>>>(
      rates, step, host_step, lr, host_lr, beta1, beta2, seed, most, count);
  return cudaGetLastError();
}

cudaError_t fp8moe_launch_weight_codes(const float* p, int E, int K, int N, bool vec, bool have_most,
                                       uint32_t* most, uint8_t* codes, float* scale,
                                       cudaStream_t s) {
  const dim3 grid((N + kTileCols - 1) / kTileCols, (K + kTileRows - 1) / kTileRows, E);
  if (!have_most) column_max_kernel<<<grid, kThreads, 0, s>>>(p, K, N, most);
  if (vec) weight_codes_kernel<true><<<grid, kThreads, 0, s>>>(p, K, N, most, codes, scale);
  else weight_codes_kernel<false><<<grid, kThreads, 0, s>>>(p, K, N, most, codes, scale);
  return cudaGetLastError();
}
