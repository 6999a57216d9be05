// adamw.cu -- one AdamW step over many tensors, with the moments in 32 bits or in 8, and what
// the next forward takes: a bf16 copy, or the experts' 8-bit codes with their channel scales.
//
//   m = b1 m + (1 - b1) g        v = b2 v + (1 - b2) g g
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every product, sum, root and quotient is rounded by itself to f32 (no contraction), and how a root
// or quotient is found depends on that value alone, so that a step has one result, however the
// tensors lie and are cut into units. Moments in 8 bits: e4m3
// codes of m and of sqrt(v), with an f32 scale for 128 values, rounded up or down by chance in
// proportion to what is lost: rounded to nearest, a moment whose change in a step is below half
// a code's spacing (6 %; b2 = 0.999 changes v by 0.1 %) would never move.
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fp8moe_status.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "ptx.cuh"
#include "quantize.cuh"
#include "vec16.cuh"

namespace fp8moe {
namespace {

constexpr int kWarps = 8;                        // that work; one more fetches
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStage = 2048;                     // values of a stage: 16 blocks of 128
constexpr int kBlocks = kStage / 128;
constexpr int kUnitStages = 4;                   // of a linear unit, where there are many
constexpr int kTileRows = 64, kTileCols = 128;   // a unit of weights with codes
constexpr int kSlabTiles = 304;                  // tiles of a slab, at least
constexpr uint32_t kLag = 4;                     // slabs between a tile and its codes
constexpr uint32_t kAll = 0xffffffffu;

// A stage in shared memory: the blocks of each array as they lie in memory (with up to 15 bytes
// in front, where that is not on a boundary of 16), then 8-bit moments' scales. 100 KB or 63 KB
// for a CTA's ring, so that an SM has about 200 KB on their way.
constexpr int kRoomWide = kStage * 4 + 128, kRoomCodes = kStage + 128;
template <int BITS, int STAGES> struct Layout {
  static constexpr int kStages = STAGES;
  static constexpr int kG = kRoomWide, kM = 2 * kRoomWide;
  static constexpr int kV = kM + (BITS == 32 ? kRoomWide : kRoomCodes);
  static constexpr int kScales = kV + (BITS == 32 ? kRoomWide : kRoomCodes);
  static constexpr int kBytes = kScales + (BITS == 32 ? 0 : 2 * kBlocks * 4);
  static constexpr int kAll = kStages * kBytes;
  static_assert(kBytes % 128 == 0, "every stage begins on a boundary that copies may have");
};

// 32 bits for the value at `i` of a tensor, from a key of the seed, the step and the tensor:
// products with the odd numbers next to 2^32 times the fractions of the golden ratio and of the
// roots of 5, 3 and 2, and shifts between them. (Means, correlations between neighbours, steps
// and halves within the noise of 2^20 draws.) random_place() is the part that is linear in i.
constexpr uint32_t kPlace = 0x9E3779B9u;
__device__ __forceinline__ uint32_t random_place(uint64_t i, uint32_t key) {
  return (uint32_t)i * kPlace + (uint32_t)(i >> 32) * 0x3C6EF373u + key;
}
__device__ __forceinline__ uint32_t random_bits(uint32_t x) {
  x = (x ^ (x >> 16)) * 0xBB67AE85u;
  x = (x ^ (x >> 15)) * 0x6A09E667u;
  return x ^ (x >> 16);
}

// Four values of a lane: following each other (wide), or 32 apart.
struct Quad {
  float p[4], g[4], m[4], v[4];
  uint32_t mc, vc;               // 8-bit moments: codes
  float ms, vs;                  // and their scales
};

struct Rates {
  float keep, rate, root, b1, c1, b2, c2, eps, grad, minus_zero;
  float low, raised;             // kLeastMoment or more, -rate / kRaise
  uint32_t key;
  double lr;
};

// CTAs on an SM, and the stages of each: 200 KB of 32-bit moments' stages, 190 KB of 8-bit ones' in
// 3 CTAs for tensors in order (addresses of any kind: 210 us against 225 in 2 CTAs, boundaries of
// 16 bytes: 178 against 175), 169 KB in 2 for tiles, whose CTAs are one warp larger and spill
// registers as three (1238 against 1278 us).
template <int BITS> using LinearLayout = Layout<BITS, 3>;
template <int BITS> using SlabLayout = Layout<BITS, BITS == 32 ? 3 : 4>;
template <int BITS> constexpr int kLinearPer = BITS == 32 ? 2 : 3;
constexpr int kSlabPer = 2;

// What a stage holds.
enum Kind : uint32_t {
  kEnd,      // nothing: the last one
  kWide,     // values that lie on boundaries of 16 bytes in every array
  kNarrow,   // values that do not
  kDirect,   // nothing: read from memory value by value (a tensor's ends)
  kTile,     // 16 rows of a tile
  kCodes     // the new weights of 32 rows of a tile
};
struct Desc {
  int64_t base;              // the first value's place in the tensor
  Kind kind;
  uint32_t entry;            // the tensor
  uint32_t left;             // kDirect: values; kTile, kCodes: rows
  uint32_t strip, tile_k;    // kTile, kCodes
  uint32_t expert, col;      // of the strip
  uint32_t edge;             // 1: a tile's first stage, 2: its last
};

struct Ring {
  uint64_t *full, *empty;
  Desc* desc;
  uint8_t* data;
};

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// What is read once goes first when the L2 needs room: the weights of the last slabs stay.
__device__ __forceinline__ uint64_t read_once() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const void* tmap, uint64_t* bar, int32_t x,
                                                 int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;"
      ::"r"(smem_u32(dst)), "l"(tmap), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// The fetching warp: stages in the order in which it is told, each when its place is free.
template <int BITS, typename L>
struct Fetcher {
  Ring ring;
  uint32_t count = 0;

  // room() is waited for; then lane 0 names the bytes that will come, and every lane ends its part,
  // which may be a small copy of its own
  __device__ __forceinline__ bool room() {
    const uint32_t round = count / L::kStages;
    return round == 0 ||
           mbar_wait_warp(&ring.empty[count % L::kStages], (round - 1) & 1, kWhereProducer);
  }
  __device__ __forceinline__ uint32_t at() const { return count % L::kStages; }
  __device__ __forceinline__ uint8_t* data() const { return ring.data + at() * L::kBytes; }
  __device__ __forceinline__ uint64_t* full() const { return &ring.full[at()]; }
  __device__ __forceinline__ void begin(const Desc& d, uint32_t bytes) {
    ring.desc[at()] = d;
    if (bytes) mbar_arrive_expect_tx(full(), bytes);
    else mbar_arrive(full());
  }
  __device__ __forceinline__ void end() {
    mbar_arrive(full());
    ++count;
  }
  __device__ __forceinline__ void end_scale(const float* scale) {
    cp_async4(data() + L::kScales + (threadIdx.x & 31) * 4, scale);
    cp_async_mbar_arrive(full());
    ++count;
  }
  __device__ __forceinline__ bool empty_stage(const Desc& d) {
    if (!room()) return false;
    if ((threadIdx.x & 31) == 0) begin(d, 0);
    end();
    return true;
  }
  // kWide or kNarrow: kStage values from d.base on, whole blocks, all inside of the tensor
  // together with what the copies' boundaries take in around them
  __device__ __forceinline__ bool values(const AdamwEntry& e, const Desc& d) {
    if (!room()) return false;
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
      const uint8_t* src[4] = {reinterpret_cast<const uint8_t*>(e.p + d.base),
                               static_cast<const uint8_t*>(e.g) + d.base * (e.g_bf16 ? 2 : 4),
                               static_cast<const uint8_t*>(e.m) + d.base * (BITS / 8),
                               static_cast<const uint8_t*>(e.v) + d.base * (BITS / 8)};
      const uint32_t size[4] = {kStage * 4, kStage * (e.g_bf16 ? 2u : 4u), kStage * (BITS / 8),
                                kStage * (BITS / 8)};
      const uint32_t to[4] = {0, L::kG, L::kM, L::kV};
      uint32_t shift[4], bytes[4], all = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        shift[i] = (uint32_t)(reinterpret_cast<uintptr_t>(src[i]) & 15u);
        bytes[i] = (shift[i] + size[i] + 15u) & ~15u;
        all += bytes[i];
      }
      begin(d, all);
#pragma unroll
      for (int i = 0; i < 4; ++i) bulk_load(data() + to[i], src[i] - shift[i], bytes[i], full());
    }
    __syncwarp();
    if constexpr (BITS == 8)
      end_scale((lane < kBlocks ? e.m_scale : e.v_scale) + (d.base >> 7) + lane % kBlocks);
    else
      end();
    return true;
  }
  // what was on its way when a wait ran out is waited for, so that no copy outlives the CTA
  __device__ __forceinline__ void drain() {
    for (uint32_t i = 0; i < L::kStages && i < count; ++i) {
      const uint32_t c = count - 1 - i;
      mbar_wait_warp(&ring.full[c % L::kStages], (c / L::kStages) & 1, kWhereDrain);
    }
  }
};

template <int STAGES>
__device__ __forceinline__ void ring_init(const Ring& r) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&r.full[i], 33);
      mbar_init(&r.empty[i], kWarps);
    }
    fence_mbar_init();
  }
}

// Four values that follow each other, or are 32 apart, of a block in shared memory.
template <bool WIDE>
__device__ __forceinline__ void lds_f32(const uint8_t* s, float (&x)[4]) {
  const int lane = threadIdx.x & 31;
  if constexpr (WIDE) {
    const float4 v = reinterpret_cast<const float4*>(s)[lane];
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = reinterpret_cast<const float*>(s)[j * 32 + lane];
  }
}
template <bool WIDE>
__device__ __forceinline__ void lds_bf16(const uint8_t* s, float (&x)[4]) {
  const int lane = threadIdx.x & 31;
  if constexpr (WIDE) {
    const uint2 w = reinterpret_cast<const uint2*>(s)[lane];
    x[0] = bf16lo_to_f32(w.x), x[1] = bf16hi_to_f32(w.x);
    x[2] = bf16lo_to_f32(w.y), x[3] = bf16hi_to_f32(w.y);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[j] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(s)[j * 32 + lane]);
  }
}
template <bool WIDE>
__device__ __forceinline__ uint32_t lds_codes(const uint8_t* s) {
  const int lane = threadIdx.x & 31;
  if constexpr (WIDE) return reinterpret_cast<const uint32_t*>(s)[lane];
  uint32_t c = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) c |= (uint32_t)s[j * 32 + lane] << (8 * j);
  return c;
}

// shift: bytes in front of the first value, of p, g, m and v.
template <int BITS, bool WIDE>
__device__ __forceinline__ void take_quad(const uint8_t* stage, int block, bool g_bf16,
                                          const uint32_t (&shift)[4], Quad& q) {
  using L = Layout<BITS, 1>;
  lds_f32<WIDE>(stage + block * 512 + shift[0], q.p);
  if (g_bf16) lds_bf16<WIDE>(stage + L::kG + block * 256 + shift[1], q.g);
  else lds_f32<WIDE>(stage + L::kG + block * 512 + shift[1], q.g);
  if constexpr (BITS == 32) {
    lds_f32<WIDE>(stage + L::kM + block * 512 + shift[2], q.m);
    lds_f32<WIDE>(stage + L::kV + block * 512 + shift[3], q.v);
  } else {
    q.mc = lds_codes<WIDE>(stage + L::kM + block * 128 + shift[2]);
    q.vc = lds_codes<WIDE>(stage + L::kV + block * 128 + shift[3]);
    const float* scales = reinterpret_cast<const float*>(stage + L::kScales);
    q.ms = scales[block], q.vs = scales[kBlocks + block];
  }
}

// The same straight from memory, value by value: those of a block at `i` of the tensor that exist.
template <int BITS>
__device__ __forceinline__ void load_quad(const AdamwEntry& d, int64_t i, uint32_t left, Quad& q) {
  const uint32_t lane = threadIdx.x & 31;
  if constexpr (BITS == 8) {
    q.mc = q.vc = 0;
    q.ms = d.m_scale[i >> 7], q.vs = d.v_scale[i >> 7];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool in = j * 32 + lane < left;
    const int64_t at = i + j * 32 + lane;
    q.p[j] = in ? d.p[at] : 0.0f;
    if (d.g_bf16)
      q.g[j] = in ? __bfloat162float(static_cast<const __nv_bfloat16*>(d.g)[at]) : 0.0f;
    else
      q.g[j] = in ? static_cast<const float*>(d.g)[at] : 0.0f;
    if constexpr (BITS == 32) {
      q.m[j] = in ? static_cast<const float*>(d.m)[at] : 0.0f;
      q.v[j] = in ? static_cast<const float*>(d.v)[at] : 0.0f;
    } else if (in) {
      q.mc |= (uint32_t)static_cast<const uint8_t*>(d.m)[at] << (8 * j);
      q.vc |= (uint32_t)static_cast<const uint8_t*>(d.v)[at] << (8 * j);
    }
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

// |x| as an e4m3 code by chance, in the top byte: |x| / scale * 2^-120 has the code's bits on
// top of its own (both formats' subnormals included; its sign falls out on the left), and the random
// ones, 16 bits and a one behind them for the middle of their step, decide about the 20 below. The
// largest of a block is 448 to within 4 units (its scale, the inverse and two products are
// rounded), where the random bits reach the next code only from 8 units on: 0x7F, a NaN's code, is
// for spoilt blocks alone.
__device__ __forceinline__ uint32_t encode(float y, uint32_t random24) {
  return __float_as_uint(y) * 16u + random24;
}
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// The larger magnitude; a NaN stays.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float largest(const float2 (&x)[2]) {
  return max_abs(max_abs(x[0].x, x[0].y, x[1].x), x[1].y, 0.0f);
}

// A product of its own: what is added to it later can not be joined with it into one rounding, as
// the compiler does with packed products, and with those of a -0 that it knows.
__device__ __forceinline__ float2 prod2(float2 a, float2 b, float minus_zero) {
  return fma2(a, b, both(minus_zero));
}

__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Square root and quotient of two values at once by Newton steps whose last takes the exact
// remainder (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): the nearest f32 but for about one in 2^22, where the exact value lies next to
// the middle of two. x, and a and b with their quotient, well inside the range of normal numbers.
//
// Whether that holds is asked of each value by itself (within()), so that its result does not depend
// on the values beside it: second moments in [2^-100, 2^36], whose roots' remainders are exact;
// first moments up to 2^36, raised by 2^40 for the quotient and lowered again by the rate, so that
// the quotient's remainder is exact for the smallest ones, too (one whose gradient stopped falls
// below 2^-100 long before its second moment; 2 % of the time of 8-bit moments). The divisors are in
// [2^-50, 2^46] then (kMostFactor, kMostEps), the quotients below 2^126.
constexpr float kLeastMoment = 0x1p-100f, kMostMoment = 0x1p36f, kMostRoot = 0x1p18f;
constexpr float kMostEps = 0x1p20f;
// 1 / sqrt(1 - b2^t) for any b2 below 1, unless the power comes out as 1
constexpr float kMostFactor = 0x1p27f;
constexpr float kRaise = 0x1p40f, kLower = 0x1p-40f;
constexpr float kLeastRate = 0x1p-60f;           // a smaller one would not be normal when lowered
__device__ __forceinline__ float2 sqrt2(float2 x) {
  const float2 y = make_float2(rsqrt_approx(x.x), rsqrt_approx(x.y));
  const float2 s = mul2(x, y);
  const float2 rest = fma2(s, s, mul2(x, both(-1.0f)));
  return fma2(rest, mul2(y, both(-0.5f)), s);
}
__device__ __forceinline__ float2 inverse2(float2 b, float2 minus_b) {
  const float2 y = make_float2(rcp_approx(b.x), rcp_approx(b.y));
  return fma2(y, fma2(minus_b, y, both(1.0f)), y);
}
__device__ __forceinline__ float2 div2(float2 a, float2 b) {
  const float2 minus_b = mul2(b, both(-1.0f));
  const float2 y = inverse2(b, minus_b);
  const float2 q = mul2(a, y);
  return fma2(fma2(minus_b, q, a), y, q);
}

// Of one value or of several: the least second moment, the largest root (by sqrt2, whose root of
// an infinity is a NaN, as that of a NaN is), the largest first moment.
__device__ __forceinline__ bool within(float second, float root, float first, float least) {
  return second >= least && root <= kMostRoot && first <= kMostMoment;
}

__device__ __forceinline__ float2 raised_step(const Rates& r, float2 m, float2 root) {
  const float2 d = add2(prod2(root, both(r.root), r.minus_zero), both(r.eps));
  return prod2(div2(mul2(m, both(kRaise)), d), both(r.raised), r.minus_zero);
}
// The values that are not within(): by the rounded operations, unless they are all zeros (an expert
// that got no token: 0 / eps).
__device__ __forceinline__ void far_step(const Rates& r, float v, float m, float& root, float& step) {
  if (within(v, root, fabsf(m), r.low)) return;
  if (v == 0.0f && m == 0.0f && r.eps > 0.0f) {
    root = v;
    step = __fmul_rn(m, -r.rate);
    return;
  }
  root = __fsqrt_rn(v);
  const float d = __fadd_rn(__fmul_rn(root, r.root), r.eps);
  step = __fmul_rn(__fdiv_rn(m, d), -r.rate);
}

// Steps of COUNT quads, side by side; the few far values are put right behind one branch of all of
// them (a branch for each quad, in front of the quotient: 1230 us for the experts with 8-bit moments,
// 1222 so). place: of the lane's first value of each in the tensor;
// apart: between two of its values.
template <int BITS, int COUNT>
__device__ __forceinline__ void step_quads(const Rates& r, const uint64_t (&place)[COUNT],
                                           uint32_t apart, Quad (&quads)[COUNT]) {
  auto prod = [&](float2 a, float b) { return prod2(a, both(b), r.minus_zero); };
  float2 ms[COUNT][2], vs[COUNT][2], roots[COUNT][2], steps[COUNT][2];
  bool usual = true;
#pragma unroll
  for (int c = 0; c < COUNT; ++c) {
    Quad& q = quads[c];
    float2(&m)[2] = ms[c], (&v)[2] = vs[c], (&root)[2] = roots[c];
    if constexpr (BITS == 8) {
      decode4(q.mc, q.ms, q.m);
      decode4(q.vc, q.vs, q.v);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 g = mul2(make_float2(q.g[2 * h], q.g[2 * h + 1]), both(r.grad));
      m[h] = make_float2(q.m[2 * h], q.m[2 * h + 1]);
      v[h] = make_float2(q.v[2 * h], q.v[2 * h + 1]);
      if constexpr (BITS == 8) v[h] = mul2(v[h], v[h]);
      m[h] = add2(prod(m[h], r.b1), prod(g, r.c1));
      v[h] = add2(prod(v[h], r.b2), prod2(mul2(g, both(r.c2)), g, r.minus_zero));
      root[h] = sqrt2(v[h]);
      steps[c][h] = raised_step(r, m[h], root[h]);
    }
    usual &= within(fminf(fminf(v[0].x, v[0].y), fminf(v[1].x, v[1].y)), largest(root), largest(m),
                    r.low);
  }
  if (!usual) {
#pragma unroll
    for (int c = 0; c < COUNT; ++c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        far_step(r, vs[c][h].x, ms[c][h].x, roots[c][h].x, steps[c][h].x);
        far_step(r, vs[c][h].y, ms[c][h].y, roots[c][h].y, steps[c][h].y);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < COUNT; ++c) {
    Quad& q = quads[c];
    float2(&m)[2] = ms[c], (&v)[2] = vs[c], (&root)[2] = roots[c];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 p = add2(prod(make_float2(q.p[2 * h], q.p[2 * h + 1]), r.keep), steps[c][h]);
      q.p[2 * h] = p.x, q.p[2 * h + 1] = p.y;
      q.m[2 * h] = m[h].x, q.m[2 * h + 1] = m[h].y;
      q.v[2 * h] = v[h].x, q.v[2 * h + 1] = v[h].y;
    }
    if constexpr (BITS == 8) {
      // (values that do not exist are zeros, and so are their moments)
      q.ms = block_scale(__reduce_max_sync(kAll, __float_as_uint(largest(m))));
      q.vs = block_scale(__reduce_max_sync(kAll, __float_as_uint(largest(root))));
      const float2 scale = make_float2(q.ms, q.vs);
      float2 inverse = inverse2(scale, mul2(scale, both(-1.0f)));
      inverse.x = q.ms != 0.0f ? inverse.x : 0.0f;
      inverse.y = q.vs != 0.0f ? inverse.y : 0.0f;
      const uint32_t least = q.vs != 0.0f ? 0x01000000u : 0u;
      // a block lies on one side of 2^32, as its first place is a multiple of 128
      const uint32_t base = random_place(place[c], r.key);
      uint32_t mc[4], vc[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 my = mul2(mul2(m[h], both(inverse.x)), both(0x1p-120f));
        const float2 vy = mul2(mul2(root[h], both(inverse.y)), both(0x1p-120f));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = 2 * h + i;
          const uint32_t bits = random_bits(base + j * apart * kPlace);
          mc[j] = (__float_as_uint(q.m[j]) & 0x80000000u) |
                  (encode(i ? my.y : my.x, __byte_perm(bits, 0x80u, 0x7104)) & 0x7fffffffu);
          // a second moment that is not zero (its root then is at least 2^-75) never becomes zero:
          // m / eps would follow
          vc[j] = max(encode(i ? vy.y : vy.x, __byte_perm(bits, 0x80u, 0x7324)),
                      min(__float_as_uint(i ? root[h].y : root[h].x), least));
        }
      }
      q.mc = top_bytes(mc[0], mc[1], mc[2], mc[3]);
      q.vc = top_bytes(vc[0], vc[1], vc[2], vc[3]);
    }
  }
}

// i: of the block's first value in the tensor. WIDE: the lane's four follow each other.
template <int BITS, bool WIDE>
__device__ __forceinline__ void store_quad(const AdamwEntry& d, int64_t i, uint32_t left,
                                           const Quad& q) {
  const uint32_t lane = threadIdx.x & 31;
  float* p = d.p + i;
  uint8_t* m = static_cast<uint8_t*>(d.m) + i * (BITS / 8);
  uint8_t* v = static_cast<uint8_t*>(d.v) + i * (BITS / 8);
  __nv_bfloat16* copy = d.copy ? static_cast<__nv_bfloat16*>(d.copy) + i : nullptr;
  if constexpr (WIDE) {
    // p stays in the L2, where its codes are made from it
    reinterpret_cast<float4*>(p)[lane] = make_float4(q.p[0], q.p[1], q.p[2], q.p[3]);
    if constexpr (BITS == 32) {
      __stcs(reinterpret_cast<float4*>(m) + lane, make_float4(q.m[0], q.m[1], q.m[2], q.m[3]));
      __stcs(reinterpret_cast<float4*>(v) + lane, make_float4(q.v[0], q.v[1], q.v[2], q.v[3]));
    } else {
      __stcs(reinterpret_cast<uint32_t*>(m) + lane, q.mc);
      __stcs(reinterpret_cast<uint32_t*>(v) + lane, q.vc);
    }
    if (copy)
      __stcs(reinterpret_cast<uint2*>(copy) + lane,
             make_uint2(f32x2_to_bf16x2(q.p[0], q.p[1]), f32x2_to_bf16x2(q.p[2], q.p[3])));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t k = j * 32 + lane;
      if (k >= left) continue;
      p[k] = q.p[j];
      if constexpr (BITS == 32) {
        reinterpret_cast<float*>(m)[k] = q.m[j];
        reinterpret_cast<float*>(v)[k] = q.v[j];
      } else {
        m[k] = (uint8_t)(q.mc >> (8 * j));
        v[k] = (uint8_t)(q.vc >> (8 * j));
      }
      if (copy) copy[k] = __float2bfloat16_rn(q.p[j]);
    }
  }
  if constexpr (BITS == 8) {
    if (lane == 0) {
      d.m_scale[i >> 7] = q.ms;
      d.v_scale[i >> 7] = q.vs;
    }
  }
}

// A working warp's blocks of a stage of a linear unit. 60 million values with a bf16 copy: f32
// gradients and 8-bit moments in one tensor 175 us (0.92 of the copy rate), in 300 tensors at odd
// addresses 208 (0.77: byte and word accesses, 68 % of the issue slots); bf16 gradients and 32-bit
// moments in 300 tensors 271 (0.92). With loads straight into registers these took 465, 465 and 372.
template <int BITS>
__device__ __forceinline__ void linear_stage(const AdamwEntry& d, const Rates& r, const Desc& a,
                                             const uint8_t* stage) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t shift[4] = {0, 0, 0, 0};
  if (a.kind == kNarrow) {
    auto low = [](const void* p, int64_t bytes) {
      return (uint32_t)((reinterpret_cast<uintptr_t>(p) + (uint64_t)bytes) & 15u);
    };
    shift[0] = low(d.p, a.base * 4), shift[1] = low(d.g, a.base * (d.g_bf16 ? 2 : 4));
    shift[2] = low(d.m, a.base * (BITS / 8)), shift[3] = low(d.v, a.base * (BITS / 8));
  }
  auto whole = [&](auto is_wide) {
    constexpr bool kIsWide = decltype(is_wide)::value;
#pragma unroll
    for (uint32_t n = 0; n < kBlocks / kWarps; ++n) {
      const uint32_t block = n * kWarps + warp;
      const int64_t i = a.base + block * 128;
      Quad q[1];
      take_quad<BITS, kIsWide>(stage, block, d.g_bf16, shift, q[0]);
      step_quads<BITS, 1>(r, {(uint64_t)i + (kIsWide ? lane * 4 : lane)}, kIsWide ? 1 : 32, q);
      store_quad<BITS, kIsWide>(d, i, 128, q[0]);
    }
  };
  if (a.kind == kWide) return whole(std::true_type());
  if (a.kind == kNarrow) return whole(std::false_type());
#pragma unroll 1
  for (uint32_t block = warp; block * 128 < a.left; block += kWarps) {
    const int64_t i = a.base + block * 128;
    Quad q[1];
    load_quad<BITS>(d, i, a.left - block * 128, q[0]);
    step_quads<BITS, 1>(r, {(uint64_t)i + lane}, 32, q);
    store_quad<BITS, false>(d, i, a.left - block * 128, q[0]);
  }
}

// What a call's tensors share, and what is a tensor's own.
__device__ __forceinline__ Rates rates_of(const AdamwCommon& c) {
  Rates r;
  r.minus_zero = c.minus_zero;
  r.b1 = c.b1, r.c1 = c.c1, r.b2 = c.b2, r.c2 = c.c2, r.eps = c.eps;
  r.grad = c.grad_scale != nullptr ? *c.grad_scale : 1.0f;
  r.rate = c.rate, r.root = c.root, r.key = c.key, r.lr = 0.0;
  if (c.rates != nullptr) {                      // step or rate on the device
    r.rate = c.rates->rate, r.root = c.rates->root, r.key = c.rates->key, r.lr = c.rates->lr;
  }
  r.keep = 1.0f;
  const bool usual = r.eps <= kMostEps && r.root <= kMostFactor &&
                     (r.rate == 0.0f || fabsf(r.rate) >= kLeastRate);
  r.low = usual ? kLeastMoment : INFINITY;
  r.raised = -r.rate * kLower;
  return r;
}
__device__ __forceinline__ Rates rates_for(const Rates& all, const AdamwCommon& c,
                                           const AdamwEntry& d) {
  Rates r = all;
  r.keep = c.rates != nullptr ? (float)(1.0 - all.lr * d.weight_decay) : d.keep;
  r.key += 0xBB67AE85u * d.which;
  return r;
}

template <int kCapacity>
struct AdamwTable {
  AdamwCommon c;
  AdamwEntry at[kCapacity];
};

template <int BITS, int kCapacity>
__global__ void __launch_bounds__(kThreads, kLinearPer<BITS>) adamw_kernel(
    const __grid_constant__ AdamwTable<kCapacity> table) {
  using L = LinearLayout<BITS>;
  extern __shared__ __align__(128) uint8_t s_data[];
  __shared__ uint64_t s_full[L::kStages], s_empty[L::kStages];
  __shared__ Desc s_desc[L::kStages];
  const Ring ring = {s_full, s_empty, s_desc, s_data};
  ring_init<L::kStages>(ring);
  __syncthreads();
  const AdamwCommon& c = table.c;

  if (threadIdx.x >= 32 * kWarps) {
    Fetcher<BITS, L> f = {ring};
    bool going = true;
    uint32_t entry = 0;
    for (uint32_t unit = blockIdx.x; going && unit < c.units; unit += gridDim.x) {
      while ((int)entry + 1 < c.count && table.at[entry + 1].first_unit <= unit) ++entry;
      const AdamwEntry& d = table.at[entry];
      Desc a = {};
      a.entry = entry;
      const uint32_t number = unit - d.first_unit;
      if (number == 0 && d.head > 0) {             // in front of the first boundary
        a.kind = kDirect, a.base = 0;
        a.left = (uint32_t)min(d.n, (int64_t)d.head);
        going = f.empty_stage(a);
      }
      a.base = d.head + (int64_t)number * c.unit_stages * kStage;
      for (int i = 0; going && i < c.unit_stages && a.base < d.n; ++i, a.base += kStage) {
        const int64_t behind = d.n - a.base - kStage;
        a.left = (uint32_t)min((int64_t)kStage, d.n - a.base);
        a.kind = d.vec && behind >= 0 ? kWide
                 : !d.vec && behind >= 16 && a.base >= 16 ? kNarrow : kDirect;
        going = a.kind == kDirect ? f.empty_stage(a) : f.values(d, a);
      }
    }
    if (going) going = f.empty_stage(Desc{});      // kEnd
    if (!going) f.drain();
    return;
  }
  if (c.prepared) pdl_wait();                    // the fetching warp needs nothing of it
  const Rates all = rates_of(c);
  for (uint32_t n = 0;; ++n) {
    const uint32_t at = n % L::kStages;
    if (!mbar_wait_warp(&s_full[at], (n / L::kStages) & 1, kWhereEpilogue)) return;
    const Desc a = s_desc[at];
    if (a.kind == kEnd) return;
    const AdamwEntry& d = table.at[a.entry];
    linear_stage<BITS>(d, rates_for(all, c, d), a, s_data + at * L::kBytes);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&s_empty[at]);
  }
}

// What a step or rate on the device makes of the constants, in 64 bits as the host does; and
// zeros for the columns' largest magnitudes.
__global__ void adamw_prepare_kernel(AdamwRates* rates, const int64_t* step, int64_t host_step,
                                     const float* lr, double host_lr, double beta1, double beta2,
                                     uint32_t seed, uint32_t* most, int64_t count) {
  pdl_launch_dependents();
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

// The columns' largest magnitudes of weights [E, K, N], where the step's units are not tiles: 8-bit
// moments whose blocks cross rows (N no multiple of 128), or arrays off 16 bytes. This kernel and the
// next but one read the weights again, value by value: 16 x 2880 x 2880 weights with 8-bit moments
// 586 us (0.57 of the copy rate for the bytes that have to move), 16 x 2880 x 2944 by tiles 477
// (0.72); off 16 bytes 633 and 644, with 32-bit moments 787 for 601.
__global__ void __launch_bounds__(32 * kWarps) column_max_kernel(const float* p, int K, int N,
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
  for (int c = threadIdx.x; c < kTileCols && col + c < N; c += 32 * kWarps) {
    uint32_t v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = max(v, s_most[w * kTileCols + c]);
    atomicMax(most + (int64_t)blockIdx.z * N + col + c, v);
  }
}

// codes = e4m3(p / scale), scale = max(column's largest, 1e-12) / 448, both as the library's
// other quantisers have them (quantize.cuh). For four columns of a lane.
struct Columns {
  float s[4];
  float2 rl[2], rh[2];
};
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ void columns_of(const float (&top)[4], Columns& x) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x.s[j] = __fdiv_rn(top[j] < kEps ? kEps : top[j], kE4m3Max);   // a NaN stays
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    bracket(x.s[2 * h], x.rl[h].x, x.rh[h].x);
    bracket(x.s[2 * h + 1], x.rl[h].y, x.rh[h].y);
  }
}
__device__ __forceinline__ uint32_t codes_of(const float (&v)[4], const Columns& x) {
  // the ends of the bracket around each quotient, all four compared at once (quantize.cuh)
  const float2 v0 = make_float2(v[0], v[1]), v1 = make_float2(v[2], v[3]);
  uint32_t lo = e4m3x4(mul2(v0, x.rl[0]), mul2(v1, x.rl[1]));
  const uint32_t hi = e4m3x4(mul2(v0, x.rh[0]), mul2(v1, x.rh[1]));
  if (lo != hi)
    lo = e4m3x4(make_float2(__fdiv_rn(v0.x, x.s[0]), __fdiv_rn(v0.y, x.s[1])),
                make_float2(__fdiv_rn(v1.x, x.s[2]), __fdiv_rn(v1.y, x.s[3])));
  return lo;
}

// For weights that the step went through in order.
__global__ void __launch_bounds__(32 * kWarps) weight_codes_kernel(const float* p, int K, int N,
                                                                   const uint32_t* most,
                                                                   uint8_t* codes, float* scale) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * kTileCols, k0 = blockIdx.y * kTileRows;
  const int64_t e = blockIdx.z;
  float top[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = col + j * 32 + lane;
    top[j] = c < N ? __uint_as_float(most[e * N + c]) : 0.0f;
  }
  Columns x;
  columns_of(top, x);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (k0 == 0 && warp == 0 && col + j * 32 + lane < N) scale[e * N + col + j * 32 + lane] = x.s[j];
  const int64_t base = (e * K + k0) * N + col;
  for (int row = warp; row < kTileRows && k0 + row < K; row += kWarps) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = col + j * 32 + lane < N ? p[base + (int64_t)row * N + j * 32 + lane] : 0.0f;
    const uint32_t w = codes_of(v, x);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j * 32 + lane < N)
        codes[base + (int64_t)row * N + j * 32 + lane] = (uint8_t)(w >> (8 * j));
  }
}

// Weights with codes. A strip is 128 columns of an expert, a slab some strips over all their rows.
// Units in order: the tiles of slab j, then the codes of slab j - kLag, whose weights are still in
// the L2 (a slab's are 10 MB; gradients and moments are read and written to go first), so that they
// are read from there and not from memory: a value's 33 bytes of traffic become 29.3. CTAs take
// units in this order from a counter. Codes wait until their slab's tiles are done; those have been
// taken before, by CTAs that wait for nothing or for earlier tiles still, so that the wait ends
// whatever else runs, and as two slabs have as many tiles as CTAs can have taken, it hardly ever
// begins. 8 x 7168 x 4096 and 8 x 2048 x 7168 weights, 32-bit moments: 1607 us (6.36 TB/s of the
// bytes that have to move), bound by memory; two kernels one after the other, 1796; slabs by a
// launch each, 1701. 8-bit moments: 1224 us, bound by instructions (96 a value, 65 % of the issue
// slots); 2153 at first, with the same arithmetic one value at a time.
// Waits until a slab's tiles are done; false (and a status bit) after two seconds.
__device__ __forceinline__ bool wait_slab(const uint32_t* done, uint32_t tiles) {
  const uint64_t began = globaltimer_ns();
  for (;;) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(done) : "memory");
    if (v >= tiles) break;
    if (globaltimer_ns() - began > kWaitLimitNs) {
      status_set(kStatusWaitTimeout | kWhereDrain);
      return false;
    }
    __nanosleep(200);
  }
  // the tiles were written by ordinary stores; the copies that follow read them another way
  asm volatile("fence.proxy.async.global;" ::: "memory");
  return true;
}

// The units in their order: phase j has the tiles of slab j, then the codes of slab j - kLag.
struct Order {
  uint32_t whole, rest, last, strips, rest_strips;   // units of a slab, of the last one; its number
  uint32_t phase = 0, begin = 0;                     // of the unit that was asked for last
  uint32_t slab, strip, tile_k;
  bool tiles;

  __device__ __forceinline__ Order(const AdamwSlabArgs& a, uint32_t tiles_k) {
    last = a.slabs - 1;
    strips = a.per_slab, rest_strips = a.strips - last * a.per_slab;
    whole = strips * tiles_k, rest = rest_strips * tiles_k;
  }
  __device__ __forceinline__ uint32_t units(uint32_t s) const {
    return s < last ? whole : s == last ? rest : 0u;
  }
  __device__ __forceinline__ uint32_t codes(uint32_t p) const {
    return p >= kLag ? units(p - kLag) : 0u;
  }
  // ascending units
  __device__ __forceinline__ void find(uint32_t unit) {
    while (unit - begin >= units(phase) + codes(phase)) begin += units(phase) + codes(phase), ++phase;
    unit -= begin;
    tiles = unit < units(phase);
    slab = tiles ? phase : phase - kLag;
    if (!tiles) unit -= units(phase);
    const uint32_t n = slab == last ? rest_strips : strips;
    strip = slab * strips + unit % n;
    tile_k = unit / n;
  }
};

// The arrays' warps: kWarps that work, one that fetches, one that closes tiles.
constexpr int kSlabThreads = kThreads + 32;
template <int BITS>
__global__ void __launch_bounds__(kSlabThreads, kSlabPer) adamw_slab_kernel(
    const __grid_constant__ AdamwSlabArgs a) {
  using L = SlabLayout<BITS>;
  extern __shared__ __align__(128) uint8_t s_data[];
  __shared__ uint64_t s_full[L::kStages], s_empty[L::kStages], s_tile[2], s_closed[2];
  __shared__ Desc s_desc[L::kStages];
  __shared__ float s_most[2][kWarps * kTileCols];    // of two tiles, in turn
  __shared__ uint32_t s_strip[2];
  constexpr uint32_t kNoStrip = 0xffffffffu;
  const Ring ring = {s_full, s_empty, s_desc, s_data};
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_tile[i], kWarps);
      mbar_init(&s_closed[i], 1);
    }
  }
  ring_init<L::kStages>(ring);
  __syncthreads();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int K = a.d.K, N = a.d.N;
  const uint32_t tiles_k = (K + kTileRows - 1) / kTileRows;
  const uint32_t tiles_n = (N + kTileCols - 1) / kTileCols;
  constexpr int kRows = kStage / kTileCols;      // of a box
  // a stage of codes has two boxes, the second one where the gradients would be, and the columns'
  // largest magnitudes in the place of the first moments
  constexpr int kCodesMost = L::kM;

  if (warp == kWarps) {
    Fetcher<BITS, L> f = {ring};
    bool going = true;
    const uint64_t once = read_once();
    Order u(a, tiles_k);
    uint32_t next = lane == 0 ? atomicAdd(a.counters, 1u) : 0u;
    while (going) {
      const uint32_t unit = __shfl_sync(kAll, next, 0);
      if (unit >= a.units) break;
      if (lane == 0) next = atomicAdd(a.counters, 1u);
      u.find(unit);
      if (!u.tiles) {
        bool ready = true;
        if (lane == 0) ready = wait_slab(a.counters + 1 + u.slab, u.units(u.slab));
        going = __shfl_sync(kAll, (int)ready, 0);
      }
      const int e = u.strip / tiles_n, col = (u.strip % tiles_n) * kTileCols;
      const int rows = min(kTileRows, K - (int)u.tile_k * kTileRows);
      const int each = u.tiles ? kRows : 2 * kRows;
      for (int row = 0; going && row < rows; row += each) {
        Desc d;
        d.kind = u.tiles ? kTile : kCodes;
        d.entry = 0, d.strip = u.strip, d.tile_k = u.tile_k, d.expert = e, d.col = col;
        d.left = min(each, rows - row);
        d.edge = (row == 0 ? 1 : 0) + (row + each >= rows ? 2 : 0);
        const int k = u.tile_k * kTileRows + row;
        d.base = ((int64_t)e * K + k) * N + col;
        going = f.room();
        if (!going) break;
        if (u.tiles) {
          if (lane == 0) {
            f.begin(d, kStage * (4 + (a.d.g_bf16 ? 2 : 4) + 2 * BITS / 8));
            tma_load_3d_hint(f.data(), &a.tm_p, f.full(), col, k, e, once);
            tma_load_3d_hint(f.data() + L::kG, &a.tm_g, f.full(), col, k, e, once);
            tma_load_3d_hint(f.data() + L::kM, &a.tm_m, f.full(), col, k, e, once);
            tma_load_3d_hint(f.data() + L::kV, &a.tm_v, f.full(), col, k, e, once);
          }
          __syncwarp();
          if constexpr (BITS == 8) {
            const int r = lane % kBlocks < (int)d.left ? lane % kBlocks : 0;
            f.end_scale((lane < kBlocks ? a.d.m_scale : a.d.v_scale) + (d.base >> 7) +
                        (int64_t)r * (N >> 7));
          } else {
            f.end();
          }
        } else {
          if (lane == 0) {
            f.begin(d, 2 * kStage * 4);
            tma_load_3d_hint(f.data(), &a.tm_p, f.full(), col, k, e, once);
            tma_load_3d_hint(f.data() + L::kG, &a.tm_p, f.full(), col, k + kRows, e, once);
          }
          __syncwarp();
          // 16 bytes of four columns, past the L1; N is a multiple of 16
          const uint32_t here = (d.edge & 1) && col + lane * 4 < N ? 16 : 0;
          cp_async16(f.data() + kCodesMost + lane * 16,
                     a.d.most + (int64_t)e * N + col + (here ? lane * 4 : 0), here);
          cp_async_mbar_arrive(f.full());
          ++f.count;
        }
      }
    }
    if (going) going = f.empty_stage(Desc{});      // kEnd
    if (!going) f.drain();
    return;
  }

  if (warp == kWarps + 1) {
    // closes tiles: their columns' largest magnitudes, then, when all of a tile's stores can be
    // seen, its slab's count (the working warps go on meanwhile)
    for (uint32_t n = 0;; ++n) {
      if (!mbar_wait_warp(&s_tile[n & 1], (n >> 1) & 1, kWhereDrain)) return;
      const uint32_t strip = s_strip[n & 1];
      if (strip == kNoStrip) return;
      const int64_t e = strip / tiles_n;
      const int col = (strip % tiles_n) * kTileCols;
#pragma unroll
      for (int j = 0; j < kTileCols / 32; ++j) {
        const int c = j * 32 + lane;
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; w += 2)
          m = max_abs(m, s_most[n & 1][w * kTileCols + c], s_most[n & 1][(w + 1) * kTileCols + c]);
        if (col + c < N) atomicMax(a.d.most + e * N + col + c, __float_as_uint(m));
      }
      __threadfence();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s_closed[n & 1]);
        atomicAdd(a.counters + 1 + strip / a.per_slab, 1u);
      }
    }
  }

  const Rates rates = rates_for(rates_of(a.c), a.c, a.d);
  float most[4];
  Columns x;
  uint32_t tiles = 0;                                // closed by this warp
  for (uint32_t n = 0;; ++n) {
    const uint32_t at = n % L::kStages;
    if (!mbar_wait_warp(&s_full[at], (n / L::kStages) & 1, kWhereEpilogue)) return;
    const Desc& d = s_desc[at];
    const Kind kind = d.kind;
    const uint32_t strip = kind == kEnd ? kNoStrip : d.strip, edge = d.edge, rows = d.left;
    if (kind == kTile || kind == kCodes) {
      const int col = d.col;
      const int64_t base = d.base;
      const bool in = col + lane * 4 < N;            // N is a multiple of 16
      const uint8_t* stage = s_data + at * L::kBytes;
      const uint32_t none[4] = {0, 0, 0, 0};
      if (kind == kTile) {
        if (edge & 1) most[0] = most[1] = most[2] = most[3] = 0.0f;
        constexpr int kEach = kRows / kWarps;      // rows past the last: zeros, worked on for nothing
        Quad q[kEach];
        uint64_t place[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          take_quad<BITS, true>(stage, i * kWarps + warp, a.d.g_bf16, none, q[i]);
          place[i] = base + (int64_t)(i * kWarps + warp) * N + lane * 4;
        }
        step_quads<BITS, kEach>(rates, place, 1, q);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const uint32_t row = i * kWarps + warp;
          if (in && row < rows) {
            store_quad<BITS, true>(a.d, base + (int64_t)row * N, 128, q[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) most[j] = max_abs(most[j], q[i].p[j], 0.0f);
          }
        }
      } else {
        if (edge & 1) {
          float top[4];
          lds_f32<true>(stage + kCodesMost, top);
          columns_of(top, x);
          if (d.tile_k == 0 && warp == 0 && in) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              a.scale[(int64_t)d.expert * N + col + lane * 4 + j] = x.s[j];
          }
        }
        uint8_t* codes = a.codes + base + lane * 4;
#pragma unroll
        for (uint32_t i = 0; i < 2 * kRows / kWarps; ++i) {
          const uint32_t row = i * kWarps + warp;
          float v[4];
          lds_f32<true>(stage + (i < kRows / kWarps ? row * 512 : L::kG + (row - kRows) * 512), v);
          const uint32_t w = codes_of(v, x);
          if (row < rows && in) __stcs(reinterpret_cast<uint32_t*>(codes + (int64_t)row * N), w);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[at]);
    }
    if (kind != kEnd && !(kind == kTile && (edge & 2))) continue;
    // a tile's last rows, or the end: to the warp that closes tiles, when it is done with the last
    // but one
    const uint32_t b = tiles & 1;
    if (tiles >= 2 && !mbar_wait_warp(&s_closed[b], ((tiles >> 1) - 1) & 1, kWhereEpilogue)) return;
    if (kind == kTile) {
#pragma unroll
      for (int j = 0; j < 4; ++j) s_most[b][warp * kTileCols + lane * 4 + j] = most[j];
    }
    if (threadIdx.x == 0) s_strip[b] = strip;
    __syncwarp();
    if (lane == 0) mbar_arrive(&s_tile[b]);
    ++tiles;
    if (kind == kEnd) return;
  }
}

// The same limit for every call of a kernel.
template <typename F>
cudaError_t allow_ring(F kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// behind: may start before the kernel in front of it (adamw_prepare_kernel) has ended.
template <typename A>
cudaError_t launch_behind(void (*kernel)(A), uint32_t grid, int threads, int bytes, bool behind,
                          const A& args, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  pdl_attribute(attr[0]);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)bytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

template <int BITS, int kCapacity>
cudaError_t launch_table(const AdamwCommon& c, const AdamwEntry* at, int num_sms, cudaStream_t s) {
  static thread_local AdamwTable<kCapacity> t;   // up to 32 KB: not on the stack
  t.c = c;
  for (int i = 0; i < c.count; ++i) t.at[i] = at[i];
  auto* kernel = adamw_kernel<BITS, kCapacity>;
  const cudaError_t e = allow_ring(kernel, LinearLayout<BITS>::kAll);
  if (e != cudaSuccess) return e;
  const uint32_t most = (uint32_t)(num_sms * kLinearPer<BITS>);
  return launch_behind(kernel, c.units < most ? c.units : most, kThreads, LinearLayout<BITS>::kAll,
                       c.prepared != 0, t, s);
}

uint32_t strips_of(int64_t n, int64_t K, int64_t N) {
  return (uint32_t)(n / (K * N) * ((N + kTileCols - 1) / kTileCols));
}
uint32_t strips_per_slab(int64_t K) {
  const int64_t tiles_k = (K + kTileRows - 1) / kTileRows;
  return (uint32_t)((kSlabTiles + tiles_k - 1) / tiles_k);
}

}  // namespace
}  // namespace fp8moe

using namespace fp8moe;

FP8MOE_DEFINE_STATUS_TAKE(fp8moe_status_take_adamw)

static uint64_t units_of(const AdamwEntry& d, int64_t values) {
  return d.n <= d.head ? 1 : (uint64_t)((d.n - d.head + values - 1) / values);
}
uint64_t fp8moe_adamw_units(const AdamwEntry& d) { return units_of(d, kUnitStages * kStage); }

cudaError_t fp8moe_launch_adamw(const AdamwCommon& common, AdamwEntry* at, int count, int bits,
                                int num_sms, cudaStream_t s) {
  AdamwCommon c = common;
  // units of four stages; of one, where that leaves CTAs without work
  uint64_t units = 0;
  for (int i = 0; i < count; ++i) units += fp8moe_adamw_units(at[i]);
  c.unit_stages = units < (uint64_t)num_sms ? 1 : kUnitStages;
  units = 0;
  for (int i = 0; i < count; ++i) {
    at[i].first_unit = (uint32_t)units;
    units += units_of(at[i], (int64_t)c.unit_stages * kStage);
  }
  c.count = count, c.units = (uint32_t)units;
  // a table of 16 entries is a launch's usual few KB of parameters, the other nearly all of them
  if (count <= 16)
    return bits == 8 ? launch_table<8, 16>(c, at, num_sms, s) : launch_table<32, 16>(c, at, num_sms, s);
  return bits == 8 ? launch_table<8, kAdamwEntries>(c, at, num_sms, s)
                   : launch_table<32, kAdamwEntries>(c, at, num_sms, s);
}

uint32_t fp8moe_adamw_slab_counters(int64_t n, int64_t K, int64_t N) {
  return 1 + (strips_of(n, K, N) + strips_per_slab(K) - 1) / strips_per_slab(K);
}
void fp8moe_adamw_tile(int* cols, int* rows) {
  *cols = kTileCols;
  *rows = kStage / kTileCols;
}

cudaError_t fp8moe_launch_adamw_slabs(const AdamwSlabArgs& args, int bits, int num_sms,
                                      cudaStream_t s) {
  AdamwSlabArgs a = args;
  a.strips = strips_of(a.d.n, a.d.K, a.d.N);
  a.per_slab = strips_per_slab(a.d.K);
  a.slabs = fp8moe_adamw_slab_counters(a.d.n, a.d.K, a.d.N) - 1;
  a.units = 2 * a.strips * ((a.d.K + kTileRows - 1) / kTileRows);
  auto launch = [&](auto* kernel, int bytes) {
    const cudaError_t e = allow_ring(kernel, bytes);
    if (e != cudaSuccess) return e;
    const uint32_t most = (uint32_t)(num_sms * kSlabPer);
    return launch_behind(kernel, a.units < most ? a.units : most, kSlabThreads, bytes,
                         a.c.prepared != 0, a, s);
  };
  return bits == 8 ? launch(adamw_slab_kernel<8>, SlabLayout<8>::kAll)
                   : launch(adamw_slab_kernel<32>, SlabLayout<32>::kAll);
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

cudaError_t fp8moe_launch_weight_codes(const float* p, int E, int K, int N, uint32_t* most,
                                       uint8_t* codes, float* scale, cudaStream_t s) {
  const dim3 grid((N + kTileCols - 1) / kTileCols, (K + kTileRows - 1) / kTileRows, E);
  column_max_kernel<<<grid, 32 * kWarps, 0, s>>>(p, K, N, most);
  weight_codes_kernel<<<grid, 32 * kWarps, 0, s>>>(p, K, N, most, codes, scale);
  return cudaGetLastError();
}
