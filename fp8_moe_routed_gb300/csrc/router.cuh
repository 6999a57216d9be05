// router.cuh -- what the router's choice and its gradient share: a token's logits in a
// warp's registers, and the experts' scores on a scale on which they cannot all vanish.
#pragma once
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "vec16.cuh"

namespace fp8moe {

constexpr uint32_t kAllLanes = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// Many tokens, at most 128 experts, at most 8 chosen, and no bias: eight lanes take a token, so that
// an instruction works for four. A choice of 65536 tokens (128 experts, bf16, with the balance loss)
// takes 25.0 us then and 46.8 by a warp for a token, of 4096 tokens 7.8 and 10.5, of 2048 7.4 and
// 8.0; its gradient 16.5 and 25.0, 4.1 and 4.3, and 3.9 and 3.5. Versions of this kernel with a bias
// had more tokens to settle one by one (f32, 32768 tokens: 51 us, by a warp 36), and with 256 experts
// so many registers that an SM had one CTA (f32, 32768: 66 and 40; the gradient 57 and 37).
constexpr int64_t kManyTokens = 4096;
constexpr int kGroup = 8, kGroups = 4;
inline bool by_groups(int64_t T, int E, int k, bool bias) {
  return T >= kManyTokens && E <= 128 && k <= kGroup && !bias;
}

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// The V experts that a lane of the G of a token holds: pieces of P, which is 16 bytes (or all of a
// lane's) where rows are whole pieces, so that the lanes' pieces follow each other in memory, and 1
// where they are not.
template <int G, int V, int P>
struct Row {
  static_assert(V % P == 0, "whole pieces");
  static __device__ __forceinline__ int expert(int lane, int j) {
    return (j / P * G + lane) * P + j % P;
  }
  // where expert e stands in [V][G] values, in the order of the lanes' registers
  static __device__ __forceinline__ int place(int e) {
    return (e / (G * P) * P + e % P) * G + e / P % G;
  }
  // past E: `fill`
  template <typename T>
  static __device__ __forceinline__ void load(const T* row, int E, int lane, float fill,
                                              float (&x)[V]) {
    constexpr int kBytes = P * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < V / P; ++i) {
      const T* p = row + expert(lane, i * P);
      const bool in = expert(lane, i * P) < E;
      float (&y)[P] = *reinterpret_cast<float (*)[P]>(&x[i * P]);
      if constexpr (P == 1) {
        y[0] = in ? load_f32(p) : fill;
      } else {
        uint32_t w[kBytes / 4];
        words<kBytes / 4>(p, in, w);
#pragma unroll
        for (int j = 0; j < kBytes / 4; ++j) {
          if constexpr (sizeof(T) == 4) {
            y[j] = in ? __uint_as_float(w[j]) : fill;
          } else {
            y[2 * j] = in ? bf16lo_to_f32(w[j]) : fill;
            y[2 * j + 1] = in ? bf16hi_to_f32(w[j]) : fill;
          }
        }
      }
    }
  }
  template <typename T>
  static __device__ __forceinline__ void store(T* row, int E, int lane, const float (&x)[V]) {
    constexpr int kWords = P * (int)sizeof(T) / 4;
#pragma unroll
    for (int i = 0; i < V / P; ++i) {
      T* p = row + expert(lane, i * P);
      if (expert(lane, i * P) >= E) continue;
      if constexpr (P == 1) {
        *p = T(x[i]);
      } else {
        uint32_t w[kWords];
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(x[i * P + j]);
          else w[j] = f32x2_to_bf16x2(x[i * P + 2 * j], x[i * P + 2 * j + 1]);
        }
        if constexpr (kWords == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kWords == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(p) = w[0];
      }
    }
  }

 private:
  template <int N>
  static __device__ __forceinline__ void words(const void* p, bool in, uint32_t (&w)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const uint4 v = in ? static_cast<const uint4*>(p)[i] : make_uint4(0, 0, 0, 0);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (N == 2) {
      const uint2 v = in ? *static_cast<const uint2*>(p) : make_uint2(0, 0);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = in ? *static_cast<const uint32_t*>(p) : 0;
    }
  }
};
// Values of a piece of a lane's V.
template <typename T, int V, bool VECT>
constexpr int kPiece = !VECT ? 1 : V * (int)sizeof(T) < 16 ? V : 16 / (int)sizeof(T);

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAllLanes, v, o);
  return v;
}
// Of lanes 0 to n - 1, for these lanes; the others hold 0.
__device__ __forceinline__ float first_sum(float v, int n) {
  for (int o = 1; o < n; o *= 2) v += __shfl_xor_sync(kAllLanes, v, o);
  return v;
}
// A NaN anywhere gives NaN.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float clamp_nan(float x, float limit) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(max_nan(x, -limit)), "f"(limit));
  return r;
}

// exp(x) for x <= 0 (and NaN), two at a time: by the exponential unit (within 2^-22 of itself) on x
// times log2 e, with what the product's rounding and the constant's lose put back to first order:
// hi is the f32 nearest to log2 e, lo the one nearest to log2 e - hi.
// Within 6 * 2^-24; 0 below 2^-126.
__device__ __forceinline__ float2 exp_neg(float2 x) {
  const float hi = 1.4426950216293335f, lo = 1.9259629911266175e-8f, ln2 = 0.6931471805599453f;
  x = make_float2(max_nan(x.x, -200.0f), max_nan(x.y, -200.0f));
  const float2 t = mul2(x, both(hi));
  const float2 rest = fma2(x, both(lo), fma2(x, both(hi), mul2(t, both(-1.0f))));
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  return fma2(mul2(e, both(ln2)), rest, e);
}
__device__ __forceinline__ float exp_neg(float x) { return exp_neg(make_float2(x, x)).x; }

// 1 / d, by a Newton step from the approximate one (within 2^-24 and a little of it).
__device__ __forceinline__ float2 inverse(float2 d) {
  float2 y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(d.y));
  return fma2(y, fma2(mul2(d, both(-1.0f)), y, both(1.0f)), y);
}
__device__ __forceinline__ float inverse(float d) { return inverse(make_float2(d, d)).x; }

// s = sigmoid(x) and q = sigmoid(-x) without cancellation, by t = exp(-|x|): 1 / (1 + t) and
// t / (1 + t). Each within 5 * 2^-24 (of 1), and within 8 * 2^-24 of itself.
__device__ __forceinline__ void sigmoids(float2 x, float2& s, float2& q) {
  const float2 t = exp_neg(make_float2(-fabsf(x.x), -fabsf(x.y)));
  const float2 large = inverse(add2(t, both(1.0f))), small = mul2(t, large);
  s = make_float2(x.x < 0.0f ? small.x : large.x, x.y < 0.0f ? small.y : large.y);
  q = make_float2(x.x < 0.0f ? large.x : small.x, x.y < 0.0f ? large.y : small.y);
}
// sigmoid(x) = 1 / (1 + exp(-x)) alone, in half of the instructions, as precise (the
// approximate inverse is within 2^-23); 0 below -88, 1 from 17 on, the infinities' too.
__device__ __forceinline__ float2 sigmoid(float2 x) {
  const float hi = 1.4426950216293335f, lo = 1.9259629911266175e-8f, ln2 = 0.6931471805599453f;
  // exp(88.5) has a zero inverse; an infinity would make a NaN of its own rounding
  x = make_float2(clamp_nan(x.x, 88.5f), clamp_nan(x.y, 88.5f));
  const float2 t = mul2(x, both(-hi));
  const float2 rest = fma2(x, both(-lo), fma2(x, both(-hi), mul2(t, both(-1.0f))));
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  const float2 d = add2(fma2(mul2(e, both(ln2)), rest, e), both(1.0f));
  float2 s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
  return s;
}
__device__ __forceinline__ float sigmoid(float x) { return sigmoid(make_float2(x, x)).x; }

// A score on the row's scale, n(x) = score(x) * exp(-top): top = the largest logit, or, with
// sigmoid scores, the largest one below zero (0 if there is one above). The scores themselves may
// all round to zero (sigmoid below -104); their ratios, which is what weights and shares are,
// do not depend on the scale, and the largest n is at least 1/2. Experts at -inf have 0.
__device__ __forceinline__ float2 scaled_scores(float2 x, float top, bool sig) {
  const float2 y = add2(x, both(-top));
  if (!sig) return exp_neg(y);
  if (top == 0.0f) return sigmoid(x);
  return mul2(exp_neg(y), sigmoid(make_float2(-x.x, -x.y)));   // sigmoid(x) = exp(x) sigmoid(-x)
}
__device__ __forceinline__ float scaled_score(float x, float top, bool sig) {
  return scaled_scores(make_float2(x, x), top, sig).x;
}
__device__ __forceinline__ float scale_top(float largest, bool sig) {
  return sig && largest > 0.0f ? 0.0f : largest;
}

// Of a token's eight lanes.
template <typename F>
__device__ __forceinline__ F group_max(F v) {
#pragma unroll
  for (int o = 1; o < kGroup; o *= 2) {
    const F w = __shfl_xor_sync(kAllLanes, v, o);
    if constexpr (std::is_same<F, float>::value) v = max_nan(v, w);
    else v = max(v, w);
  }
  return v;
}
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < kGroup; o *= 2) v += __shfl_xor_sync(kAllLanes, v, o);
  return v;
}

// Of the G lanes that have a token.
template <int G>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (G == 32) return warp_max(v);
  else return group_max(v);
}
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (G == 32) return warp_sum(v);
  else return group_sum(v);
}

template <typename T, int V>
bool whole_pieces(int E) { return E % kPiece<T, V, true> == 0; }
template <int N> using Int = std::integral_constant<int, N>;
// f(experts of a lane), where a warp or where eight lanes have a token.
template <typename F>
cudaError_t with_width(int E, F f) {
  if (E <= 64) return f(Int<2>());
  if (E <= 128) return f(Int<4>());
  if (E <= 256) return f(Int<8>());
  if (E <= 512) return f(Int<16>());
  return f(Int<32>());
}
template <typename F>
cudaError_t with_group_width(int E, F f) {
  if (E <= 32) return f(Int<4>());
  if (E <= 64) return f(Int<8>());
  return f(Int<16>());
}

// The sequence that token t belongs to, with offsets[b] <= t < offsets[b + 1] (the first b
// with offsets[b + 1] > t); B behind the last one, -1 before the first.
__device__ __forceinline__ int find_sequence(const int32_t* offsets, int B, int64_t t) {
  if (t < offsets[0]) return -1;
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

}  // namespace fp8moe
