// router_choice.cuh -- how the experts of a token are put in order, for the kernels that choose
// (router.cu, router_group.cu).
#pragma once
#include <utility>

#include "fp8moe_status.cuh"
#include "kernels.h"
#include "router.cuh"

namespace fp8moe {
namespace {

// Ascending with the value; a NaN is the largest. -inf lies below kNone: it is no candidate.
constexpr uint32_t kNone = 0x00800000u;
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));    // -0 is 0, a NaN the positive one
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// The upper 22 bits, then the expert, the lowest first.
__device__ __forceinline__ uint32_t choice_key(float v, int e) {
  return (order_key(v) & ~1023u) | (uint32_t)(1023 - e);
}

// The smallest value of a key's upper 22 bits.
__device__ __forceinline__ float key_value(uint32_t key) {
  const uint32_t o = key & ~1023u;
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// What decides the choice, in f32: the logit, or score + bias (-inf stays out either way).
__device__ __forceinline__ float choice_value(float x, float b, bool has_bias, bool sig, float top,
                                              float inv_sum) {
  if (!has_bias) return x;
  if (x == -INFINITY) return x;
  return __fadd_rn(sig ? sigmoid(x) : __fmul_rn(exp_neg(x - top), inv_sum), b);
}
__device__ __forceinline__ double choice_value_64(float x, float b, bool has_bias, bool sig,
                                                  float top, double sum) {
  if (!has_bias) return (double)x;
  const double s = sig ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) / sum;
  return s + (double)b;
}

// Twice the error of a score and of its sum with the bias: 5 * 2^-24 of a sigmoid; of a softmax
// score the argument's rounding, at most .4 of the largest score, the exponential's and the sum's
// of 37 terms; half a unit of the sum.
__device__ __forceinline__ float choice_slack(uint32_t largest, uint32_t least, bool sig,
                                              float inv_sum) {
  return (sig ? 0x1p-20f : 0x1p-17f * inv_sum) +
         0x1p-22f * (fabsf(key_value(largest)) + fabsf(key_value(least)));
}

// The choice in 64 bits, among the experts whose f32 value is at least `cut`: lane j's j-th
// expert (-1 for none). For the few tokens on which 32 bits leave the order open.
template <typename T>
__device__ __noinline__ int choose_exactly(const T* row, const float* bias, int E, int k, bool sig,
                                           float top, float inv_sum, float cut, uint16_t* list) {
  const int lane = threadIdx.x & 31;
  const bool has_bias = bias != nullptr;
  double sum = 0.0;
  int n = 0;
  for (int base = 0; base < E; base += 32) {
    const int e = base + lane;
    const float x = e < E ? load_f32(row + e) : -INFINITY;
    const float b = has_bias && e < E ? bias[e] : 0.0f;
    if (has_bias && !sig && e < E) sum += exp((double)x - (double)top);
    const float c = choice_value(x, b, has_bias, sig, top, inv_sum);
    const bool in = e < E && order_key(c) >= kNone && !(c < cut);
    const uint32_t who = __ballot_sync(kAllLanes, in);
    if (in) list[n + __popc(who & ((1u << lane) - 1u))] = (uint16_t)e;
    n += __popc(who);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAllLanes, sum, o);
  __syncwarp();
  constexpr int kTaken = 0xffff;
  // a NaN counts as the largest, as in order_key
  auto value = [&](int e) {
    const double v = choice_value_64(load_f32(row + e), has_bias ? bias[e] : 0.0f, has_bias, sig,
                                     top, sum);
    return v != v ? (double)INFINITY : v;
  };
  const double first = lane < n ? value(list[lane]) : -(double)INFINITY;
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    double best = -(double)INFINITY;
    int expert = kTaken, place = -1;
    for (int i = lane; i < n; i += 32) {
      const int e = list[i];
      if (e == kTaken) continue;
      const double v = i == lane ? first : value(e);
      if (place < 0 || v > best) best = v, expert = e, place = i;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double v = __shfl_xor_sync(kAllLanes, best, o);
      const int e = __shfl_xor_sync(kAllLanes, expert, o);
      const int at = __shfl_xor_sync(kAllLanes, place, o);
      if (at >= 0 && (place < 0 || v > best || (v == best && e < expert)))
        best = v, expert = e, place = at;
    }
    if (place < 0) break;
    if (lane == j) mine = expert;
    if (lane == 0) list[place] = kTaken;
    __syncwarp();
  }
  return mine;
}

// Descending, by Batcher's odd-even merge sort: its comparisons, written out by the compiler.
template <int V>
struct Network {
  int count = 0, first[192] = {}, second[192] = {};
  constexpr Network() {
    for (int p = 1; p < V; p *= 2)
      for (int d = p; d >= 1; d /= 2)
        for (int i = 0; i + d < V; ++i)
          if (i >= d % p && (i - d % p) % (2 * d) < d && i / (2 * p) == (i + d) / (2 * p))
            first[count] = i, second[count] = i + d, ++count;
  }
};
template <int V> constexpr Network<V> kNetwork{};
template <int V, size_t... I>
__device__ __forceinline__ void sort_steps(uint32_t (&key)[V], std::index_sequence<I...>) {
  auto step = [&](auto i, auto j) {
    const uint32_t large = max(key[i], key[j]);
    key[j] = min(key[i], key[j]);
    key[i] = large;
  };
  (step(std::integral_constant<int, kNetwork<V>.first[I]>(),
        std::integral_constant<int, kNetwork<V>.second[I]>()), ...);
}
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[V]) {
  sort_steps<V>(key, std::make_index_sequence<kNetwork<V>.count>());
}

// For lane i: the lane among the first n whose (value, expert) comes at place i, larger values and
// lower experts first (a NaN value in place of the largest); its own for lanes from n on.
template <typename F>
__device__ __forceinline__ int sorted_from(F value, int id, int n) {
  const int lane = threadIdx.x & 31;
  if (value != value) value = (F)INFINITY;
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const F v = __shfl_sync(kAllLanes, value, i);
    const int e = __shfl_sync(kAllLanes, id, i);
    rank += v > value || (v == value && e < id);
  }
  int from = lane;
  for (int i = 0; i < n; ++i)
    if (__shfl_sync(kAllLanes, rank, i) == lane) from = i;
  return from;
}

// This CTA's chunk of tokens, one run after the other: of each sequence that has a part in it.
// What lies outside of the sequences is padding.
template <bool GIVEN, typename Clear, typename Run, typename Flush>
__device__ __forceinline__ void walk_chunk(const RouterArgs& a, Clear clear, Run run, Flush flush) {
  const int64_t begin = (int64_t)blockIdx.x * a.chunk;
  const int64_t end = begin + a.chunk < a.T ? begin + a.chunk : a.T;
  auto padding = [&](int64_t from, int64_t to) {
    if constexpr (!GIVEN) {
      for (int64_t i = from * a.k + threadIdx.x; i < to * a.k; i += kThreads) {
        a.ids[i] = -1;
        a.weights[i] = 0.0f;
      }
    }
  };
  int64_t at = begin;
  int b = 0;
  const int B = a.offsets != nullptr ? a.B : 1;
  if (a.offsets != nullptr) {
    at = max(begin, min((int64_t)a.offsets[0], end));
    padding(begin, at);
    b = at < end ? max(0, find_sequence(a.offsets, B, at)) : B;
  }
  for (; at < end && b < B; ++b) {
    const int64_t stop = a.offsets != nullptr ? min((int64_t)a.offsets[b + 1], end) : end;
    if (stop <= at) continue;
    clear();
    run(at, stop);
    flush((int64_t)blockIdx.x + b);
    at = stop;
  }
  padding(at, end);
}

}  // namespace
}  // namespace fp8moe
