// router.cu -- the router's choice of experts with its weights, the balance loss with the
// experts' counts, and the gradient of both into the logits.
//
//   s = softmax(x) or sigmoid(x) over a token's E logits;  chosen: the topk largest of x, or,
//   with a bias b, of s + b;  weight: scale * s / (sum of the chosen s), or scale * s
//   share p_i = s_i / sum s;  for a sequence of n tokens with C choices, c_i of them expert i:
//   loss = sum_i slope_i * sum_t p_ti,  slope_i = E c_i / (C n)
//
// A warp takes a token: lane l holds experts [l V, l V + V) in registers, so that one pass over
// the logits gives the maximum, the sum, the choice and the shares.
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <utility>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fp8moe_status.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "ptx.cuh"
#include "router.cuh"

namespace fp8moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kJoinThreads = 1024;
constexpr int64_t kManyTokens = 16384;          // from here on eight lanes take a token

__device__ __forceinline__ uint32_t load_peer(const void* p, int cta) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), cta))
               : "memory");
  return v;
}

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

template <typename T, int V, bool VECT, bool GIVEN>
__global__ void __launch_bounds__(kThreads, V <= 16 ? 4 : 1) router_kernel(const __grid_constant__ RouterArgs a) {
  extern __shared__ float s_mem[];
  float* s_share = s_mem;                                           // [kWarps][32 V]
  int32_t* s_count = reinterpret_cast<int32_t*>(s_mem + kWarps * 32 * V);   // [32 V]
  __shared__ int32_t s_tokens[kWarps];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E, k = a.k;
  const bool sig = a.sig, has_bias = !GIVEN && a.bias != nullptr;
  const T* logits = static_cast<const T*>(a.logits);
  const bool balance = a.part_share != nullptr;
  uint16_t* list = reinterpret_cast<uint16_t*>(s_mem) + warp * 32 * V;

  float acc[V];
  int tokens = 0;

  auto token = [&](int64_t t) {
    const T* row = logits + t * E;
    float x[V];
    load_row<T, V, VECT>(row, E, lane, -INFINITY, x);
    int id = -1;
    if (GIVEN && lane < k) id = a.given[t * k + lane];
    auto row_max = [&]() {
      float m = x[0];
#pragma unroll
      for (int j = 1; j < V; ++j) m = max_nan(m, x[j]);
      return warp_max(m);
    };
    // the scores, where shares, unnormalised weights or a bias ask for them
    float n[V], top = 0.0f, inv_sum = 0.0f;
    auto scores = [&](float largest) {
      top = scale_top(largest, sig);
      const bool none = largest == -INFINITY;
      float2 sum = both(0.0f);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float2 s = none ? both(0.0f)
                              : scaled_scores(make_float2(x[j], x[j + 1]), top, sig);
        n[j] = s.x, n[j + 1] = s.y;
        sum = add2(sum, s);
      }
      inv_sum = none ? 0.0f : inverse(warp_sum(sum.x + sum.y));
    };

    if constexpr (GIVEN) {
      scores(row_max());
    } else {
      float largest = 0.0f;
      if (has_bias) {
        largest = row_max();
        if (!sig || balance) scores(largest);
      }
      // keys: the value's upper 22 bits of order, then the expert, the lowest first; they
      // differ from each other, so that the largest of a warp names its expert
      uint32_t key[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = lane * V + j;
        float c = x[j];
        if (has_bias && c != -INFINITY) {
          const float b = e < E ? a.bias[e] : 0.0f;
          // (with a balance loss the scores are at hand, on their own scale if that is 0's)
          if (!sig) c = __fadd_rn(__fmul_rn(n[j], inv_sum), b);
          else c = __fadd_rn(balance && top == 0.0f ? n[j] : sigmoid(c), b);
        }
        key[j] = choice_key(c, e);
      }
      sort_keys(key);
      // The topk largest keys, and those behind them whose values may be as large: with the same
      // upper bits, or, with a bias, within the error of two scores.
      uint32_t mine = 0, m = 0, top_key = 0;
      auto take = [&](int place) {               // the largest key, out of its lane
        m = __reduce_max_sync(kAllLanes, key[0]);
        const bool here = key[0] == m;
#pragma unroll
        for (int j = 0; j + 1 < V; ++j) key[j] = here ? key[j + 1] : key[j];
        key[V - 1] = here ? 0u : key[V - 1];
        if (lane == place) mine = m;
      };
      take(0);
      top_key = m;
#pragma unroll 1
      for (int r = 1; r < k; ++r) take(r);
      int found = k;
      float slack = 0.0f;
      const uint32_t k_th = m;
      if (m < kNone) {
        found = __popc(__ballot_sync(kAllLanes, mine >= kNone));
      } else {
        uint32_t floor = m & ~1023u;
        if (has_bias) {
          slack = choice_slack(top_key, m, sig, inv_sum);
          floor = order_key(key_value(m) - slack) & ~1023u;
        }
        while (found <= 32) {
          const uint32_t next = __reduce_max_sync(kAllLanes, key[0]);
          if (next < kNone || next < floor) break;
          take(found++);
        }
      }
      if (mine >= kNone) id = 1023 - (int)(mine & 1023u);
      float xc = id >= 0 ? load_f32(row + id) : -INFINITY;
      if (!has_bias) largest = __shfl_sync(kAllLanes, xc, 0);   // but for equal upper bits
      if (k > 1 || found > 1) {
        const float b = has_bias && id >= 0 ? a.bias[id] : 0.0f;
        float c = id >= 0 ? choice_value(xc, b, has_bias, sig, top, inv_sum) : -INFINITY;
        // into the order of the whole values
        float next = __shfl_down_sync(kAllLanes, c, 1);
        const bool wrong = __any_sync(kAllLanes, lane + 1 < found && c < next);
        if (wrong && found <= 32) {
          const int from = sorted_from(c, id, found);
          c = __shfl_sync(kAllLanes, c, from);
          xc = __shfl_sync(kAllLanes, xc, from);
          id = __shfl_sync(kAllLanes, id, from);
          next = __shfl_down_sync(kAllLanes, c, 1);
        }
        if (!has_bias) largest = __shfl_sync(kAllLanes, xc, 0);
        bool open = false;
        if (has_bias) {
          const float bc = id >= 0 ? a.bias[id] : 0.0f;
          const float next_x = __shfl_down_sync(kAllLanes, xc, 1);
          const float next_b = __shfl_down_sync(kAllLanes, bc, 1);
          open = lane < k && lane + 1 < found && !(c - next > slack) &&
                 !(xc == next_x && bc == next_b);
        }
        open = __any_sync(kAllLanes, open);
        if (found > 32 || (open && !sig)) {
          // cut: the last that can belong to the choice
          const float cut = key_value(k_th) - slack;
          id = choose_exactly(row, a.bias, E, k, sig, top, inv_sum, cut, list);
          __syncwarp();
          xc = id >= 0 ? load_f32(row + id) : -INFINITY;
          if (!has_bias) largest = __shfl_sync(kAllLanes, xc, 0);
        } else if (open) {
          const float bc = id >= 0 ? a.bias[id] : 0.0f;
          const double v = id >= 0 ? choice_value_64(xc, bc, true, true, 0.0f, 0.0)
                                   : -(double)INFINITY;
          const int from = sorted_from(v, id, found);
          xc = __shfl_sync(kAllLanes, xc, from);
          id = __shfl_sync(kAllLanes, id, from);
        }
      }
      if (lane >= k) id = -1, xc = -INFINITY;
      if (!has_bias && (balance || (!sig && !a.normalize))) scores(largest);

      float w = 0.0f;
      if (a.normalize) {
        const float most = has_bias ? warp_max(xc) : largest;
        const float nc = id >= 0 ? scaled_score(xc, scale_top(most, sig), sig) : 0.0f;
        w = nc / first_sum(nc, k);
      } else if (id >= 0) {
        w = sig ? sigmoid(xc) : exp_neg(xc - top) * inv_sum;
      }
      if (largest != largest) w = largest;       // a NaN among the logits, chosen or not
      if (lane < k) {
        a.ids[t * k + lane] = id;
        a.weights[t * k + lane] = id >= 0 ? a.scale * w : 0.0f;
      }
    }
    if (!balance) return;
    if (GIVEN && id >= E) {
      status_set(kStatusBadExpert);
      id = -1;
    }
    if (!__any_sync(kAllLanes, id >= 0)) return;
    if (id >= 0) atomicAdd(&s_count[id], 1);
    ++tokens;
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 s = fma2(make_float2(n[j], n[j + 1]), both(inv_sum),
                            make_float2(acc[j], acc[j + 1]));
      acc[j] = s.x, acc[j + 1] = s.y;
    }
  };
  auto clear = [&]() {
    tokens = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
    if (balance) {
      for (int i = threadIdx.x; i < 32 * V; i += kThreads) s_count[i] = 0;
      __syncthreads();
    }
  };
  // the sums of this CTA's tokens of one sequence, added up in the order of the warps
  auto flush = [&](int64_t slot) {
    if (!balance) return;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) s_share[warp * 32 * V + j * 32 + lane] = acc[j];
    if (lane == 0) s_tokens[warp] = tokens;
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += kThreads) {
      const int e = (i & 31) * V + (i >> 5);
      if (e >= E) continue;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += s_share[w * 32 * V + i];
      a.part_share[slot * E + e] = sum;
      a.part_count[slot * E + e] = s_count[e];
    }
    if (threadIdx.x == 0) {
      int n = 0;
      for (int w = 0; w < kWarps; ++w) n += s_tokens[w];
      a.part_tokens[slot] = n;
    }
    __syncthreads();
  };
  walk_chunk<GIVEN>(a, clear, [&](int64_t from, int64_t to) {
    for (int64_t t = from + warp; t < to; t += kWarps) token(t);
  }, flush);
}

// Many tokens and at most 256 experts, of which 8 are chosen: eight lanes take a token, so that an
// instruction of the choice works for four. Lane l of a group holds experts [l V, l V + V). What
// is as above is not explained again; a token whose border is not settled by the upper 22 bits
// (or, with a bias, by f32) is chosen by the whole warp in choose_exactly. (65536 tokens, 128
// experts, bf16: 632 instructions a token in the kernel above.)
constexpr int kGroup = 8, kGroups = 4;

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

template <typename T, int V, bool VECT, bool GIVEN>
__global__ void __launch_bounds__(kThreads) router_group_kernel(
    const __grid_constant__ RouterArgs a) {
  constexpr int W = kGroup * V;
  extern __shared__ float s_mem[];
  float* s_share = s_mem;                                           // [kWarps][W]
  int32_t* s_count = reinterpret_cast<int32_t*>(s_mem + kWarps * W);   // [W]
  __shared__ int32_t s_tokens[kWarps];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane & (kGroup - 1), g = lane / kGroup;
  const uint32_t group_lanes = 0xffu << (g * kGroup);
  const int E = a.E, k = a.k;
  const bool sig = a.sig, has_bias = !GIVEN && a.bias != nullptr;
  const T* logits = static_cast<const T*>(a.logits);
  const bool balance = a.part_share != nullptr;
  uint16_t* list = reinterpret_cast<uint16_t*>(s_mem) + warp * 2 * W;

  float acc[V];
  int tokens = 0;
  auto group_any = [&](bool x) { return (__ballot_sync(kAllLanes, x) & group_lanes) != 0u; };

  // four tokens of the warp; `on`: this group's exists (its lanes go along all the same)
  auto four = [&](int64_t first, int64_t to) {
    const bool on = first + g < to;
    const int64_t t = on ? first + g : first;
    const T* row = logits + t * E;
    float x[V];
    load_row<T, V, VECT>(row, E, l, -INFINITY, x);
    int id = -1;
    if (GIVEN && on && l < k) id = a.given[t * k + l];
    auto row_max = [&]() {
      float m = x[0];
#pragma unroll
      for (int j = 1; j < V; ++j) m = max_nan(m, x[j]);
      return group_max(m);
    };
    float n[V], top = 0.0f, inv_sum = 0.0f;
    auto scores = [&](float largest) {
      top = scale_top(largest, sig);
      const bool none = largest == -INFINITY;
      float2 sum = both(0.0f);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float2 s = none ? both(0.0f)
                              : scaled_scores(make_float2(x[j], x[j + 1]), top, sig);
        n[j] = s.x, n[j + 1] = s.y;
        sum = add2(sum, s);
      }
      const float all = group_sum(sum.x + sum.y);
      inv_sum = none ? 0.0f : inverse(all);
    };

    if constexpr (GIVEN) {
      scores(row_max());
    } else {
      float largest = 0.0f;
      if (has_bias) {
        largest = row_max();
        if (!sig || balance) scores(largest);
      }
      uint32_t key[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = l * V + j;
        float c = x[j];
        if (has_bias && c != -INFINITY) {
          const float b = e < E ? a.bias[e] : 0.0f;
          if (!sig) c = __fadd_rn(__fmul_rn(n[j], inv_sum), b);
          else c = __fadd_rn(balance && top == 0.0f ? n[j] : sigmoid(c), b);
        }
        key[j] = choice_key(c, e);
      }
      sort_keys(key);
      uint32_t mine = 0, m = 0, top_key = 0;
#pragma unroll 1
      for (int r = 0; r < k; ++r) {
        m = group_max(key[0]);
        const bool here = key[0] == m;
#pragma unroll
        for (int j = 0; j + 1 < V; ++j) key[j] = here ? key[j + 1] : key[j];
        key[V - 1] = here ? 0u : key[V - 1];
        if (l == r) mine = m;
        if (r == 0) top_key = m;
      }
      const uint32_t next_key = group_max(key[0]);
      const float slack = has_bias && m >= kNone ? choice_slack(top_key, m, sig, inv_sum) : 0.0f;
      const uint32_t floor = (has_bias ? order_key(key_value(m) - slack) : m) & ~1023u;
      // (the upper 22 bits are all that a bf16 logit has)
      bool hard = (has_bias || sizeof(T) == 4) && on && m >= kNone && next_key >= kNone &&
                  next_key >= floor;

      if (mine >= kNone) id = 1023 - (int)(mine & 1023u);
      float xc = id >= 0 ? load_f32(row + id) : -INFINITY;
      const float b = has_bias && id >= 0 ? a.bias[id] : 0.0f;
      float c = id >= 0 ? choice_value(xc, b, has_bias, sig, top, inv_sum) : -INFINITY;
      float next = __shfl_down_sync(kAllLanes, c, 1);
      if (__any_sync(kAllLanes, l + 1 < k && c < next)) {
        // by the whole values; a NaN in place of the largest, those without an expert at the end
        const float value = c != c ? INFINITY : c;
        const int order = id >= 0 ? id : 2048 + l;
        int rank = 0;
#pragma unroll
        for (int o = 1; o < kGroup; ++o) {
          const float v = __shfl_xor_sync(kAllLanes, value, o);
          const int e = __shfl_xor_sync(kAllLanes, order, o);
          rank += v > value || (v == value && e < order);
        }
        int from = lane;
#pragma unroll
        for (int o = 0; o < kGroup; ++o)
          if (__shfl_xor_sync(kAllLanes, rank, o) == l) from = lane ^ o;
        c = __shfl_sync(kAllLanes, c, from);
        xc = __shfl_sync(kAllLanes, xc, from);
        id = __shfl_sync(kAllLanes, id, from);
        next = __shfl_down_sync(kAllLanes, c, 1);
      }
      if (has_bias) {
        const float bc = id >= 0 ? a.bias[id] : 0.0f;
        const float next_x = __shfl_down_sync(kAllLanes, xc, 1);
        const float next_b = __shfl_down_sync(kAllLanes, bc, 1);
        const int next_id = __shfl_down_sync(kAllLanes, id, 1);
        hard |= group_any(on && l + 1 < k && next_id >= 0 && !(c - next > slack) &&
                          !(xc == next_x && bc == next_b));
      }
      const float cut = key_value(m) - slack;
      for (uint32_t left = __ballot_sync(kAllLanes, hard && l == 0); left != 0u; left &= left - 1u) {
        const int who = __ffs(left) - 1;
        const int64_t th = __shfl_sync(kAllLanes, t, who);
        const int exact = choose_exactly(
            logits + th * E, a.bias, E, k, sig, __shfl_sync(kAllLanes, top, who),
            __shfl_sync(kAllLanes, inv_sum, who), __shfl_sync(kAllLanes, cut, who), list);
        const int found = __shfl_sync(kAllLanes, exact, l);
        if (g == who / kGroup) id = l < k ? found : -1;
        __syncwarp();
      }
      if (__any_sync(kAllLanes, hard)) xc = id >= 0 ? load_f32(row + id) : -INFINITY;

      if (!has_bias) {
        largest = __shfl_sync(kAllLanes, xc, g * kGroup);
        if (balance || (!sig && !a.normalize)) scores(largest);
      }
      float w = 0.0f;
      if (a.normalize) {
        const float most = has_bias ? group_max(xc) : largest;
        const float nc = id >= 0 ? scaled_score(xc, scale_top(most, sig), sig) : 0.0f;
        w = nc / group_sum(nc);
      } else if (id >= 0) {
        w = sig ? sigmoid(xc) : exp_neg(xc - top) * inv_sum;
      }
      if (largest != largest) w = largest;
      if (on && l < k) {
        a.ids[t * k + l] = id;
        a.weights[t * k + l] = id >= 0 ? a.scale * w : 0.0f;
      }
    }
    if (!balance) return;
    if (GIVEN && id >= E) {
      status_set(kStatusBadExpert);
      id = -1;
    }
    const bool chosen = group_any(id >= 0);        // a vote of all lanes: not behind a condition
    const bool counts = on && chosen;
    if (counts && id >= 0) atomicAdd(&s_count[id], 1);
    if (counts) {
      tokens += l == 0;
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float2 s = fma2(make_float2(n[j], n[j + 1]), both(inv_sum),
                              make_float2(acc[j], acc[j + 1]));
        acc[j] = s.x, acc[j + 1] = s.y;
      }
    }
  };
  auto clear = [&]() {
    tokens = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
    if (balance) {
      for (int i = threadIdx.x; i < W; i += kThreads) s_count[i] = 0;
      __syncthreads();
    }
  };
  auto flush = [&](int64_t slot) {
    if (!balance) return;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float s = acc[j];
      s += __shfl_xor_sync(kAllLanes, s, kGroup);
      s += __shfl_xor_sync(kAllLanes, s, 2 * kGroup);
      if (g == 0) s_share[warp * W + j * kGroup + l] = s;
    }
    const int all = __reduce_add_sync(kAllLanes, tokens);
    if (lane == 0) s_tokens[warp] = all;
    __syncthreads();
    for (int i = threadIdx.x; i < W; i += kThreads) {
      const int e = (i % kGroup) * V + i / kGroup;
      if (e >= E) continue;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += s_share[w * W + i];
      a.part_share[slot * E + e] = sum;
      a.part_count[slot * E + e] = s_count[e];
    }
    if (threadIdx.x == 0) {
      int n = 0;
      for (int w = 0; w < kWarps; ++w) n += s_tokens[w];
      a.part_tokens[slot] = n;
    }
    __syncthreads();
  };
  walk_chunk<GIVEN>(a, clear, [&](int64_t from, int64_t to) {
    for (int64_t t = from + warp * kGroups; t < to; t += kWarps * kGroups) four(t, to);
  }, flush);
}

// Adds up a sequence's parts in a fixed order: counts, slope and loss. A cluster a sequence, of
// one CTA or of eight; CTA r takes the parts r, r + CTAs, ... of a sequence, its thread t column
// t % width of every (1024 / width)-th of these. (One CTA for the 586 parts of a batch of 65536
// tokens and 128 experts took 20 us.)
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(const int32_t* offsets, int64_t T,
                                                         int B, int E, int width, int chunk, int ctas,
                                                         const float* part_share,
                                                         const int32_t* part_count,
                                                         const int32_t* part_tokens,
                                                         int32_t* counts, float* loss,
                                                         float* slope) {
  __shared__ float s_share[kJoinThreads];
  __shared__ int32_t s_count[kJoinThreads];
  __shared__ int32_t s_chosen[32], s_tokens[33];
  __shared__ float s_loss[32];
  const int b = blockIdx.x / ctas, cta = blockIdx.x % ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int e = tid % width, groups = kJoinThreads / width;
  int64_t first = 0, last = T;
  if (offsets != nullptr) {
    const int64_t o0 = offsets[b], o1 = offsets[b + 1];
    if (tid == 0 && cta == 0 && (o0 < 0 || o1 < o0 || o1 > T)) status_set(kStatusBadOffsets);
    first = min(max(o0, (int64_t)0), T);
    last = min(max(o1, first), T);
  }
  const int64_t s0 = first / chunk + b, s1 = last > first ? (last - 1) / chunk + b + 1 : s0;
  pdl_wait();
  float share = 0.0f;
  int32_t count = 0, tokens = 0;
  if (e < E) {
#pragma unroll 4
    for (int64_t s = s0 + cta + (int64_t)(tid / width) * ctas; s < s1; s += groups * ctas) {
      share += part_share[s * E + e];
      count += part_count[s * E + e];
    }
  }
  for (int64_t s = s0 + cta + (int64_t)tid * ctas; s < s1; s += kJoinThreads * ctas)
    tokens += part_tokens[s];
  s_share[tid] = share;
  s_count[tid] = count;
  tokens = __reduce_add_sync(kAllLanes, tokens);
  if (lane == 0) s_tokens[warp] = tokens;
  __syncthreads();
  // this CTA's sums of the columns in s_share and s_count [width], its tokens in s_tokens[32]
  if (tid < width) {
    for (int g = 1; g < groups; ++g) {
      share += s_share[g * width + e];
      count += s_count[g * width + e];
    }
    s_share[tid] = share;
    s_count[tid] = count;
  }
  if (warp == 0) {
    tokens = __reduce_add_sync(kAllLanes, s_tokens[lane]);
    if (lane == 0) s_tokens[32] = tokens;
  }
  if (ctas > 1) {
    cluster_sync();
    if (cta == 0 && tid < width) {
      for (int r = 1; r < ctas; ++r) {
        share += __uint_as_float(load_peer(&s_share[tid], r));
        count += (int32_t)load_peer(&s_count[tid], r);
      }
    }
    tokens = 0;
    if (cta == 0 && tid < ctas) tokens = (int32_t)load_peer(&s_tokens[32], tid);
    cluster_sync();
    if (cta != 0) return;
    if (warp == 0) {
      tokens = __reduce_add_sync(kAllLanes, tokens);
      if (lane == 0) s_tokens[32] = tokens;
    }
  }
  const int32_t chosen = __reduce_add_sync(kAllLanes, tid < width ? count : 0);
  if (lane == 0) s_chosen[warp] = chosen;
  __syncthreads();
  const float C = (float)__reduce_add_sync(kAllLanes, s_chosen[lane]);
  const float n = (float)s_tokens[32];
  float part = 0.0f;
  if (tid < width && e < E) {
    const float d = C > 0.0f ? (float)count * (float)E / C / n : 0.0f;
    counts[(int64_t)b * E + e] = count;
    slope[(int64_t)b * E + e] = d;
    part = d * share;
  }
  part = warp_sum(part);
  if (lane == 0) s_loss[warp] = part;
  __syncthreads();
  if (warp == 0) {
    const float all = warp_sum(s_loss[lane]);
    if (lane == 0) loss[b] = all;
  }
}

// dx = q * (w (dw - sum dw w) + p (D - sum D p)),  q = 1 (softmax) or sigmoid(-x),
// D = dloss * slope. Weights that are not normalised: of softmax scores their gradient joins
// D, of sigmoid scores it is dw s.
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

template <typename T, int G, int V, bool VECT>
__global__ void __launch_bounds__(kThreads, V <= 16 ? 4 : 1) router_bwd_kernel(
    const __grid_constant__ RouterBwdArgs a) {
  extern __shared__ float s_mem[];
  const int lane = threadIdx.x % G, warp = threadIdx.x / 32;
  float* s_row = s_mem + (threadIdx.x / G) * G * V;
  const int E = a.E, k = a.k;
  const bool sig = a.sig;
  const int64_t warp_first = ((int64_t)blockIdx.x * kWarps + warp) * (32 / G);
  if (warp_first >= a.T) return;
  // the lanes of a group past the last token go along with its work and write nothing
  const int64_t mine = warp_first + threadIdx.x % 32 / G;
  const bool on = mine < a.T;
  const int64_t t = on ? mine : a.T - 1;
  const T* row = static_cast<const T*>(a.logits) + t * E;
  T* out = static_cast<T*>(a.dlogits) + t * E;
  float x[V], dx[V];
  load_row<T, V, VECT>(row, E, lane, -INFINITY, x);
  int id = lane < k ? a.ids[t * k + lane] : -1;
  if (id >= E) {
    status_set(kStatusBadExpert);
    id = -1;
  }
  const float dw = a.dweights != nullptr && id >= 0 ? a.scale * a.dweights[t * k + lane] : 0.0f;
  int b = 0;
  if (a.offsets != nullptr) b = find_sequence(a.offsets, a.B, t);
  float largest = x[0];
#pragma unroll
  for (int j = 1; j < V; ++j) largest = max_nan(largest, x[j]);
  largest = lanes_max<G>(largest);
  // nothing was chosen for this token: padding, or no expert was left
  const uint32_t whole = G == 32 ? kAllLanes : ((1u << (G & 31)) - 1u) << (threadIdx.x % 32 / G * G);
  const bool chosen = (__ballot_sync(kAllLanes, id >= 0) & whole) != 0u;
  const bool none = b < 0 || b >= a.B || largest == -INFINITY || !chosen;
  if (__all_sync(kAllLanes, none)) {
#pragma unroll
    for (int j = 0; j < V; ++j) dx[j] = 0.0f;
    if (on) store_row<T, V, VECT>(out, E, lane, dx);
    return;
  }
  if (none) b = 0;
  const float xc = id >= 0 ? load_f32(row + id) : -INFINITY;
  const float top = scale_top(largest, sig);
#pragma unroll
  for (int j = 0; j < V; ++j) s_row[j * G + lane] = 0.0f;
  __syncwarp();

  // each choice's part, put to its expert
  float part = 0.0f;
  const bool joins = !a.normalize && !sig;
  if (a.normalize) {
    const float most = lanes_max<G>(xc);
    const float nc = id >= 0 && xc != -INFINITY ? scaled_score(xc, scale_top(most, sig), sig) : 0.0f;
    const float sum = lanes_sum<G>(nc);
    const float total = largest != largest ? largest : sum;
    const float w = total > 0.0f || total != total ? nc / total : 0.0f;
    part = w * (dw - lanes_sum<G>(dw * w));
  } else {
    part = joins ? dw : dw * sigmoid(xc);
  }
  const int place = id >= 0 ? (id % V) * G + id / V : 0;
  // is an expert among the choices twice?
  const int self = threadIdx.x % 32;
  const int key = id >= 0 ? self / G * 1024 + id : -1 - self;
  const bool alone = __match_any_sync(kAllLanes, key) == (1u << self);
  if (__all_sync(kAllLanes, alone)) {
    if (id >= 0) s_row[place] = part;
  } else {                                    // an expert twice: in the order of the choices
    for (int j = 0; j < k; ++j) {
      if (lane == j && id >= 0) s_row[place] += part;
      __syncwarp();
    }
  }
  __syncwarp();

  float2 d[V / 2], q[V / 2], p[V / 2], shares_sum = both(0.0f);
  const bool shares = a.dloss != nullptr || joins;
#pragma unroll
  for (int h = 0; h < V / 2; ++h) {
    const float2 v = make_float2(x[2 * h], x[2 * h + 1]);
    d[h] = make_float2(s_row[2 * h * G + lane], s_row[(2 * h + 1) * G + lane]);
    if (sig) {
      sigmoids(v, p[h], q[h]);
      if (top != 0.0f)                           // every x is below 0: sigmoid(x) = exp(x) q
        p[h] = mul2(exp_neg(make_float2(v.x - top, v.y - top)), q[h]);
    } else if (shares) {
      p[h] = exp_neg(make_float2(v.x - top, v.y - top));
    }
    if (shares) shares_sum = add2(shares_sum, p[h]);
  }
  if (shares) {
    const float inv_sum = inverse(lanes_sum<G>(shares_sum.x + shares_sum.y));
    float D[V];
    float2 dot = both(0.0f);
    if (a.dloss != nullptr) load_row<float, V, VECT>(a.slope + (int64_t)b * E, E, lane, 0.0f, D);
    const float dl = a.dloss != nullptr ? a.dloss[b] : 0.0f;
#pragma unroll
    for (int h = 0; h < V / 2; ++h) {
      float2 g = both(0.0f);
      if (a.dloss != nullptr) g = mul2(make_float2(D[2 * h], D[2 * h + 1]), both(dl));
      if (joins) g = add2(g, d[h]), d[h] = both(0.0f);
      p[h] = mul2(p[h], both(inv_sum));
      dot = fma2(g, p[h], dot);
      D[2 * h] = g.x, D[2 * h + 1] = g.y;
    }
    const float all = lanes_sum<G>(dot.x + dot.y);
#pragma unroll
    for (int h = 0; h < V / 2; ++h)
      d[h] = fma2(p[h], make_float2(D[2 * h] - all, D[2 * h + 1] - all), d[h]);
  }
#pragma unroll
  for (int h = 0; h < V / 2; ++h) {
    if (sig) d[h] = mul2(d[h], q[h]);
    dx[2 * h] = none ? 0.0f : d[h].x, dx[2 * h + 1] = none ? 0.0f : d[h].y;
  }
  if (on) store_row<T, V, VECT>(out, E, lane, dx);
}

// Rows of whole pieces for 16-byte accesses (load_row); V: experts of a lane.
template <typename T>
bool whole_pieces(int E, int V) {
  const int values = (V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16) / (int)sizeof(T);
  return E % values == 0;
}

template <typename F>
cudaError_t with_width(int E, F f) {
  if (E <= 64) return f(std::integral_constant<int, 2>());
  if (E <= 128) return f(std::integral_constant<int, 4>());
  if (E <= 256) return f(std::integral_constant<int, 8>());
  if (E <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

bool by_groups(int64_t T, int E, int k) { return T >= kManyTokens && E <= 256 && k <= kGroup; }

template <typename T, bool GIVEN>
cudaError_t launch_router(const RouterArgs& a, cudaStream_t s) {
  const int64_t grid = (a.T + a.chunk - 1) / a.chunk;
  if (by_groups(a.T, a.E, a.k)) {
    auto launch = [&](auto width) {
      constexpr int V = decltype(width)::value;
      const size_t smem = (size_t)(kWarps + 1) * kGroup * V * sizeof(float);
      if (whole_pieces<T>(a.E, V))
        router_group_kernel<T, V, true, GIVEN><<<(unsigned)grid, kThreads, smem, s>>>(a);
      else
        router_group_kernel<T, V, false, GIVEN><<<(unsigned)grid, kThreads, smem, s>>>(a);
      return cudaGetLastError();
    };
    if (a.E <= 32) return launch(std::integral_constant<int, 4>());
    if (a.E <= 64) return launch(std::integral_constant<int, 8>());
    if (a.E <= 128) return launch(std::integral_constant<int, 16>());
    return launch(std::integral_constant<int, 32>());
  }
  return with_width(a.E, [&](auto width) {
    constexpr int V = decltype(width)::value;
    const size_t smem = (size_t)(kWarps + 1) * 32 * V * sizeof(float);
    if (whole_pieces<T>(a.E, V))
      router_kernel<T, V, true, GIVEN><<<(unsigned)grid, kThreads, smem, s>>>(a);
    else
      router_kernel<T, V, false, GIVEN><<<(unsigned)grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace
}  // namespace fp8moe

using namespace fp8moe;

FP8MOE_DEFINE_STATUS_TAKE(fp8moe_status_take_router)

static int chunk_of(int64_t T, int ctas, int step, int most) {
  const int64_t c = (T / ctas + step - 1) / step * step;
  return (int)(c < step ? step : c > most ? most : c);
}
// The smallest there are: four CTAs on an SM, a token for a warp at a time.
int fp8moe_balance_chunk(int64_t T) { return chunk_of(T, 608, kWarps, 128); }
// Two CTAs on an SM, four tokens for a warp.
static int group_chunk(int64_t T) { return chunk_of(T, 304, kWarps * kGroups, 256); }

cudaError_t fp8moe_launch_router(const RouterArgs& args, cudaStream_t s) {
  RouterArgs a = args;
  const bool balance = a.part_share != nullptr;
  a.chunk = by_groups(a.T, a.E, a.k) ? group_chunk(a.T) : balance ? fp8moe_balance_chunk(a.T) : kWarps;
  cudaError_t e = cudaSuccess;
  if (a.T > 0) {
    if (a.given != nullptr)
      e = a.f32 ? launch_router<float, true>(a, s) : launch_router<__nv_bfloat16, true>(a, s);
    else
      e = a.f32 ? launch_router<float, false>(a, s) : launch_router<__nv_bfloat16, false>(a, s);
  }
  if (e != cudaSuccess || !balance) return e;
  int width = 32;
  while (width < a.E) width *= 2;
  const int64_t parts = (a.T + a.chunk - 1) / a.chunk;
  const int ctas = parts / a.B > 16 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  pdl_attribute(attr[1]);
  cfg.gridDim = dim3((unsigned)(a.B * ctas));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = a.T > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, balance_join_kernel, a.offsets, a.T, a.B, a.E, width, a.chunk, ctas,
                            (const float*)a.part_share, (const int32_t*)a.part_count,
                            (const int32_t*)a.part_tokens, a.counts, a.loss, a.slope);
}

cudaError_t fp8moe_launch_router_bwd(const RouterBwdArgs& a, cudaStream_t s) {
  auto launch = [&](auto type, auto lanes, auto width) {
    using T = decltype(type);
    constexpr int G = decltype(lanes)::value, V = decltype(width)::value;
    const int64_t tokens = kWarps * (32 / G);    // of a CTA
    const unsigned grid = (unsigned)((a.T + tokens - 1) / tokens);
    const size_t smem = (size_t)tokens * G * V * sizeof(float);
    // slope rows are f32: their pieces have to be whole, too
    if (whole_pieces<T>(a.E, V) && whole_pieces<float>(a.E, V))
      router_bwd_kernel<T, G, V, true><<<grid, kThreads, smem, s>>>(a);
    else
      router_bwd_kernel<T, G, V, false><<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
  };
  auto of_type = [&](auto type) {
    if (by_groups(a.T, a.E, a.k)) {
      const std::integral_constant<int, kGroup> lanes;
      if (a.E <= 32) return launch(type, lanes, std::integral_constant<int, 4>());
      if (a.E <= 64) return launch(type, lanes, std::integral_constant<int, 8>());
      if (a.E <= 128) return launch(type, lanes, std::integral_constant<int, 16>());
      return launch(type, lanes, std::integral_constant<int, 32>());
    }
    return with_width(a.E, [&](auto width) {
      return launch(type, std::integral_constant<int, 32>(), width);
    });
  };
  return a.f32 ? of_type(float()) : of_type(__nv_bfloat16());
}
