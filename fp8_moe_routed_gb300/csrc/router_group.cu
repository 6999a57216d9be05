// router_group.cu -- the router's choice without a bias, and the balance sums, for many tokens
// (router.cuh): eight lanes take a token, each of them pieces of a row that follow the other lanes'
// (Row::expert). What is as in router.cu is not explained again; a token whose border is not settled
// by the keys' upper 22 bits is chosen by the whole warp in choose_exactly. 65536 tokens of 128 bf16
// logits: 19.5 us for the choice, 25.0 with the balance loss (0.8 TB/s), at half of the issue slots
// (194 instructions a token, 630 by a warp): eight rounds of three dependent shuffles, with 16 warps
// on an SM to hide them.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fp8moe_status.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "ptx.cuh"
#include "router.cuh"
#include "router_choice.cuh"

namespace fp8moe {
namespace {

template <typename T, int V, bool VECT, bool GIVEN>
__global__ void __launch_bounds__(kThreads) router_group_kernel(
    const __grid_constant__ RouterArgs a) {
  constexpr int W = kGroup * V;
  using R = Row<kGroup, V, kPiece<T, V, VECT>>;
  extern __shared__ float s_mem[];
  float* s_share = s_mem;                                           // [kWarps][W]
  int32_t* s_count = reinterpret_cast<int32_t*>(s_mem + kWarps * W);   // [W]
  __shared__ int32_t s_tokens[kWarps];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane & (kGroup - 1), g = lane / kGroup;
  const uint32_t group_lanes = 0xffu << (g * kGroup);
  const int E = a.E, k = a.k;
  const bool sig = a.sig;
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
    R::load(row, E, l, -INFINITY, x);
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
      uint32_t key[V];
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = choice_key(x[j], R::expert(l, j));
      sort_keys(key);
      // a lane's first nine are all that eight choices and the next one can come from
      constexpr int kDepth = V < kGroup + 1 ? V : kGroup + 1;
      uint32_t mine = 0, m = 0;
#pragma unroll 1
      for (int r = 0; r < k; ++r) {
        m = group_max(key[0]);
        const bool here = key[0] == m;
#pragma unroll
        for (int j = 0; j + 1 < kDepth; ++j) key[j] = here ? key[j + 1] : key[j];
        key[kDepth - 1] = here ? 0u : key[kDepth - 1];
        if (l == r) mine = m;
      }
      const uint32_t next_key = group_max(key[0]);
      // (the upper 22 bits are all that a bf16 logit has)
      const bool hard = sizeof(T) == 4 && on && m >= kNone && next_key >= (m & ~1023u);

      if (mine >= kNone) id = 1023 - (int)(mine & 1023u);
      float xc = id >= 0 ? load_f32(row + id) : -INFINITY;
      const float next = __shfl_down_sync(kAllLanes, xc, 1);
      if (__any_sync(kAllLanes, l + 1 < k && xc < next)) {
        // by the whole values; a NaN in place of the largest, those without an expert at the end
        const float value = xc != xc ? INFINITY : xc;
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
        xc = __shfl_sync(kAllLanes, xc, from);
        id = __shfl_sync(kAllLanes, id, from);
      }
      const float cut = key_value(m);
      for (uint32_t left = __ballot_sync(kAllLanes, hard && l == 0); left != 0u; left &= left - 1u) {
        const int who = __ffs(left) - 1;
        const int64_t th = __shfl_sync(kAllLanes, t, who);
        const int exact = choose_exactly(logits + th * E, static_cast<const float*>(nullptr), E, k, sig,
                                         0.0f, 0.0f, __shfl_sync(kAllLanes, cut, who), list);
        const int found = __shfl_sync(kAllLanes, exact, l);
        if (g == who / kGroup) id = l < k ? found : -1;
        __syncwarp();
      }
      if (__any_sync(kAllLanes, hard)) xc = id >= 0 ? load_f32(row + id) : -INFINITY;

      const float largest = __shfl_sync(kAllLanes, xc, g * kGroup);
      if (balance || (!sig && !a.normalize)) scores(largest);
      float w = 0.0f;
      if (a.normalize) {
        const float nc = id >= 0 ? scaled_score(xc, scale_top(largest, sig), sig) : 0.0f;
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
      const int e = R::expert(i % kGroup, i / kGroup);
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

template <typename T, bool GIVEN>
cudaError_t launch_groups(const RouterArgs& a, cudaStream_t s) {
  const int64_t grid = (a.T + a.chunk - 1) / a.chunk;
  return with_group_width(a.E, [&](auto width) {
    constexpr int V = decltype(width)::value;
    const size_t smem = (size_t)(kWarps + 1) * kGroup * V * sizeof(float);
    if (whole_pieces<T, V>(a.E))
      router_group_kernel<T, V, true, GIVEN><<<(unsigned)grid, kThreads, smem, s>>>(a);
    else
      router_group_kernel<T, V, false, GIVEN><<<(unsigned)grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace
}  // namespace fp8moe

using namespace fp8moe;

FP8MOE_DEFINE_STATUS_TAKE(fp8moe_status_take_router_group)

cudaError_t fp8moe_launch_router_groups(const RouterArgs& a, cudaStream_t s) {
  if (a.given != nullptr)
    return a.f32 ? launch_groups<float, true>(a, s) : launch_groups<__nv_bfloat16, true>(a, s);
  return a.f32 ? launch_groups<float, false>(a, s) : launch_groups<__nv_bfloat16, false>(a, s);
}
