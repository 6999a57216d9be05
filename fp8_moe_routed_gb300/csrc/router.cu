// router.cu -- the router's choice of experts with its weights, and the balance loss with the
// experts' counts (router_bwd.cu: the gradient of both).
//
//   s = softmax(x) or sigmoid(x) over a token's E logits;  chosen: the topk largest of x, or,
//   with a bias b, of s + b;  weight: scale * s / (sum of the chosen s), or scale * s
//   share p_i = s_i / sum s;  for a sequence of n tokens with C choices, c_i of them expert i:
//   loss = sum_i slope_i * sum_t p_ti,  slope_i = E c_i / (C n)
//
// A warp takes a token, its logits in registers, so that one pass over them gives the maximum, the
// sum, the choice and the shares. Bytes are nothing to it: 4096 tokens of 256 f32 logits with a bias
// (0.66 us of bytes) take 9.7 us for the choice and 16.3 with the balance loss: one wave, so that it
// is the chain of a token's dependent steps (about 900 instructions; k rounds of a maximum over the
// lanes; with the 64 registers of four CTAs, 176 bytes of spills) and the join. One token takes
// 4.1 us, most of it the launch's. 32768 tokens of 512 logits with given choices 21.7 us (3.1 TB/s), bound by the
// instructions of the scores.
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

constexpr int kJoinThreads = 1024, kJoinCtas = 8;

__device__ __forceinline__ uint32_t load_peer(const void* p, int cta) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), cta))
               : "memory");
  return v;
}

template <typename T, int V, bool VECT, bool GIVEN>
__global__ void __launch_bounds__(kThreads, GIVEN ? V <= 16 ? 4 : 3 : V <= 8 ? 4 : 2)
    router_kernel(const __grid_constant__ RouterArgs a) {
  using R = Row<32, V, kPiece<T, V, VECT>>;
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
    R::load(row, E, lane, -INFINITY, x);
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
        const int e = R::expert(lane, j);
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
      const int e = R::expert(i & 31, i >> 5);
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
    if (cta == 0 && tid < width) {               // all on their way before the first is added
      uint32_t shares[kJoinCtas - 1], those[kJoinCtas - 1];
#pragma unroll
      for (int r = 1; r < kJoinCtas; ++r) {
        shares[r - 1] = load_peer(&s_share[tid], r);
        those[r - 1] = load_peer(&s_count[tid], r);
      }
#pragma unroll
      for (int r = 0; r < kJoinCtas - 1; ++r) {
        share += __uint_as_float(shares[r]);
        count += (int32_t)those[r];
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

template <typename T, bool GIVEN>
cudaError_t launch_router(const RouterArgs& a, cudaStream_t s) {
  const int64_t grid = (a.T + a.chunk - 1) / a.chunk;
  return with_width(a.E, [&](auto width) {
    constexpr int V = decltype(width)::value;
    const size_t smem = (size_t)(kWarps + 1) * 32 * V * sizeof(float);
    if (whole_pieces<T, V>(a.E))
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
  const bool groups = by_groups(a.T, a.E, a.k, a.bias != nullptr);
  a.chunk = groups ? group_chunk(a.T) : balance ? fp8moe_balance_chunk(a.T) : kWarps;
  cudaError_t e = cudaSuccess;
  if (a.T > 0) {
    if (groups)
      e = fp8moe_launch_router_groups(a, s);
    else if (a.given != nullptr)
      e = a.f32 ? launch_router<float, true>(a, s) : launch_router<__nv_bfloat16, true>(a, s);
    else
      e = a.f32 ? launch_router<float, false>(a, s) : launch_router<__nv_bfloat16, false>(a, s);
  }
  if (e != cudaSuccess || !balance) return e;
  int width = 32;
  while (width < a.E) width *= 2;
  const int64_t parts = (a.T + a.chunk - 1) / a.chunk;
  const int ctas = parts / a.B > 64 ? kJoinCtas : 1;
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
