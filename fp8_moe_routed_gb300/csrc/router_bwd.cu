// router_bwd.cu -- the gradient of the router's weights and of the balance loss into the logits:
//
// dx = q * (w (dw - sum dw w) + p (D - sum D p)),  q = 1 (softmax) or sigmoid(-x),
// D = dloss * slope. Weights that are not normalised: of softmax scores their gradient joins
// D, of sigmoid scores it is dw s.
//
// One pass: a warp, or of a large batch eight lanes, take a token; the choices' parts meet the
// experts' in a row of shared memory. 65536 tokens of 128 bf16 logits 16.4 us (2.3 TB/s, bound by
// the latency of a token's chain), 24.8 by a warp for each; 32768 of 512 f32 logits 38 (3.6 TB/s).
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fp8moe_status.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "router.cuh"

namespace fp8moe {
namespace {

template <typename T, int G, int V, bool VECT>
__global__ void __launch_bounds__(kThreads, V <= 16 ? 4 : 2) router_bwd_kernel(
    const __grid_constant__ RouterBwdArgs a) {
  using R = Row<G, V, kPiece<T, V, VECT>>;
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
  R::load(row, E, lane, -INFINITY, x);
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
    if (on) R::store(out, E, lane, dx);
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
  const int place = id >= 0 ? R::place(id) : 0;
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
    if (a.dloss != nullptr) R::load(a.slope + (int64_t)b * E, E, lane, 0.0f, D);
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
  if (on) R::store(out, E, lane, dx);
}

}  // namespace
}  // namespace fp8moe

using namespace fp8moe;

FP8MOE_DEFINE_STATUS_TAKE(fp8moe_status_take_router_bwd)

cudaError_t fp8moe_launch_router_bwd(const RouterBwdArgs& a, cudaStream_t s) {
  auto launch = [&](auto type, auto lanes, auto width) {
    using T = decltype(type);
    constexpr int G = decltype(lanes)::value, V = decltype(width)::value;
    const int64_t tokens = kWarps * (32 / G);    // of a CTA
    const unsigned grid = (unsigned)((a.T + tokens - 1) / tokens);
    const size_t smem = (size_t)tokens * G * V * sizeof(float);
    if (whole_pieces<T, V>(a.E))
      router_bwd_kernel<T, G, V, true><<<grid, kThreads, smem, s>>>(a);
    else
      router_bwd_kernel<T, G, V, false><<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
  };
  auto of_type = [&](auto type) {
    if (by_groups(a.T, a.E, a.k, false))
      return with_group_width(a.E, [&](auto width) { return launch(type, Int<kGroup>(), width); });
    return with_width(a.E, [&](auto width) { return launch(type, Int<32>(), width); });
  };
  return a.f32 ? of_type(float()) : of_type(__nv_bfloat16());
}
