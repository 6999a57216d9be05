// norm.cu -- the RMS norms after and before a block, fused with the block's gate
// and the scaled residual sum, and their gradient.
//
// Forward, per row of H values (n(z) = z * rstd(z), rstd(z) = 1/sqrt(mean(z^2) + eps)):
//   r = a * x + b * g * (w_post * n(y))         (without y: r = x, only h is written)
//   h = w_pre * n(r)                            (r in f32, before it is rounded)
// with g = 1, a value per row, per column or per element, taken as it is or through
// a sigmoid. Backward, with rh = r * rstd_pre, yh = y * rstd_post and the incoming
// gradients dr (of r) and dh (of h):
//   D  = dr + rstd_pre * (w_pre dh - rh c1),   c1 = mean(w_pre dh rh)
//   dx = a D;  dn = b D g;  dy = rstd_post * (w_post dn - yh c2),  c2 = mean(w_post dn yh)
//   dw_pre = sum_rows dh rh;  dw_post = sum_rows dn yh;  dgate = sum over what shares it
//   of b D w_post yh (times g (1 - g) behind a sigmoid)
// D enters c2 linearly, so with q = b g w_post yh
//   H c2 = sum q D = sum q (dr + rstd_pre w_pre dh) - c1 rstd_pre sum q rh,
// and every row needs one reduction (three sums), not two in a row.
//
// Bound by HBM: 4 (forward) or 6 (backward) row vectors per row, each moved once. A
// persistent CTA per SM streams rows through a ring of shared-memory stages filled
// by bulk copies, which keeps two stages (57 KB each at H = 7168) in flight without
// holding registers; rows are contiguous, so one copy per tensor fills a stage. All
// sums and the column sums of the weight gradients are f32; the latter stay in
// registers over all rows of a CTA and are joined by a second small kernel in a
// fixed order, so results do not change from run to run.
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fp8moe_status.cuh"
#include "kernels.h"
#include "vec16.cuh"

namespace fp8moe {
namespace norm {

constexpr int kCols = 16;            // columns a thread holds: 2 vectors of bf16 or 4 of f32
constexpr int kTeamThreads = 512;    // threads of a CTA when rows are short (several teams)
constexpr int kRingBytes = 200 * 1024;
constexpr int kMaxStages = 4;
constexpr int kMaxTensors = 5;

enum { kGateNone = 0, kGateRow = 1, kGateCol = 2, kGateFull = 3 };

struct Shape {
  int64_t T;
  int H, nvec;
  int warps;       // of a team: one row per team
  int teams;       // rows of a stage
  int stages, tensors;
  uint32_t row_bytes;
};

// The inputs of a stage that are there, in order.
struct Loads {
  const uint8_t* p[kMaxTensors];
};

// exp and reciprocal by the fast units: a relative error of a few 2^-23, that of one or
// two of the f32 operations that follow.
__device__ __forceinline__ float sigmoid(float z) {
  return __fdividef(1.0f, 1.0f + __expf(-z));
}
__device__ __forceinline__ float2 sigmoid2(float2 z) { return make_float2(sigmoid(z.x), sigmoid(z.y)); }

// A ring of stages in shared memory, a stage the rows of one item.
struct Ring {
  uint8_t* base;
  uint64_t* full;
  __device__ __forceinline__ const uint4* row(const Shape& sh, int stage, int tensor, int team) const {
    return reinterpret_cast<const uint4*>(
        base + ((size_t)(stage * sh.tensors + tensor) * sh.teams + team) * sh.row_bytes);
  }
  // one thread: the rows of item `it` into `stage`
  __device__ __forceinline__ void fill(const Shape& sh, const Loads& in, int64_t it, int stage) const {
    const int64_t r0 = it * sh.teams;
    const int64_t left = sh.T - r0;
    const uint32_t bytes = (uint32_t)(left < sh.teams ? left : sh.teams) * sh.row_bytes;
    mbar_arrive_expect_tx(&full[stage], bytes * sh.tensors);
#pragma unroll
    for (int i = 0; i < kMaxTensors; ++i)
      if (i < sh.tensors)
        bulk_load(const_cast<uint4*>(row(sh, stage, i, 0)), in.p[i] + r0 * sh.row_bytes, bytes,
                  &full[stage]);
  }
};

// Sums of NS values over a team's warps, for every thread of the team. `buf`
// alternates between two areas: a slow reader of one call's sums is past them
// before the call after the next writes there again.
template <int NS>
__device__ __forceinline__ void team_sum(float (&v)[NS], float* s_red, int buf, int warp,
                                         int team_warp0, int team_warps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  float4* const area = reinterpret_cast<float4*>(s_red) + buf * 32;
  if ((threadIdx.x & 31) == 0)
    area[warp] = make_float4(v[0], NS > 1 ? v[NS > 1 ? 1 : 0] : 0.0f, NS > 2 ? v[NS - 1] : 0.0f, 0.0f);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = 0.0f;
#pragma unroll 4
  for (int w = 0; w < team_warps; ++w) {
    const float4 p = area[team_warp0 + w];
    v[0] += p.x;
    if (NS > 1) v[NS > 1 ? 1 : 0] += p.y;
    if (NS > 2) v[NS - 1] += p.z;
  }
}

template <int P>
__device__ __forceinline__ void load_f32(const float* __restrict__ p, float2 (&f)[P]) {
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
    f[2 * i] = make_float2(v.x, v.y);
    f[2 * i + 1] = make_float2(v.z, v.w);
  }
}

// A per-column parameter: in registers for all rows of a thread (HOIST), or, when rows
// are so long that a CTA needs more than 512 threads, loaded for every row.
template <typename T, bool HOIST>
struct Param {
  static constexpr int P = Vec<T>::kP, NV = kCols / Vec<T>::kN;
  float2 v[HOIST ? NV : 1][P];
  const float* p;
  __device__ __forceinline__ void init(const float* src, int tt, int stride, int nvec) {
    p = src;
    if (HOIST && src) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tt + i * stride < nvec) load_f32<P>(src + (size_t)(tt + i * stride) * Vec<T>::kN, v[i]);
    }
  }
  __device__ __forceinline__ void get(int i, int vec, float2 (&o)[P]) const {
    if (HOIST) {
#pragma unroll
      for (int k = 0; k < P; ++k) o[k] = v[HOIST ? i : 0][k];
    } else {
      load_f32<P>(p + (size_t)vec * Vec<T>::kN, o);
    }
  }
};

struct FwdArgs {
  Loads in;                    // x, y, gate (each only if it is there)
  const float* w_post;
  const float* w_pre;
  const float* gate;           // per row or per column
  int gate_kind, sigmoid;
  float residual_scale, branch_scale, eps;
  void* r;
  void* h;
  float* rstd_post;
  float* rstd_pre;
};

// COL: a gate per column (its registers are not spent otherwise).
template <typename T, int MAXT, bool COL>
__global__ void __launch_bounds__(MAXT, 1)
norm_fwd_kernel(const __grid_constant__ FwdArgs a, const __grid_constant__ Shape sh) {
  constexpr int P = Vec<T>::kP, NV = kCols / Vec<T>::kN;
  constexpr bool HOIST = MAXT <= kTeamThreads;
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ uint64_t s_full[kMaxStages];
  __shared__ __align__(16) float s_red[2 * 32 * 4];
  const Ring ring{ring_mem, s_full};
  const int warp = threadIdx.x >> 5;
  const int team = warp / sh.warps, team_warp0 = team * sh.warps;
  const int tt = threadIdx.x - team_warp0 * 32, stride = sh.warps * 32;
  const int64_t items = (sh.T + sh.teams - 1) / sh.teams;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  if (threadIdx.x == 0) {
    for (int i = 0; i < sh.stages; ++i) mbar_init(&s_full[i], 1);
    fence_mbar_init();
    for (int i = 0; i < sh.stages; ++i) {
      const int64_t it = blockIdx.x + (int64_t)i * gridDim.x;
      if (it < items) ring.fill(sh, a.in, it, i);
    }
  }
  Param<T, HOIST> w_post, w_pre, gate;
  w_post.init(a.w_post, tt, stride, sh.nvec);
  w_pre.init(a.w_pre, tt, stride, sh.nvec);
  if (COL) gate.init(a.gate, tt, stride, sh.nvec);
  __syncthreads();
  const float inv_h = 1.0f / (float)sh.H;
  int stage = 0, buf = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t row = it * sh.teams + team;
    const bool live = row < sh.T;
    float grow = 1.0f;
    if (post && a.gate_kind == kGateRow && live) {
      grow = __ldg(a.gate + row);
      if (a.sigmoid) grow = sigmoid(grow);
    }
    ok = ok && mbar_wait(&s_full[stage], phase, kWhereEpilogue);
    const uint4* const xs = ring.row(sh, stage, 0, team);
    const uint4* const ys = ring.row(sh, stage, 1, team);
    const uint4* const gs = ring.row(sh, stage, 2, team);
    float rp = 0.0f;
    if (post) {
      float2 s2 = both(0.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tt + i * stride;
        if (!live || v >= sh.nvec) continue;
        float2 y[P];
        Vec<T>::unpack(ys[v], y);
#pragma unroll
        for (int k = 0; k < P; ++k) s2 = fma2(y[k], y[k], s2);
      }
      float ss[1] = {s2.x + s2.y};
      team_sum<1>(ss, s_red, buf, warp, team_warp0, sh.warps);
      buf ^= 1;
      rp = 1.0f / sqrtf(ss[0] * inv_h + a.eps);
    }
    float2 r[NV][P];
    float2 s2 = both(0.0f);
    const float2 scale = both(a.branch_scale * grow), rs = both(a.residual_scale);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tt + i * stride;
#pragma unroll
      for (int k = 0; k < P; ++k) r[i][k] = both(0.0f);
      if (!live || v >= sh.nvec) continue;
      float2 x[P];
      Vec<T>::unpack(xs[v], x);
      if (post) {
        float2 y[P], w[P], g[P];
        Vec<T>::unpack(ys[v], y);
        w_post.get(i, v, w);
        if (COL) gate.get(i, v, g);
        else if (a.gate_kind == kGateFull) Vec<T>::unpack(gs[v], g);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          float2 b = mul2(mul2(y[k], both(rp)), w[k]);
          if (COL || a.gate_kind == kGateFull) b = mul2(b, a.sigmoid ? sigmoid2(g[k]) : g[k]);
          r[i][k] = fma2(b, scale, mul2(rs, x[k]));
        }
        reinterpret_cast<uint4*>(a.r)[row * sh.nvec + v] = Vec<T>::pack(r[i]);
      } else {
#pragma unroll
        for (int k = 0; k < P; ++k) r[i][k] = x[k];
      }
#pragma unroll
      for (int k = 0; k < P; ++k) s2 = fma2(r[i][k], r[i][k], s2);
    }
    if (post && tt == 0 && live) a.rstd_post[row] = rp;
    // the barrier of this sum also says that every thread has read the stage
    float ss[1] = {s2.x + s2.y};
    team_sum<1>(ss, s_red, buf, warp, team_warp0, sh.warps);
    buf ^= 1;
    if (threadIdx.x == 0) {
      const int64_t next = it + (int64_t)sh.stages * gridDim.x;
      if (next < items) ring.fill(sh, a.in, next, stage);
    }
    if (pre) {
      const float rq = 1.0f / sqrtf(ss[0] * inv_h + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tt + i * stride;
        if (!live || v >= sh.nvec) continue;
        float2 w[P], h[P];
        w_pre.get(i, v, w);
#pragma unroll
        for (int k = 0; k < P; ++k) h[k] = mul2(mul2(r[i][k], both(rq)), w[k]);
        reinterpret_cast<uint4*>(a.h)[row * sh.nvec + v] = Vec<T>::pack(h);
      }
      if (tt == 0 && live) a.rstd_pre[row] = rq;
    }
    if (++stage == sh.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
}

struct BwdArgs {
  Loads in;                    // dr, dh, r, y, gate (each only if it is there)
  int i_dr, i_dh, i_r, i_y, i_gate;   // their places in a stage, -1 if absent
  const float* w_post;
  const float* w_pre;
  const float* rstd_post;
  const float* rstd_pre;
  const float* gate;
  int gate_kind, sigmoid;
  float residual_scale, branch_scale;
  void* dx;
  void* dy;
  float* dgate_row;
  void* dgate_full;
  float* part;                 // [3][gridDim.x][H]: dw_pre, dw_post, dgate per column
};

template <typename T, int MAXT, bool COL>
__global__ void __launch_bounds__(MAXT, 1)
norm_bwd_kernel(const __grid_constant__ BwdArgs a, const __grid_constant__ Shape sh) {
  constexpr int N = Vec<T>::kN, P = Vec<T>::kP, NV = kCols / N;
  constexpr bool HOIST = MAXT <= kTeamThreads && !COL;   // else too many registers
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ uint64_t s_full[kMaxStages];
  __shared__ __align__(16) float s_red[2 * 32 * 4];
  const Ring ring{ring_mem, s_full};
  const int warp = threadIdx.x >> 5;
  const int team = warp / sh.warps, team_warp0 = team * sh.warps;
  const int tt = threadIdx.x - team_warp0 * 32, stride = sh.warps * 32;
  const int64_t items = (sh.T + sh.teams - 1) / sh.teams;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const bool full = !COL && a.gate_kind == kGateFull;
  if (threadIdx.x == 0) {
    for (int i = 0; i < sh.stages; ++i) mbar_init(&s_full[i], 1);
    fence_mbar_init();
    for (int i = 0; i < sh.stages; ++i) {
      const int64_t it = blockIdx.x + (int64_t)i * gridDim.x;
      if (it < items) ring.fill(sh, a.in, it, i);
    }
  }
  Param<T, HOIST> w_post, w_pre;
  Param<T, false> gate;
  w_post.init(a.w_post, tt, stride, sh.nvec);
  w_pre.init(a.w_pre, tt, stride, sh.nvec);
  gate.init(a.gate, tt, stride, sh.nvec);
  __syncthreads();
  const float inv_h = 1.0f / (float)sh.H;
  float2 acc_pre[NV][P], acc_post[NV][P], acc_gate[COL ? NV : 1][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) acc_pre[i][k] = acc_post[i][k] = acc_gate[COL ? i : 0][k] = both(0.0f);
  int stage = 0, buf = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t row = it * sh.teams + team;
    const bool live = row < sh.T;
    float rp = 0.0f, rq = 0.0f, grow = 1.0f, slope_row = 1.0f;
    if (live) {
      if (post) rp = __ldg(a.rstd_post + row);
      if (pre) rq = __ldg(a.rstd_pre + row);
      if (a.gate_kind == kGateRow) {
        grow = __ldg(a.gate + row);
        if (a.sigmoid) {
          grow = sigmoid(grow);
          slope_row = grow * (1.0f - grow);
        }
      }
    }
    ok = ok && mbar_wait(&s_full[stage], phase, kWhereEpilogue);
    auto tensor = [&](int i) { return ring.row(sh, stage, i < 0 ? 0 : i, team); };
    const uint4* const drs = tensor(a.i_dr);
    const uint4* const dhs = tensor(a.i_dh);
    const uint4* const rs = tensor(a.i_r);
    const uint4* const ys = tensor(a.i_y);
    const uint4* const gs = tensor(a.i_gate);
    // the branch factor q = b g w_post yh of a vector, with g as far as it is per element
    auto gate_of = [&](int i, int v, float2 (&g)[P]) {
      if (COL) gate.get(i, v, g);
      else Vec<T>::unpack(gs[v], g);
      if (a.sigmoid) {
#pragma unroll
        for (int k = 0; k < P; ++k) g[k] = sigmoid2(g[k]);
      }
    };
    // first pass: sum u rh, sum q (dr + rq u), sum q rh
    float2 s0 = both(0.0f), s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tt + i * stride;
      if (!live || v >= sh.nvec) continue;
      float2 d[P], rh[P];
#pragma unroll
      for (int k = 0; k < P; ++k) d[k] = rh[k] = both(0.0f);
      if (a.i_dr >= 0) Vec<T>::unpack(drs[v], d);
      if (pre) {
        float2 u[P], w[P];
        Vec<T>::unpack(dhs[v], u);
        Vec<T>::unpack(rs[v], rh);
        w_pre.get(i, v, w);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          u[k] = mul2(u[k], w[k]);
          rh[k] = mul2(rh[k], both(rq));
          s0 = fma2(u[k], rh[k], s0);
          d[k] = fma2(both(rq), u[k], d[k]);
        }
      }
      if (post) {
        float2 y[P], w[P];
        Vec<T>::unpack(ys[v], y);
        w_post.get(i, v, w);
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] = mul2(mul2(y[k], both(rp)), w[k]);
        if (COL || full) {
          float2 g[P];
          gate_of(i, v, g);
#pragma unroll
          for (int k = 0; k < P; ++k) y[k] = mul2(y[k], g[k]);
        }
#pragma unroll
        for (int k = 0; k < P; ++k) {
          s1 = fma2(y[k], d[k], s1);
          s2 = fma2(y[k], rh[k], s2);
        }
      }
    }
    float s3[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
    team_sum<3>(s3, s_red, buf, warp, team_warp0, sh.warps);
    buf ^= 1;
    // Past this barrier every thread has finished with the stage of the item before.
    if (threadIdx.x == 0 && it >= gridDim.x && sh.stages > 1) {
      const int64_t next = it + (int64_t)(sh.stages - 1) * gridDim.x;
      if (next < items) ring.fill(sh, a.in, next, stage == 0 ? sh.stages - 1 : stage - 1);
    }
    const float c1 = s3[0] * inv_h;
    const float qd = a.branch_scale * (s3[1] - c1 * rq * s3[2]);
    const float c2 = qd * grow * inv_h;
    if (a.gate_kind == kGateRow && tt == 0 && live) a.dgate_row[row] = qd * slope_row;
    // second pass: the outputs and the column sums
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tt + i * stride;
      if (!live || v >= sh.nvec) continue;
      float2 d[P], o[P];
#pragma unroll
      for (int k = 0; k < P; ++k) d[k] = both(0.0f);
      if (a.i_dr >= 0) Vec<T>::unpack(drs[v], d);
      if (pre) {
        float2 dh[P], rh[P], w[P];
        Vec<T>::unpack(dhs[v], dh);
        Vec<T>::unpack(rs[v], rh);
        w_pre.get(i, v, w);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          rh[k] = mul2(rh[k], both(rq));
          acc_pre[i][k] = fma2(dh[k], rh[k], acc_pre[i][k]);
          d[k] = fma2(both(rq), fma2(rh[k], both(-c1), mul2(dh[k], w[k])), d[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < P; ++k) o[k] = mul2(both(a.residual_scale), d[k]);
      reinterpret_cast<uint4*>(a.dx)[row * sh.nvec + v] = Vec<T>::pack(o);
      if (post) {
        float2 y[P], w[P], g[P];
        Vec<T>::unpack(ys[v], y);
        w_post.get(i, v, w);
        if (COL || full) gate_of(i, v, g);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const float2 yh = mul2(y[k], both(rp));
          float2 dn = mul2(both(a.branch_scale), d[k]);
          if (COL || full) {
            const float2 dg = mul2(mul2(dn, w[k]), yh);
            dn = mul2(dn, g[k]);
            if (COL) acc_gate[COL ? i : 0][k] = add2(acc_gate[COL ? i : 0][k], dg);
            else if (a.sigmoid) g[k] = mul2(dg, fma2(mul2(g[k], both(-1.0f)), g[k], g[k]));
            else g[k] = dg;
          } else {
            dn = mul2(dn, both(grow));
          }
          acc_post[i][k] = fma2(dn, yh, acc_post[i][k]);
          o[k] = mul2(both(rp), fma2(yh, both(-c2), mul2(w[k], dn)));
        }
        reinterpret_cast<uint4*>(a.dy)[row * sh.nvec + v] = Vec<T>::pack(o);
        if (full) reinterpret_cast<uint4*>(a.dgate_full)[row * sh.nvec + v] = Vec<T>::pack(g);
      }
    }
    if (sh.stages == 1) {      // the longest rows: this item's stage is also the next one's
      __syncthreads();
      const int64_t next = it + gridDim.x;
      if (threadIdx.x == 0 && next < items) ring.fill(sh, a.in, next, 0);
    }
    if (++stage == sh.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  // the column sums of this CTA: its teams' are joined in shared memory (the ring
  // is idle: every stage that was filled has been read)
  auto join = [&](float2 (&acc)[NV][P], int which) {
    float* const out = a.part + ((size_t)which * gridDim.x + blockIdx.x) * sh.H;
    float* const s = reinterpret_cast<float*>(ring_mem);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tt + i * stride;
      if (v >= sh.nvec) continue;
#pragma unroll
      for (int k = 0; k < P; ++k)
        *reinterpret_cast<float2*>(s + (size_t)team * sh.H + v * N + 2 * k) = acc[i][k];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < sh.H; c += blockDim.x) {
      float sum = 0.0f;
      for (int q = 0; q < sh.teams; ++q) sum += s[(size_t)q * sh.H + c];
      out[c] = sum;
    }
  };
  if (pre) join(acc_pre, 0);
  if (post) join(acc_post, 1);
  if constexpr (COL) join(acc_gate, 2);
}

// Joins the CTAs' column sums: 16 threads per column take every 16th CTA.
constexpr int kJoinCols = 32, kJoinRows = 16;

__global__ void __launch_bounds__(kJoinCols * kJoinRows)
norm_join_kernel(const float* __restrict__ part, int ctas, int H, const float* __restrict__ gate,
                 int sigmoid_gate, float* __restrict__ dw_pre, float* __restrict__ dw_post,
                 float* __restrict__ dgate) {
  __shared__ float s[kJoinRows][kJoinCols + 1];
  float* const out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
  if (!out) return;
  const int cx = threadIdx.x % kJoinCols, ry = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + cx;
  const float* p = part + (size_t)blockIdx.y * ctas * H;
  float sum = 0.0f;
  if (c < H) {
#pragma unroll 4
    for (int i = ry; i < ctas; i += kJoinRows) sum += __ldg(p + (size_t)i * H + c);
  }
  s[ry][cx] = sum;
  __syncthreads();
  if (ry == 0 && c < H) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) t += s[i][cx];
    if (blockIdx.y == 2 && sigmoid_gate) {
      const float g = sigmoid(__ldg(gate + c));
      t *= g * (1.0f - g);
    }
    out[c] = t;
  }
}

Shape make_shape(int64_t T, int H, int f32, int tensors) {
  Shape s;
  s.T = T;
  s.H = H;
  s.nvec = H / (f32 ? 4 : 8);
  s.row_bytes = (uint32_t)H * (f32 ? 4 : 2);
  const int per_warp = 32 * (kCols / (f32 ? 4 : 8));
  s.warps = (s.nvec + per_warp - 1) / per_warp;
  s.teams = kTeamThreads / (32 * s.warps);
  if (s.teams < 1) s.teams = 1;
  s.tensors = tensors;
  const int64_t stage = (int64_t)s.teams * s.row_bytes * tensors;
  s.stages = (int)(kRingBytes / stage);
  if (s.stages > kMaxStages) s.stages = kMaxStages;
  return s;      // H * element size <= 32768 leaves at least one stage
}

size_t ring_bytes(const Shape& s) {
  size_t b = (size_t)s.stages * s.tensors * s.teams * s.row_bytes;
  const size_t join = (size_t)s.teams * s.H * sizeof(float);
  return b > join ? b : join;
}

}  // namespace norm
}  // namespace fp8moe

FP8MOE_DEFINE_STATUS_TAKE(fp8moe_status_take_norm)

cudaError_t fp8moe_launch_norm_fwd(const NormFwdArgs& p, int num_sms, cudaStream_t s) {
  using namespace fp8moe::norm;
  FwdArgs a = {};
  int n = 0;
  a.in.p[n++] = static_cast<const uint8_t*>(p.x);
  if (p.y) a.in.p[n++] = static_cast<const uint8_t*>(p.y);
  if (p.y && p.gate_kind == kGateFull) a.in.p[n++] = static_cast<const uint8_t*>(p.gate);
  a.w_post = p.w_post;
  a.w_pre = p.w_pre;
  a.gate = static_cast<const float*>(p.gate);
  a.gate_kind = p.gate_kind;
  a.sigmoid = p.sigmoid;
  a.residual_scale = p.residual_scale;
  a.branch_scale = p.branch_scale;
  a.eps = p.eps;
  a.r = p.r;
  a.h = p.h;
  a.rstd_post = p.rstd_post;
  a.rstd_pre = p.rstd_pre;
  const Shape sh = make_shape(p.T, p.H, p.f32, n);
  const int64_t items = (sh.T + sh.teams - 1) / sh.teams;
  const int grid = (int)(items < num_sms ? items : num_sms);
  const size_t smem = ring_bytes(sh);
  auto run = [&](auto kern) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<grid, sh.teams * sh.warps * 32, smem, s>>>(a, sh);
    return cudaGetLastError();
  };
  // rows past 8192 columns need more than 512 threads, which halves the registers
  const bool small = sh.teams * sh.warps * 32 <= kTeamThreads;
  const bool col = p.gate_kind == kGateCol;
  using bf16 = __nv_bfloat16;
  if (p.f32)
    return small ? (col ? run(norm_fwd_kernel<float, kTeamThreads, true>)
                        : run(norm_fwd_kernel<float, kTeamThreads, false>))
                 : (col ? run(norm_fwd_kernel<float, 1024, true>)
                        : run(norm_fwd_kernel<float, 1024, false>));
  return small ? (col ? run(norm_fwd_kernel<bf16, kTeamThreads, true>)
                      : run(norm_fwd_kernel<bf16, kTeamThreads, false>))
               : (col ? run(norm_fwd_kernel<bf16, 1024, true>)
                      : run(norm_fwd_kernel<bf16, 1024, false>));
}

int fp8moe_norm_bwd_ctas(int64_t T) {
  // workspace bound: a CTA's column sums; the grid is one CTA per SM
  constexpr int kMost = 256;
  return (int)(T < kMost ? T : kMost);
}

cudaError_t fp8moe_launch_norm_bwd(const NormBwdArgs& p, int num_sms, cudaStream_t s) {
  using namespace fp8moe::norm;
  BwdArgs a = {};
  int n = 0;
  auto add = [&](const void* t) {
    if (!t) return -1;
    a.in.p[n] = static_cast<const uint8_t*>(t);
    return n++;
  };
  const bool post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  a.i_dr = add(p.dr);
  a.i_dh = add(p.dh);
  a.i_r = add(pre ? p.r : nullptr);
  a.i_y = add(p.y);
  a.i_gate = add(post && p.gate_kind == kGateFull ? p.gate : nullptr);
  a.w_post = p.w_post;
  a.w_pre = p.w_pre;
  a.rstd_post = p.rstd_post;
  a.rstd_pre = p.rstd_pre;
  a.gate = static_cast<const float*>(p.gate);
  a.gate_kind = p.gate_kind;
  a.sigmoid = p.sigmoid;
  a.residual_scale = p.residual_scale;
  a.branch_scale = p.branch_scale;
  a.dx = p.dx;
  a.dy = p.dy;
  a.dgate_row = p.gate_kind == kGateRow ? static_cast<float*>(p.dgate) : nullptr;
  a.dgate_full = p.gate_kind == kGateFull ? p.dgate : nullptr;
  a.part = p.part;
  const Shape sh = make_shape(p.T, p.H, p.f32, n);
  const int64_t items = (sh.T + sh.teams - 1) / sh.teams;
  int grid = (int)(items < num_sms ? items : num_sms);
  if (grid > fp8moe_norm_bwd_ctas(p.T)) grid = fp8moe_norm_bwd_ctas(p.T);
  if (grid > 0) {
    const size_t smem = ring_bytes(sh);
    auto run = [&](auto kern) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)smem);
      if (e != cudaSuccess) return e;
      kern<<<grid, sh.teams * sh.warps * 32, smem, s>>>(a, sh);
      return cudaGetLastError();
    };
    const bool small = sh.teams * sh.warps * 32 <= kTeamThreads;
    const bool col = p.gate_kind == kGateCol;
    using bf16 = __nv_bfloat16;
    cudaError_t e;
    if (p.f32)
      e = small ? (col ? run(norm_bwd_kernel<float, kTeamThreads, true>)
                       : run(norm_bwd_kernel<float, kTeamThreads, false>))
                : (col ? run(norm_bwd_kernel<float, 1024, true>)
                       : run(norm_bwd_kernel<float, 1024, false>));
    else
      e = small ? (col ? run(norm_bwd_kernel<bf16, kTeamThreads, true>)
                       : run(norm_bwd_kernel<bf16, kTeamThreads, false>))
                : (col ? run(norm_bwd_kernel<bf16, 1024, true>)
                       : run(norm_bwd_kernel<bf16, 1024, false>));
    if (e != cudaSuccess) return e;
  }
  const dim3 jg((unsigned)((p.H + kJoinCols - 1) / kJoinCols), 3, 1);
  norm_join_kernel<<<jg, kJoinCols * kJoinRows, 0, s>>>(
      p.part, grid, p.H, p.gate_kind == kGateCol ? a.gate : nullptr, p.sigmoid,
      pre ? p.dw_pre : nullptr, post ? p.dw_post : nullptr,
      p.gate_kind == kGateCol ? static_cast<float*>(p.dgate) : nullptr);
  return cudaGetLastError();
}
