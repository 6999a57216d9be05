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
// persistent CTA per SM streams rows through rings of shared-memory stages filled by
// bulk copies (one per tensor and row), which keeps 100 to 150 KB on their way without
// holding registers. A row belongs to a team of warps; short rows get several teams,
// each with a ring of its own and at its own pace. All sums and the column sums of the
// weight gradients are f32; the latter stay in registers over all rows of a CTA and are
// joined by a second small kernel in a fixed order, so results do not change from run
// to run. 4096 x 7168 bf16, a gate per token: forward 42 us (5.6 TB/s), backward with the
// join's 4 us 68 us (5.2 TB/s); what is left is the latency of a row's chain (copy,
// reduction, stores), which 14 to 16 warps do not hide completely.
#include <cstdint>
#include <initializer_list>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fp8moe_status.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "vec16.cuh"

namespace fp8moe {
namespace norm {

// A thread holds 16 columns of a row, a row of up to 8192 columns takes at most 512
// threads, whose 128 registers hold the weights and the column sums as well. Rows past
// that take up to 1024 threads, whose 64 registers do not. (8 columns a thread and
// twice the warps measured slower, 54 against 44 us forward and 110 against 96 us
// backward for 4096 x 7168 bf16: the reductions' share grows with the warps.)
constexpr int kCols = 16;
constexpr int kShort = 512, kLong = 1024;
constexpr int kRingBytes = 200 * 1024;
constexpr int kMaxStages = 4;       // of a team
constexpr int kMaxTeams = 16;
constexpr int kMaxTensors = 5;

enum { kGateNone = 0, kGateRow = 1, kGateCol = 2, kGateFull = 3 };

struct Shape {
  int64_t T;
  int H, nvec;
  int warps;       // of a team: one row per team
  int teams;       // of a CTA, each at its own pace
  int stages;      // rows that a team has in shared memory, in use or on their way
  int tensors;
  uint32_t row_bytes;
  bool is_long;
};

// The inputs of a row that are there, in order.
struct Loads {
  const uint8_t* p[kMaxTensors];
};

// exp(x), x = -|z|, within seven steps of 2^-24: for any h near x / (2 ln 2),
//   exp(x) = (2^h)^2 exp(r) = (2^h)^2 (1 + r),  r = x - h 2 ln 2  (under 1e-5: r^2 is nothing)
// with 2^h by the exponential unit (measured 2.4 steps) and r by two exact fused products.
// A plain fast exponential leaves r out and is off by 1.2 |z| units in the last place; the
// library's is exact to one, but its branches and registers cost 63.5 us where this takes 48
// (5003 x 1544 f32, a gate per element). The square keeps results below 2^-126 from being
// flushed. NaN stays NaN.
__device__ __forceinline__ float2 exp_minus_abs2(float2 z) {
  constexpr double kTwoLn2 = 1.3862943611198906;
  constexpr float kHi = (float)kTwoLn2, kLo = (float)(kTwoLn2 - (double)kHi);
  float2 x, e;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.x) : "f"(-fabsf(z.x)), "f"(-128.0f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.y) : "f"(-fabsf(z.y)), "f"(-128.0f));
  const float2 h = mul2(x, both((float)(1.0 / kTwoLn2)));
  const float2 r = fma2(h, both(-kLo), fma2(h, both(-kHi), x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(h.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(h.y));
  const float2 t = mul2(e, e);
  return fma2(t, r, t);
}

// 1 / (1 + t), t >= 0, within three steps of 2^-24.
__device__ __forceinline__ float2 one_over_one_plus2(float2 t) {
  const float2 s = add2(t, both(1.0f));
  float2 d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d.x) : "f"(s.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d.y) : "f"(s.y));
  return d;
}

// g = 1 / (1 + exp(-z)) and its slope g (1 - g) = exp(-z) g^2, which unlike that product does
// not cancel where g is near one; through t = exp(-|z|), nothing can overflow. FAST, for
// what is rounded to bf16 (what a gate per element or per channel makes of bf16 rows): the
// plain fast exponential, off by a hundredth of that rounding at most, and a quotient that
// is zero below 2^-126. (4096 x 7168 bf16, a gate per element: backward 108 us against 118.)
template <bool FAST>
__device__ __forceinline__ float2 sigmoid2(float2 z, float2& slope) {
  if (FAST) {
    constexpr float kLog2e = 1.4426950408889634f;
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(-z.x * kLog2e));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(-z.y * kLog2e));
    const float2 g = one_over_one_plus2(e);
    slope = mul2(mul2(make_float2(fminf(e.x, 1e38f), fminf(e.y, 1e38f)), g), g);
    return g;
  }
  const float2 t = exp_minus_abs2(z), d = one_over_one_plus2(t), td = mul2(t, d);
  slope = mul2(td, d);
  return make_float2(z.x >= 0.0f ? d.x : td.x, z.y >= 0.0f ? d.y : td.y);
}
template <bool FAST>
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  float2 slope;
  return sigmoid2<FAST>(z, slope);
}
__device__ __forceinline__ float sigmoid(float z, float& slope) {
  float2 slopes;
  const float g = sigmoid2<false>(both(z), slopes).x;
  slope = slopes.x;
  return g;
}
__device__ __forceinline__ float sigmoid(float z) { return sigmoid2<false>(both(z)).x; }

// A team's ring of rows in shared memory, by 32-bit shared addresses.
struct Ring {
  uint32_t base, row_bytes;
  uint64_t* full;
  int tensors;
  __device__ __forceinline__ Ring(const Shape& sh, const uint8_t* mem, uint64_t* bars, int team)
      : base(smem_u32(mem) + (uint32_t)(team * sh.stages * sh.tensors) * sh.row_bytes),
        row_bytes(sh.row_bytes), full(bars + team * kMaxStages), tensors(sh.tensors) {}
  __device__ __forceinline__ uint32_t at(int stage, int tensor) const {
    return base + (uint32_t)(stage * tensors + tensor) * row_bytes;
  }
  // one thread: row `row` into `stage`
  __device__ __forceinline__ void fill(const Loads& in, uint32_t row, int stage) const {
    mbar_arrive_expect_tx(&full[stage], row_bytes * tensors);
#pragma unroll
    for (int i = 0; i < kMaxTensors; ++i)
      if (i < tensors)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
            ::"r"(at(stage, i)), "l"(in.p[i] + (size_t)row * row_bytes), "r"(row_bytes),
              "r"(smem_u32(&full[stage])) : "memory");
  }
};

// What a thread knows of its ring, in one word: bit 0 the parity of its stage's barrier, above
// it the waits that have run out (each sets the status word). After the first of them the
// thread that fills the ring fetches no row any more, but goes on waiting, as every thread
// does until it has given up on as many as there are stages: so whatever was on its way to
// the ring has been waited for, with the same limit, before the CTA leaves its shared memory.
constexpr uint32_t kOneLost = 2, kAllLost = kOneLost * kMaxStages;

__device__ __forceinline__ void wait_row(const Ring& ring, int stage, uint32_t& state) {
  if (state < kAllLost && !mbar_wait(&ring.full[stage], state & 1, kWhereEpilogue)) state += kOneLost;
}

// Vector v of a row, zeros past its end.
__device__ __forceinline__ uint4 row_vec(uint32_t row, int v, bool in) {
  uint4 x = make_uint4(0, 0, 0, 0);
  if (in)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(row + 16u * (uint32_t)v));
  return x;
}

// Barrier of a team's warps.
__device__ __forceinline__ void team_sync(int team, int warps) {
  if (warps == 1) __syncwarp();
  else named_bar_sync(1 + team, warps * 32);
}

// Sums of NS values over a team's warps, for every thread of the team. The warps' sums
// lie in groups of four (zeros behind a team's last), `buf` alternates between two
// areas: a slow reader of one call's sums is past them before the call after the next
// writes there again.
constexpr int kRedTeam = 64;         // most words of all teams: teams * (warps rounded up to 4)
constexpr int kRedWords = 2 * 3 * kRedTeam;

template <int NS>
__device__ __forceinline__ void team_sum(float (&v)[NS], float* s_red, int buf, int slot, int first,
                                         int quads, int team, int warps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  float* const area = s_red + buf * (3 * kRedTeam);
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < NS; ++i) area[i * kRedTeam + slot] = v[i];
  }
  team_sync(team, warps);
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = 0.0f;
#pragma unroll 4
  for (int q = 0; q < quads; ++q)
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float4 p = reinterpret_cast<const float4*>(area + i * kRedTeam + first)[q];
      v[i] += (p.x + p.y) + (p.z + p.w);
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

// A norm's weight, times the block's gate where that is one per column: in registers for
// all rows of a thread (HOIST), or loaded for every row.
template <typename T, bool HOIST>
struct Param {
  static constexpr int P = Vec<T>::kP, NV = kCols / Vec<T>::kN;
  static constexpr bool FAST = Vec<T>::kN == 8;
  float2 v[HOIST ? NV : 1][P];
  const float* w;
  const float* g;      // null: no gate
  int sig, nvec;
  // zeros past the row
  __device__ __forceinline__ void load(int vec, float2 (&o)[P]) const {
#pragma unroll
    for (int k = 0; k < P; ++k) o[k] = both(0.0f);
    if (vec >= nvec) return;
    load_f32<P>(w + (size_t)vec * Vec<T>::kN, o);
    if (g) {
      float2 z[P];
      load_f32<P>(g + (size_t)vec * Vec<T>::kN, z);
#pragma unroll
      for (int k = 0; k < P; ++k) o[k] = mul2(o[k], sig ? sigmoid2<FAST>(z[k]) : z[k]);
    }
  }
  __device__ __forceinline__ void init(const float* weight, const float* gate, int sigmoid, int tt,
                                       int stride, int n) {
    w = weight;
    g = gate;
    sig = sigmoid;
    nvec = n;
    if (HOIST) {
#pragma unroll
      for (int i = 0; i < NV; ++i) load(tt + i * stride, v[HOIST ? i : 0]);
    }
  }
  __device__ __forceinline__ void get(int i, int vec, float2 (&o)[P]) const {
    if (HOIST) {
#pragma unroll
      for (int k = 0; k < P; ++k) o[k] = v[HOIST ? i : 0][k];
    } else {
      load(vec, o);
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

// What a kernel variant does: the norm after the block, the one before it, a gate value
// per element (the other gates are a factor of the row's or of the weight's).
// EXACT: a row is as long as its threads' 16 columns each, so no column is out of range
// (the common lengths, multiples of 512 up to 8192).
template <typename T, int MAXT, bool POST, bool PRE, bool FULL, bool EXACT>
__global__ void __launch_bounds__(MAXT, 1)
norm_fwd_kernel(const __grid_constant__ FwdArgs a, const __grid_constant__ Shape sh) {
  constexpr int P = Vec<T>::kP, NV = kCols / Vec<T>::kN;
  constexpr bool HOIST = MAXT == kShort, FAST = Vec<T>::kN == 8;
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ uint64_t s_full[kMaxTeams * kMaxStages];
  __shared__ __align__(16) float s_red[kRedWords];
  const int warp = threadIdx.x >> 5;
  const int team = warp / sh.warps;
  const Ring ring(sh, ring_mem, s_full, team);
  const int tt = threadIdx.x - team * sh.warps * 32, stride = sh.warps * 32;
  const int quads = (sh.warps + 3) / 4, first = team * quads * 4;
  const int slot = first + warp - team * sh.warps;
  // the team's first row, and on to its next (T < 2^31: the sums stay below 2^32)
  const uint32_t row0 = blockIdx.x * sh.teams + team, step = gridDim.x * sh.teams;
  const uint32_t rows = (uint32_t)sh.T;
  if (tt == 0) {
    for (int i = 0; i < sh.stages; ++i) mbar_init(&ring.full[i], 1);
    fence_mbar_init();
    for (int i = 0; i < sh.stages; ++i)
      if (row0 + i * step < rows) ring.fill(a.in, row0 + i * step, i);
  }
  for (int i = threadIdx.x; i < kRedWords; i += blockDim.x) s_red[i] = 0.0f;
  Param<T, HOIST> w_post, w_pre;
  if (POST)
    w_post.init(a.w_post, a.gate_kind == kGateCol ? a.gate : nullptr, a.sigmoid, tt, stride, sh.nvec);
  if (PRE) w_pre.init(a.w_pre, nullptr, 0, tt, stride, sh.nvec);
  __syncthreads();
  const float inv_h = 1.0f / (float)sh.H;
  int stage = 0, buf = 0;
  uint32_t state = 0;
  const bool row_gate = POST && a.gate_kind == kGateRow;
  float next_g = 1.0f;                     // the next item's gate, fetched an item ahead
  auto fetch = [&](uint32_t row) {
    if (row_gate && row < rows) next_g = __ldg(a.gate + row);
  };
  fetch(row0);
  for (uint32_t row = row0; row < rows; row += step) {
    float grow = next_g;
    if (row_gate && a.sigmoid) grow = sigmoid(grow);
    fetch(row + step);
    wait_row(ring, stage, state);
    const uint32_t xs = ring.at(stage, 0);
    const uint32_t ys = ring.at(stage, 1);
    const uint32_t gs = ring.at(stage, 2);
    float2 r[NV][P];
    float rp = 0.0f;
    if (POST) {
      float2 s2 = both(0.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tt + i * stride;
        Vec<T>::unpack(row_vec(ys, v, EXACT || v < sh.nvec), r[i]);
#pragma unroll
        for (int k = 0; k < P; ++k) s2 = fma2(r[i][k], r[i][k], s2);
      }
      float ss[1] = {s2.x + s2.y};
      team_sum<1>(ss, s_red, buf, slot, first, quads, team, sh.warps);
      buf ^= 1;
      rp = rsqrtf(fmaf(ss[0], inv_h, a.eps));
    }
    float2 s2 = both(0.0f);
    const float2 scale = both(a.branch_scale * grow * rp), rs = both(a.residual_scale);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tt + i * stride;
      const bool in = EXACT || v < sh.nvec;
      float2 x[P];
      Vec<T>::unpack(row_vec(xs, v, in), x);
      if (POST) {
        float2 w[P], g[P];
        w_post.get(i, v, w);
        if (FULL) Vec<T>::unpack(row_vec(gs, v, in), g);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          float2 b = mul2(r[i][k], w[k]);
          if (FULL) b = mul2(b, a.sigmoid ? sigmoid2<FAST>(g[k]) : g[k]);
          r[i][k] = fma2(b, scale, mul2(rs, x[k]));
        }
        if (in) reinterpret_cast<uint4*>(a.r)[(size_t)row * sh.nvec + v] = Vec<T>::pack(r[i]);
      } else {
#pragma unroll
        for (int k = 0; k < P; ++k) r[i][k] = x[k];
      }
      // columns past the row are zeros, so they add nothing
#pragma unroll
      for (int k = 0; k < P; ++k) s2 = fma2(r[i][k], r[i][k], s2);
    }
    if (POST && tt == 0) a.rstd_post[row] = rp;
    float ss[1] = {s2.x + s2.y};
    if (PRE) {
      team_sum<1>(ss, s_red, buf, slot, first, quads, team, sh.warps);
      buf ^= 1;
    } else {
      team_sync(team, sh.warps);
    }
    // past that barrier every thread has read the stage
    if (tt == 0 && state < kOneLost && row + sh.stages * step < rows) ring.fill(a.in, row + sh.stages * step, stage);
    if (PRE) {
      const float rq = rsqrtf(fmaf(ss[0], inv_h, a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tt + i * stride;
        float2 w[P], h[P];
        w_pre.get(i, v, w);
#pragma unroll
        for (int k = 0; k < P; ++k) h[k] = mul2(mul2(r[i][k], both(rq)), w[k]);
        if (EXACT || v < sh.nvec) reinterpret_cast<uint4*>(a.h)[(size_t)row * sh.nvec + v] = Vec<T>::pack(h);
      }
      if (tt == 0) a.rstd_pre[row] = rq;
    }
    if (++stage == sh.stages) {
      stage = 0;
      state ^= 1;
    }
  }
}

struct BwdArgs {
  Loads in;                    // dr, dh, r, y, gate (each only if it is there)
  int i_dr, i_dh, i_y;         // places in a stage (-1: absent); r follows dh, the gate y
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
  float* part;                 // [2][gridDim.x][H]: the sums of dh rh, and of b D g yh (g without a
                               // gate per column)
};

template <typename T, int MAXT, bool POST, bool PRE, bool FULL, bool EXACT>
__global__ void __launch_bounds__(MAXT, 1)
norm_bwd_kernel(const __grid_constant__ BwdArgs a, const __grid_constant__ Shape sh) {
  constexpr int N = Vec<T>::kN, P = Vec<T>::kP, NV = kCols / N;
  constexpr bool HOIST = MAXT == kShort, FAST = Vec<T>::kN == 8;
  extern __shared__ __align__(128) uint8_t ring_mem[];
  __shared__ uint64_t s_full[kMaxTeams * kMaxStages];
  __shared__ __align__(16) float s_red[kRedWords];
  const int warp = threadIdx.x >> 5;
  const int team = warp / sh.warps;
  const Ring ring(sh, ring_mem, s_full, team);
  const int tt = threadIdx.x - team * sh.warps * 32, stride = sh.warps * 32;
  const int quads = (sh.warps + 3) / 4, first = team * quads * 4;
  const int slot = first + warp - team * sh.warps;
  // the team's first row, and on to its next (T < 2^31: the sums stay below 2^32)
  const uint32_t row0 = blockIdx.x * sh.teams + team, step = gridDim.x * sh.teams;
  const uint32_t rows = (uint32_t)sh.T;
  pdl_launch_dependents();
  if (tt == 0) {
    for (int i = 0; i < sh.stages; ++i) mbar_init(&ring.full[i], 1);
    fence_mbar_init();
    for (int i = 0; i < sh.stages; ++i)
      if (row0 + i * step < rows) ring.fill(a.in, row0 + i * step, i);
  }
  for (int i = threadIdx.x; i < kRedWords; i += blockDim.x) s_red[i] = 0.0f;
  Param<T, HOIST> w_post, w_pre;
  if (POST)
    w_post.init(a.w_post, a.gate_kind == kGateCol ? a.gate : nullptr, a.sigmoid, tt, stride, sh.nvec);
  if (PRE) w_pre.init(a.w_pre, nullptr, 0, tt, stride, sh.nvec);
  __syncthreads();
  const float inv_h = 1.0f / (float)sh.H;
  const bool row_gate = POST && a.gate_kind == kGateRow;
  float2 acc_pre[PRE ? NV : 1][P], acc_post[POST ? NV : 1][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) acc_pre[PRE ? i : 0][k] = acc_post[POST ? i : 0][k] = both(0.0f);
  float next_p = 0.0f, next_q = 0.0f, next_g = 1.0f;   // the next item's, fetched an item ahead
  auto fetch = [&](uint32_t row) {
    if (row < rows) {
      if (POST) next_p = __ldg(a.rstd_post + row);
      if (PRE) next_q = __ldg(a.rstd_pre + row);
      if (row_gate) next_g = __ldg(a.gate + row);
    }
  };
  fetch(row0);
  int stage = 0, buf = 0;
  uint32_t state = 0;
  for (uint32_t row = row0; row < rows; row += step) {
    const float rp = next_p, rq = next_q;
    float grow = next_g, slope_row = 1.0f;
    fetch(row + step);
    wait_row(ring, stage, state);
    const uint32_t drs = ring.at(stage, 0);
    const uint32_t dhs = ring.at(stage, PRE ? a.i_dh : 0);
    const uint32_t rs = ring.at(stage, PRE ? a.i_dh + 1 : 0);
    const uint32_t ys = ring.at(stage, POST ? a.i_y : 0);
    const uint32_t gs = ring.at(stage, FULL ? a.i_y + 1 : 0);
    // With u = w_pre dh and p = w_post y (times a gate per column or element):
    // sum u r, sum p (dr + rq u), sum p r. The row's factors come in afterwards.
    float2 s0 = both(0.0f), s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tt + i * stride;
      const bool in = EXACT || v < sh.nvec;
      float2 d[P], r[P], w[P];
      Vec<T>::unpack(row_vec(drs, v, in && a.i_dr >= 0), d);
      if (PRE) {
        float2 u[P];
        Vec<T>::unpack(row_vec(dhs, v, in), u);
        Vec<T>::unpack(row_vec(rs, v, in), r);
        w_pre.get(i, v, w);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          u[k] = mul2(u[k], w[k]);
          s0 = fma2(u[k], r[k], s0);
          d[k] = fma2(both(rq), u[k], d[k]);
        }
      }
      if (POST) {
        float2 y[P];
        Vec<T>::unpack(row_vec(ys, v, in), y);
        w_post.get(i, v, w);
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] = mul2(y[k], w[k]);
        if (FULL) {
          float2 g[P];
          Vec<T>::unpack(row_vec(gs, v, in), g);
#pragma unroll
          for (int k = 0; k < P; ++k) y[k] = mul2(y[k], a.sigmoid ? sigmoid2<FAST>(g[k]) : g[k]);
        }
#pragma unroll
        for (int k = 0; k < P; ++k) {
          s1 = fma2(y[k], d[k], s1);
          if (PRE) s2 = fma2(y[k], r[k], s2);
        }
      }
    }
    float s3[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
    if (row_gate && a.sigmoid) grow = sigmoid(grow, slope_row);
    team_sum<3>(s3, s_red, buf, slot, first, quads, team, sh.warps);
    buf ^= 1;
    // Past this barrier every thread has finished with the stage of the row before.
    if (tt == 0 && state < kOneLost && sh.stages > 2 && row != row0 &&
        row + (sh.stages - 1) * step < rows)
      ring.fill(a.in, row + (sh.stages - 1) * step, stage == 0 ? sh.stages - 1 : stage - 1);
    // D = dr + rq u - k1 rh;  dn = bg g D;  dy = k2 (w_post g D) - k3 yh. No factor is a higher
    // power of rstd than the result: rows of 1e15, or of 1e-15, keep their precision.
    const float k1 = rq * (rq * s3[0] * inv_h);
    const float qd = a.branch_scale * rp * (s3[1] - k1 * (rq * s3[2]));   // sum q D without the row's gate
    const float bg = a.branch_scale * grow, k2 = bg * rp;
    const float k3 = rp * (grow * qd * inv_h);
    if (row_gate && tt == 0) a.dgate_row[row] = qd * slope_row;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tt + i * stride;
      const bool in = EXACT || v < sh.nvec;
      float2 d[P], o[P], w[P];
      Vec<T>::unpack(row_vec(drs, v, in && a.i_dr >= 0), d);
      if (PRE) {
        float2 dh[P], r[P];
        Vec<T>::unpack(row_vec(dhs, v, in), dh);
        Vec<T>::unpack(row_vec(rs, v, in), r);
        w_pre.get(i, v, w);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          r[k] = mul2(r[k], both(rq));
          d[k] = fma2(r[k], both(-k1), fma2(both(rq), mul2(dh[k], w[k]), d[k]));
          acc_pre[PRE ? i : 0][k] = fma2(dh[k], r[k], acc_pre[PRE ? i : 0][k]);
        }
      }
#pragma unroll
      for (int k = 0; k < P; ++k) o[k] = mul2(both(a.residual_scale), d[k]);
      if (in) reinterpret_cast<uint4*>(a.dx)[(size_t)row * sh.nvec + v] = Vec<T>::pack(o);
      if (POST) {
        float2 y[P], g[P];
        Vec<T>::unpack(row_vec(ys, v, in), y);
        w_post.get(i, v, w);
        if (FULL) Vec<T>::unpack(row_vec(gs, v, in), g);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          y[k] = mul2(y[k], both(rp));
          float2 dy = mul2(d[k], y[k]), wd = mul2(w[k], d[k]);
          if (FULL) {
            float2 slope = both(1.0f);
            const float2 s = a.sigmoid ? sigmoid2<FAST>(g[k], slope) : g[k];
            g[k] = mul2(mul2(mul2(dy, w[k]), both(bg)), slope);
            dy = mul2(dy, s);
            wd = mul2(wd, s);
          }
          acc_post[POST ? i : 0][k] = fma2(dy, both(bg), acc_post[POST ? i : 0][k]);
          o[k] = fma2(wd, both(k2), mul2(y[k], both(-k3)));
        }
        if (in) reinterpret_cast<uint4*>(a.dy)[(size_t)row * sh.nvec + v] = Vec<T>::pack(o);
        if (FULL && in) reinterpret_cast<uint4*>(a.dgate_full)[(size_t)row * sh.nvec + v] = Vec<T>::pack(g);
      }
    }
    if (sh.stages <= 2) {      // long rows: a stage is too dear to wait for the next barrier
      team_sync(team, sh.warps);
      if (tt == 0 && state < kOneLost && row + sh.stages * step < rows) ring.fill(a.in, row + sh.stages * step, stage);
    }
    if (++stage == sh.stages) {
      stage = 0;
      state ^= 1;
    }
  }
  // the column sums of this CTA: its teams' are joined in shared memory (the ring
  // is idle: every stage that was filled has been read)
  auto join = [&](const auto& acc, int which) {
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
  if constexpr (PRE) join(acc_pre, 0);
  if constexpr (POST) join(acc_post, 1);
}

// Joins the CTAs' column sums: 16 threads per column take every 16th CTA. A gate per
// column shares its sum with the weight: with S = sum b D yh, dw_post = g S and
// dgate = w_post S (times g (1 - g) behind a sigmoid).
constexpr int kJoinCols = 32, kJoinRows = 16;

__global__ void __launch_bounds__(kJoinCols * kJoinRows)
norm_join_kernel(const float* __restrict__ part, int ctas, int H, const float* __restrict__ gate,
                 const float* __restrict__ w_post, int sigmoid_gate, float* __restrict__ dw_pre,
                 float* __restrict__ dw_post, float* __restrict__ dgate) {
  __shared__ float s[kJoinRows][kJoinCols + 1];
  if (!(blockIdx.y == 0 ? dw_pre : dw_post)) return;
  const int cx = threadIdx.x % kJoinCols, ry = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + cx;
  const float* p = part + (size_t)blockIdx.y * ctas * H;
  pdl_wait();          // the sums are the backward kernel's
  float sum = 0.0f;
  if (c < H) {
    // plain loads: the kernel that writes them may still run when this one starts
#pragma unroll 4
    for (int i = ry; i < ctas; i += kJoinRows)
      sum += *static_cast<const volatile float*>(p + (size_t)i * H + c);
  }
  s[ry][cx] = sum;
  __syncthreads();
  if (ry != 0 || c >= H) return;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinRows; ++i) t += s[i][cx];
  if (blockIdx.y == 0) {
    dw_pre[c] = t;
  } else if (gate) {
    float slope = 1.0f;
    const float z = __ldg(gate + c), g = sigmoid_gate ? sigmoid(z, slope) : z;
    dw_post[c] = t * g;
    dgate[c] = t * __ldg(w_post + c) * slope;
  } else {
    dw_post[c] = t;
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
  s.is_long = s.warps * 32 > kShort;
  // rows that fit into shared memory: two at least for a team if there is more than one
  const int64_t rows = kRingBytes / ((int64_t)s.row_bytes * tensors);
  s.teams = s.is_long ? 1 : kShort / (32 * s.warps);
  if (s.teams > rows / 2) s.teams = rows < 4 ? 1 : (int)(rows / 2);
  s.tensors = tensors;
  s.stages = (int)(rows / s.teams);
  if (s.stages > kMaxStages) s.stages = kMaxStages;
  return s;      // H * element size <= 32768 leaves at least one stage
}

// A kernel variant as a type, and the choice of one.
template <typename TT, int MAXT, bool POST, bool PRE, bool FULL, bool EXACT>
struct Variant {
  using T = TT;
  static constexpr int kMaxT = MAXT;
  static constexpr bool kPost = POST, kPre = PRE, kFull = FULL, kExact = EXACT;
};
template <typename T, int MAXT, bool EXACT, typename F>
cudaError_t pick_parts(bool post, bool pre, int gate, F f) {
  if (!post) return f(Variant<T, MAXT, false, true, false, EXACT>());
  if (gate == kGateFull)
    return pre ? f(Variant<T, MAXT, true, true, true, EXACT>())
               : f(Variant<T, MAXT, true, false, true, EXACT>());
  return pre ? f(Variant<T, MAXT, true, true, false, EXACT>())
             : f(Variant<T, MAXT, true, false, false, EXACT>());
}
template <typename T, typename F>
cudaError_t pick_length(const Shape& sh, bool post, bool pre, int gate, F f) {
  // rows of at most 32768 bytes: only bf16 ones are longer than kShort threads' columns
  if constexpr (32768 / sizeof(T) > kShort * kCols)
    if (sh.is_long) return pick_parts<T, kLong, false>(post, pre, gate, f);
  const bool exact = sh.nvec * Vec<T>::kN == sh.warps * 32 * kCols;
  return exact ? pick_parts<T, kShort, true>(post, pre, gate, f)
               : pick_parts<T, kShort, false>(post, pre, gate, f);
}
template <typename F>
cudaError_t pick_norm(bool f32, const Shape& sh, bool post, bool pre, int gate, F f) {
  return f32 ? pick_length<float>(sh, post, pre, gate, f)
             : pick_length<__nv_bfloat16>(sh, post, pre, gate, f);
}

size_t ring_bytes(const Shape& s) {
  size_t b = (size_t)s.stages * s.tensors * s.teams * s.row_bytes;
  const size_t join = (size_t)s.teams * s.H * sizeof(float);
  return b > join ? b : join;
}

// The same limit for every call: another thread's call or a captured graph of the same
// kernel may need more than this one does. (A join takes at most 64 KB.)
template <typename K>
cudaError_t allow_ring(K kern) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
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
  const bool post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  const size_t smem = ring_bytes(sh);
  auto run = [&](auto kern) {
    cudaError_t e = allow_ring(kern);
    if (e != cudaSuccess) return e;
    kern<<<grid, sh.teams * sh.warps * 32, smem, s>>>(a, sh);
    return cudaGetLastError();
  };
  return pick_norm(p.f32, sh, post, pre, p.gate_kind, [&](auto v) {
    using V = decltype(v);
    return run(norm_fwd_kernel<typename V::T, V::kMaxT, V::kPost, V::kPre, V::kFull, V::kExact>);
  });
}

int fp8moe_norm_bwd_ctas(int64_t T) {
  // workspace bound: a CTA's column sums; the grid is one CTA per SM
  constexpr int kMost = 256;
  return (int)(T < kMost ? T : kMost);
}

cudaError_t fp8moe_launch_norm_bwd(const NormBwdArgs& p, int num_sms, cudaStream_t s) {
  using namespace fp8moe::norm;
  if (p.T == 0) {
    // No rows: no kernel shape either (empty tensors have no address, so nothing to stream).
    // Sums over nothing are zeros, whatever the weights and the gate hold.
    for (float* sum : {p.w_pre ? p.dw_pre : nullptr, p.w_post ? p.dw_post : nullptr,
                       p.gate_kind == kGateCol ? static_cast<float*>(p.dgate) : nullptr}) {
      const cudaError_t e = sum ? cudaMemsetAsync(sum, 0, (size_t)p.H * sizeof(float), s) : cudaSuccess;
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
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
  add(pre ? p.r : nullptr);
  a.i_y = add(p.y);
  add(post && p.gate_kind == kGateFull ? p.gate : nullptr);
  a.w_post = p.w_post;
  a.w_pre = p.w_pre;
  a.rstd_post = p.rstd_post;
  a.rstd_pre = p.rstd_pre;
  a.gate = static_cast<const float*>(p.gate);
  a.gate_kind = p.gate_kind;
  a.sigmoid = p.sigmoid;
  a.residual_scale = post ? p.residual_scale : 1.0f;
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
  const size_t smem = ring_bytes(sh);
  auto run = [&](auto kern) {
    cudaError_t e = allow_ring(kern);
    if (e != cudaSuccess) return e;
    kern<<<grid, sh.teams * sh.warps * 32, smem, s>>>(a, sh);
    return cudaGetLastError();
  };
  cudaError_t e = pick_norm(p.f32, sh, post, pre, p.gate_kind, [&](auto v) {
    using V = decltype(v);
    return run(norm_bwd_kernel<typename V::T, V::kMaxT, V::kPost, V::kPre, V::kFull, V::kExact>);
  });
  if (e != cudaSuccess) return e;
  const dim3 jg((unsigned)((p.H + kJoinCols - 1) / kJoinCols), 2, 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = jg;
  cfg.blockDim = dim3(kJoinCols * kJoinRows, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  fp8moe::pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(
      &cfg, norm_join_kernel, static_cast<const float*>(p.part), grid, p.H,
      p.gate_kind == kGateCol ? a.gate : nullptr, p.w_post, p.sigmoid, pre ? p.dw_pre : nullptr,
      post ? p.dw_post : nullptr,
      p.gate_kind == kGateCol ? static_cast<float*>(p.dgate) : nullptr);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}
