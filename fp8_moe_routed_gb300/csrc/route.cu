// route.cu -- tokens sorted by expert and back: the stable counting sort of the
// router's choices, the copy of each token to its rows (dispatch), the weighted
// sum of a token's rows (combine), and their gradients.
//
// A slot s = t * topk + j is token t's j-th choice. With key(s) its expert id
// (a slot whose id is outside [0, E) has no row):
//   row(s) = #{s': key(s') < key(s)} + #{s' < s: key(s') = key(s)},  dropped if >= M
//   rows[row(t, j)]  = x[t]                                   (dispatch)
//   out[t]           = sum_j w[t, j] * rows[row(t, j)]        (combine; w = 1: dispatch's gradient)
//   drows[row(t, j)] = w[t, j] * dout[t],  dw[t, j] = <dout[t], rows[row(t, j)]>
// Everything but the sort is bound by HBM: each kernel reads and writes every row
// once. Work is laid out by token, so a token's vector is read once for its topk
// rows, and no two threads ever write (or add to) the same element of a row: the sums
// run in the order of j and the results do not depend on scheduling. (4096 tokens, top-8,
// H = 7168 bf16: dispatch 85 us = 6.2 TB/s, combine's gradient 153 us = 6.5 TB/s,
// dispatch's 77 us = 6.9 TB/s.)
#include <cstdint>
#include <type_traits>
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "fp8moe_status.cuh"
#include "groups.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "vec16.cuh"

namespace cg = cooperative_groups;

namespace fp8moe {
namespace route {

__device__ __forceinline__ int warp_incl_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// ------------------------------------------------------------------------ sort
// One cluster of kSortCtas CTAs (one CTA when there are few slots). The slots are
// cut into one contiguous run per warp. First pass: every warp counts its run per
// expert in its own shared-memory counters, 32 slots at a time (votes on the keys' bits
// give the lanes that share an expert, their lowest lane adds their number). Then each
// counter becomes the first row of that (warp, expert): an exclusive scan over the
// warps of a CTA, over the CTAs (their totals read through distributed shared
// memory) and over the experts. Second pass: a slot's row is its warp's counter
// plus the number of lower lanes with the same expert. Bound by latency and by the
// passes' issue rate on eight SMs: 8.2 us for 32768 slots; the dispatch that follows moves
// H / 2 times the bytes.
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortHeld = 8;      // batches of a warp kept in registers between the passes

__global__ void __launch_bounds__(kSortThreads, 1)
sort_kernel(const int32_t* __restrict__ ids, uint32_t n, int E, int32_t M,
            int32_t* __restrict__ group_sizes, int32_t* __restrict__ slot_row,
            int32_t* __restrict__ row_slot) {
  extern __shared__ int32_t sm[];
  int32_t* const counts = sm;                           // [kSortWarps][E]
  int32_t* const cta_total = sm + (size_t)kSortWarps * E;   // [E], read by the other CTAs
  __shared__ int32_t s_warp[kSortWarps];
  __shared__ int32_t s_base[kMaxExperts];    // first row of this CTA's slots of an expert
  __shared__ int64_t s_rows;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) counts[i] = 0;
  __syncthreads();

  // (n < 2^31: slots and batches past the end stay below 2^32)
  const uint32_t batches = (n + 31) / 32;
  const uint32_t per = (batches + ctas * kSortWarps - 1) / (ctas * kSortWarps);
  const uint32_t b0 = (rank * kSortWarps + warp) * per;
  const uint32_t b1 = min(b0 + per, batches);
  int32_t* const mine = counts + (size_t)warp * E;
  const int bits = 32 - __clz(E - 1);        // of a key; 0 for one expert
  bool bad = false;
  auto fetch = [&](uint32_t b) -> int32_t {
    const uint32_t s = b * 32 + lane;
    const int32_t e = b < b1 && s < n ? __ldg(ids + s) : -1;
    bad |= e >= E;
    return e >= 0 && e < E ? e : -1;
  };
  // key, the lower lanes with the same one and, for the lowest of them, their number: a
  // vote per bit of the key (match_any takes a step per different key, 45 cycles a batch
  // on an SM, and twice as long in all)
  auto ranked = [&](int32_t key) -> int32_t {
    uint32_t same = __ballot_sync(0xffffffffu, key >= 0);
    for (int i = 0; i < bits; ++i) {
      const bool one = (key >> i) & 1;
      const uint32_t ones = __ballot_sync(0xffffffffu, one);
      same &= one ? ones : ~ones;
    }
    if (key < 0) return -1;
    const int below = __popc(same & ((1u << lane) - 1u));
    return key | below << 10 | (below ? 0 : __popc(same)) << 15;
  };
  auto advance = [&](int32_t packed) {
    if (packed >= 0 && packed >> 15) mine[packed & 1023] += packed >> 15;
    __syncwarp();
  };
  int32_t held[kSortHeld];       // of the first batches, all loads in flight at once
#pragma unroll
  for (int i = 0; i < kSortHeld; ++i) held[i] = fetch(b0 + i);
#pragma unroll
  for (int i = 0; i < kSortHeld; ++i)
    if (b0 + i < b1) advance(held[i] = ranked(held[i]));
  for (uint32_t b = b0 + kSortHeld; b < b1; ++b) advance(ranked(fetch(b)));
  __syncthreads();
  // thread e: exclusive scan of expert e over this CTA's warps
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int32_t run = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t c = counts[(size_t)w * E + e];
      counts[(size_t)w * E + e] = run;
      run += c;
    }
    cta_total[e] = run;
  }
  cluster.sync();
  // experts: E <= 1024 = one per thread
  {
    const int e = threadIdx.x;
    int32_t before = 0, total = 0;
    if (e < E) {
      for (int c = 0; c < ctas; ++c) {
        const int32_t v = cluster.map_shared_rank(cta_total, c)[e];
        if (c < rank) before += v;
        total += v;
      }
    }
    const int32_t incl = warp_incl_scan(total, lane);
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int32_t base = 0;
    for (int w = 0; w < warp; ++w) base += s_warp[w];
    const int32_t start = base + incl - total;
    if (e < E) {
      s_base[e] = start + before;
      if (rank == 0) {
        const int64_t lo = start < M ? start : M;
        const int64_t hi = (int64_t)start + total < M ? (int64_t)start + total : M;
        group_sizes[e] = (int32_t)(hi - lo);
      }
    }
    if (threadIdx.x == kSortThreads - 1) {
      s_rows = (int64_t)base + incl;
      if (rank == 0 && s_rows > M) status_set(kStatusGroupsExceedM);
    }
  }
  __syncthreads();
  auto place = [&](uint32_t b, int32_t packed) {
    const uint32_t s = b * 32 + lane;
    int32_t row = -1;
    if (packed >= 0) {
      const int key = packed & 1023;
      row = s_base[key] + mine[key] + (packed >> 10 & 31);
    }
    __syncwarp();
    advance(packed);
    if (row >= M) row = -1;
    if (s < n) {
      slot_row[s] = row;
      if (row >= 0 && row_slot) row_slot[row] = (int32_t)s;
    }
  };
#pragma unroll
  for (int i = 0; i < kSortHeld; ++i)
    if (b0 + i < b1) place(b0 + i, held[i]);
  for (uint32_t b = b0 + kSortHeld; b < b1; ++b) place(b, ranked(fetch(b)));
  if (row_slot) {
    for (int64_t r = s_rows + (int64_t)rank * kSortThreads + threadIdx.x; r < M;
         r += (int64_t)ctas * kSortThreads)
      row_slot[r] = -1;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) status_set(kStatusBadExpert);
  cluster.sync();   // no CTA leaves while another may still read its totals
}

// The row of a slot, -1 for none. A caller's entry past the buffer (a slot_row
// made for a larger one) counts as none: it is never followed out of bounds.
__device__ __forceinline__ int32_t row_of(const int32_t* slot_row, int64_t s, int64_t M) {
  const int32_t r = __ldg(slot_row + s);
  return r < M ? r : -1;
}

// -------------------------------------------------------------------- dispatch
// A warp moves 128 16-byte vectors of one token: four loads in flight per lane,
// then the stores to each of the token's rows (512 contiguous bytes per store).
constexpr int kMoveVecs = 4;
constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads)
dispatch_kernel(const uint4* __restrict__ x, int64_t T, int topk, int nvec, int chunks,
                const int32_t* __restrict__ slot_row, int64_t M, uint4* __restrict__ rows) {
  const int lane = threadIdx.x & 31;
  const int64_t items = T * chunks;
  const int64_t step = (int64_t)gridDim.x * (kMoveThreads / 32);
  for (int64_t it = (int64_t)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); it < items;
       it += step) {
    const int64_t t = it / chunks;
    const int v0 = (int)(it - t * chunks) * (32 * kMoveVecs) + lane;
    uint4 v[kMoveVecs];
#pragma unroll
    for (int i = 0; i < kMoveVecs; ++i)
      if (v0 + 32 * i < nvec) v[i] = __ldg(x + t * nvec + v0 + 32 * i);
    pdl_wait();            // the row numbers are the sort's
    // (not by row_of: its load may use a cache that does not see a kernel still running)
    int32_t r = lane < topk ? __ldcg(slot_row + t * topk + lane) : -1;
    if (r >= M) r = -1;
    for (int j = 0; j < topk; ++j) {
      const int32_t row = __shfl_sync(0xffffffffu, r, j);
      if (row < 0) continue;
      uint4* d = rows + (int64_t)row * nvec + v0;
#pragma unroll
      for (int i = 0; i < kMoveVecs; ++i)
        if (v0 + 32 * i < nvec) d[32 * i] = v[i];
    }
  }
}

// --------------------------------------------------------- dispatch of few slots
// Up to 1024 slots sort and copy in one launch: every CTA holds all keys in shared
// memory and counts the rows of its own token's slots, row(s) = #{key < key(s)} +
// #{s' < s: key = key(s)}, a warp per slot, 32 keys at a time. A CTA copies 256 vectors
// of one token; the first of a token also writes its row numbers, one more CTA the group
// sizes and the empty tail of row_slot. (One token to eight experts: 4 us against 10 us
// for the two launches.)
constexpr int kFewSlots = 1024;

__global__ void __launch_bounds__(kMoveThreads)
dispatch_few_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ ids, int T, int topk,
                    int E, int64_t M, int nvec, int chunks, uint4* __restrict__ rows,
                    int32_t* __restrict__ group_sizes, int32_t* __restrict__ slot_row,
                    int32_t* __restrict__ row_slot) {
  __shared__ int32_t s_key[kFewSlots];
  __shared__ int32_t s_row[32];
  __shared__ int32_t s_count[kMaxExperts];
  const int n = T * topk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / chunks, chunk = blockIdx.x - t * chunks;
  const int vec = chunk * kMoveThreads + threadIdx.x;
  const bool copies = t < T && vec < nvec;
  uint4 v;
  if (copies) v = __ldg(x + (int64_t)t * nvec + vec);
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += kMoveThreads) {
    const int32_t e = __ldg(ids + i);
    bad |= e >= E;
    s_key[i] = e >= 0 && e < E ? e : E;
  }
  if (t < T) {
    __syncthreads();
    for (int j = warp; j < topk; j += kMoveThreads / 32) {
      const int s = t * topk + j, key = s_key[s];
      int before = 0;
      for (int i = lane; i < n; i += 32) before += s_key[i] < key || (s_key[i] == key && i < s);
      int row = __reduce_add_sync(0xffffffffu, before);
      if (key == E || row >= M) row = -1;
      if (lane == 0) {
        s_row[j] = row;
        if (chunk == 0) {
          slot_row[s] = row;
          if (row >= 0 && row_slot) row_slot[row] = s;
        }
      }
    }
    __syncthreads();
    if (!copies) return;
    for (int j = 0; j < topk; ++j)
      if (s_row[j] >= 0) rows[(int64_t)s_row[j] * nvec + vec] = v;
    return;
  }
  for (int e = threadIdx.x; e < E; e += kMoveThreads) s_count[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kMoveThreads)
    if (s_key[i] < E) atomicAdd(&s_count[s_key[i]], 1);
  const bool any_bad = __syncthreads_or(bad);
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + lane;
      const int c = e < E ? s_count[e] : 0;
      const int incl = warp_incl_scan(c, lane);
      const int64_t lo = carry + incl - c, hi = carry + incl;
      if (e < E) group_sizes[e] = (int32_t)((hi < M ? hi : M) - (lo < M ? lo : M));
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      s_row[0] = carry;
      if (carry > M) status_set(kStatusGroupsExceedM);
      if (any_bad) status_set(kStatusBadExpert);
    }
  }
  __syncthreads();
  if (row_slot)
    for (int64_t r = s_row[0] + (int64_t)threadIdx.x; r < M; r += kMoveThreads) row_slot[r] = -1;
}

// --------------------------------------------------------------------- combine
// A CTA sums one token's rows (several tokens' when rows are short), a thread 16 bytes at
// a time with up to eight row loads in flight; four CTAs of 256 threads on an SM keep
// 128 KB in flight, and the token's row numbers are read once. A slot without a row adds
// nothing: neither its vector nor its weight is read (zeros stand for them), so what lies
// there, or a NaN weight, cannot reach the sum. Bound by HBM: 4093 x 8 x 4096 bf16 with a
// quarter of the slots dropped 37 us = 6.3 TB/s. (Warps that walked 512-byte pieces of
// all tokens waited for row numbers and rows in turn: 72 us; weights read beside their
// row's sum, which is skipped without a row: 42.6, two waits where one does; 128 or 512
// threads a CTA measured the same or slower.)

// BATCH row loads in flight (the rows of up to four or eight choices at once); SHORT: rows
// of at most 128 vectors, per_token threads each, else a token has the whole CTA.
template <typename T, bool WEIGHTED, int BATCH, bool SHORT>
__global__ void __launch_bounds__(kMoveThreads, 4)
combine_kernel(const uint4* __restrict__ rows, int64_t tokens, int topk, int nvec, int per_token,
               const int32_t* __restrict__ slot_row, int64_t M, const float* __restrict__ weights,
               uint4* __restrict__ out) {
  constexpr int P = Vec<T>::kP;
  int64_t t = blockIdx.x;
  int v = threadIdx.x, step = blockDim.x;
  if (SHORT) {
    const int group = threadIdx.x / per_token;
    t = t * (kMoveThreads / per_token) + group;
    v -= group * per_token;
    step = per_token;
    if (t >= tokens) return;
  }
  const int32_t* const sr = slot_row + t * topk;
  for (; v < nvec; v += step) {
    float2 acc[P];
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i] = both(0.0f);
    for (int j0 = 0; j0 < topk; j0 += BATCH) {
      uint4 x[BATCH];
      float w[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const int32_t row = j0 + j < topk ? row_of(sr, j0 + j, M) : -1;
        x[j] = make_uint4(0, 0, 0, 0);
        w[j] = 0.0f;
        if (row >= 0) {
          if (WEIGHTED) w[j] = __ldg(weights + t * topk + j0 + j);
          x[j] = __ldg(rows + (int64_t)row * nvec + v);
        }
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        float2 f[P];
        Vec<T>::unpack(x[j], f);
#pragma unroll
        for (int i = 0; i < P; ++i)
          acc[i] = WEIGHTED ? fma2(both(w[j]), f[i], acc[i]) : add2(acc[i], f[i]);
      }
    }
    out[t * nvec + v] = Vec<T>::pack(acc);
  }
}

// ---------------------------------------------------------- combine's gradient
// A CTA takes a token (several when rows are short): every thread walks its share of the
// token's vectors, reads
// dout once and each row once (BATCH at a time), writes the row's gradient and
// keeps the partial dot products; one reduction per BATCH rows ends it.
constexpr int kBwdThreads = 256;

template <typename T, int BATCH>
__global__ void __launch_bounds__(kBwdThreads, BATCH == 8 ? 2 : 4)
combine_bwd_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ rows, int64_t tokens,
                   int topk, int nvec, int per_token, const int32_t* __restrict__ slot_row, int64_t M,
                   const float* __restrict__ weights, uint4* __restrict__ drows,
                   float* __restrict__ dweights) {
  constexpr int P = Vec<T>::kP;
  __shared__ float s_part[kBwdThreads / 32][BATCH];
  const int group = threadIdx.x / per_token, tid = threadIdx.x - group * per_token;
  const int64_t t = (int64_t)blockIdx.x * (kBwdThreads / per_token) + group;
  const bool live = t < tokens;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j0 = 0; j0 < topk; j0 += BATCH) {
    int32_t row[BATCH];
    float w[BATCH];
    float2 dot[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const bool have = live && j0 + j < topk;
      row[j] = have ? row_of(slot_row, t * topk + j0 + j, M) : -1;
      w[j] = have ? __ldg(weights + t * topk + j0 + j) : 0.0f;
      dot[j] = both(0.0f);
    }
    for (int v = live ? tid : nvec; v < nvec; v += per_token) {
      const uint4 dv = __ldg(dout + t * nvec + v);
      uint4 y[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (row[j] >= 0) y[j] = __ldg(rows + (int64_t)row[j] * nvec + v);
      float2 d[P];
      Vec<T>::unpack(dv, d);
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        if (row[j] < 0) continue;
        float2 f[P], o[P];
        Vec<T>::unpack(y[j], f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          dot[j] = fma2(d[i], f[i], dot[j]);
          o[i] = mul2(both(w[j]), d[i]);
        }
        drows[(int64_t)row[j] * nvec + v] = Vec<T>::pack(o);
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      float sum = dot[j].x + dot[j].y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) s_part[warp][j] = sum;
    }
    __syncthreads();
    if (live && tid < BATCH && j0 + tid < topk) {
      float sum = 0.0f;
      for (int k = 0; k < per_token / 32; ++k) sum += s_part[group * (per_token / 32) + k][tid];
      dweights[t * topk + j0 + tid] = sum;   // 0 where the slot has no row
    }
    __syncthreads();
  }
}

// Threads of a 256-thread CTA that share a token: a power of two of warps.
int threads_per_token(int nvec) {
  int n = 32;
  while (n < 256 && n < nvec) n *= 2;
  return n;
}

int grid_for(int64_t items, int per_cta, int num_sms, int ctas_per_sm) {
  const int64_t want = (items + per_cta - 1) / per_cta;
  const int64_t most = (int64_t)num_sms * ctas_per_sm;
  return (int)(want < most ? want : most);
}

}  // namespace route
}  // namespace fp8moe

FP8MOE_DEFINE_STATUS_TAKE(fp8moe_status_take_route)

cudaError_t fp8moe_launch_sort_tokens(const int32_t* ids, int64_t n, int E, int64_t M,
                                      int32_t* group_sizes, int32_t* slot_row, int32_t* row_slot,
                                      cudaStream_t s) {
  using namespace fp8moe::route;
  const size_t smem = (size_t)(kSortWarps + 1) * E * sizeof(int32_t);
  // the limit is the same for every call: another thread's call or a captured graph may
  // need more than this one does
  constexpr size_t most = (size_t)(kSortWarps + 1) * fp8moe::kMaxExperts * sizeof(int32_t);
  cudaError_t err = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)most);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  // up to 2048 slots one CTA has at most two 32-slot batches per warp (8192 slots: 11.5 us
  // on one CTA, 32768 slots 8.2 us on eight)
  const unsigned ctas = n <= 2048 ? 1 : kSortCtas;
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kSortThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, sort_kernel, ids, (uint32_t)n, E, (int32_t)M, group_sizes, slot_row,
                           row_slot);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

cudaError_t fp8moe_launch_dispatch(const void* x, const int32_t* ids, int64_t T, int topk, int E,
                                   int64_t M, int nvec, void* rows, int32_t* group_sizes,
                                   int32_t* slot_row, int32_t* row_slot, int num_sms,
                                   cudaStream_t s) {
  using namespace fp8moe::route;
  if (T * topk <= kFewSlots) {
    const int chunks = (nvec + kMoveThreads - 1) / kMoveThreads;
    dispatch_few_kernel<<<(unsigned)(T * chunks + 1), kMoveThreads, 0, s>>>(
        static_cast<const uint4*>(x), ids, (int)T, topk, E, M, nvec, chunks,
        static_cast<uint4*>(rows), group_sizes, slot_row, row_slot);
    return cudaGetLastError();
  }
  cudaError_t err = fp8moe_launch_sort_tokens(ids, T * topk, E, M, group_sizes, slot_row, row_slot, s);
  if (err != cudaSuccess || M == 0) return err;
  const int chunks = (nvec + 32 * kMoveVecs - 1) / (32 * kMoveVecs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid_for(T * chunks, kMoveThreads / 32, num_sms, 8), 1, 1);
  cfg.blockDim = dim3(kMoveThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  fp8moe::pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, dispatch_kernel, static_cast<const uint4*>(x), T, topk, nvec, chunks,
                           static_cast<const int32_t*>(slot_row), M, static_cast<uint4*>(rows));
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

cudaError_t fp8moe_launch_combine(const void* rows, int64_t T, int topk, int nvec, int f32,
                                  const int32_t* slot_row, int64_t M, const float* weights,
                                  void* out, cudaStream_t s) {
  using namespace fp8moe::route;
  const bool is_short = nvec <= 128;
  const int per_token = is_short ? threads_per_token(nvec) : kMoveThreads;
  const int tokens = kMoveThreads / per_token;
  auto run = [&](auto kern) {
    kern<<<(unsigned)((T + tokens - 1) / tokens), kMoveThreads, 0, s>>>(
        static_cast<const uint4*>(rows), T, topk, nvec, per_token, slot_row, M, weights,
        static_cast<uint4*>(out));
  };
  auto pick = [&](auto type, auto weighted) {
    using R = decltype(type);
    constexpr bool W = decltype(weighted)::value;
    if (topk <= 4) is_short ? run(combine_kernel<R, W, 4, true>) : run(combine_kernel<R, W, 4, false>);
    else is_short ? run(combine_kernel<R, W, 8, true>) : run(combine_kernel<R, W, 8, false>);
  };
  if (f32) weights ? pick(float(), std::true_type()) : pick(float(), std::false_type());
  else weights ? pick(__nv_bfloat16(), std::true_type()) : pick(__nv_bfloat16(), std::false_type());
  return cudaGetLastError();
}

cudaError_t fp8moe_launch_combine_bwd(const void* dout, const void* rows, int64_t T, int topk,
                                      int nvec, int f32, const int32_t* slot_row, int64_t M,
                                      const float* weights, void* drows, float* dweights,
                                      cudaStream_t s) {
  using namespace fp8moe::route;
  const int per_token = threads_per_token(nvec), tokens = kBwdThreads / per_token;
  auto run = [&](auto kern) {
    kern<<<(unsigned)((T + tokens - 1) / tokens), kBwdThreads, 0, s>>>(
        static_cast<const uint4*>(dout), static_cast<const uint4*>(rows), T, topk, nvec, per_token,
        slot_row, M, weights, static_cast<uint4*>(drows), dweights);
  };
  if (f32) topk <= 4 ? run(combine_bwd_kernel<float, 4>) : run(combine_bwd_kernel<float, 8>);
  else topk <= 4 ? run(combine_bwd_kernel<__nv_bfloat16, 4>) : run(combine_bwd_kernel<__nv_bfloat16, 8>);
  return cudaGetLastError();
}
