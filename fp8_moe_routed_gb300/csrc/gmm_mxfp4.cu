// gmm_mxfp4.cu -- the ragged grouped product of microscaled 4-bit operands,
//   y[m, n] = sum_blocks 2^(ex[m, b] + ew[e(m), n, b]) * sum_{k in b} qx[m, k] * qw[e(m), n, k]
// (f32 accumulation), out = bf16(y), or with SwiGLU bf16(silu(y[m, f]) * y[m, F + f]).
//
// The product is computed transposed, D[n, m]: the weight rows are the MMA's M side
// and the tokens its N side, whose size an instruction can choose in steps of 16.
// An expert's rows are cut into equal tiles of at most 208 tokens (a group of 1024
// into five of 208, not four of 208 and one of 192; a group of one token into one
// tile of 16), so few tokens cost few tensor cycles and the weight's bytes bound.
//
// CTA pairs, tcgen05.mma.cta_group::2 kind::mxf4: M = 256 weight rows (128 per CTA),
// N = the token tile (half of its rows in each CTA's shared memory), K = 64. Roles:
//   warp 0       TMA: 256 k per stage: this CTA's 128 weight rows (16 KB) and its half
//                of the token rows, 128-byte swizzle, 6 to 9 stages, counted on the even
//                CTA's barrier. Three token boxes (16, 48, 104 rows): a small tile
//                does not fetch rows that it does not multiply.
//   warp 1       TMEM; in the even CTA the MMA-issuing thread.
//   warp 2       TMA: the scale words of the stages (8 stages of their own, counted on
//                this CTA's barriers).
//   warp 3       idle.
//   warps 4..19  scales: four groups of four that take every fourth stage. The words of a
//                stage (2 words of each of 128 weight rows and up to 208 token rows) go
//                from shared memory through registers into tensor memory (tcgen05.st),
//                one warp per lane quarter, the same data in all four. Passing them
//                through registers lets a token tile start at any row: the box starts at
//                the next lower multiple of four (a copy starts on 16 bytes) and the
//                warps read from the remainder on. A group's chain per stage (two waits,
//                the TMEM store's round trip) takes about 900 cycles, a stage of MMAs 416.
//   warps 20..27 epilogue: two groups of four (one warp per lane quarter) alternate over
//                16-token chunks of one of two accumulators.
// The peer's threads, copies or commits arrive on full, empty, tfull, tempty and drain:
// these are waited for at cluster scope (no difference in time to CTA scope).
// TMEM (512 columns): two accumulators of 208, four scale slots of 24.
//
// SwiGLU: a CTA's 128 weight rows are 4 x (16 gate rows, 16 up rows), fetched by one
// five-dimensional box, so the two 16-lane halves of a warp's lane quarter hold the gate
// and up rows of the same 16 columns and two loads give a thread both.
//
// What bounds it (32 experts, balanced, K = 7168, N = 4096, SwiGLU: 275 us = 7.0 PFLOP/s
// at a power-capped 1.75 GHz; 68 % of a stage's time the tensor pipe is busy): with many
// tokens per expert the MMA thread's chain per stage (wait, four products, commit: 450 to
// 525 cycles against 416 of tensor time) and shared-memory traffic (codes in and out 142
// bytes a cycle at the tensor rate; without the code loads 13 % less time, without the
// scale warps' reads 4 %); with K = 2048 also the epilogue's share of it (205 against 156
// us without). With few tokens the weight's bytes, at 5.7 TB/s for 32 experts of one tile
// each; eight experts' 128 units make two uneven rounds on 76 pairs.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "groups.cuh"
#include "kernels.h"
#include "mxfp4.cuh"
#include "pdl.cuh"
#include "ptx_mx.cuh"

namespace fp8moe {
namespace mxgmm {

constexpr int kBK = 256;                     // k per stage: 128 bytes of codes
constexpr int kKBytes = kBK / 2;
constexpr int kRowsA = 128;                  // weight rows per CTA
constexpr int kUnitN = 2 * kRowsA;           // weight rows per unit = MMA M
constexpr int kMaxTok = 208;                 // token rows per unit = largest MMA N
// token rows per CTA of the three TMA boxes
constexpr int kBox0 = 16, kBox1 = 48, kBox2 = 104;
constexpr int kABytes = kRowsA * kKBytes;    // 16 KB
constexpr int kBBytes = kBox2 * kKBytes;
constexpr int kSaBytes = 2 * kRowsA * 4;     // scale words of a stage: weight rows
constexpr int kSbWords = kMaxTok + 4;        // token rows, from a multiple of four on
constexpr int kSbBytes = 2 * kSbWords * 4;
constexpr int kScaleBytes = (kSaBytes + kSbBytes + 127) / 128 * 128;
// The code stages share this much memory: 6 stages when a tile of the call has more than
// 96 token rows, 7 or 9 when every tile is small. A few tokens are bound by how many
// weight bytes are in flight: with 6 stages a pair got 84 GB/s.
constexpr int kCodeBytes = 6 * (kABytes + kBBytes);
constexpr int kMaxStages = 9;
static_assert(kCodeBytes / (kABytes + kBox0 * kKBytes) == kMaxStages, "barriers for every stage");
constexpr int kWords = 8;                    // scale-word stages
constexpr int kSlots = 4;
constexpr int kSfA = 8, kSfB = 16;           // TMEM columns of a stage's scales
constexpr int kSfCols = kSfA + kSfB;
constexpr int kDCols = kMaxTok;
constexpr int kSfBase = 2 * kDCols;
static_assert(kSfBase + kSlots * kSfCols <= 512, "TMEM budget");
static_assert(kSlots < 6, "a slot comes round before its step's code stage does");
static_assert(kBBytes % 1024 == 0, "swizzle atoms start on 1024-byte boundaries");
// A parity wait tells a phase from the one before it, not from the one before that: a
// scale group has to take part in every use of its stages and slots.
constexpr int kSfGroups = 4;
static_assert(kWords % kSfGroups == 0 && kSlots == kSfGroups, "a group owns a slot and its words");
constexpr int kTokWords = (kMaxTok + 31) / 32;   // scale columns of the token rows per 128 k
constexpr int kFirstSf = 4, kFirstEpi = kFirstSf + 4 * kSfGroups;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kFirstEpi + kEpiWarps) * 32;   // 896
constexpr int kChunk = 16;                   // token rows that four epilogue warps turn at a time
constexpr int kTurnBytes = kChunk * (kRowsA * 2 + 16);

struct Smem {
  uint64_t full[kMaxStages];   // even CTA: the stage's four code boxes landed and both CTAs'
                               // scales are in TMEM
  uint64_t empty[kMaxStages];  // the MMAs of the stage completed (and of its scale slot)
  uint64_t words[kWords];      // this CTA's scale words landed
  uint64_t wempty[kWords];     // and were read
  uint64_t tfull[2];           // accumulator complete
  uint64_t tempty[2];          // even CTA: both CTAs' epilogues loaded it
  uint64_t drain;
  uint32_t tmem_base;
  int32_t T;
  int32_t tiles;               // token tiles of all experts
  int32_t stage_bytes, stages;
  int32_t begin[kMaxExperts + 1];    // [e + 1] is also where expert e ends
  int32_t prefix[kMaxExperts + 1];   // token tiles before expert e
  uint8_t tok[kMaxExperts];          // token rows of its tiles
};
constexpr size_t kSmemBytes = 1024 + (size_t)kCodeBytes + (size_t)kWords * kScaleBytes + 4 * kTurnBytes + sizeof(Smem);
static_assert(kSmemBytes <= 232448, "shared memory per CTA exceeds 227 KB");

struct Unit {
  int e, m0, rows, tok, w0;    // rows: valid token rows; tok: MMA N; w0: first weight tile index
};

__device__ __forceinline__ int token_tiles(int rows) { return (rows + kMaxTok - 1) / kMaxTok; }

// Token rows of an expert's tiles: equal tiles, t = ceil(rows / 208) of ceil(rows / t)
// rounded up to 16. That is <= 208, so the last of the t tiles is never empty.
__device__ __forceinline__ int tile_rows(int rows) {
  const int t = max(1, token_tiles(rows));
  return ((rows + t - 1) / t + 15) & ~15;
}

// Units: expert by expert, token tiles, weight tiles fastest (their shared token tile
// stays in L2). A pair walks units cluster, cluster + nclusters, ...: `tile` counts token
// tiles over all experts, w0 the weight tile; steps and wraps, no division per unit.
struct Walk {
  int tile, w0, e, step_t, step_w, wt;
  __device__ __forceinline__ Walk(int first, int step, int weight_tiles)
      : tile(first / weight_tiles), w0(first % weight_tiles), e(0), step_t(step / weight_tiles),
        step_w(step % weight_tiles), wt(weight_tiles) {}
  __device__ __forceinline__ void next() {
    tile += step_t;
    w0 += step_w;
    if (w0 >= wt) { w0 -= wt; ++tile; }
  }
  __device__ __forceinline__ int expert(const Smem& s) {
    while (tile >= s.prefix[e + 1]) ++e;
    return e;
  }
  __device__ __forceinline__ Unit unit(const Smem& s) {
    Unit r;
    r.e = expert(s);
    r.w0 = w0;
    r.tok = s.tok[r.e];
    r.m0 = s.begin[r.e] + (tile - s.prefix[r.e]) * r.tok;
    r.rows = min(r.tok, s.begin[r.e + 1] - r.m0);
    return r;
  }
};

// The smallest box that holds half of a tile.
__device__ __forceinline__ int box_rows(int tok) {
  return tok <= 2 * kBox0 ? kBox0 : tok <= 2 * kBox1 ? kBox1 : kBox2;
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
gmm_mxfp4_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX0,
                 const __grid_constant__ CUtensorMap tmX1, const __grid_constant__ CUtensorMap tmX2,
                 const __grid_constant__ CUtensorMap tmSw, const __grid_constant__ CUtensorMap tmSx,
                 const int32_t* __restrict__ gs, __nv_bfloat16* __restrict__ out, int64_t M, int K,
                 int N, int E) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t* const scales = ring + kCodeBytes;
  uint8_t* const turn = scales + (size_t)kWords * kScaleBytes;
  Smem& s = *reinterpret_cast<Smem*>(turn + 4 * kTurnBytes);
  auto sa_tile = [&](int i) -> uint8_t* { return scales + i * kScaleBytes; };
  auto sb_tile = [&](int i) -> uint8_t* { return scales + i * kScaleBytes + kSaBytes; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  const int F = N / 2;                                  // SwiGLU: gate and up rows
  const int wt = SWIGLU ? (F + kRowsA - 1) / kRowsA : (N + kUnitN - 1) / kUnitN;
  const int nkb = (K + kBK - 1) / kBK;

  if (warp == 0) {
    load_groups_warp0(gs, E, M, s.begin, s.begin + 1, &s.T, blockIdx.x == 0);
    __syncwarp();
    int32_t carry = 0, most = 16;
    for (int base = 0; base < E; base += 32) {
      const int e = base + lane;
      int32_t n = 0;
      if (e < E) {
        const int rows = s.begin[e + 1] - s.begin[e], tok = tile_rows(rows);
        n = token_tiles(rows);
        s.tok[e] = (uint8_t)tok;
        most = max(most, tok);
      }
      int32_t incl = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      if (e < E) s.prefix[e] = carry + incl - n;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      s.stage_bytes = kABytes + box_rows(most) * kKBytes;
      s.stages = kCodeBytes / s.stage_bytes;
      s.prefix[E] = carry;
      s.tiles = carry;
      prefetch_tmap(&tmW);
      prefetch_tmap(&tmX0);
      prefetch_tmap(&tmX1);
      prefetch_tmap(&tmX2);
      prefetch_tmap(&tmSw);
      prefetch_tmap(&tmSx);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      for (int i = 0; i < kMaxStages; ++i) {
        mbar_init(&s.full[i], 1 + 8);    // the producer's bytes + a group of scale warps per CTA
        mbar_init(&s.empty[i], 1);
      }
      for (int i = 0; i < kWords; ++i) {
        mbar_init(&s.words[i], 1);
        mbar_init(&s.wempty[i], 4);      // one group of scale warps
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s.tfull[i], 1);
        mbar_init(&s.tempty[i], 2 * kEpiWarps);
      }
      mbar_init(&s.drain, 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc_pair(&s.tmem_base, 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();      // the peer's barriers exist before anyone signals them
  tc_fence_after();
  const int tiles = s.tiles;
  const uint32_t tmem = s.tmem_base;
  const int stages = s.stages, stage_bytes = s.stage_bytes;
  auto a_tile = [&](int i) -> uint8_t* { return ring + i * stage_bytes; };
  auto b_tile = [&](int i) -> uint8_t* { return ring + i * stage_bytes + kABytes; };

  if (warp == 0) {
    // ========================= TMA producer: codes ========================
    pdl_wait();        // the activations' codes and scales are the quantiser's
    // Like the MMA warp: the whole warp walks the steps, one thread issues.
    const bool leader = elect_one();
    int st = 0;
    uint32_t ph = 0;
    int64_t issued = 0;
    bool ok = true;
    for (Walk at(cluster, nclusters, wt); at.tile < tiles && ok; at.next()) {
      const Unit t = at.unit(s);
      const int box = box_rows(t.tok);
      const CUtensorMap* tmX = box == kBox0 ? &tmX0 : box == kBox1 ? &tmX1 : &tmX2;
      const uint32_t bytes = 2u * (uint32_t)(kABytes + box * kKBytes);
      const int m = t.m0 + rank * (t.tok / 2);
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait_warp_cluster(&s.empty[st], ph ^ 1, kWhereProducer)) { ok = false; break; }
        if (leader) {
          if (rank == 0) mbar_arrive_expect_tx(&s.full[st], bytes);
          const uint32_t bar = mapa_shared(smem_u32(&s.full[st]), 0);
          if (SWIGLU)
            tma_load_5d_pair(a_tile(st), &tmW, bar, kb * kKBytes, 0, 0,
                             t.w0 * (kRowsA / 16) + rank * 4, t.e);
          else
            tma_load_3d_pair(a_tile(st), &tmW, bar, kb * kKBytes, t.w0 * kUnitN + rank * kRowsA,
                             t.e);
          tma_load_2d_pair(b_tile(st), tmX, bar, kb * kKBytes, m);
        }
        __syncwarp();
        ++issued;
        if (++st == stages) { st = 0; ph ^= 1; }
      }
    }
    // drain: every copy landed before either CTA may exit
    if (lane == 0 && rank == 0) {
      const int64_t n_last = issued < stages ? issued : stages;
      for (int64_t i = 1; i <= n_last; ++i) {
        const int64_t idx = issued - i;
        mbar_wait_cluster(&s.full[idx % stages], (uint32_t)((idx / stages) & 1), kWhereDrain);
      }
    }
  } else if (warp == 1) {
    // ============================== MMA issuer ============================
    // One elected thread walks the steps: a branch on elect.sync (unlike one on the lane
    // number) tells the compiler that a single thread runs it, so that descriptors and
    // addresses go to uniform registers without a loop over the warp's values.
    if (rank == 0 && elect_one()) {
      int st = 0, sl = 0, ab = 0;
      uint32_t ph = 0, tph = 0;
      bool ok = true, ready = false;
      Walk at(cluster, nclusters, wt);
      uint32_t tok = at.tile < tiles ? s.tok[at.expert(s)] : 16u;
      while (at.tile < tiles && ok) {
        const uint32_t idesc0 = make_idesc_mxf4(kUnitN, tok, 0);
        const uint32_t idesc2 = make_idesc_mxf4(kUnitN, tok, 2);
        const uint32_t d = tmem + (uint32_t)(ab * kDCols);
        if (!mbar_wait_cluster(&s.tempty[ab], tph ^ 1, kWhereMma)) { ok = false; break; }
        tc_fence_after();
        for (int kb = 0; kb < nkb; ++kb) {
          // a wait costs its latency even when there is nothing to wait for, so the next
          // step's barrier is tested before this step's products are issued
          if (!ready && !mbar_wait_cluster(&s.full[st], ph, kWhereMma)) { ok = false; break; }
          tc_fence_after();
          const uint64_t ad = make_desc(smem_u32(a_tile(st)), 16, 1024, kSwizzle128B);
          const uint64_t bd = make_desc(smem_u32(b_tile(st)), 16, 1024, kSwizzle128B);
          const uint32_t sf = tmem + (uint32_t)(kSfBase + sl * kSfCols);
          uint64_t* const done = &s.empty[st];
          if (++st == stages) { st = 0; ph ^= 1; }
          if (++sl == kSlots) sl = 0;
          ready = mbar_test_cluster(&s.full[st], ph);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            // the descriptors' address field counts 16 bytes: 64 values are two. Past K
            // codes and scales are zeros; leaving those products out (a predicate on every
            // one) doubles the issue time.
              mma_mxf4_pair(d, ad + 2 * kk, bd + 2 * kk, (kk & 1) ? idesc2 : idesc0,
                            sf + (kk >> 1) * (kSfA / 2), sf + kSfA + (kk >> 1) * (kSfB / 2),
                            (kb | kk) != 0);
          }
          mma_commit_pair(done);
          if (kb == 0) {                     // the next unit's tile size, while this one runs
            at.next();
            if (at.tile < tiles) tok = s.tok[at.expert(s)];
          }
        }
        if (!ok) break;
        mma_commit_pair(&s.tfull[ab]);
        if (++ab == 2) { ab = 0; tph ^= 1; }
      }
      // all MMAs complete (in both CTAs' TMEM) before TMEM may be released
      mma_commit_pair(&s.drain);
    }
    __syncwarp();
    if (lane == 0) mbar_wait_cluster(&s.drain, 0, kWhereDrain);
  } else if (warp == 2) {
    // ===================== TMA producer: scale words ======================
    pdl_wait();
    const bool leader = elect_one();
    int st = 0;
    uint32_t ph = 0;
    int64_t issued = 0;
    bool ok = true;
    for (Walk at(cluster, nclusters, wt); at.tile < tiles && ok; at.next()) {
      const Unit t = at.unit(s);
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait_warp(&s.wempty[st], ph ^ 1, kWhereProducer)) { ok = false; break; }
        if (leader) {
          mbar_arrive_expect_tx(&s.words[st], kSaBytes + kSbBytes);
          if (SWIGLU)
            tma_load_5d(sa_tile(st), &tmSw, &s.words[st], 0, 0, t.w0 * (kRowsA / 16) + rank * 4,
                        2 * kb, t.e);
          else
            tma_load_3d(sa_tile(st), &tmSw, &s.words[st], t.w0 * kUnitN + rank * kRowsA, 2 * kb,
                        t.e);
          tma_load_2d(sb_tile(st), &tmSx, &s.words[st], t.m0 & ~3, 2 * kb);
        }
        __syncwarp();
        ++issued;
        if (++st == kWords) { st = 0; ph ^= 1; }
      }
    }
    if (lane == 0) {
      const int64_t n_last = issued < kWords ? issued : kWords;
      for (int64_t i = 1; i <= n_last; ++i) {
        const int64_t idx = issued - i;
        mbar_wait(&s.words[idx % kWords], (uint32_t)((idx / kWords) & 1), kWhereDrain);
      }
    }
  } else if (warp < kFirstSf) {
    // idle
  } else if (warp < kFirstEpi) {
    // =============================== scales ===============================
    const int quarter = warp & 3;
    const int group = (warp - kFirstSf) >> 2;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)kSfBase;
    const uint32_t even_full = mapa_shared(smem_u32(&s.full[0]), 0);
    const int words = (K + kMxWord - 1) / kMxWord;
    const int last_blocks = (K - (words - 1) * kMxWord) / kMxBlock;     // of the last word: 1..4
    const uint32_t last_mask = last_blocks == 4 ? 0xFFFFFFFFu : (1u << (8 * last_blocks)) - 1u;
    uint32_t i = 0;                                // global step index (word stages and slots)
    // the code stage of this group's step and of its step before, which had the same slot
    int cs = group, before = 0;
    uint32_t cph = 0, before_ph = 0;
    bool ok = true;
    for (Walk at(cluster, nclusters, wt); at.tile < tiles && ok; at.next()) {
      const Unit t = at.unit(s);
      const int shift = t.m0 & 3;
      for (int kb = 0; kb < nkb; ++kb, ++i) {
        if ((int)(i % kSfGroups) != group) continue;
        const int st = (int)(i % kWords), sl = (int)(i % kSlots);
        if (!mbar_wait_warp(&s.words[st], (i / kWords) & 1, kWhereDequant)) { ok = false; break; }
        const uint32_t* const pa = reinterpret_cast<const uint32_t*>(sa_tile(st)) + lane;
        const uint32_t* const pb = reinterpret_cast<const uint32_t*>(sb_tile(st)) + shift + lane;
        uint32_t wa[8], wb[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // past the last word the boxes are filled with zeros
          const uint32_t mask = 2 * kb + h == words - 1 ? last_mask : 0xFFFFFFFFu;
#pragma unroll
          for (int j = 0; j < 4; ++j) wa[h * 4 + j] = pa[h * kRowsA + j * 32] & mask;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            wb[h * 8 + j] = j < kTokWords && j * 32 + lane < kMaxTok
                                ? pb[h * kSbWords + j * 32] & mask : 0u;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.wempty[st]);     // words read
        // The slot was last read by the products of step i - kSlots, this group's step
        // before: their stage's barrier tells when they are done. (The phase that it could
        // be mistaken for, two uses of the stage earlier, was waited for in its turn.)
        if (i >= kSlots && !mbar_wait_warp_cluster(&s.empty[before], before_ph, kWhereDequant)) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_st8(tq + (uint32_t)(sl * kSfCols), wa);
        tmem_st16(tq + (uint32_t)(sl * kSfCols + kSfA), wb);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        // Relaxed: what the product reads is in tensor memory, ordered by the store's wait and the
        // fences on both sides of the barrier, not by a release (which would also wait for
        // every earlier access of this thread: balanced wi 552 against 418 us).
        if (lane == 0) mbar_arrive_cluster_relaxed(even_full + (uint32_t)(cs * sizeof(uint64_t)));
        before = cs;
        before_ph = cph;
        cs += kSfGroups;
        if (cs >= stages) { cs -= stages; cph ^= 1; }
      }
    }
  } else {
    // =============================== epilogue =============================
    const int quarter = warp & 3;
    const int half = (warp - kFirstEpi) >> 2;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t even_tempty = mapa_shared(smem_u32(&s.tempty[0]), 0);
    // The accumulator has a column per token; the output wants whole rows. Four warps turn
    // 16 tokens x their 128 weight rows through shared memory and store 16 bytes a lane,
    // 256 (SwiGLU: 128) contiguous bytes of a token.
    constexpr int kCols = SWIGLU ? kRowsA / 2 : kRowsA;     // outputs of a token in this CTA
    constexpr int kPieces = kCols / 8;
    constexpr uint32_t kPitch = kCols * 2 + 16;             // rows of 16 bytes fall into all banks
    const uint32_t turn_addr = smem_u32(turn);
    // this lane's row of the four 8 x 8 pieces: pieces (tokens 0..7, rows 0..7), (0..7, 8..15),
    // (8..15, 0..7), (8..15, 8..15)
    const uint32_t st_row = (uint32_t)((lane >> 4) * 8 + (lane & 7));
    const uint32_t st_col = (uint32_t)(((lane >> 3) & 1) * 16);
    const int width = SWIGLU ? F : N;
    int ab = 0, buf = 0;
    uint32_t tph = 0;
    uint16_t* const o16 = reinterpret_cast<uint16_t*>(out);
    for (Walk at(cluster, nclusters, wt); at.tile < tiles; at.next()) {
      const Unit t = at.unit(s);
      // the four warps leave together: a named barrier's wait has no limit
      if (!named_bar_all(1 + half, 128, mbar_wait_warp_cluster(&s.tfull[ab], tph, kWhereEpilogue)))
        break;
      tc_fence_after();
      const int col0 = SWIGLU ? t.w0 * kRowsA + rank * 64 : t.w0 * kUnitN + rank * kRowsA;
      for (int c0 = half * kChunk; c0 < t.tok; c0 += 2 * kChunk) {
        // rows 0..15 and 16..31 of the quarter: a thread holds, of row (lane / 4) and the row
        // 8 below it, tokens 2 (lane % 4), + 1 and the same 8 further on. The transposing
        // matrix store turns 8 x 8 pieces of such pairs into 16 bytes of a token's row.
        uint32_t lo[8], hi[8];
        tmem_ld_16x256b_x2(tq + (uint32_t)(ab * kDCols + c0), lo);
        tmem_ld_16x256b_x2(tq + (16u << 16) + (uint32_t)(ab * kDCols + c0), hi);
        tmem_ld_wait();
        const uint32_t mine = turn_addr + (uint32_t)((2 * half + buf) * kTurnBytes);
        uint32_t pk[4];
        if (SWIGLU) {
          // gate rows and the up rows of the same columns
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float h[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // fast exponential and division: at most 2 + 1.2 |g| f32 steps and 2 of error, far
              // below the bf16 rounding that follows (the exact ones: 385 against 371 us). Below
              // g = -87 the quotient, under 2e-36 in magnitude, is zero.
              const float g = __uint_as_float(lo[j + i]), v = __uint_as_float(hi[j + i]);
              h[i] = __fmul_rn(__fdividef(g, __fadd_rn(1.0f, __expf(-g))), v);
            }
            pk[j / 2] = f32x2_to_bf16x2(h[0], h[1]);
          }
          stmatrix_x4_trans(mine + st_row * kPitch + (uint32_t)(quarter * 32) + st_col, pk);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j += 2)
            pk[j / 2] = f32x2_to_bf16x2(__uint_as_float(lo[j]), __uint_as_float(lo[j + 1]));
          stmatrix_x4_trans(mine + st_row * kPitch + (uint32_t)(quarter * 64) + st_col, pk);
#pragma unroll
          for (int j = 0; j < 8; j += 2)
            pk[j / 2] = f32x2_to_bf16x2(__uint_as_float(hi[j]), __uint_as_float(hi[j + 1]));
          stmatrix_x4_trans(mine + st_row * kPitch + (uint32_t)(quarter * 64) + 32u + st_col, pk);
        }
        // the barrier also orders this turn's writes after the reads of the one before
        // the last, which had the same buffer
        named_bar_sync(1 + half, 128);
#pragma unroll
        for (int i = 0; i < kChunk * kPieces / 128; ++i) {
          const int q = i * 128 + quarter * 32 + lane;
          const int j = q / kPieces, col = col0 + (q % kPieces) * 8;
          if (c0 + j < t.rows && col < width)
            *reinterpret_cast<uint4*>(o16 + ((int64_t)t.m0 + c0 + j) * width + col) =
                ld_shared_16B(mine + (uint32_t)(j * kPitch + (q % kPieces) * 16));
        }
        buf ^= 1;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(even_tempty + (uint32_t)(ab * sizeof(uint64_t)));
      if (++ab == 2) { ab = 0; tph ^= 1; }
    }
  }

  __syncthreads();
  cluster_sync();      // both CTAs done with TMEM, shared memory and barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool SWIGLU>
cudaError_t launch(const GmmMxfp4Args& a, int num_sms, cudaStream_t s) {
  auto kern = gmm_mxfp4_kernel<SWIGLU>;
  cudaError_t err =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_sms & ~1), 1, 1);   // whole CTA pairs, one CTA per SM
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  pdl_attribute(attr[1]);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, kern, a.tmW, a.tmX[0], a.tmX[1], a.tmX[2], a.tmSw,
                           a.tmSx, a.gs,
                           static_cast<__nv_bfloat16*>(a.out), a.M, a.K, a.N, a.E);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

}  // namespace mxgmm
}  // namespace fp8moe

FP8MOE_DEFINE_STATUS_TAKE(fp8moe_status_take_gmm_mxfp4)

void fp8moe_gmm_mxfp4_boxes(int rows[3], int* scale_rows) {
  using namespace fp8moe::mxgmm;
  rows[0] = kBox0;
  rows[1] = kBox1;
  rows[2] = kBox2;
  *scale_rows = kSbWords;
}

cudaError_t fp8moe_launch_gmm_mxfp4(const GmmMxfp4Args& a, int num_sms, cudaStream_t s) {
  using namespace fp8moe::mxgmm;
  return a.swiglu ? launch<true>(a, num_sms, s) : launch<false>(a, num_sms, s);
}
