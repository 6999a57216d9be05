/* fp8moe.h -- C ABI of libfp8moe.so: native-FP8 grouped matmuls for the routed
 * experts of a mixture-of-experts layer, on one GB300 (sm_103a).
 *
 * Sources (web pages):
 *   [NQ] "MoE: native FP8 QAT for routed-expert GMMs (FP8 forward + FP8-weight
 *        backward dLHS)" -- Description, Data flow, Implementation, Tests.
 *   [DQ] "MoE fp8 backward: in-kernel drhs operand quantization + configurable
 *        gradient dtype" -- What.
 *   [SM] "Fix fp8 MoE on the sparse_matmul path" -- Fix (forward dtype is
 *        float8_e4m3fn).
 *
 * Common conventions
 *   - All array pointers are DEVICE pointers on the current CUDA device,
 *     row-major and contiguous, 16-byte aligned.  bf16 arrays are passed as
 *     void* (IEEE bfloat16 bit patterns).  FP8 codes are OCP float8_e4m3fn bit
 *     patterns in uint8_t.
 *   - The ragged buffer has a static number of rows M.  group_sizes (int32 [E],
 *     device memory) gives the rows of each expert, in order: expert e owns rows
 *     [off[e], off[e] + group_sizes[e]) with off the exclusive prefix sum.
 *     T = sum(group_sizes) may be smaller than M; rows >= T are never read and
 *     never written.  A negative size counts as 0 and ranges are clipped at M;
 *     both are recorded in the device status word (fp8moe_read_status).
 *   - Weights: codes[E, K, N] (N contiguous) with per-output-channel f32
 *     scale[E, N] (the pages' [g, 1, n] scale); weight w = code * scale.
 *   - K is whole in every call: the activation scale always spans all K.
 *   - Calls only enqueue work on `stream`; they never synchronize and never
 *     copy group_sizes to the host.  The caller owns every buffer, including the
 *     workspace (size from fp8moe_workspace_size); the library allocates no
 *     memory.
 *   - Shapes: 1 <= E <= 1024; K, N > 0 and multiples of 16 (TMA stride rule);
 *     0 <= M < 2^31 (M == 0 returns FP8MOE_OK without launching).
 *   - Return value: FP8MOE_OK (0) or a negative FP8MOE_E* code; nothing is
 *     launched when an argument check fails.  fp8moe_last_cuda_error() gives the
 *     CUDA error behind FP8MOE_ECUDA.
 */
#ifndef FP8MOE_H_
#define FP8MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* fp8moe_stream_t;

enum {
  FP8MOE_OK = 0,
  FP8MOE_EINVAL = -1,       /* null pointer, bad dimension, odd N for SwiGLU, E out of range */
  FP8MOE_EALIGN = -2,       /* pointer not 16-byte aligned, or K / N not a multiple of 16 */
  FP8MOE_EWORKSPACE = -3,   /* workspace missing or smaller than fp8moe_workspace_size() */
  FP8MOE_ECUDA = -4,        /* a CUDA call or launch failed; see fp8moe_last_cuda_error() */
  FP8MOE_EUNSUPPORTED = -5  /* the current device is not an sm_103 GPU */
};

/* Operation ids for fp8moe_workspace_size. */
enum {
  FP8MOE_OP_GMM_FP8_FWD = 1,
  FP8MOE_OP_GMM_SILU_FP8_FWD = 2,
  FP8MOE_OP_GMM_DLHS_FP8 = 3,
  FP8MOE_OP_TGMM_DRHS_QUANT = 4,
  FP8MOE_OP_GMM_BF16_FWD = 5,
  FP8MOE_OP_DEQUANTIZE = 6,
  FP8MOE_OP_GMM_FP8_FWD_BLOCK = 7,
  FP8MOE_OP_GMM_MXFP4_FWD = 8,
  FP8MOE_OP_GMM_SILU_MXFP4_FWD = 9,
  FP8MOE_OP_NORM_BWD = 10,       /* M = T rows, K = H columns; N and E unused */
  FP8MOE_OP_BALANCE = 11         /* M = T tokens, N = B sequences, E experts; K unused */
};

/* Element types of the rows that the token and norm operators move. */
enum {
  FP8MOE_TYPE_BF16 = 0,
  FP8MOE_TYPE_F32 = 1
};

/* A router's scores (fp8moe_router_fwd). */
enum {
  FP8MOE_SCORE_SOFTMAX = 0,
  FP8MOE_SCORE_SIGMOID = 1
};

/* What a block's gate is shared by (fp8moe_norm_fwd). */
enum {
  FP8MOE_GATE_NONE = 0,  /* no gate (1) */
  FP8MOE_GATE_TOKEN = 1,   /* f32 [T], one value per token */
  FP8MOE_GATE_CHANNEL = 2, /* f32 [H], one value per column */
  FP8MOE_GATE_FULL = 3     /* [T, H] of the rows' type */
};

/* fp8 formats of the tgmm's dout (gradient) operand -- [DQ] What: the
 * gradient fp8 dtype is configurable, e5m2 (the recipe's default) or e4m3. */
enum {
  FP8MOE_FMT_E4M3 = 0,   /* OCP float8_e4m3fn, max 448 */
  FP8MOE_FMT_E5M2 = 1    /* OCP float8_e5m2, max 57344 */
};

/* Bits of the device status word. */
#define FP8MOE_STATUS_NEGATIVE_GROUP 0x1u    /* some group_sizes[e] < 0 (taken as 0) */
#define FP8MOE_STATUS_GROUPS_EXCEED_M 0x2u   /* sum(group_sizes) > M (clipped at M) */
#define FP8MOE_STATUS_WAIT_TIMEOUT 0x4u      /* a kernel pipeline wait gave up; bits 8..15 say where */
#define FP8MOE_STATUS_TOO_MANY_SEGMENTS 0x8u /* internal: segment bound exceeded */
#define FP8MOE_STATUS_BAD_EXPERT 0x10u       /* an expert id >= E (its slot was dropped) */
#define FP8MOE_STATUS_BAD_OFFSETS 0x20u      /* sequence offsets below 0, falling, or past T */

/* Workspace bytes the operation needs for these sizes (0 if none); the
 * workspace pointer must be 256-byte aligned.  Depends on M, K, N, E only. */
size_t fp8moe_workspace_size(int op, int64_t M, int64_t K, int64_t N, int32_t E);

/* Forward FP8 GMM, no epilogue (wo forward; also the ring-of-experts down
 * projection forward) -- [NQ] Implementation (gmm_dswiglu_fp8 forward,
 * gmm_fp8_forward).  For row m of expert e:
 *   sx[m]  = max(max_k |lhs[m,k]|, 1e-12) / 448          (f32, full K)
 *   qx     = e4m3(lhs[m,k] / sx[m])                       (RNE, saturating)
 *   out[m,n] = bf16( sx[m] * scale[e,n] * sum_k qx[m,k] * codes[e,k,n] )  (f32 accumulation)
 * lhs: bf16 [M, K].  codes: u8 [E, K, N].  scale: f32 [E, N].
 * out: bf16 [M, N]; rows >= T untouched.  Workspace: FP8MOE_OP_GMM_FP8_FWD
 * (holds the activation codes and row scales). */
int fp8moe_gmm_fp8_fwd(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                       const float* scale, int32_t E, int64_t N, const int32_t* group_sizes,
                       void* out, void* workspace, size_t workspace_bytes,
                       fp8moe_stream_t stream);

/* Forward FP8 GMM with the fused SwiGLU epilogue (wi forward) -- [NQ]
 * Implementation (gmm_silu_fp8).  Same as fp8moe_gmm_fp8_fwd; the N columns
 * are gate | up halves (N a multiple of 32, else FP8MOE_EALIGN: the up half
 * must start on a 16-byte boundary) and, with y the scaled f32 accumulator,
 *   out[m, j] = bf16( silu(y[m, j]) * y[m, N/2 + j] ),  silu(z) = z / (1 + exp(-z)).
 * out: bf16 [M, N/2].  Workspace: FP8MOE_OP_GMM_SILU_FP8_FWD. */
int fp8moe_gmm_silu_fp8_fwd(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                            const float* scale, int32_t E, int64_t N,
                            const int32_t* group_sizes, void* out, void* workspace,
                            size_t workspace_bytes, fp8moe_stream_t stream);

/* Backward dLHS GMM from the FP8 weight -- [NQ] Description and Implementation
 * (rhs_contract_dequant): each weight tile is dequantized on chip,
 *   w[e,k,n] = bf16(f32(codes[e,k,n]) * scale[e,n]),
 *   dlhs[m,k] = bf16( sum_n dout[m,n] * w[e,k,n] )   (f32 accumulation),
 * bit-identical whichever internal path is taken (contraction N <= 256: the
 * dequantized weight block cached in shared memory; N > 256: CTA pairs with the
 * dequantized weight tile in tensor memory).
 * dout: bf16 [M, N] (the forward output's cotangent).  dlhs: bf16 [M, K];
 * rows >= T untouched.  No workspace (pass NULL, 0). */
int fp8moe_gmm_dlhs_fp8(const void* dout, int64_t M, int64_t N, const uint8_t* codes,
                        const float* scale, int32_t E, int64_t K, const int32_t* group_sizes,
                        void* dlhs, void* workspace, size_t workspace_bytes,
                        fp8moe_stream_t stream);

/* Same as fp8moe_gmm_dlhs_fp8 with the internal path forced: path 0 streams
 * and dequantizes every weight tile per output tile; path 1 keeps the
 * dequantized weight block of an (expert, k tile) on chip across the expert's
 * m tiles (needs N <= 256, else FP8MOE_EINVAL); path 2 computes the transposed
 * product on CTA pairs with the dequantized weight tile held in tensor memory
 * (the default for N > 256).  Any other path: FP8MOE_EINVAL.  All paths give
 * identical bits. */
int fp8moe_gmm_dlhs_fp8_path(const void* dout, int64_t M, int64_t N, const uint8_t* codes,
                             const float* scale, int32_t E, int64_t K,
                             const int32_t* group_sizes, void* dlhs, int32_t path,
                             fp8moe_stream_t stream);

/* wo dLHS with the SwiGLU backward fused into its epilogue -- [NQ]
 * Implementation (gmm_dswiglu_fp8, the wo op whose backward also undoes the wi
 * SwiGLU).  With codes/scale the wo weight [E, F, N] / [E, N]:
 *   dh[m,f]  = sum_n dout[m,n] * w[e,f,n]   (as fp8moe_gmm_dlhs_fp8, f32, not rounded)
 *   g = gu[m,f], u = gu[m,F+f], sig(z) = 1 / (1 + exp(-z))
 *   dgu[m,f]   = bf16( dh * u * sig(g) * (1 + g * (1 - sig(g))) )     (dg)
 *   dgu[m,F+f] = bf16( dh * g * sig(g) )                              (du)
 * gu: bf16 [M, 2F], the wi forward output before SwiGLU (gate | up halves).
 * dgu: bf16 [M, 2F]; rows >= T untouched; dh is never written to memory.
 * Pointers 16-byte aligned; F % 16 == 0 and N % 16 == 0 (FP8MOE_EALIGN);
 * gu NULL with M > 0: FP8MOE_EINVAL.  No workspace (pass NULL, 0). */
int fp8moe_gmm_dlhs_dswiglu_fp8(const void* dout, int64_t M, int64_t N, const uint8_t* codes,
                                const float* scale, int32_t E, int64_t F, const void* gu,
                                const int32_t* group_sizes, void* dgu, void* workspace,
                                size_t workspace_bytes, fp8moe_stream_t stream);

/* fp8moe_gmm_dlhs_dswiglu_fp8 with the internal path forced (0 streaming,
 * 1 on-chip weight cache, N <= 256, 2 CTA pairs with the weight in tensor
 * memory); all give identical bits. */
int fp8moe_gmm_dlhs_dswiglu_fp8_path(const void* dout, int64_t M, int64_t N, const uint8_t* codes,
                                     const float* scale, int32_t E, int64_t F, const void* gu,
                                     const int32_t* group_sizes, void* dgu, int32_t path,
                                     fp8moe_stream_t stream);

/* Weight-gradient tgmm with in-kernel per-tile operand quantization -- [DQ]
 * What.  Segments: the global 128-row tiles [128t, 128t+128) intersected with
 * each group.  Per segment q and channel:
 *   sx[q,k] = max(max_{m in q} |lhs[m,k]|, 1e-12) / 448,  qx = e4m3(lhs / sx)
 *   sd[q,n] = max(max_{m in q} |dout[m,n]|, 1e-12) / 448, qd = e4m3(dout / sd)
 *   dW[e,k,n] = sum_{q of e} sx[q,k] * sd[q,n] * sum_{m in q} qx[m,k] * qd[m,n]
 * lhs: bf16 [M, K]; dout: bf16 [M, N]; dW: f32 [E, K, N], fully written
 * (experts without rows get 0).  Rows >= T are never read, so garbage there
 * (NaN, Inf) cannot reach dW.  Workspace: FP8MOE_OP_TGMM_DRHS_QUANT. */
int fp8moe_tgmm_drhs_quant(const void* lhs, const void* dout, int64_t M, int64_t K, int64_t N,
                           int32_t E, const int32_t* group_sizes, float* dW, void* workspace,
                           size_t workspace_bytes, fp8moe_stream_t stream);

/* fp8moe_tgmm_drhs_quant with the dout operand's fp8 format chosen -- [DQ]
 * What (configurable gradient dtype).  FP8MOE_FMT_E5M2:
 *   sd[q,n] = max(max_{m in q} |dout[m,n]|, 1e-12) / 57344, qd = e5m2(dout / sd)
 * (round to nearest even, saturating at +-57344); lhs stays e4m3 and the MMA
 * multiplies e4m3 x e5m2.  FP8MOE_FMT_E4M3 is fp8moe_tgmm_drhs_quant.  Any
 * other dout_fmt: FP8MOE_EINVAL.  Same workspace. */
int fp8moe_tgmm_drhs_quant_fmt(const void* lhs, const void* dout, int64_t M, int64_t K, int64_t N,
                               int32_t E, const int32_t* group_sizes, float* dW, void* workspace,
                               size_t workspace_bytes, int32_t dout_fmt, fp8moe_stream_t stream);

/* dequantize_fp8_codes -- [NQ] Implementation: out[e,k,n] =
 * bf16(f32(codes[e,k,n]) * scale[e,n]) (one f32 multiply, round to nearest
 * even).  out: bf16 [E, K, N]. */
int fp8moe_dequantize_fp8_codes(const uint8_t* codes, const float* scale, int32_t E, int64_t K,
                                int64_t N, void* out, fp8moe_stream_t stream);

/* BF16 grouped matmul, the fake-QAT comparison arm ([NQ] Tests: the BF16 GMM
 * takes a weight dequantized beforehand): out = bf16(lhs x w[e]) with f32
 * accumulation, w: bf16 [E, K, N]; swiglu != 0 applies the same SwiGLU
 * epilogue as fp8moe_gmm_silu_fp8_fwd (out [M, N/2]). */
int fp8moe_gmm_bf16_fwd(const void* lhs, int64_t M, int64_t K, const void* w, int32_t E,
                        int64_t N, const int32_t* group_sizes, int32_t swiglu, void* out,
                        fp8moe_stream_t stream);

/* Forward GMM with per-block activation quantization -- [NQ] Implementation:
 * the ops-level lhs_quant_block_size = 512 option (the pages' earlier default;
 * the production forward is fp8moe_gmm_fp8_fwd's full-K f32 scale).  Per row m
 * and block b of 512 columns (the last one may be shorter):
 *   sb[m,b] = bf16( max(max_{k in b} |lhs[m,k]|, 1e-12) / 448 ),  q = e4m3(lhs / sb)
 *   acc = 0 (bf16); for each block b:  acc = bf16( acc + sb[m,b] * P_b[m,n] ),
 *     P_b = the f32 product of the block's codes,  sum_{k in b} q[m,k] * codes[e,k,n]
 *   out[m,n] = bf16( acc * scale[e,n] ), or with swiglu = 1 the SwiGLU of the
 *   gate | up halves as fp8moe_gmm_silu_fp8_fwd (out [M, N/2]).
 * block must be 512 (FP8MOE_EINVAL otherwise).  Workspace:
 * FP8MOE_OP_GMM_FP8_FWD_BLOCK (codes and block scales).  Rows >= T untouched. */
int fp8moe_gmm_fp8_fwd_block(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                             const float* scale, int32_t E, int64_t N,
                             const int32_t* group_sizes, void* out, void* workspace,
                             size_t workspace_bytes, int32_t block, int32_t swiglu,
                             fp8moe_stream_t stream);

/* Parity export of the block quantization above: q u8 [M, K] and the
 * bf16-valued f32 scales sb [M, ceil(K/512)] for rows < T. */
int fp8moe_quantize_rows_block(const void* lhs, int64_t M, int64_t K, const int32_t* group_sizes,
                               int32_t E, int32_t block, uint8_t* q, float* sb,
                               fp8moe_stream_t stream);

/* Parity export of the forward activation quantization: q u8 [M, K] and
 * sx f32 [M] for rows < T (rows >= T untouched). */
int fp8moe_quantize_rows(const void* lhs, int64_t M, int64_t K, const int32_t* group_sizes,
                         int32_t E, uint8_t* q, float* sx, fp8moe_stream_t stream);

/* Parity export of the tgmm operand quantization.  Segments are numbered
 * expert by expert, tiles ascending; S = the segment bound ceil(M/128) + E.
 * Segment q of tile t fills slot q: slot row r holds buffer row 128t + r if it
 * belongs to the segment, else zero codes.  qx u8 [S, 128, K], sx f32 [S, K],
 * qd u8 [S, 128, N], sd f32 [S, N]; slots past the last segment untouched. */
int fp8moe_tgmm_quantize_tiles(const void* lhs, const void* dout, int64_t M, int64_t K,
                               int64_t N, int32_t E, const int32_t* group_sizes, uint8_t* qx,
                               float* sx, uint8_t* qd, float* sd, fp8moe_stream_t stream);

/* fp8moe_tgmm_quantize_tiles with the dout format chosen (FP8MOE_FMT_*): qd
 * holds e5m2 codes and sd the e5m2 scales when dout_fmt = FP8MOE_FMT_E5M2. */
int fp8moe_tgmm_quantize_tiles_fmt(const void* lhs, const void* dout, int64_t M, int64_t K,
                                   int64_t N, int32_t E, const int32_t* group_sizes, uint8_t* qx,
                                   float* sx, uint8_t* qd, float* sd, int32_t dout_fmt,
                                   fp8moe_stream_t stream);

/* Exercises the failure path of the bounded pipeline waits: one thread waits on
 * an mbarrier that nothing ever completes, gives up after limit_us
 * microseconds (1 .. 2,000,000, else FP8MOE_EINVAL), records
 * FP8MOE_STATUS_WAIT_TIMEOUT with where = 6 (bits 8..15) in the status word and
 * exits; the context stays usable.  For tests of failure detection; the paper
 * has no counterpart. */
int fp8moe_selftest_wait_timeout(uint32_t limit_us, fp8moe_stream_t stream);

/* The f32 -> fp8 cast that every quantizer of the library ends in, on
 * arbitrary inputs: codes[i] = RN_sat(x[i]) in the format fmt (FP8MOE_FMT_E4M3:
 * round to nearest even, saturating at +-448, NaN -> NaN code; FP8MOE_FMT_E5M2:
 * the same at +-57344), converted two values at a time by the same
 * cvt.rn.satfinite helpers as the quantizers ("MoE: native FP8 QAT for
 * routed-expert GMMs", Implementation: the e4m3 activation codes; "MoE fp8
 * backward: in-kernel drhs operand quantization", What: the e5m2 gradient
 * codes).  x f32 [n] and codes u8 [n] are device pointers, x 4-byte aligned;
 * the caller owns both.  n = 0 does nothing.  FP8MOE_EINVAL: n < 0, an unknown
 * fmt, or a null pointer with n > 0.  For parity tests of the cast over whole
 * binades of bit patterns. */
int fp8moe_selftest_cast_f32(const float* x, int64_t n, int32_t fmt, uint8_t* codes,
                             fp8moe_stream_t stream);

/* Waits for `stream`, returns in *flags the OR of the FP8MOE_STATUS_* bits set
 * since the last call, and clears them.  A bit that is set meanwhile, by work on
 * another stream, is in this call's flags or in a later one's, never lost. */
int fp8moe_read_status(fp8moe_stream_t stream, uint32_t* flags);

/* The wi forward of fp8moe_gmm_silu_fp8_fwd for callers that cannot allocate
 * device memory (a plugin inside a framework whose caching allocator holds
 * nearly all of it, or a runtime that forbids allocations after start-up).  The
 * pages have no counterpart: it is an interface variant, not a step of the
 * method.  Arguments and results are those of fp8moe_gmm_silu_fp8_fwd minus the
 * workspace, which comes from a fixed 32 MiB device array that the library holds
 * on every GPU it is loaded on until the process exits; sizes whose workspace
 * (fp8moe_workspace_size(FP8MOE_OP_GMM_SILU_FP8_FWD, ...)) exceeds it return
 * FP8MOE_EWORKSPACE and launch nothing.  Argument errors are checked first and
 * return what fp8moe_gmm_silu_fp8_fwd would (FP8MOE_EINVAL, FP8MOE_EALIGN),
 * whatever the size.  The first call on a device looks up the array's device
 * address and keeps it (make that call before any stream capture); after a
 * cudaDeviceReset the kept address is stale, so do not call this again in that
 * process.  All calls share the array, so calls that overlap on the GPU race;
 * each call rewrites everything it reads, so nothing needs clearing between
 * calls.  Allocates nothing. */
int fp8moe_gmm_silu_fp8_fwd_noalloc(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                                    const float* scale, int32_t E, int64_t N,
                                    const int32_t* group_sizes, void* out,
                                    fp8moe_stream_t stream);

/* ---- Tokens sorted by expert and back (no counterpart on the pages: the layer
 * around the routed experts that the ragged buffer above belongs to).
 *
 * ids int32 [T, topk]: the experts that a router chose for each token, 1 <= topk
 * <= 32, T * topk < 2^31.  Slot s = t * topk + j is token t's j-th choice.  A slot
 * whose id is negative has no row (an expert of another rank, a padding token); so
 * has one whose id is >= E, which also sets FP8MOE_STATUS_BAD_EXPERT.  The rows of
 * the other slots are sorted by expert and, inside an expert, by slot: the order
 * does not depend on scheduling.  Rows that would be at or past M are dropped,
 * group_sizes is clipped accordingly and FP8MOE_STATUS_GROUPS_EXCEED_M set.
 *   group_sizes int32 [E]        rows of each expert (what the grouped products take)
 *   slot_row    int32 [T, topk]  the row of a slot, -1 for none
 *   row_slot    int32 [M]        the slot of a row, -1 past the last (NULL: not written)
 * All three are fully written, also when T = 0.  4-byte aligned. */
int fp8moe_sort_tokens(const int32_t* ids, int64_t T, int32_t topk, int32_t E, int64_t M,
                       int32_t* group_sizes, int32_t* slot_row, int32_t* row_slot,
                       fp8moe_stream_t stream);

/* fp8moe_sort_tokens, and the copy of each token to its rows:
 *   rows[slot_row[t, j]] = x[t].   x: [T, H] of `type` (FP8MOE_TYPE_*), rows: [M, H];
 * rows past the last are not written.  H * element size must be a multiple of 16
 * (FP8MOE_EALIGN). */
int fp8moe_dispatch_tokens(const void* x, const int32_t* ids, int64_t T, int32_t topk, int64_t H,
                           int32_t type, int32_t E, int64_t M, void* rows, int32_t* group_sizes,
                           int32_t* slot_row, int32_t* row_slot, fp8moe_stream_t stream);

/* The weighted sum of a token's rows, f32 in the order of j, rounded once:
 *   out[t] = sum_j weights[t, j] * rows[slot_row[t, j]]       (weights f32 [T, topk])
 * weights NULL: all 1, which is also the gradient of fp8moe_dispatch_tokens (rows:
 * the rows' gradient, out: x's).  A slot without a row, or with one outside
 * [0, M), adds nothing, whatever its weight; a token without rows gives 0.  No other
 * row is read. */
int fp8moe_combine_tokens(const void* rows, int64_t M, int64_t H, int32_t type,
                          const int32_t* slot_row, const float* weights, int64_t T, int32_t topk,
                          void* out, fp8moe_stream_t stream);

/* Gradient of fp8moe_combine_tokens:
 *   drows[slot_row[t, j]] = weights[t, j] * dout[t]
 *   dweights[t, j]        = sum_h dout[t, h] * rows[slot_row[t, j], h]   (f32; 0 without a row)
 * A row belongs to one slot at most (as fp8moe_sort_tokens makes it); rows that no slot
 * names are not written. */
int fp8moe_combine_tokens_bwd(const void* dout, const void* rows, int64_t M, int64_t H,
                              int32_t type, const int32_t* slot_row, const float* weights,
                              int64_t T, int32_t topk, void* drows, float* dweights,
                              fp8moe_stream_t stream);

/* ---- Norms after and before a block, with the block's gate and the scaled
 * residual sum (no counterpart on the pages).  x (residual stream), y (block
 * output), r, h: [T, H] of `type`; norm weights f32 [H]; rstd f32 [T].
 *   rstd(z) = 1 / sqrt(mean_h z^2 + eps)
 *   r = residual_scale * x + branch_scale * g * (w_post * y * rstd(y))
 *   h = w_pre * r * rstd(r)                 (of r before it is rounded to `type`)
 * g: 1, or `gate` by gate_kind (FP8MOE_GATE_*), through 1 / (1 + exp(-gate)) with
 * sigmoid = 1.  w_post NULL: no block output (y NULL, no gate, the scales are not
 * used); r is x, is not written, and only h is.  w_pre NULL: no h.  At least one of them is given.
 * rstd_post and rstd_pre are what the gradient takes.  eps >= 0 (FP8MOE_EINVAL; with 0 a
 * row of zeros gives NaN).  H * element size: a multiple of 16 (FP8MOE_EALIGN), at most
 * 32768 (FP8MOE_EINVAL).  All sums are f32: a row keeps f32's relative precision, in
 * both directions, while its sum of squares is a normal f32 number (or eps holds it up). */
int fp8moe_norm_fwd(const void* x, const void* y, int64_t T, int64_t H, int32_t type,
                    const float* w_post, const float* w_pre, const void* gate, int32_t gate_kind,
                    int32_t sigmoid, float residual_scale, float branch_scale, float eps, void* r,
                    void* h, float* rstd_post, float* rstd_pre, fp8moe_stream_t stream);

/* Gradient of fp8moe_norm_fwd.  dr: the gradient of r from the residual stream (NULL:
 * 0, only with w_pre); dh: of h (with w_pre); r: the forward's r (without w_post: x).
 *   D  = dr + rstd_pre * (w_pre dh - rh * mean(w_pre dh rh)),      rh = r rstd_pre
 *   dx = residual_scale * D,   dn = branch_scale * D * g,          yh = y rstd_post
 *   dy = rstd_post * (w_post dn - yh * mean(w_post dn yh))
 *   dw_pre = sum_t dh rh,   dw_post = sum_t dn yh                  (f32 [H])
 *   dgate = branch_scale * D * w_post * yh, summed over what shares a gate value, times
 *   g (1 - g) with sigmoid = 1: f32 [T], f32 [H] or [T, H] of `type`, by gate_kind
 * Without w_post dx = D (r is x; the scales are not used).  Column sums are joined in a fixed order.
 * T = 0 writes zeros to dw_post, dw_pre and a per-channel dgate, whatever the weights and
 * the gate hold.  Workspace: FP8MOE_OP_NORM_BWD with M = T, K = H. */
int fp8moe_norm_bwd(const void* dr, const void* dh, const void* r, const void* y, int64_t T,
                    int64_t H, int32_t type, const float* w_post, const float* w_pre,
                    const float* rstd_post, const float* rstd_pre, const void* gate,
                    int32_t gate_kind, int32_t sigmoid, float residual_scale, float branch_scale,
                    void* dx, void* dy, float* dw_post, float* dw_pre, void* dgate,
                    void* workspace, size_t workspace_bytes, fp8moe_stream_t stream);

/* ---- Microscaled 4-bit floating point (OCP MXFP4; no counterpart on the pages):
 * e2m1 elements (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) in blocks of 32
 * along K, each block with a power-of-two scale X:
 *   X = 2^(floor(log2 max|v|) - 2), at least 2^-127;  scale byte = log2 X + 127
 *   code = e2m1(v / X), round to nearest even, saturating
 * A block with an infinity or a NaN gets scale byte 0xFF (NaN) and codes 0: what is
 * computed from it is NaN.  K must be a multiple of 32, N of 16 (FP8MOE_EALIGN).
 *   codes of weights      u8 [E, N, K/2], two a byte along K, even k in the low half
 *   scales of weights     u8 [E, ceil(K/128), N, 4]: four consecutive blocks of a row
 *                         together; bytes past K/32 mean nothing and are never used
 *   codes, scales of rows u8 [M, K/2], u8 [ceil(K/128), M, 4] */

/* Rows < T of lhs bf16 [M, K] (what the products do with their activations);
 * codes and scales of rows >= T untouched. */
int fp8moe_mxfp4_quantize_rows(const void* lhs, int64_t M, int64_t K, const int32_t* group_sizes,
                               int32_t E, uint8_t* codes, uint8_t* scales, fp8moe_stream_t stream);

/* Expert weights w bf16 [E, K, N] (N contiguous, as every weight of this library). */
int fp8moe_mxfp4_quantize_weights(const void* w, int32_t E, int64_t K, int64_t N, uint8_t* codes,
                                  uint8_t* scales, fp8moe_stream_t stream);

/* out bf16 [E, N, K] = code * X (exact wherever bf16 can hold it).  As the weight of
 * fp8moe_gmm_bf16_fwd, with its K and N exchanged, it gives the gradient of a
 * product's activations taken as if they were not rounded (straight through). */
int fp8moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t E, int64_t N,
                            int64_t K, void* out, fp8moe_stream_t stream);

/* The grouped product on 4-bit weights: the activation rows are quantised as above
 * (into the workspace), then for row m of expert e
 *   out[m, n] = bf16( sum_k (qx Xx)[m, k] * (qw Xw)[e, n, k] )        (f32 accumulation)
 * lhs: bf16 [M, K]; out: bf16 [M, N]; rows >= T untouched.  Any number of rows per
 * expert, from none to all.  Workspace: FP8MOE_OP_GMM_MXFP4_FWD. */
int fp8moe_gmm_mxfp4_fwd(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                         const uint8_t* scales, int32_t E, int64_t N, const int32_t* group_sizes,
                         void* out, void* workspace, size_t workspace_bytes,
                         fp8moe_stream_t stream);

/* The same with the SwiGLU of fp8moe_gmm_silu_fp8_fwd (gate | up halves of N, N a
 * multiple of 32): out bf16 [M, N/2].  Workspace: FP8MOE_OP_GMM_SILU_MXFP4_FWD. */
int fp8moe_gmm_silu_mxfp4_fwd(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                              const uint8_t* scales, int32_t E, int64_t N,
                              const int32_t* group_sizes, void* out, void* workspace,
                              size_t workspace_bytes, fp8moe_stream_t stream);

/* ---- The router in front of the experts (no counterpart on the pages): the choice of experts
 * with its weights, the balance loss with the experts' counts, and the gradient of both.
 *
 * logits: [T, E] of `type` (FP8MOE_TYPE_*), 1 <= E <= 1024, 1 <= topk <= min(32, E).
 *   s      = softmax over the token's E logits, or sigmoid of each (`score`, FP8MOE_SCORE_*)
 *   chosen = the topk experts with the largest logit, or, with bias f32 [E], with the largest
 *            s + bias; equal ones by number. Values that f32 cannot tell apart are compared in
 *            64 bits. An expert whose logit (or bias) is -inf is never chosen.
 *   weights[t, j] = scale * s_j / (sum of the chosen s), or scale * s_j with normalize = 0
 * The bias takes part in the choice alone. Slots without an expert have id -1 and weight 0, as
 * have all slots of a token that belongs to no sequence; a NaN logit ranks first and spoils the
 * token's weights.
 *
 * seq_offsets: int32 [B + 1], where the batch's B sequences begin and end (token t belongs to
 * sequence b if seq_offsets[b] <= t < seq_offsets[b + 1]; what lies before the first and behind
 * the last is padding), or NULL with B = 1: all tokens are one sequence. Offsets below 0, falling
 * or past T are clipped, what depends on them is unspecified, and FP8MOE_STATUS_BAD_OFFSETS is
 * set where the balance loss is computed.
 *
 * Balance loss of each sequence, over the n tokens with a choice and their C choices:
 *   p_i = s_i / sum s (a token's share of expert i);  counts_i = choices of expert i
 *   slope_i = E * counts_i / (C * n),   loss = sum_i slope_i * sum_t p_ti
 * which is 1 when choices or shares are even. counts int32 [B, E], loss f32 [B], slope f32 [B, E]
 * (the loss's derivative by a token's share; what the gradient takes); zeros for a sequence without
 * choices. Sums are f32 and added up in a fixed order.
 *
 * fp8moe_router_fwd: ids int32 [T, topk], weights f32 [T, topk], and, unless counts, loss and
 * slope are NULL, the balance loss. Workspace: FP8MOE_OP_BALANCE with M = T, N = B (with the
 * balance loss; else NULL, 0). */
int fp8moe_router_fwd(const void* logits, int64_t T, int32_t E, int32_t type, int32_t score,
                      const float* bias, int32_t topk, int32_t normalize, float scale,
                      const int32_t* seq_offsets, int32_t B, int32_t* ids, float* weights,
                      int32_t* counts, float* loss, float* slope, void* workspace,
                      size_t workspace_bytes, fp8moe_stream_t stream);

/* The balance loss of choices that were made elsewhere: ids int32 [T, topk]. A negative id is
 * no choice; one >= E is none either and sets FP8MOE_STATUS_BAD_EXPERT. */
int fp8moe_balance_fwd(const void* logits, const int32_t* ids, int64_t T, int32_t E, int32_t type,
                       int32_t score, int32_t topk, const int32_t* seq_offsets, int32_t B,
                       int32_t* counts, float* loss, float* slope, void* workspace,
                       size_t workspace_bytes, fp8moe_stream_t stream);

/* Gradient of the weights (dweights f32 [T, topk]; NULL: 0) and of the balance losses (dloss
 * f32 [B], with the forward's slope; both NULL: 0) into the logits, dlogits [T, E] of `type`:
 *   dx_i = q_i * (scale w_i (dw_i - sum dw w) + p_i (D_i - sum D p)),   D = dloss_b * slope_b,
 *   w: the normalised weights without `scale`, q = 1 (softmax) or sigmoid(-x_i)
 * (normalize = 0: of softmax scores scale * dw joins D, of sigmoid scores the first term is
 * scale * dw_i * s_i). ids: the forward's, or given ones (one that occurs twice counts twice).
 * The choice and the bias have no gradient. dlogits is fully written: zeros for a token without
 * a choice or outside the sequences. No workspace. */
int fp8moe_router_bwd(const float* dweights, const void* logits, const int32_t* ids, int64_t T,
                      int32_t E, int32_t type, int32_t score, int32_t topk, int32_t normalize,
                      float scale, const float* dloss, const float* slope,
                      const int32_t* seq_offsets, int32_t B, void* dlogits,
                      fp8moe_stream_t stream);

/* ---- AdamW over many tensors at once (no counterpart on the pages): what turns the gradients
 * into the next step's weights. For each value, g = grad_scale * g (where one is given):
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * p is f32 (master weights), g bf16 or f32. Every operation is rounded to f32 by itself (root and
 * quotient to the nearest, but for about one in 2^22 that lies next to the middle of two values; a
 * quotient below 2^-126 may keep more bits than f32 has there): a step has one result for a value,
 * which depends neither on its neighbours (but for those in the block of an 8-bit moment), nor on
 * where its tensor lies, nor on what else is in the call.
 *
 * Moments are f32 (state_bits = 32), or (8) e4m3 codes of m and of sqrt(v) with an f32 scale for
 * each 128 consecutive values (the last block may be shorter): scale = largest magnitude / 448,
 * or 0 where that is below 2^-126; code * scale is the value. A value between two codes takes
 * the upper one with the probability that keeps the mean, by 16 bits of a hash of its place, of
 * the tensor's number in the call, t and seed: the same inputs give the same result. The code of
 * a second moment above zero is never zero. Codes and scales of zero are moments of zero.
 * A NaN or an infinity in a block's moments makes the block NaN or infinite in the next step.
 *
 * copy (may be NULL): bf16 of the new p. codes with code_scale (may be NULL): p is expert weights
 * [E, K, N], n = E K N, E at most 1024, K and N multiples of 16 up to 2^21, and the new weights
 * come as the forward takes them, code_scale f32 [E, N] = max(max_k |p|, 1e-12) / 448, codes u8
 * [E, K, N] = e4m3(p / code_scale), round to nearest even. */
typedef struct fp8moe_adamw_tensor {
  float* p;
  const void* g;
  void* m;               /* f32 or u8 [n] */
  void* v;
  float* m_scale;        /* f32 [ceil(n / 128)] with 8 bits, else NULL */
  float* v_scale;
  void* copy;            /* bf16 [n] or NULL */
  uint8_t* codes;        /* u8 [n] or NULL */
  float* code_scale;     /* f32 [E, N] with codes */
  int64_t n;             /* values; 0: skipped, no pointer is looked at */
  int64_t K, N;          /* with codes */
  double weight_decay;
  int32_t g_type;        /* FP8MOE_TYPE_* */
  int32_t state_bits;    /* 32 or 8 */
} fp8moe_adamw_tensor;

/* `tensors` is a HOST array of `count` entries, read during the call (its pointers are device
 * pointers); no two entries may overlap, nor may a gradient overlap what a step writes. Values need
 * the alignment of their type only. t: `step` >= 1, or *step_dev (int64 on the device, NULL: `step`);
 * the rate: `lr`, or *lr_dev (f32 on the device, NULL: `lr`): a captured step follows what they hold
 * when it is replayed. grad_scale: f32 on the device or NULL. 0 <= beta < 1, eps >= 0 (with 0 a value
 * that never had a gradient becomes NaN). Workspace: fp8moe_adamw_workspace_size (256-byte aligned),
 * with on_device = 1 if step_dev or lr_dev is given; calls that overlap on the GPU need one each. */
size_t fp8moe_adamw_workspace_size(const fp8moe_adamw_tensor* tensors, int32_t count,
                                   int32_t on_device);
int fp8moe_adamw_step(const fp8moe_adamw_tensor* tensors, int32_t count, int64_t step,
                      const int64_t* step_dev, double lr, const float* lr_dev, double beta1,
                      double beta2, double eps, const float* grad_scale, uint32_t seed,
                      void* workspace, size_t workspace_bytes, fp8moe_stream_t stream);

/* Text for a return code. */
const char* fp8moe_status_string(int code);

/* The cudaError_t value behind the last FP8MOE_ECUDA of this thread. */
int fp8moe_last_cuda_error(void);

/* Number of SMs the kernels size their grids for (0 if no device). */
int fp8moe_num_sms(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8MOE_H_ */
