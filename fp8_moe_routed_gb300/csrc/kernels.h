// kernels.h -- internal launchers of the CUDA library (host side).  The public
// C ABI lives in include/fp8moe.h; these are the per-file entry points that
// api.cu calls after validating arguments and building tensor maps.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

// Rows of experts [e0, e1); ctas_per_sm bounds the grid (resident CTAs per SM).
cudaError_t fp8moe_launch_quantize_rows(const void* lhs, int64_t M, int K, const int32_t* gs,
                                        int E, int e0, int e1, uint8_t* q, float* sx, int num_sms,
                                        int ctas_per_sm, int report, cudaStream_t s);
// Per-512-column block quantization: codes q [M, K], bf16-valued scales sb [M, ceil(K/512)].
cudaError_t fp8moe_launch_quantize_rows_block(const void* lhs, int64_t M, int K, const int32_t* gs,
                                              int E, uint8_t* q, float* sb, int num_sms, int report,
                                              cudaStream_t s);
cudaError_t fp8moe_launch_tgmm_quantize_tiles(const void* lhs, const void* dout, int64_t M, int K,
                                              int N, const int32_t* gs, int E, int64_t Smax,
                                              uint8_t* qx, float* sx, uint8_t* qd, float* sd,
                                              int num_sms, int report, int d_fmt,
                                              cudaStream_t s);
cudaError_t fp8moe_launch_dequantize(const uint8_t* codes, const float* scale, int E, int64_t K,
                                     int64_t N, void* out, int num_sms, cudaStream_t s);

// Forward grouped matmul (FP8 x FP8 or the BF16 comparison arm).
struct GmmFwdArgs {
  CUtensorMap tmA;        // A operand tiles (codes [M, K] u8, or lhs [M, K] bf16)
  CUtensorMap tmB;        // B operand tiles (weights [E, K, N], N contiguous)
  const float* sx;        // [M] row scales (FP8 arm) or nullptr
  const float* scale;     // [E, N] channel scales (FP8 arm) or nullptr
  const int32_t* gs;      // [E]
  void* out;              // bf16 [M, Nout]
  int64_t M;
  int K, N, E, swiglu;
  int e0, e1;             // only the units of experts [e0, e1)
  int blk;                // 1: sx holds per-512-column block scales [M, ceil(K/512)] and the
                          //    accumulation across blocks is bf16 (FP8 arm only)
};
cudaError_t fp8moe_launch_gmm_fp8_fwd(const GmmFwdArgs& a, int num_sms, cudaStream_t s);
cudaError_t fp8moe_launch_gmm_bf16_fwd(const GmmFwdArgs& a, int num_sms, cudaStream_t s);

struct GmmDlhsArgs {
  CUtensorMap tmA;        // dout [M, N] bf16 tiles
  CUtensorMap tmC;        // codes [E, K, N] u8 tiles [256 k x 64 n], no swizzle
  CUtensorMap tmCp;       // the same codes as [128 k x 64 n] tiles, 64-byte swizzle (pair path)
  const float* scale;     // [E, N]
  const int32_t* gs;
  const void* gu;         // bf16 [M, 2K] wi output (gate | up) for the dSwiGLU epilogue, or null
  void* dlhs;             // bf16 [M, K], or [M, 2K] dgu with the dSwiGLU epilogue
  int64_t M;
  int N, K, E;
};
// path: 0 streaming, 1 on-chip weight cache (N <= 256), 2 CTA pairs with the
// dequantized weight in tensor memory.
cudaError_t fp8moe_launch_gmm_dlhs(const GmmDlhsArgs& a, int num_sms, int path, cudaStream_t s);
// The pair kernel alone (gmm_dlhs_pair.cu); fp8moe_launch_gmm_dlhs routes path 2 here.
cudaError_t fp8moe_launch_gmm_dlhs_pair(const GmmDlhsArgs& a, int num_sms, cudaStream_t s);

struct TgmmArgs {
  CUtensorMap tmX;        // qx slots [S, 128, K] u8
  CUtensorMap tmD;        // qd slots [S, 128, N] u8
  CUtensorMap tmW;        // dW [E, K, N] f32 (store)
  const float* sx;        // [S, K]
  const float* sd;        // [S, N]
  const int32_t* gs;
  float* dW;              // [E, K, N]
  int64_t M;
  int K, N, E;
  int d_fmt;              // qd codes: 0 e4m3, 1 e5m2
};
cudaError_t fp8moe_launch_tgmm(const TgmmArgs& a, int num_sms, cudaStream_t s);

// Records the CUDA error that fp8moe_last_cuda_error() reports (api.cu).
extern "C" void fp8moe_internal_set_cuda_error(int e);
extern "C" int fp8moe_internal_check_fwd_args(const void* lhs, int64_t M, int64_t K,
                                              const uint8_t* codes, const float* scale, int32_t E,
                                              int64_t N, const int32_t* gs, const void* out,
                                              int swiglu, int* empty);

// Waits for the stream; *flags receives the OR of all status words, which are cleared
// (status.cu).
cudaError_t fp8moe_collect_status(uint32_t* flags, cudaStream_t s);
// Addresses of the translation units' status words on the current device.
cudaError_t fp8moe_status_take_quant(uint32_t** word);
cudaError_t fp8moe_status_take_dequant(uint32_t** word);
cudaError_t fp8moe_status_take_gmm_fwd(uint32_t** word);
cudaError_t fp8moe_status_take_dlhs(uint32_t** word);
cudaError_t fp8moe_status_take_dlhs_pair(uint32_t** word);
cudaError_t fp8moe_status_take_tgmm(uint32_t** word);
cudaError_t fp8moe_status_take_selftest(uint32_t** word);

// One thread waits on an mbarrier that nothing completes for limit_ns, then
// records a wait timeout (selftest.cu).
cudaError_t fp8moe_launch_selftest_wait(uint64_t limit_ns, cudaStream_t s);
// Converts n f32 values to fp8 codes (fmt 0 e4m3, 1 e5m2) with the quantizers'
// cast (selftest.cu).
cudaError_t fp8moe_launch_selftest_cast(const float* x, int64_t n, int fmt, uint8_t* out,
                                        int num_sms, cudaStream_t s);

// Tokens sorted by expert and back (route.cu). n = T * topk slots; nvec = 16-byte
// vectors of a row; f32: rows hold f32 instead of bf16.
cudaError_t fp8moe_status_take_route(uint32_t** word);
cudaError_t fp8moe_launch_sort_tokens(const int32_t* ids, int64_t n, int E, int64_t M,
                                      int32_t* group_sizes, int32_t* slot_row, int32_t* row_slot,
                                      cudaStream_t s);
// The sort and the copy; rows is not touched when M == 0.
cudaError_t fp8moe_launch_dispatch(const void* x, const int32_t* ids, int64_t T, int topk, int E,
                                   int64_t M, int nvec, void* rows, int32_t* group_sizes,
                                   int32_t* slot_row, int32_t* row_slot, int num_sms,
                                   cudaStream_t s);
cudaError_t fp8moe_launch_combine(const void* rows, int64_t T, int topk, int nvec, int f32,
                                  const int32_t* slot_row, int64_t M, const float* weights,
                                  void* out, cudaStream_t s);
cudaError_t fp8moe_launch_combine_bwd(const void* dout, const void* rows, int64_t T, int topk,
                                      int nvec, int f32, const int32_t* slot_row, int64_t M,
                                      const float* weights, void* drows, float* dweights,
                                      cudaStream_t s);

// Norms around a block (norm.cu). gate_kind: 0 none, 1 per row, 2 per column, 3 per element.
struct NormFwdArgs {
  const void* x;
  const void* y;          // null: no block output, only h = norm(x)
  const float* w_post;    // with y
  const float* w_pre;     // null: no h
  const void* gate;
  int gate_kind, sigmoid;
  float residual_scale, branch_scale, eps;
  int64_t T;
  int H, f32;
  void* r;
  void* h;
  float* rstd_post;
  float* rstd_pre;
};
cudaError_t fp8moe_launch_norm_fwd(const NormFwdArgs& a, int num_sms, cudaStream_t s);

struct NormBwdArgs {
  const void* dr;         // may be null (with dh)
  const void* dh;         // null: no pre norm
  const void* r;
  const void* y;          // null: no post norm
  const float* w_post;
  const float* w_pre;
  const float* rstd_post;
  const float* rstd_pre;
  const void* gate;
  int gate_kind, sigmoid;
  float residual_scale, branch_scale;
  int64_t T;
  int H, f32;
  void* dx;
  void* dy;
  float* dw_post;
  float* dw_pre;
  void* dgate;
  float* part;            // 2 * fp8moe_norm_bwd_ctas(T) * H
};
int fp8moe_norm_bwd_ctas(int64_t T);
cudaError_t fp8moe_launch_norm_bwd(const NormBwdArgs& a, int num_sms, cudaStream_t s);
cudaError_t fp8moe_status_take_norm(uint32_t** word);

// Microscaled 4-bit quantisation (mxfp4.cu).
// scale_stride: words between the scale words of consecutive 128 k (>= M).
cudaError_t fp8moe_launch_mxfp4_quantize_rows(const void* x, int64_t M, int K, const int32_t* gs,
                                              int E, uint8_t* codes, uint8_t* scales,
                                              int64_t scale_stride, int num_sms, int report,
                                              cudaStream_t s);
cudaError_t fp8moe_launch_mxfp4_quantize_weights(const void* w, int E, int K, int N, uint8_t* codes,
                                                 uint8_t* scales, cudaStream_t s);
cudaError_t fp8moe_launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int E,
                                           int N, int K, void* out, int num_sms, cudaStream_t s);
cudaError_t fp8moe_status_take_mxfp4(uint32_t** word);

// Grouped product of MXFP4 operands (gmm_mxfp4.cu).
struct GmmMxfp4Args {
  CUtensorMap tmW;          // weight codes: [E, N, K/2] boxes of 128 rows, or with SwiGLU
                            // [E, F/16, 2, 16, K/2] boxes of 4 x 2 x 16 rows
  CUtensorMap tmX[3];       // activation codes [M, K/2], boxes of fp8moe_gmm_mxfp4_boxes() rows
  CUtensorMap tmSw;         // weight scale words [E, ceil(K/128), N], boxes of 2 x 128, or with
                            // SwiGLU [E, ceil(K/128), F/16, 2, 16], boxes of 2 x 4 x 2 x 16
  CUtensorMap tmSx;         // activation scale words [ceil(K/128), M], boxes of 2 x scale_rows
  const int32_t* gs;
  void* out;                // bf16 [M, N] or [M, N/2]
  int64_t M;
  int K, N, E, swiglu;
};
void fp8moe_gmm_mxfp4_boxes(int rows[3], int* scale_rows);
cudaError_t fp8moe_launch_gmm_mxfp4(const GmmMxfp4Args& a, int num_sms, cudaStream_t s);
cudaError_t fp8moe_status_take_gmm_mxfp4(uint32_t** word);

// The router (router.cu). given: the choices, made elsewhere (null: chosen here, into ids and
// weights). part_*: the parts of the balance sums, (chunks + B) rows (null: no balance).
struct RouterArgs {
  const void* logits;
  const int32_t* given;
  const float* bias;
  int32_t* ids;
  float* weights;
  const int32_t* offsets;   // [B + 1], or null: one sequence
  float* part_share;
  int32_t* part_count;
  int32_t* part_tokens;
  int32_t* counts;
  float* loss;
  float* slope;
  int64_t T;
  int E, k, B, f32, sig, normalize;
  float scale;
  int chunk;                // set by the launcher
};
// Tokens of a CTA, whose balance sums are one part for each sequence among them.
int fp8moe_balance_chunk(int64_t T);
cudaError_t fp8moe_launch_router(const RouterArgs& a, cudaStream_t s);
// Many tokens (router_group.cu): without the join of the balance sums.
cudaError_t fp8moe_launch_router_groups(const RouterArgs& a, cudaStream_t s);

struct RouterBwdArgs {
  const void* logits;
  const int32_t* ids;
  const float* dweights;    // null: only the balance loss
  const int32_t* offsets;
  const float* dloss;       // null: only the weights
  const float* slope;
  void* dlogits;
  int64_t T;
  int E, k, B, f32, sig, normalize;
  float scale;
};
cudaError_t fp8moe_launch_router_bwd(const RouterBwdArgs& a, cudaStream_t s);
cudaError_t fp8moe_status_take_router(uint32_t** word);
cudaError_t fp8moe_status_take_router_group(uint32_t** word);
cudaError_t fp8moe_status_take_router_bwd(uint32_t** word);

// AdamW (adamw.cu): a tensor in a launch's table.
struct AdamwEntry {
  float* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  void* copy;               // bf16, or null
  int64_t n;
  double weight_decay;
  float keep;               // 1 - lr * weight_decay, unless the rates are on the device
  uint32_t first_unit;      // set by the launcher
  uint32_t which;           // the tensor's number in the call
  uint8_t g_bf16;
  uint8_t vec, head;        // from the value number `head` on, all arrays lie on 16 bytes
};
struct AdamwRates {         // from a step or a rate on the device
  double lr;
  float rate, root;
  uint32_t key;
};
struct AdamwCommon {
  const AdamwRates* rates;  // null: the values below
  const float* grad_scale;
  float rate, root, b1, c1, b2, c2, eps;
  float minus_zero;         // -0, of which the compiler knows nothing
  uint32_t key;
  int prepared;             // the kernel right in front of this launch is the preparation
  int count, unit_stages;   // set by the launcher, as is the next
  uint32_t units;
};
constexpr int kAdamwEntries = 360;     // of 88 bytes: a launch has 32764 bytes of parameters
uint64_t fp8moe_adamw_units(const AdamwEntry& d);
cudaError_t fp8moe_launch_adamw(const AdamwCommon& common, AdamwEntry* at, int count, int bits,
                                int num_sms, cudaStream_t s);

// One tensor of expert weights [E, K, N] with its codes; all arrays on 16 bytes, and with 8 bits N
// a multiple of 128.
struct AdamwSlabEntry : AdamwEntry {
  uint32_t* most;           // [E, N] on 16 bytes, the columns' largest magnitudes: zeros first
  int32_t K, N;
};
struct AdamwSlabArgs {
  CUtensorMap tm_p, tm_g, tm_m, tm_v;  // [E, K, N] boxes of fp8moe_adamw_tile()
  AdamwCommon c;
  AdamwSlabEntry d;
  uint8_t* codes;
  float* scale;
  uint32_t* counters;       // fp8moe_adamw_slab_counters(), zeros to begin with: the next unit,
                            // then the tiles done of each slab
  uint32_t strips, per_slab, slabs, units;   // set by the launcher
};
uint32_t fp8moe_adamw_slab_counters(int64_t n, int64_t K, int64_t N);
void fp8moe_adamw_tile(int* cols, int* rows);
cudaError_t fp8moe_launch_adamw_slabs(const AdamwSlabArgs& args, int bits, int num_sms,
                                      cudaStream_t s);
cudaError_t fp8moe_launch_adamw_prepare(AdamwRates* rates, const int64_t* step, int64_t host_step,
                                        const float* lr, double host_lr, double beta1,
                                        double beta2, uint32_t seed, uint32_t* most, int64_t count,
                                        cudaStream_t s);
// The codes of weights that the step went through in order. most: zeros to begin with.
cudaError_t fp8moe_launch_weight_codes(const float* p, int E, int K, int N, uint32_t* most,
                                       uint8_t* codes, float* scale, cudaStream_t s);
cudaError_t fp8moe_status_take_adamw(uint32_t** word);
