// api.cu -- the C ABI of libfp8moe.so (declared in include/fp8moe.h): argument
// checks, workspace carving, TMA tensor maps and kernel launches.  Every step of
// the path runs in the kernels of this library; there is no host fallback.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "fp8moe.h"
#include "kernels.h"

namespace {

thread_local int t_last_cuda_error = 0;

constexpr int kMaxDevices = 64;
struct DeviceInfo {
  int ready = 0;
  int num_sms = 0;
  int supported = 0;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_mu;

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

int cuda_fail(cudaError_t e) {
  t_last_cuda_error = (int)e;
  (void)cudaGetLastError();   // do not leave a non-sticky error for the caller's next call
  return FP8MOE_ECUDA;
}

// Lazy per-device set-up: SM count, architecture check, the driver's tensor-map
// encoder.  Returns FP8MOE_OK or an error code; *sms receives the SM count.
int device_init(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return FP8MOE_EUNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    cudaDeviceProp p;
    e = cudaGetDeviceProperties(&p, dev);
    if (e != cudaSuccess) return cuda_fail(e);
    d.num_sms = p.multiProcessorCount;
    d.supported = (p.major == 10 && p.minor == 3);
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                           cudaEnableDefault, &q);
      if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn)
        return cuda_fail(e != cudaSuccess ? e : cudaErrorNotSupported);
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    d.ready = 1;
  }
  if (!d.supported) return FP8MOE_EUNSUPPORTED;
  *sms = d.num_sms;
  return FP8MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }


size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int64_t segment_bound(int64_t M, int32_t E) { return (M + 127) / 128 + E; }

// rank-2 to rank-5 tiled tensor map; dims[0] is the contiguous one.
int make_tmap(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base,
              const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
              CUtensorMapSwizzle sw) {
  cuuint64_t gd[5];
  cuuint64_t gs[4];
  cuuint32_t bx[5];
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    gd[i] = dims[i];
    bx[i] = box[i];
  }
  for (int i = 0; i < rank - 1; ++i) gs[i] = strides_bytes[i];
  CUresult r = g_encode(m, dt, (cuuint32_t)rank, const_cast<void*>(base), gd, gs, bx, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    t_last_cuda_error = (int)r;
    return FP8MOE_ECUDA;
  }
  return FP8MOE_OK;
}

int check_common(int64_t M, int64_t K, int64_t N, int32_t E) {
  if (M < 0 || M >= (int64_t(1) << 31)) return FP8MOE_EINVAL;
  if (K <= 0 || N <= 0 || K >= (int64_t(1) << 31) || N >= (int64_t(1) << 31)) return FP8MOE_EINVAL;
  if (E < 1 || E > 1024) return FP8MOE_EINVAL;
  if (K % 16 != 0 || N % 16 != 0) return FP8MOE_EALIGN;
  return FP8MOE_OK;
}

struct FwdWorkspace {
  uint8_t* q;
  float* sx;
};

size_t fwd_ws_bytes(int64_t M, int64_t K) {
  return round_up((size_t)M * (size_t)K, 256) + round_up((size_t)M * 4, 256);
}

constexpr int64_t kQuantBlock = 512;
size_t fwd_block_ws_bytes(int64_t M, int64_t K) {
  const int64_t nb = (K + kQuantBlock - 1) / kQuantBlock;
  return round_up((size_t)M * (size_t)K, 256) + round_up((size_t)M * (size_t)nb * 4, 256);
}

struct TgmmWorkspace {
  uint8_t* qx;
  uint8_t* qd;
  float* sx;
  float* sd;
};

size_t tgmm_ws_bytes(int64_t M, int64_t K, int64_t N, int32_t E) {
  const size_t S = (size_t)segment_bound(M, E);
  return round_up(S * 128 * (size_t)K, 256) + round_up(S * 128 * (size_t)N, 256) +
         round_up(S * (size_t)K * 4, 256) + round_up(S * (size_t)N * 4, 256);
}

TgmmWorkspace carve_tgmm(void* ws, int64_t M, int64_t K, int64_t N, int32_t E) {
  const size_t S = (size_t)segment_bound(M, E);
  uint8_t* p = static_cast<uint8_t*>(ws);
  TgmmWorkspace w;
  w.qx = p;
  p += round_up(S * 128 * (size_t)K, 256);
  w.qd = p;
  p += round_up(S * 128 * (size_t)N, 256);
  w.sx = reinterpret_cast<float*>(p);
  p += round_up(S * (size_t)K * 4, 256);
  w.sd = reinterpret_cast<float*>(p);
  return w;
}

int gmm_fp8_fwd_impl(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                     const float* scale, int32_t E, int64_t N, const int32_t* gs, void* out,
                     void* ws, size_t ws_bytes, cudaStream_t stream, int swiglu) {
  int rc = check_common(M, K, N, E);
  if (rc) return rc;
  // SwiGLU: the up half starts at byte N/2 of each weight row, and a TMA copy's
  // inner coordinate must be a multiple of 16 bytes.
  if (swiglu && (N % 32 != 0)) return FP8MOE_EALIGN;
  if (M == 0) return FP8MOE_OK;
  if (!lhs || !codes || !scale || !gs || !out || !ws) return ws ? FP8MOE_EINVAL : FP8MOE_EWORKSPACE;
  if (!aligned16(lhs) || !aligned16(codes) || !aligned16(scale) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u) || (reinterpret_cast<uintptr_t>(gs) & 3u))
    return FP8MOE_EALIGN;
  if (ws_bytes < fwd_ws_bytes(M, K)) return FP8MOE_EWORKSPACE;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  uint8_t* q = static_cast<uint8_t*>(ws);
  float* sx = reinterpret_cast<float*>(q + round_up((size_t)M * (size_t)K, 256));
  GmmFwdArgs a;
  {
    const uint64_t dims[2] = {(uint64_t)K, (uint64_t)M};
    const uint64_t st[1] = {(uint64_t)K};
    const uint32_t box[2] = {128, 128};
    rc = make_tmap(&a.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  {
    const uint64_t dims[3] = {(uint64_t)N, (uint64_t)K, (uint64_t)E};
    const uint64_t st[2] = {(uint64_t)N, (uint64_t)N * (uint64_t)K};
    const uint32_t box[3] = {128, 128, 1};
    rc = make_tmap(&a.tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  a.sx = sx;
  a.scale = scale;
  a.gs = gs;
  a.out = out;
  a.M = M;
  a.K = (int)K;
  a.N = (int)N;
  a.E = E;
  a.swiglu = swiglu;
  cudaError_t e = fp8moe_launch_quantize_rows(lhs, M, (int)K, gs, E, 0, E, q, sx, sms, 8, 1,
                                              stream);
  if (e != cudaSuccess) return cuda_fail(e);
  a.e0 = 0;
  a.e1 = E;
  a.blk = 0;
  e = fp8moe_launch_gmm_fp8_fwd(a, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

// gu != nullptr selects the dSwiGLU epilogue: dlhs is then dgu [M, 2K].
int dlhs_impl(const void* dout, int64_t M, int64_t N, const uint8_t* codes, const float* scale,
              int32_t E, int64_t K, const int32_t* gs, const void* gu, void* dlhs, int path,
              cudaStream_t stream) {
  int rc = check_common(M, K, N, E);
  if (rc) return rc;
  if (path == 1 && N > 256) return FP8MOE_EINVAL;
  if (M == 0) return FP8MOE_OK;
  if (!dout || !codes || !scale || !gs || !dlhs) return FP8MOE_EINVAL;
  if (!aligned16(dout) || !aligned16(codes) || !aligned16(scale) || !aligned16(dlhs) ||
      (gu && !aligned16(gu)) || (reinterpret_cast<uintptr_t>(gs) & 3u))
    return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  GmmDlhsArgs a;
  a.gu = gu;
  {
    const uint64_t dims[2] = {(uint64_t)N, (uint64_t)M};
    const uint64_t st[1] = {(uint64_t)N * 2};
    const uint32_t box[2] = {64, 128};
    rc = make_tmap(&a.tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dout, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  {
    const uint64_t dims[3] = {(uint64_t)N, (uint64_t)K, (uint64_t)E};
    const uint64_t st[2] = {(uint64_t)N, (uint64_t)N * (uint64_t)K};
    const uint32_t box[3] = {64, 256, 1};
    rc = make_tmap(&a.tmC, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc) return rc;
    // pair path: 128 k rows x 64 bytes, 64-byte swizzle (conflict-free row reads)
    const uint32_t box_p[3] = {64, 128, 1};
    rc = make_tmap(&a.tmCp, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, st, box_p,
                   CU_TENSOR_MAP_SWIZZLE_64B);
    if (rc) return rc;
  }
  a.scale = scale;
  a.gs = gs;
  a.dlhs = dlhs;
  a.M = M;
  a.N = (int)N;
  a.K = (int)K;
  a.E = E;
  cudaError_t e = fp8moe_launch_gmm_dlhs(a, sms, path, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

int tgmm_quantize_impl(const void* lhs, const void* dout, int64_t M, int64_t K, int64_t N,
                       int32_t E, const int32_t* gs, uint8_t* qx, float* sx, uint8_t* qd,
                       float* sd, cudaStream_t stream, int sms, int d_fmt) {
  cudaError_t e = fp8moe_launch_tgmm_quantize_tiles(lhs, dout, M, (int)K, (int)N, gs, E,
                                                    segment_bound(M, E), qx, sx, qd, sd, sms, 1,
                                                    d_fmt, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

// ---- tokens sorted by expert, norms around the block, MXFP4

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Bytes per element of a row type, 0 if it is not one.
int type_bytes(int32_t type) {
  return type == FP8MOE_TYPE_BF16 ? 2 : type == FP8MOE_TYPE_F32 ? 4 : 0;
}

int check_route(int64_t T, int32_t topk, int64_t M) {
  if (T < 0 || M < 0 || M >= (int64_t(1) << 31)) return FP8MOE_EINVAL;
  if (topk < 1 || topk > 32 || T >= (int64_t(1) << 31) / topk) return FP8MOE_EINVAL;
  return FP8MOE_OK;
}

// Row length and type; *nvec receives the 16-byte vectors of a row.
int check_row(int64_t H, int32_t type, int* nvec) {
  const int b = type_bytes(type);
  if (!b || H <= 0 || H >= (int64_t(1) << 31)) return FP8MOE_EINVAL;
  if (H * b % 16 != 0) return FP8MOE_EALIGN;
  *nvec = (int)(H * b / 16);
  return FP8MOE_OK;
}

int check_sort(const int32_t* ids, int64_t T, int32_t topk, int32_t E, int64_t M,
               const int32_t* group_sizes, const int32_t* slot_row, const int32_t* row_slot) {
  int rc = check_route(T, topk, M);
  if (rc) return rc;
  if (E < 1 || E > 1024 || !group_sizes || (T > 0 && (!ids || !slot_row))) return FP8MOE_EINVAL;
  if (!aligned4(ids) || !aligned4(group_sizes) || !aligned4(slot_row) || !aligned4(row_slot))
    return FP8MOE_EALIGN;
  return FP8MOE_OK;
}

int check_norm(int64_t T, int64_t H, int32_t type, int32_t gate_kind, int32_t sigmoid) {
  int nvec = 0;
  if (T < 0 || T >= (int64_t(1) << 31)) return FP8MOE_EINVAL;
  int rc = check_row(H, type, &nvec);
  if (rc) return rc;
  if (nvec > 2048) return FP8MOE_EINVAL;     // H * element size <= 32768
  if (gate_kind < FP8MOE_GATE_NONE || gate_kind > FP8MOE_GATE_FULL) return FP8MOE_EINVAL;
  if (sigmoid != 0 && sigmoid != 1) return FP8MOE_EINVAL;
  return FP8MOE_OK;
}

size_t norm_bwd_ws_bytes(int64_t T, int64_t H) {
  return (size_t)2 * (size_t)fp8moe_norm_bwd_ctas(T) * (size_t)H * sizeof(float);
}

int64_t mxfp4_words(int64_t K) { return (K + 127) / 128; }

// The products' scale words of 128 k start on 16 bytes (a TMA stride).
int64_t mxfp4_scale_stride(int64_t M) { return (M + 3) / 4 * 4; }

size_t mxfp4_ws_bytes(int64_t M, int64_t K) {
  return round_up((size_t)M * (size_t)(K / 2), 256) +
         round_up((size_t)mxfp4_scale_stride(M) * (size_t)mxfp4_words(K) * 4, 256);
}

int check_mxfp4(int64_t M, int64_t K, int64_t N, int32_t E) {
  int rc = check_common(M, K, N, E);
  if (rc) return rc;
  return K % 32 != 0 ? FP8MOE_EALIGN : FP8MOE_OK;
}

int gmm_mxfp4_impl(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                   const uint8_t* scales, int32_t E, int64_t N, const int32_t* gs, void* out,
                   void* ws, size_t ws_bytes, cudaStream_t stream, int swiglu) {
  int rc = check_mxfp4(M, K, N, E);
  if (rc) return rc;
  if (swiglu && N % 32 != 0) return FP8MOE_EALIGN;
  if (M == 0) return FP8MOE_OK;
  if (!lhs || !codes || !scales || !gs || !out) return FP8MOE_EINVAL;
  if (!ws) return FP8MOE_EWORKSPACE;
  if (!aligned16(lhs) || !aligned16(codes) || !aligned16(scales) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u) || !aligned4(gs))
    return FP8MOE_EALIGN;
  if (ws_bytes < mxfp4_ws_bytes(M, K)) return FP8MOE_EWORKSPACE;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  uint8_t* const qx = static_cast<uint8_t*>(ws);
  uint8_t* const sx = qx + round_up((size_t)M * (size_t)(K / 2), 256);
  const uint64_t kb = (uint64_t)K / 2;
  GmmMxfp4Args a;
  if (swiglu) {
    const uint64_t F = (uint64_t)N / 2;
    const uint64_t dims[5] = {kb, 16, 2, F / 16, (uint64_t)E};
    const uint64_t st[4] = {kb, F * kb, 16 * kb, (uint64_t)N * kb};
    const uint32_t box[5] = {128, 16, 2, 4, 1};
    rc = make_tmap(&a.tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, codes, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    const uint64_t dims[3] = {kb, (uint64_t)N, (uint64_t)E};
    const uint64_t st[2] = {kb, (uint64_t)N * kb};
    const uint32_t box[3] = {128, 128, 1};
    rc = make_tmap(&a.tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (rc) return rc;
  const uint64_t words = (uint64_t)mxfp4_words(K), stride = (uint64_t)mxfp4_scale_stride(M);
  int rows[3], scale_rows = 0;
  fp8moe_gmm_mxfp4_boxes(rows, &scale_rows);
  if (swiglu) {
    const uint64_t F = (uint64_t)N / 2;
    const uint64_t dims[5] = {16, 2, F / 16, words, (uint64_t)E};
    const uint64_t st[4] = {F * 4, 64, (uint64_t)N * 4, words * (uint64_t)N * 4};
    const uint32_t box[5] = {16, 2, 4, 2, 1};
    rc = make_tmap(&a.tmSw, CU_TENSOR_MAP_DATA_TYPE_UINT32, 5, scales, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_NONE);
  } else {
    const uint64_t dims[3] = {(uint64_t)N, words, (uint64_t)E};
    const uint64_t st[2] = {(uint64_t)N * 4, words * (uint64_t)N * 4};
    const uint32_t box[3] = {128, 2, 1};
    rc = make_tmap(&a.tmSw, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, scales, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  if (rc) return rc;
  {
    const uint64_t dims[2] = {stride, words};
    const uint64_t st[1] = {stride * 4};
    const uint32_t box[2] = {(uint32_t)scale_rows, 2};
    rc = make_tmap(&a.tmSx, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, sx, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc) return rc;
  }
  for (int i = 0; i < 3; ++i) {
    const uint64_t dims[2] = {kb, (uint64_t)M};
    const uint64_t st[1] = {kb};
    const uint32_t box[2] = {128, (uint32_t)rows[i]};
    rc = make_tmap(&a.tmX[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, qx, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  a.gs = gs;
  a.out = out;
  a.M = M;
  a.K = (int)K;
  a.N = (int)N;
  a.E = E;
  a.swiglu = swiglu;
  cudaError_t e = fp8moe_launch_mxfp4_quantize_rows(lhs, M, (int)K, gs, E, qx, sx,
                                                    (int64_t)stride, sms, 1, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  e = fp8moe_launch_gmm_mxfp4(a, sms, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int check_router(int64_t T, int32_t E, int32_t type, int32_t score, int32_t topk,
                 const int32_t* offsets, int32_t B) {
  if (E < 1 || E > 1024 || topk < 1 || topk > 32 || topk > E || B < 1) return FP8MOE_EINVAL;
  if (T < 0 || T >= ((int64_t)1 << 31) || T * topk >= ((int64_t)1 << 31)) return FP8MOE_EINVAL;
  if (!type_bytes(type)) return FP8MOE_EINVAL;
  if (score != FP8MOE_SCORE_SOFTMAX && score != FP8MOE_SCORE_SIGMOID) return FP8MOE_EINVAL;
  if (!offsets && B != 1) return FP8MOE_EINVAL;
  return aligned4(offsets) ? FP8MOE_OK : FP8MOE_EALIGN;
}

// Parts of the balance sums: one for each chunk of tokens and sequence that has a part in it.
int64_t balance_slots(int64_t T, int64_t B) {
  const int64_t chunk = fp8moe_balance_chunk(T);
  return (T + chunk - 1) / chunk + B;
}

size_t balance_ws_bytes(int64_t T, int64_t B, int32_t E) {
  const size_t slots = (size_t)balance_slots(T, B);
  return 2 * round_up(slots * (size_t)E * 4, 256) + round_up(slots * 4, 256);
}

// Checks the balance loss's outputs and workspace and enters them into `a`.
int set_balance(RouterArgs& a, int32_t* counts, float* loss, float* slope, void* ws,
                size_t ws_bytes) {
  if (!counts || !loss || !slope) return FP8MOE_EINVAL;
  if (!ws) return FP8MOE_EWORKSPACE;
  if (!aligned4(counts) || !aligned4(loss) || !aligned4(slope) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u))
    return FP8MOE_EALIGN;
  if (ws_bytes < balance_ws_bytes(a.T, a.B, a.E)) return FP8MOE_EWORKSPACE;
  const size_t slots = (size_t)balance_slots(a.T, a.B);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.part_share = reinterpret_cast<float*>(w);
  a.part_count = reinterpret_cast<int32_t*>(w + round_up(slots * (size_t)a.E * 4, 256));
  a.part_tokens = reinterpret_cast<int32_t*>(w + 2 * round_up(slots * (size_t)a.E * 4, 256));
  a.counts = counts;
  a.loss = loss;
  a.slope = slope;
  return FP8MOE_OK;
}

bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

int check_adamw(const fp8moe_adamw_tensor& d) {
  if (d.n < 0 || d.n > ((int64_t)1 << 42)) return FP8MOE_EINVAL;
  if (d.n == 0) return FP8MOE_OK;
  if (!type_bytes(d.g_type) || (d.state_bits != 32 && d.state_bits != 8)) return FP8MOE_EINVAL;
  if (!d.p || !d.g || !d.m || !d.v) return FP8MOE_EINVAL;
  const bool eight = d.state_bits == 8;
  if ((d.m_scale != nullptr) != eight || (d.v_scale != nullptr) != eight) return FP8MOE_EINVAL;
  if ((d.codes != nullptr) != (d.code_scale != nullptr)) return FP8MOE_EINVAL;
  if (!(d.weight_decay == d.weight_decay)) return FP8MOE_EINVAL;
  if (!aligned4(d.p) || !aligned4(d.m_scale) || !aligned4(d.v_scale) || !aligned4(d.code_scale) ||
      !aligned2(d.copy) || (d.g_type == FP8MOE_TYPE_F32 ? !aligned4(d.g) : !aligned2(d.g)) ||
      (!eight && (!aligned4(d.m) || !aligned4(d.v))))
    return FP8MOE_EALIGN;
  if (d.codes) {
    if (d.K < 1 || d.N < 1 || d.K > (1 << 21) || d.N > (1 << 21)) return FP8MOE_EINVAL;
    if (d.n % (d.K * d.N) != 0 || d.n / (d.K * d.N) > 1024) return FP8MOE_EINVAL;
    if (d.K % 16 != 0 || d.N % 16 != 0) return FP8MOE_EALIGN;
  }
  return FP8MOE_OK;
}

// Words of the workspace for weights with codes: of each column, and the units' counters. Each
// tensor's begin on 256 bytes (columns are copied by 16).
int64_t adamw_columns(const fp8moe_adamw_tensor& d) { return d.n / d.K; }
int64_t adamw_words(const fp8moe_adamw_tensor& d) {
  if (d.n <= 0 || !d.codes || check_adamw(d) != FP8MOE_OK) return 0;
  return (adamw_columns(d) + fp8moe_adamw_slab_counters(d.n, d.K, d.N) + 63) / 64 * 64;
}

// The first value from which on every array lies on a boundary that wide accesses need (16 bytes
// for what is copied to shared memory, 8 for the stores of a copy), -1 if there is none: parts of one
// flat buffer lie alike, wherever they begin. A block of an 8-bit moment begins with the tensor,
// so that only 0 will do there.
int adamw_head(const fp8moe_adamw_tensor& d) {
  auto at = [](const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) + bytes; };
  const int g = d.g_type == FP8MOE_TYPE_BF16 ? 2 : 4, state = d.state_bits / 8;
  for (int h = 0; h < (d.state_bits == 32 ? 8 : 1); ++h)
    if (at(d.p, 4 * h) % 16 == 0 && at(d.g, g * h) % 16 == 0 && at(d.m, state * h) % 16 == 0 &&
        at(d.v, state * h) % 16 == 0 && (!d.copy || at(d.copy, 2 * h) % 8 == 0))
      return h;
  return -1;
}
// Weights whose step goes by tiles, together with the codes. A block of an 8-bit moment has to lie
// in one row of a tile.
bool adamw_slabs(const fp8moe_adamw_tensor& d) {
  return d.n > 0 && d.codes && aligned4(d.codes) && adamw_head(d) == 0 &&
         (d.state_bits == 32 || d.N % 128 == 0);
}
int adamw_tmap(CUtensorMap* m, const void* base, int bytes, const fp8moe_adamw_tensor& d) {
  int cols, rows;
  fp8moe_adamw_tile(&cols, &rows);
  const uint64_t K = (uint64_t)d.K, N = (uint64_t)d.N;
  const uint64_t dims[3] = {N, K, (uint64_t)d.n / (K * N)};
  const uint64_t strides[2] = {N * bytes, K * N * bytes};
  const uint32_t box[3] = {(uint32_t)cols, (uint32_t)rows, 1};
  return make_tmap(m, bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                      : bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                   3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}
AdamwEntry adamw_entry(const fp8moe_adamw_tensor& d, int32_t which, double lr) {
  AdamwEntry w = {};
  w.p = d.p, w.g = d.g, w.m = d.m, w.v = d.v, w.m_scale = d.m_scale, w.v_scale = d.v_scale;
  w.copy = d.copy, w.n = d.n, w.weight_decay = d.weight_decay;
  w.keep = (float)(1.0 - lr * d.weight_decay);
  w.which = (uint32_t)which;
  const int head = adamw_head(d);
  w.g_bf16 = d.g_type == FP8MOE_TYPE_BF16, w.vec = head >= 0, w.head = (uint8_t)(head > 0 ? head : 0);
  return w;
}

// The rates of a step on the device lie in front of the words of the weights with codes.
constexpr size_t kAdamwRatesBytes = 256;
static_assert(sizeof(AdamwRates) <= kAdamwRatesBytes, "the words of the weights with codes begin behind");

size_t adamw_ws_bytes(const fp8moe_adamw_tensor* tensors, int32_t count, bool on_device) {
  size_t words = 0;
  for (int32_t i = 0; i < count; ++i) words += (size_t)adamw_words(tensors[i]);
  return words || on_device ? kAdamwRatesBytes + words * 4 : 0;
}

}  // namespace

extern "C" {

size_t fp8moe_workspace_size(int op, int64_t M, int64_t K, int64_t N, int32_t E) {
  if (M < 0 || K < 0 || N < 0 || E < 0) return 0;
  switch (op) {
    case FP8MOE_OP_GMM_FP8_FWD:
    case FP8MOE_OP_GMM_SILU_FP8_FWD:
      return fwd_ws_bytes(M, K);
    case FP8MOE_OP_TGMM_DRHS_QUANT:
      return tgmm_ws_bytes(M, K, N, E);
    case FP8MOE_OP_GMM_FP8_FWD_BLOCK:
      return fwd_block_ws_bytes(M, K);
    case FP8MOE_OP_GMM_MXFP4_FWD:
    case FP8MOE_OP_GMM_SILU_MXFP4_FWD:
      return mxfp4_ws_bytes(M, K);
    case FP8MOE_OP_NORM_BWD:
      return norm_bwd_ws_bytes(M, K);
    case FP8MOE_OP_BALANCE:
      return balance_ws_bytes(M, N, E);
    default:
      return 0;
  }
}

int fp8moe_gmm_fp8_fwd(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                       const float* scale, int32_t E, int64_t N, const int32_t* group_sizes,
                       void* out, void* workspace, size_t workspace_bytes,
                       fp8moe_stream_t stream) {
  return gmm_fp8_fwd_impl(lhs, M, K, codes, scale, E, N, group_sizes, out, workspace,
                          workspace_bytes, stream, 0);
}

int fp8moe_gmm_silu_fp8_fwd(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                            const float* scale, int32_t E, int64_t N,
                            const int32_t* group_sizes, void* out, void* workspace,
                            size_t workspace_bytes, fp8moe_stream_t stream) {
  return gmm_fp8_fwd_impl(lhs, M, K, codes, scale, E, N, group_sizes, out, workspace,
                          workspace_bytes, stream, 1);
}

int fp8moe_gmm_dlhs_fp8(const void* dout, int64_t M, int64_t N, const uint8_t* codes,
                        const float* scale, int32_t E, int64_t K, const int32_t* group_sizes,
                        void* dlhs, void* workspace, size_t workspace_bytes,
                        fp8moe_stream_t stream) {
  (void)workspace;
  (void)workspace_bytes;
  // the on-chip cache path when the whole contraction fits one cached block,
  // otherwise CTA pairs with the dequantized weight in tensor memory
  const int path = (N <= 256) ? 1 : 2;
  return dlhs_impl(dout, M, N, codes, scale, E, K, group_sizes, nullptr, dlhs, path, stream);
}

int fp8moe_gmm_dlhs_fp8_path(const void* dout, int64_t M, int64_t N, const uint8_t* codes,
                             const float* scale, int32_t E, int64_t K,
                             const int32_t* group_sizes, void* dlhs, int32_t path,
                             fp8moe_stream_t stream) {
  if (path < 0 || path > 2) return FP8MOE_EINVAL;
  return dlhs_impl(dout, M, N, codes, scale, E, K, group_sizes, nullptr, dlhs, path, stream);
}

int fp8moe_gmm_dlhs_dswiglu_fp8(const void* dout, int64_t M, int64_t N, const uint8_t* codes,
                                const float* scale, int32_t E, int64_t F, const void* gu,
                                const int32_t* group_sizes, void* dgu, void* workspace,
                                size_t workspace_bytes, fp8moe_stream_t stream) {
  (void)workspace;
  (void)workspace_bytes;
  if (M > 0 && !gu) return FP8MOE_EINVAL;
  // the pair path has one accumulator and must hold it through the SwiGLU
  // backward, which stalls its MMAs; the streaming path is the faster one here
  const int path = (N <= 256) ? 1 : 0;
  return dlhs_impl(dout, M, N, codes, scale, E, F, group_sizes, gu, dgu, path, stream);
}

int fp8moe_gmm_dlhs_dswiglu_fp8_path(const void* dout, int64_t M, int64_t N, const uint8_t* codes,
                                     const float* scale, int32_t E, int64_t F, const void* gu,
                                     const int32_t* group_sizes, void* dgu, int32_t path,
                                     fp8moe_stream_t stream) {
  if (path < 0 || path > 2) return FP8MOE_EINVAL;
  if (M > 0 && !gu) return FP8MOE_EINVAL;
  return dlhs_impl(dout, M, N, codes, scale, E, F, group_sizes, gu, dgu, path, stream);
}

static int tgmm_drhs_impl(const void* lhs, const void* dout, int64_t M, int64_t K, int64_t N,
                          int32_t E, const int32_t* group_sizes, float* dW, void* workspace,
                          size_t workspace_bytes, int d_fmt, fp8moe_stream_t stream) {
  int rc = check_common(M, K, N, E);
  if (rc) return rc;
  if (d_fmt != FP8MOE_FMT_E4M3 && d_fmt != FP8MOE_FMT_E5M2) return FP8MOE_EINVAL;
  if (!dW || !group_sizes) return FP8MOE_EINVAL;
  if (M > 0 && (!lhs || !dout)) return FP8MOE_EINVAL;
  if (!workspace) return FP8MOE_EWORKSPACE;
  if (!aligned16(lhs) || !aligned16(dout) || !aligned16(dW) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      (reinterpret_cast<uintptr_t>(group_sizes) & 3u))
    return FP8MOE_EALIGN;
  if (workspace_bytes < tgmm_ws_bytes(M, K, N, E)) return FP8MOE_EWORKSPACE;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  TgmmWorkspace w = carve_tgmm(workspace, M, K, N, E);
  const int64_t S = segment_bound(M, E);
  if (M > 0) {
    rc = tgmm_quantize_impl(lhs, dout, M, K, N, E, group_sizes, w.qx, w.sx, w.qd, w.sd, stream, sms,
                            d_fmt);
    if (rc) return rc;
  }
  TgmmArgs a;
  {
    const uint64_t dims[2] = {(uint64_t)K, (uint64_t)(S * 128)};
    const uint64_t st[1] = {(uint64_t)K};
    const uint32_t box[2] = {128, 128};
    rc = make_tmap(&a.tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, w.qx, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  {
    const uint64_t dims[2] = {(uint64_t)N, (uint64_t)(S * 128)};
    const uint64_t st[1] = {(uint64_t)N};
    const uint32_t box[2] = {128, 128};
    rc = make_tmap(&a.tmD, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, w.qd, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  {
    // dW as [E][K][N] so that a box's rows past K (ragged k tile) are clipped
    const uint64_t dims[3] = {(uint64_t)N, (uint64_t)K, (uint64_t)E};
    const uint64_t st[2] = {(uint64_t)N * 4, (uint64_t)K * (uint64_t)N * 4};
    const uint32_t box[3] = {32, 32, 1};
    rc = make_tmap(&a.tmW, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, dW, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  a.sx = w.sx;
  a.sd = w.sd;
  a.gs = group_sizes;
  a.dW = dW;
  a.M = M;
  a.K = (int)K;
  a.N = (int)N;
  a.E = E;
  a.d_fmt = d_fmt;
  cudaError_t e = fp8moe_launch_tgmm(a, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

int fp8moe_tgmm_drhs_quant(const void* lhs, const void* dout, int64_t M, int64_t K, int64_t N,
                           int32_t E, const int32_t* group_sizes, float* dW, void* workspace,
                           size_t workspace_bytes, fp8moe_stream_t stream) {
  return tgmm_drhs_impl(lhs, dout, M, K, N, E, group_sizes, dW, workspace, workspace_bytes,
                        FP8MOE_FMT_E4M3, stream);
}

int fp8moe_tgmm_drhs_quant_fmt(const void* lhs, const void* dout, int64_t M, int64_t K, int64_t N,
                               int32_t E, const int32_t* group_sizes, float* dW, void* workspace,
                               size_t workspace_bytes, int32_t dout_fmt, fp8moe_stream_t stream) {
  return tgmm_drhs_impl(lhs, dout, M, K, N, E, group_sizes, dW, workspace, workspace_bytes,
                        dout_fmt, stream);
}

int fp8moe_dequantize_fp8_codes(const uint8_t* codes, const float* scale, int32_t E, int64_t K,
                                int64_t N, void* out, fp8moe_stream_t stream) {
  int rc = check_common(0, K, N, E);
  if (rc) return rc;
  if (!codes || !scale || !out) return FP8MOE_EINVAL;
  if (!aligned16(codes) || !aligned16(scale) || !aligned16(out)) return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_dequantize(codes, scale, E, K, N, out, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

int fp8moe_gmm_bf16_fwd(const void* lhs, int64_t M, int64_t K, const void* w, int32_t E,
                        int64_t N, const int32_t* group_sizes, int32_t swiglu, void* out,
                        fp8moe_stream_t stream) {
  int rc = check_common(M, K, N, E);
  if (rc) return rc;
  if (M == 0) return FP8MOE_OK;
  if (!lhs || !w || !group_sizes || !out) return FP8MOE_EINVAL;
  if (!aligned16(lhs) || !aligned16(w) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(group_sizes) & 3u))
    return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  GmmFwdArgs a;
  {
    const uint64_t dims[2] = {(uint64_t)K, (uint64_t)M};
    const uint64_t st[1] = {(uint64_t)K * 2};
    const uint32_t box[2] = {64, 128};
    rc = make_tmap(&a.tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, lhs, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  {
    const uint64_t dims[3] = {(uint64_t)N, (uint64_t)K, (uint64_t)E};
    const uint64_t st[2] = {(uint64_t)N * 2, (uint64_t)N * (uint64_t)K * 2};
    const uint32_t box[3] = {64, 64, 1};
    rc = make_tmap(&a.tmB, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, w, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  a.sx = nullptr;
  a.scale = nullptr;
  a.gs = group_sizes;
  a.out = out;
  a.M = M;
  a.K = (int)K;
  a.N = (int)N;
  a.E = E;
  a.swiglu = swiglu ? 1 : 0;
  a.e0 = 0;
  a.e1 = E;
  a.blk = 0;
  cudaError_t e = fp8moe_launch_gmm_bf16_fwd(a, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

int fp8moe_gmm_fp8_fwd_block(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                             const float* scale, int32_t E, int64_t N,
                             const int32_t* group_sizes, void* out, void* workspace,
                             size_t workspace_bytes, int32_t block, int32_t swiglu,
                             fp8moe_stream_t stream) {
  int rc = check_common(M, K, N, E);
  if (rc) return rc;
  if (block != kQuantBlock || (swiglu != 0 && swiglu != 1)) return FP8MOE_EINVAL;
  if (swiglu && (N % 32 != 0)) return FP8MOE_EALIGN;
  if (M == 0) return FP8MOE_OK;
  if (!workspace) return FP8MOE_EWORKSPACE;
  if (!lhs || !codes || !scale || !group_sizes || !out) return FP8MOE_EINVAL;
  if (!aligned16(lhs) || !aligned16(codes) || !aligned16(scale) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      (reinterpret_cast<uintptr_t>(group_sizes) & 3u))
    return FP8MOE_EALIGN;
  if (workspace_bytes < fwd_block_ws_bytes(M, K)) return FP8MOE_EWORKSPACE;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  uint8_t* q = static_cast<uint8_t*>(workspace);
  float* sb = reinterpret_cast<float*>(q + round_up((size_t)M * (size_t)K, 256));
  cudaError_t e = fp8moe_launch_quantize_rows_block(lhs, M, (int)K, group_sizes, E, q, sb, sms, 1,
                                                    stream);
  if (e != cudaSuccess) return cuda_fail(e);
  GmmFwdArgs a;
  {
    const uint64_t dims[2] = {(uint64_t)K, (uint64_t)M};
    const uint64_t st[1] = {(uint64_t)K};
    const uint32_t box[2] = {128, 128};
    rc = make_tmap(&a.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  {
    const uint64_t dims[3] = {(uint64_t)N, (uint64_t)K, (uint64_t)E};
    const uint64_t st[2] = {(uint64_t)N, (uint64_t)N * (uint64_t)K};
    const uint32_t box[3] = {128, 128, 1};
    rc = make_tmap(&a.tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, st, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  a.sx = sb;
  a.scale = scale;
  a.gs = group_sizes;
  a.out = out;
  a.M = M;
  a.K = (int)K;
  a.N = (int)N;
  a.E = E;
  a.swiglu = swiglu;
  a.e0 = 0;
  a.e1 = E;
  a.blk = 1;
  e = fp8moe_launch_gmm_fp8_fwd(a, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

int fp8moe_quantize_rows_block(const void* lhs, int64_t M, int64_t K, const int32_t* group_sizes,
                               int32_t E, int32_t block, uint8_t* q, float* sb,
                               fp8moe_stream_t stream) {
  int rc = check_common(M, K, 16, E);
  if (rc) return rc;
  if (block != kQuantBlock) return FP8MOE_EINVAL;
  if (M == 0) return FP8MOE_OK;
  if (!lhs || !group_sizes || !q || !sb) return FP8MOE_EINVAL;
  if (!aligned16(lhs) || !aligned16(q) || (reinterpret_cast<uintptr_t>(sb) & 3u) ||
      (reinterpret_cast<uintptr_t>(group_sizes) & 3u))
    return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_quantize_rows_block(lhs, M, (int)K, group_sizes, E, q, sb, sms, 1,
                                                    stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

int fp8moe_quantize_rows(const void* lhs, int64_t M, int64_t K, const int32_t* group_sizes,
                         int32_t E, uint8_t* q, float* sx, fp8moe_stream_t stream) {
  int rc = check_common(M, K, 16, E);
  if (rc) return rc;
  if (M == 0) return FP8MOE_OK;
  if (!lhs || !group_sizes || !q || !sx) return FP8MOE_EINVAL;
  if (!aligned16(lhs) || !aligned16(q) || (reinterpret_cast<uintptr_t>(sx) & 3u) ||
      (reinterpret_cast<uintptr_t>(group_sizes) & 3u))
    return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_quantize_rows(lhs, M, (int)K, group_sizes, E, 0, E, q, sx, sms, 8,
                                              1, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

int fp8moe_tgmm_quantize_tiles(const void* lhs, const void* dout, int64_t M, int64_t K,
                               int64_t N, int32_t E, const int32_t* group_sizes, uint8_t* qx,
                               float* sx, uint8_t* qd, float* sd, fp8moe_stream_t stream) {
  return fp8moe_tgmm_quantize_tiles_fmt(lhs, dout, M, K, N, E, group_sizes, qx, sx, qd, sd,
                                        FP8MOE_FMT_E4M3, stream);
}

int fp8moe_tgmm_quantize_tiles_fmt(const void* lhs, const void* dout, int64_t M, int64_t K,
                                   int64_t N, int32_t E, const int32_t* group_sizes, uint8_t* qx,
                                   float* sx, uint8_t* qd, float* sd, int32_t dout_fmt,
                                   fp8moe_stream_t stream) {
  int rc = check_common(M, K, N, E);
  if (rc) return rc;
  if (dout_fmt != FP8MOE_FMT_E4M3 && dout_fmt != FP8MOE_FMT_E5M2) return FP8MOE_EINVAL;
  if (M == 0) return FP8MOE_OK;
  if (!lhs || !dout || !group_sizes || !qx || !sx || !qd || !sd) return FP8MOE_EINVAL;
  if (!aligned16(lhs) || !aligned16(dout) || !aligned16(qx) || !aligned16(qd) ||
      !aligned16(sx) || !aligned16(sd) || (reinterpret_cast<uintptr_t>(group_sizes) & 3u))
    return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  return tgmm_quantize_impl(lhs, dout, M, K, N, E, group_sizes, qx, sx, qd, sd, stream, sms,
                            dout_fmt);
}

int fp8moe_selftest_wait_timeout(uint32_t limit_us, fp8moe_stream_t stream) {
  if (limit_us == 0 || limit_us > 2000000u) return FP8MOE_EINVAL;
  int sms = 0;
  int rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_selftest_wait((uint64_t)limit_us * 1000u, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

int fp8moe_selftest_cast_f32(const float* x, int64_t n, int32_t fmt, uint8_t* codes,
                             fp8moe_stream_t stream) {
  if (n < 0 || (fmt != FP8MOE_FMT_E4M3 && fmt != FP8MOE_FMT_E5M2)) return FP8MOE_EINVAL;
  if (n == 0) return FP8MOE_OK;
  if (!x || !codes) return FP8MOE_EINVAL;
  if (reinterpret_cast<uintptr_t>(x) & 3u) return FP8MOE_EALIGN;
  int sms = 0;
  int rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_selftest_cast(x, n, fmt, codes, sms, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return FP8MOE_OK;
}

int fp8moe_sort_tokens(const int32_t* ids, int64_t T, int32_t topk, int32_t E, int64_t M,
                       int32_t* group_sizes, int32_t* slot_row, int32_t* row_slot,
                       fp8moe_stream_t stream) {
  int rc = check_sort(ids, T, topk, E, M, group_sizes, slot_row, row_slot);
  if (rc) return rc;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_sort_tokens(ids, T * topk, E, M, group_sizes, slot_row, row_slot,
                                            stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_dispatch_tokens(const void* x, const int32_t* ids, int64_t T, int32_t topk, int64_t H,
                           int32_t type, int32_t E, int64_t M, void* rows, int32_t* group_sizes,
                           int32_t* slot_row, int32_t* row_slot, fp8moe_stream_t stream) {
  int nvec = 0, sms = 0;
  int rc = check_sort(ids, T, topk, E, M, group_sizes, slot_row, row_slot);
  if (rc) return rc;
  rc = check_row(H, type, &nvec);
  if (rc) return rc;
  if (T > 0 && (!x || (M > 0 && !rows))) return FP8MOE_EINVAL;
  if (!aligned16(x) || !aligned16(rows)) return FP8MOE_EALIGN;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_dispatch(x, ids, T, topk, E, M, nvec, rows, group_sizes, slot_row,
                                         row_slot, sms, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_combine_tokens(const void* rows, int64_t M, int64_t H, int32_t type,
                          const int32_t* slot_row, const float* weights, int64_t T, int32_t topk,
                          void* out, fp8moe_stream_t stream) {
  int nvec = 0, sms = 0;
  int rc = check_route(T, topk, M);
  if (rc) return rc;
  rc = check_row(H, type, &nvec);
  if (rc) return rc;
  if (T == 0) return FP8MOE_OK;
  if (!slot_row || !out || (M > 0 && !rows)) return FP8MOE_EINVAL;
  if (!aligned16(rows) || !aligned16(out) || !aligned4(slot_row) || !aligned4(weights))
    return FP8MOE_EALIGN;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_combine(rows, T, topk, nvec, type == FP8MOE_TYPE_F32, slot_row, M,
                                        weights, out, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_combine_tokens_bwd(const void* dout, const void* rows, int64_t M, int64_t H,
                              int32_t type, const int32_t* slot_row, const float* weights,
                              int64_t T, int32_t topk, void* drows, float* dweights,
                              fp8moe_stream_t stream) {
  int nvec = 0, sms = 0;
  int rc = check_route(T, topk, M);
  if (rc) return rc;
  rc = check_row(H, type, &nvec);
  if (rc) return rc;
  if (T == 0) return FP8MOE_OK;
  if (!dout || !slot_row || !weights || !dweights || (M > 0 && (!rows || !drows)))
    return FP8MOE_EINVAL;
  if (!aligned16(dout) || !aligned16(rows) || !aligned16(drows) || !aligned4(slot_row) ||
      !aligned4(weights) || !aligned4(dweights))
    return FP8MOE_EALIGN;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_combine_bwd(dout, rows, T, topk, nvec, type == FP8MOE_TYPE_F32,
                                            slot_row, M, weights, drows, dweights, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_norm_fwd(const void* x, const void* y, int64_t T, int64_t H, int32_t type,
                    const float* w_post, const float* w_pre, const void* gate, int32_t gate_kind,
                    int32_t sigmoid, float residual_scale, float branch_scale, float eps, void* r,
                    void* h, float* rstd_post, float* rstd_pre, fp8moe_stream_t stream) {
  int rc = check_norm(T, H, type, gate_kind, sigmoid);
  if (rc) return rc;
  const bool post = w_post != nullptr, pre = w_pre != nullptr;
  if (!post && !pre) return FP8MOE_EINVAL;
  if (!post && (y || gate_kind != FP8MOE_GATE_NONE)) return FP8MOE_EINVAL;
  if (!(eps >= 0.0f)) return FP8MOE_EINVAL;
  if (T == 0) return FP8MOE_OK;
  if (!x || (post && (!y || !r || !rstd_post)) || (pre && (!h || !rstd_pre))) return FP8MOE_EINVAL;
  if ((gate_kind != FP8MOE_GATE_NONE) != (gate != nullptr)) return FP8MOE_EINVAL;
  // a token's gate is read value by value, the other kinds by 16 bytes
  if (!aligned16(x) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) ||
      !aligned16(r) || !aligned16(h) || !aligned4(rstd_post) || !aligned4(rstd_pre) ||
      (gate_kind == FP8MOE_GATE_TOKEN ? !aligned4(gate) : !aligned16(gate)))
    return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  NormFwdArgs a = {x, y, w_post, w_pre, gate, gate_kind, sigmoid, residual_scale, branch_scale,
                   eps, T, (int)H, type == FP8MOE_TYPE_F32, r, h, rstd_post, rstd_pre};
  cudaError_t e = fp8moe_launch_norm_fwd(a, sms, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_norm_bwd(const void* dr, const void* dh, const void* r, const void* y, int64_t T,
                    int64_t H, int32_t type, const float* w_post, const float* w_pre,
                    const float* rstd_post, const float* rstd_pre, const void* gate,
                    int32_t gate_kind, int32_t sigmoid, float residual_scale, float branch_scale,
                    void* dx, void* dy, float* dw_post, float* dw_pre, void* dgate,
                    void* workspace, size_t workspace_bytes, fp8moe_stream_t stream) {
  int rc = check_norm(T, H, type, gate_kind, sigmoid);
  if (rc) return rc;
  const bool post = w_post != nullptr, pre = w_pre != nullptr;
  if (!post && !pre) return FP8MOE_EINVAL;
  if (!post && (y || gate_kind != FP8MOE_GATE_NONE)) return FP8MOE_EINVAL;
  if (!pre && dh) return FP8MOE_EINVAL;
  if ((post && !dw_post) || (pre && !dw_pre)) return FP8MOE_EINVAL;
  if (T > 0 && (gate_kind != FP8MOE_GATE_NONE) != (gate != nullptr)) return FP8MOE_EINVAL;
  if (gate_kind != FP8MOE_GATE_NONE && !dgate && (T > 0 || gate_kind == FP8MOE_GATE_CHANNEL))
    return FP8MOE_EINVAL;
  if (T > 0) {
    if (!dx || (!dr && !pre)) return FP8MOE_EINVAL;
    if (post && (!y || !rstd_post || !dy)) return FP8MOE_EINVAL;
    if (pre && (!dh || !r || !rstd_pre)) return FP8MOE_EINVAL;
    if (!workspace) return FP8MOE_EWORKSPACE;
  }
  if (!aligned16(dr) || !aligned16(dh) || !aligned16(r) || !aligned16(y) || !aligned16(w_post) ||
      !aligned16(w_pre) || !aligned4(rstd_post) || !aligned4(rstd_pre) || !aligned16(dx) ||
      !aligned16(dy) || !aligned4(dw_post) || !aligned4(dw_pre) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      (gate_kind == FP8MOE_GATE_TOKEN ? !aligned4(gate) || !aligned4(dgate)
                                    : !aligned16(gate) || !aligned16(dgate)))
    return FP8MOE_EALIGN;
  if (T > 0 && workspace_bytes < norm_bwd_ws_bytes(T, H)) return FP8MOE_EWORKSPACE;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  NormBwdArgs a = {dr, dh, r, y, w_post, w_pre, rstd_post, rstd_pre, gate, gate_kind, sigmoid,
                   residual_scale, branch_scale, T, (int)H, type == FP8MOE_TYPE_F32, dx, dy,
                   dw_post, dw_pre, dgate, static_cast<float*>(workspace)};
  cudaError_t e = fp8moe_launch_norm_bwd(a, sms, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_mxfp4_quantize_rows(const void* lhs, int64_t M, int64_t K, const int32_t* group_sizes,
                               int32_t E, uint8_t* codes, uint8_t* scales, fp8moe_stream_t stream) {
  int rc = check_mxfp4(M, K, 16, E);
  if (rc) return rc;
  if (M == 0) return FP8MOE_OK;
  if (!lhs || !group_sizes || !codes || !scales) return FP8MOE_EINVAL;
  if (!aligned16(lhs) || !aligned16(codes) || !aligned16(scales) || !aligned4(group_sizes))
    return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_mxfp4_quantize_rows(lhs, M, (int)K, group_sizes, E, codes, scales,
                                                    M, sms, 1, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_mxfp4_quantize_weights(const void* w, int32_t E, int64_t K, int64_t N, uint8_t* codes,
                                  uint8_t* scales, fp8moe_stream_t stream) {
  int rc = check_mxfp4(0, K, N, E);
  if (rc) return rc;
  if (!w || !codes || !scales) return FP8MOE_EINVAL;
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scales)) return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_mxfp4_quantize_weights(w, E, (int)K, (int)N, codes, scales, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t E, int64_t N,
                            int64_t K, void* out, fp8moe_stream_t stream) {
  int rc = check_mxfp4(0, K, N, E);
  if (rc) return rc;
  if (!codes || !scales || !out) return FP8MOE_EINVAL;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out)) return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  cudaError_t e = fp8moe_launch_mxfp4_dequantize(codes, scales, E, (int)N, (int)K, out, sms, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_gmm_mxfp4_fwd(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                         const uint8_t* scales, int32_t E, int64_t N, const int32_t* group_sizes,
                         void* out, void* workspace, size_t workspace_bytes,
                         fp8moe_stream_t stream) {
  return gmm_mxfp4_impl(lhs, M, K, codes, scales, E, N, group_sizes, out, workspace,
                        workspace_bytes, stream, 0);
}

int fp8moe_gmm_silu_mxfp4_fwd(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                              const uint8_t* scales, int32_t E, int64_t N,
                              const int32_t* group_sizes, void* out, void* workspace,
                              size_t workspace_bytes, fp8moe_stream_t stream) {
  return gmm_mxfp4_impl(lhs, M, K, codes, scales, E, N, group_sizes, out, workspace,
                        workspace_bytes, stream, 1);
}

int fp8moe_router_fwd(const void* logits, int64_t T, int32_t E, int32_t type, int32_t score,
                      const float* bias, int32_t topk, int32_t normalize, float scale,
                      const int32_t* seq_offsets, int32_t B, int32_t* ids, float* weights,
                      int32_t* counts, float* loss, float* slope, void* workspace,
                      size_t workspace_bytes, fp8moe_stream_t stream) {
  int rc = check_router(T, E, type, score, topk, seq_offsets, B);
  if (rc) return rc;
  if (normalize != 0 && normalize != 1) return FP8MOE_EINVAL;
  if (T > 0 && (!logits || !ids || !weights)) return FP8MOE_EINVAL;
  if (!aligned16(logits) || !aligned4(bias) || !aligned4(ids) || !aligned4(weights))
    return FP8MOE_EALIGN;
  RouterArgs a = {};
  a.logits = logits, a.bias = bias, a.ids = ids, a.weights = weights, a.offsets = seq_offsets;
  a.T = T, a.E = E, a.k = topk, a.B = B, a.f32 = type == FP8MOE_TYPE_F32;
  a.sig = score == FP8MOE_SCORE_SIGMOID, a.normalize = normalize, a.scale = scale;
  if (counts || loss || slope) {
    rc = set_balance(a, counts, loss, slope, workspace, workspace_bytes);
    if (rc) return rc;
  } else if (T == 0) {
    return FP8MOE_OK;
  }
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  const cudaError_t e = fp8moe_launch_router(a, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_balance_fwd(const void* logits, const int32_t* ids, int64_t T, int32_t E, int32_t type,
                       int32_t score, int32_t topk, const int32_t* seq_offsets, int32_t B,
                       int32_t* counts, float* loss, float* slope, void* workspace,
                       size_t workspace_bytes, fp8moe_stream_t stream) {
  int rc = check_router(T, E, type, score, topk, seq_offsets, B);
  if (rc) return rc;
  if (T > 0 && (!logits || !ids)) return FP8MOE_EINVAL;
  if (!aligned16(logits) || !aligned4(ids)) return FP8MOE_EALIGN;
  RouterArgs a = {};
  a.logits = logits, a.given = ids, a.offsets = seq_offsets;
  a.T = T, a.E = E, a.k = topk, a.B = B, a.f32 = type == FP8MOE_TYPE_F32;
  a.sig = score == FP8MOE_SCORE_SIGMOID;
  rc = set_balance(a, counts, loss, slope, workspace, workspace_bytes);
  if (rc) return rc;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  const cudaError_t e = fp8moe_launch_router(a, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

int fp8moe_router_bwd(const float* dweights, const void* logits, const int32_t* ids, int64_t T,
                      int32_t E, int32_t type, int32_t score, int32_t topk, int32_t normalize,
                      float scale, const float* dloss, const float* slope,
                      const int32_t* seq_offsets, int32_t B, void* dlogits,
                      fp8moe_stream_t stream) {
  int rc = check_router(T, E, type, score, topk, seq_offsets, B);
  if (rc) return rc;
  if (normalize != 0 && normalize != 1) return FP8MOE_EINVAL;
  if ((dloss != nullptr) != (slope != nullptr)) return FP8MOE_EINVAL;
  if (T == 0) return FP8MOE_OK;
  if (!logits || !ids || !dlogits) return FP8MOE_EINVAL;
  if (!aligned16(logits) || !aligned16(dlogits) || !aligned16(slope) || !aligned4(ids) ||
      !aligned4(dweights) || !aligned4(dloss))
    return FP8MOE_EALIGN;
  int sms = 0;
  rc = device_init(&sms);
  if (rc) return rc;
  RouterBwdArgs a = {logits, ids, dweights, seq_offsets, dloss, slope, dlogits, T, E, topk, B,
                     type == FP8MOE_TYPE_F32, score == FP8MOE_SCORE_SIGMOID, normalize, scale};
  const cudaError_t e = fp8moe_launch_router_bwd(a, stream);
  return e == cudaSuccess ? FP8MOE_OK : cuda_fail(e);
}

size_t fp8moe_adamw_workspace_size(const fp8moe_adamw_tensor* tensors, int32_t count,
                                   int32_t on_device) {
  return tensors && count > 0 ? adamw_ws_bytes(tensors, count, on_device != 0) : 0;
}

int fp8moe_adamw_step(const fp8moe_adamw_tensor* tensors, int32_t count, int64_t step,
                      const int64_t* step_dev, double lr, const float* lr_dev, double beta1,
                      double beta2, double eps, const float* grad_scale, uint32_t seed,
                      void* workspace, size_t workspace_bytes, fp8moe_stream_t stream) {
  if (count < 0 || (count > 0 && !tensors)) return FP8MOE_EINVAL;
  if (!step_dev && step < 1) return FP8MOE_EINVAL;
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0 && eps >= 0.0) ||
      (!lr_dev && !(lr == lr)))
    return FP8MOE_EINVAL;
  if (!aligned4(grad_scale) || !aligned4(lr_dev) || (reinterpret_cast<uintptr_t>(step_dev) & 7u))
    return FP8MOE_EALIGN;
  bool any = false;
  for (int32_t i = 0; i < count; ++i) {
    const int rc = check_adamw(tensors[i]);
    if (rc) return rc;
    any |= tensors[i].n > 0;
  }
  if (!any) return FP8MOE_OK;
  const bool on_device = step_dev || lr_dev;
  const size_t need = adamw_ws_bytes(tensors, count, on_device);
  if (need) {
    if (!workspace) return FP8MOE_EWORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return FP8MOE_EALIGN;
    if (workspace_bytes < need) return FP8MOE_EWORKSPACE;
  }
  int sms = 0;
  int rc = device_init(&sms);
  if (rc) return rc;

  AdamwRates* rates = on_device ? static_cast<AdamwRates*>(workspace) : nullptr;
  uint32_t* most = need ? reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) +
                                                      kAdamwRatesBytes)
                        : nullptr;
  cudaError_t e = cudaSuccess;
  if (need) {
    e = fp8moe_launch_adamw_prepare(rates, step_dev, step, lr_dev, lr, beta1, beta2, seed, most,
                                    (int64_t)((need - kAdamwRatesBytes) / 4), stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  AdamwCommon c = {};
  c.rates = rates;
  c.grad_scale = grad_scale;
  if (!on_device) {
    c.rate = (float)(lr / (1.0 - pow(beta1, (double)step)));
    c.root = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
    c.key = seed + 0x6A09E667u * (uint32_t)step;
  }
  c.b1 = (float)beta1, c.c1 = (float)(1.0 - beta1);
  c.b2 = (float)beta2, c.c2 = (float)(1.0 - beta2);
  c.eps = (float)eps;
  c.minus_zero = -0.0f;
  c.prepared = need > 0;

  // A launch for each table of tensors (at most 360 of them, or 2^30 units) with moments of the same kind, then
  // the weights with codes, one after the other.
  for (int bits = 8; bits <= 32; bits += 24) {
    AdamwEntry at[kAdamwEntries];
    int n = 0;
    uint64_t units = 0;
    for (int32_t i = 0; i < count; ++i) {
      const fp8moe_adamw_tensor& d = tensors[i];
      if (d.n == 0 || d.state_bits != bits || adamw_slabs(d)) continue;
      const AdamwEntry w = adamw_entry(d, i, lr);
      const uint64_t more = fp8moe_adamw_units(w);
      if (n == kAdamwEntries || (n > 0 && units + more > (1u << 30))) {
        e = fp8moe_launch_adamw(c, at, n, bits, sms, stream);
        if (e != cudaSuccess) return cuda_fail(e);
        c.prepared = 0;
        n = 0, units = 0;
      }
      at[n++] = w;
      units += more;
    }
    if (n == 0) continue;
    e = fp8moe_launch_adamw(c, at, n, bits, sms, stream);
    if (e != cudaSuccess) return cuda_fail(e);
    c.prepared = 0;
  }
  for (int32_t i = 0; i < count; ++i) {
    const fp8moe_adamw_tensor& d = tensors[i];
    if (d.n == 0 || !d.codes) continue;
    if (adamw_slabs(d)) {
      AdamwSlabArgs w = {};
      static_cast<AdamwEntry&>(w.d) = adamw_entry(d, i, lr);
      w.c = c, w.d.K = (int32_t)d.K, w.d.N = (int32_t)d.N, w.d.most = most;
      w.codes = d.codes, w.scale = d.code_scale, w.counters = most + adamw_columns(d);
      const int state = d.state_bits / 8;
      rc = adamw_tmap(&w.tm_p, d.p, 4, d);
      if (!rc) rc = adamw_tmap(&w.tm_g, d.g, d.g_type == FP8MOE_TYPE_BF16 ? 2 : 4, d);
      if (!rc) rc = adamw_tmap(&w.tm_m, d.m, state, d);
      if (!rc) rc = adamw_tmap(&w.tm_v, d.v, state, d);
      if (rc) return rc;
      e = fp8moe_launch_adamw_slabs(w, d.state_bits, sms, stream);
      c.prepared = 0;
    } else {
      e = fp8moe_launch_weight_codes(d.p, (int)(d.n / (d.K * d.N)), (int)d.K, (int)d.N, most,
                                     d.codes, d.code_scale, stream);
    }
    if (e != cudaSuccess) return cuda_fail(e);
    most += adamw_words(d);
  }
  return FP8MOE_OK;
}

int fp8moe_read_status(fp8moe_stream_t stream, uint32_t* flags) {
  if (!flags) return FP8MOE_EINVAL;
  uint32_t v = 0;
  const cudaError_t e = fp8moe_collect_status(&v, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  *flags = v;
  return FP8MOE_OK;
}

const char* fp8moe_status_string(int code) {
  switch (code) {
    case FP8MOE_OK: return "ok";
    case FP8MOE_EINVAL: return "invalid argument";
    case FP8MOE_EALIGN: return "misaligned pointer or dimension (16-byte rule)";
    case FP8MOE_EWORKSPACE: return "workspace missing or too small";
    case FP8MOE_ECUDA: return "CUDA error (see fp8moe_last_cuda_error)";
    case FP8MOE_EUNSUPPORTED: return "device is not sm_103";
    default: return "unknown status";
  }
}

int fp8moe_last_cuda_error(void) { return t_last_cuda_error; }

void fp8moe_internal_set_cuda_error(int e) { t_last_cuda_error = e; }

// The forward's argument checks that come before its workspace check, in the
// same order and with the same codes (for callers that supply the workspace
// themselves). FP8MOE_OK with *empty = 1: M == 0, nothing to do.
int fp8moe_internal_check_fwd_args(const void* lhs, int64_t M, int64_t K, const uint8_t* codes,
                                   const float* scale, int32_t E, int64_t N, const int32_t* gs,
                                   const void* out, int swiglu, int* empty) {
  *empty = 0;
  int rc = check_common(M, K, N, E);
  if (rc) return rc;
  if (swiglu && (N % 32 != 0)) return FP8MOE_EALIGN;
  if (M == 0) {
    *empty = 1;
    return FP8MOE_OK;
  }
  if (!lhs || !codes || !scale || !gs || !out) return FP8MOE_EINVAL;
  if (!aligned16(lhs) || !aligned16(codes) || !aligned16(scale) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(gs) & 3u))
    return FP8MOE_EALIGN;
  return FP8MOE_OK;
}

int fp8moe_num_sms(void) {
  int sms = 0;
  if (device_init(&sms) != FP8MOE_OK) return 0;
  return sms;
}

}  // extern "C"
