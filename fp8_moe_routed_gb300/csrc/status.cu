// status.cu -- the status words of all translation units, read and cleared in one launch.
//
// A warp takes every word by an exchange with zero, so a bit that another stream's kernel
// sets meanwhile is either in this reading or left for the next one, and leaves their OR in
// a word that is copied to the host: one launch, one copy and one wait, whatever the number
// of words. (A copy, a wait, a copy of zero and a wait for each of eleven words took 198 us;
// this takes 23.)
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace fp8moe {

constexpr int kMaxWords = 32;       // a lane each
// Readings in flight: each has a word of its own.
constexpr unsigned kReadings = 1024;

struct StatusWords {
  uint32_t* at[kMaxWords];
};

static __device__ uint32_t g_readings[kReadings];

__global__ void collect_status_kernel(const __grid_constant__ StatusWords words, int n,
                                      unsigned reading) {
  const uint32_t v = (int)threadIdx.x < n ? atomicExch(words.at[threadIdx.x], 0u) : 0u;
  const uint32_t all = __reduce_or_sync(0xffffffffu, v);
  if (threadIdx.x == 0) g_readings[reading] = all;
}

}  // namespace fp8moe

cudaError_t fp8moe_collect_status(uint32_t* flags, cudaStream_t s) {
  using namespace fp8moe;
  static std::atomic<unsigned> next{0};
  cudaError_t (*const units[])(uint32_t**) = {
      fp8moe_status_take_quant, fp8moe_status_take_dequant, fp8moe_status_take_gmm_fwd,
      fp8moe_status_take_dlhs, fp8moe_status_take_dlhs_pair, fp8moe_status_take_tgmm,
      fp8moe_status_take_selftest, fp8moe_status_take_route, fp8moe_status_take_norm,
      fp8moe_status_take_mxfp4, fp8moe_status_take_gmm_mxfp4, fp8moe_status_take_router,
      fp8moe_status_take_router_group, fp8moe_status_take_router_bwd,
      fp8moe_status_take_adamw};
  constexpr int n = sizeof(units) / sizeof(units[0]);
  static_assert(n <= kMaxWords, "a lane for every word");
  StatusWords words = {};
  for (int i = 0; i < n; ++i) {
    const cudaError_t e = units[i](&words.at[i]);
    if (e != cudaSuccess) return e;
  }
  const unsigned reading = next++ % kReadings;
  collect_status_kernel<<<1, 32, 0, s>>>(words, n, reading);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbolAsync(flags, g_readings, sizeof(uint32_t), reading * sizeof(uint32_t),
                                cudaMemcpyDeviceToHost, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}
