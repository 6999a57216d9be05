// pdl.cuh -- programmatic dependent launch: the second kernel of a call starts while the
// first still runs, sets itself up, and waits for the first's results only where it
// needs them. The first kernel runs as an ordinary launch, so everything that came
// before the call is complete when either of the two starts.
#pragma once
#include <cuda_runtime.h>

namespace fp8moe {

// In the first kernel: the second may start now (its CTAs take what room is left).
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// In the second kernel: returns when the first has completed and its writes are visible.
// (No effect in a kernel that was launched without the attribute.)
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

inline void pdl_attribute(cudaLaunchAttribute& a) {
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
}

}  // namespace fp8moe
