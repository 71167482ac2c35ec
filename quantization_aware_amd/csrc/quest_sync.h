// A workgroup barrier for kernels that keep loads in flight across it.
#pragma once

#include <hip/hip_runtime.h>

namespace quest {

// A workgroup barrier that waits for this wave's LDS accesses only (a
// __syncthreads would also wait for every load and store in flight).  The two
// builtins keep memory accesses on their side; arithmetic may cross.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
}

}  // namespace quest
