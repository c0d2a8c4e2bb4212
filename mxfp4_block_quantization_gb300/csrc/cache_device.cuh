// cache_device.cuh — what the cache and the attention over it share on the
// device (cache.cu, attention.cu).
#pragma once

#include <cuda_runtime.h>

namespace mxfp4 {

// A cache's global scale; a call that touches no cache may have none.
__device__ __forceinline__ float global_scale_or_one(const float* g) { return g != nullptr ? __ldg(g) : 1.0f; }

}  // namespace mxfp4
