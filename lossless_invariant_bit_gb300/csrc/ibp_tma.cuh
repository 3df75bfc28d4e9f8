// Host-side helpers of the kernels that use tensor maps (ibp_launch.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

namespace ibp {

// cuTensorMapEncodeTiled, looked up once through the runtime (the library
// links no driver library); NULL when the driver has none.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled();

// Raise a kernel's dynamic shared-memory limit to `smem` once per device (a
// call being captured into a CUDA graph then sets nothing).
cudaError_t smem_limit(const void* fn, size_t smem);

}  // namespace ibp
