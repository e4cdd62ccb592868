// Host-side services that the library's translation units share (defined in
// attn_api.cu): the per-device status word, the tensor-map encoder, the wait
// limit, and the record of the contexts a kernel's attributes were set in.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace attn {

constexpr int kApiMaxDevices = 64;

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, or nullptr when the driver has none.
EncodeTiledFn api_encode_tiled();
// Device address of the current device's status word, or nullptr on a CUDA error.
int* api_status_ptr();
// Upper bound of one internal wait, in nanoseconds.
unsigned long long api_wait_limit_ns();
// Sets a kernel's dynamic shared-memory opt-in once per context; `seen` is the
// kernel's own record (kApiMaxDevices entries, zero at first).
cudaError_t api_smem_opt_in(const void* kernel, int bytes, CUcontext* seen);

}  // namespace attn
