// tensor_map.cuh -- the driver's encoder of tensor maps (cuTensorMapEncodeTiled).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace gdn {

// The encoder, or null where the driver has none.  It fails without a current context, which a thread gets from its
// first runtime call that needs one; here a tensor map may come before any (its memory may all have been allocated
// already), so the thread's device is set once.
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool there =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess;
    return there ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr) : nullptr;
  }();
  thread_local bool current = false;
  int device = 0;
  if (!current) current = cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess;
  return fn;
}

}  // namespace gdn
