// The CUDA runtime's calls that gdn_paged_mass makes, for the tests: nothing runs, launches are counted, and the first of them
// fails where the test says so.
#include <cuda_runtime.h>

static int launches, failing;
static cudaError_t last;

extern "C" {
void fake_reset(int fail_first) { launches = 0, failing = fail_first, last = cudaSuccess; }
int fake_launches() { return launches; }

cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *, void **) {
  const bool fails = failing && launches == 0;
  ++launches;
  if (fails) last = cudaErrorLaunchOutOfResources;
  return fails ? last : cudaSuccess;
}
cudaError_t cudaGetLastError() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
cudaError_t cudaPeekAtLastError() { return last; }

void **__cudaRegisterFatBinary(void *) {
  static void *handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
}
