// The layer norm and distillation kernels in a library of their own whose
// waits run out at once (MP_WAIT_LIMIT_NS = 0; compiled by
// test_gpu_train_give_up.py), with what they need of the rest.
#include "mp_internal.h"

namespace mpk {

cudaError_t device_info(DeviceInfo* out) {
  cudaError_t e = cudaGetDevice(&out->device);
  if (e != cudaSuccess) return e;
  return cudaDeviceGetAttribute(&out->sms, cudaDevAttrMultiProcessorCount, out->device);
}

int record_cuda_error(cudaError_t) { return MP_ERR_CUDA; }

}  // namespace mpk
