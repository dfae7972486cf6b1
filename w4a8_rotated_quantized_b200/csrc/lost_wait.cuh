// lost_wait.cuh -- waits that ran out, noted beside the status word in a word of the device that outlives the call's
// workspace: a caller that keeps no workspace can still ask.  Every file that includes this has a word of its own,
// which the host reads and clears.  Included after cr_device.cuh.
#pragma once

#include <cuda_runtime.h>

namespace cr {
namespace {

__device__ int g_lost_wait;

// A wait ran out.  `status` may be null.
__device__ __forceinline__ void record_timeout(int* status) {
  record_status(status, CR_ERR_TIMEOUT);
  atomicExch(&g_lost_wait, 1);
}

// Whether one did since this was last asked, on the current device and up to here on the stream.
cudaError_t take_lost_wait(cudaStream_t stream, bool* found) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_lost_wait, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess || !v) return e;
  *found = true;
  v = 0;
  e = cudaMemcpyToSymbolAsync(g_lost_wait, &v, sizeof(v), 0, cudaMemcpyHostToDevice, stream);
  return e == cudaSuccess ? cudaStreamSynchronize(stream) : e;
}

}  // namespace
}  // namespace cr
