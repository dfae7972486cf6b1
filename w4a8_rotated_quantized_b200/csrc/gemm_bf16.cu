// gemm_bf16.cu -- the input gradient's product dX[m, k] = sum_n dY[m, n] W[n, k], bf16 operands, float32
// sums.  Simple tiled form: 64 x 64 outputs a block, 16 steps of n at a time through shared memory.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cr_device.cuh"
#include "cr_internal.h"
#include "lora_device.cuh"

namespace cr {
namespace {

__global__ void __launch_bounds__(256)
    gemm_bf16_kernel(const uint16_t* __restrict__ A, int64_t lda, const uint16_t* __restrict__ W,
                     uint16_t* __restrict__ Y, int64_t ldy, int M, int N, int K) {
  __shared__ float sa[16][65], sw[16][64];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = 64ll * blockIdx.x;
  const int k0 = 64 * blockIdx.y;
  float acc[4][4] = {};
  for (int n0 = 0; n0 < N; n0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int n = n0 + (i & 15), k = k0 + (i & 63), nw = n0 + (i >> 6);
      const int64_t m = m0 + (i >> 4);
      sa[i & 15][i >> 4] = (m < M && n < N) ? bf16_float(A[m * lda + n]) : 0.f;
      sw[i >> 6][i & 63] = (nw < N && k < K) ? bf16_float(W[static_cast<int64_t>(nw) * K + k]) : 0.f;
    }
    __syncthreads();
    for (int n = 0; n < 16; ++n)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[n][ty + 16 * i], sw[n][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i;
      const int k = k0 + tx + 16 * j;
      if (m < M && k < K) Y[m * ldy + k] = bf16_bits(acc[i][j]);
    }
}

}  // namespace

int launch_gemm_bf16(const void* A, int64_t lda, const void* W, void* Y, int64_t ldy, int M, int N, int K, int* status,
                     int num_sms, cudaStream_t stream) {
  (void)status;
  (void)num_sms;
  const dim3 grid((M + 63) / 64, (K + 63) / 64);
  gemm_bf16_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(A), lda, static_cast<const uint16_t*>(W),
                                             static_cast<uint16_t*>(Y), ldy, M, N, K);
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // namespace cr
