// lora_rows.cu -- low-rank adapters beside a projection, row by row on the CUDA cores.
//
//   V[m, j] = sum_k X[m, k] A[a][j, k]                     (the products with the rank-r rows)
//   Y[m, n] = base[m, n] + s[a] sum_j V[m, j] U[a][j, n]   (added to the projection's output)
//
// with a = adapter[m]; rows whose adapter lies outside the pool have V = 0 and Y = base.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cr_device.cuh"
#include "cr_internal.h"
#include "lora_device.cuh"

namespace cr {
namespace {

constexpr int kVWarps = 8;
constexpr int kYThreads = 64;

// One warp for each (row, four ranks, K split): every lane takes 8 values of the row and of the four rank
// rows at a time; the partial sums of the splits are added by whoever reads V.
__global__ void __launch_bounds__(32 * kVWarps)
    lora_v_rows_kernel(const uint16_t* __restrict__ X, int64_t ldx, const int32_t* __restrict__ adapter,
                       const uint16_t* __restrict__ down, float* __restrict__ V, int M, int K, int rank, int L,
                       int splits, int* __restrict__ status) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = CR_OK;
  const int lane = threadIdx.x & 31;
  const int groups = rank >> 2;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kVWarps + (threadIdx.x >> 5);
  const int64_t per_split = static_cast<int64_t>(M) * groups;
  if (task >= per_split * splits) return;
  const int sp = static_cast<int>(task / per_split);
  const int64_t rest = task - sp * per_split;
  const int64_t m = rest / groups;
  const int j = 4 * static_cast<int>(rest - m * groups);
  const int a = row_adapter(adapter, m, L);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (a >= 0) {
    const uint16_t* x = X + m * ldx;
    const uint16_t* w = down + (static_cast<int64_t>(a) * rank + j) * K;
    // split boundaries on multiples of 256 columns (one pass of the warp)
    const int passes = (K + 255) >> 8;
    const int p0 = static_cast<int>(static_cast<int64_t>(passes) * sp / splits);
    const int p1 = static_cast<int>(static_cast<int64_t>(passes) * (sp + 1) / splits);
    for (int p = p0; p < p1; ++p) {
      const int k = 256 * p + 8 * lane;
      if (k < K) {
        float xv[8];
        widen8(ldg16(x + k), xv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float wv[8];
          widen8(ldg16(w + static_cast<int64_t>(i) * K + k), wv);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[i] = fmaf(xv[e], wv[e], acc[i]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  }
  if (lane == 0)
    *reinterpret_cast<float4*>(V + (static_cast<int64_t>(sp) * M + m) * rank + j) =
        make_float4(acc[0], acc[1], acc[2], acc[3]);
}

// One block for each (row, 512 columns): the row's V (splits added in order) in shared memory, eight
// columns a thread.
__global__ void __launch_bounds__(kYThreads)
    lora_y_rows_kernel(const float* __restrict__ V, int splits, const int32_t* __restrict__ adapter,
                       const uint16_t* __restrict__ up, const float* __restrict__ scale,
                       const uint16_t* __restrict__ base, int64_t ldb, uint16_t* __restrict__ Y, int64_t ldy,
                       uint16_t* __restrict__ Vout, int M, int N, int rank, int L) {
  __shared__ float v[kMaxRank];
  const int64_t m = blockIdx.x;
  const int n = (blockIdx.y * kYThreads + threadIdx.x) * 8;
  const int a = row_adapter(adapter, m, L);
  const float s = (a >= 0 && scale) ? __ldg(scale + a) : 1.f;
  for (int j = threadIdx.x; j < rank; j += kYThreads) {
    float t = 0.f;
    if (a >= 0)
      for (int sp = 0; sp < splits; ++sp) t += V[(static_cast<int64_t>(sp) * M + m) * rank + j];
    if (Vout && blockIdx.y == 0) Vout[m * rank + j] = bf16_bits(t);
    v[j] = t * s;
  }
  __syncthreads();
  if (n >= N) return;
  float y[8] = {};
  if (a >= 0) {
    const uint16_t* u = up + static_cast<int64_t>(a) * rank * N + n;
#pragma unroll 4
    for (int j = 0; j < rank; ++j) {
      float uv[8];
      widen8(ldg16(u + static_cast<int64_t>(j) * N), uv);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(v[j], uv[e], y[e]);
    }
  }
  if (base) {
    float bv[8];
    widen8(*reinterpret_cast<const uint4*>(base + m * ldb + n), bv);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += bv[e];
  }
  *reinterpret_cast<uint4*>(Y + m * ldy + n) = narrow8(y);
}

}  // namespace

int lora_row_splits(int M, int K, int rank, int num_sms) {
  const int passes = (K + 255) / 256;
  const int64_t tasks = static_cast<int64_t>(M) * (rank / 4);
  const int64_t want = (16ll * num_sms + tasks - 1) / tasks;
  const int64_t most = (passes + 1) / 2;
  return static_cast<int>(want < 1 ? 1 : want < most ? want : most < 1 ? 1 : most);
}

cudaError_t launch_lora_v_rows(const uint16_t* X, int64_t ldx, const int32_t* adapter, const uint16_t* down, float* V,
                               int M, int K, int rank, int L, int splits, int* status, cudaStream_t stream) {
  const int64_t tasks = static_cast<int64_t>(M) * (rank / 4) * splits;
  const unsigned grid = static_cast<unsigned>((tasks + kVWarps - 1) / kVWarps);
  lora_v_rows_kernel<<<grid, 32 * kVWarps, 0, stream>>>(X, ldx, adapter, down, V, M, K, rank, L, splits, status);
  return cudaGetLastError();
}

cudaError_t launch_lora_y_rows(const float* V, int splits, const int32_t* adapter, const uint16_t* up,
                               const float* scale, const uint16_t* base, int64_t ldb, uint16_t* Y, int64_t ldy,
                               uint16_t* Vout, int M, int N, int rank, int L, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(M), static_cast<unsigned>((N + 8 * kYThreads - 1) / (8 * kYThreads)));
  lora_y_rows_kernel<<<grid, kYThreads, 0, stream>>>(V, splits, adapter, up, scale, base, ldb, Y, ldy, Vout, M, N,
                                                     rank, L);
  return cudaGetLastError();
}

}  // namespace cr
