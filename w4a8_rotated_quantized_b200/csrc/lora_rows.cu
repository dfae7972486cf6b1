// lora_rows.cu -- low-rank adapters beside a projection for few rows (single tokens of many requests), on the
// CUDA cores, one launch:
//
//   V[m, j] = sum_k X[m, k] A[a][j, k]
//   Y[m, n] = base[m, n] + s[a] sum_j V[m, j] U[a][j, n]
//
// with a = adapter[m]; rows whose adapter lies outside the pool have V = 0 and Y = base.
//
// A row has a cluster of 16 CTAs (fewer when there are more rows).  Each multiplies its part of the row by the rank rows of A and sends the
// partial sums to all the others, which add them in order; then each makes its part of the columns.  What
// costs time here is latency: a token's factors are a few hundred KB.  So the first ranks' U and the base are on
// their way before the first product, and the only other wait is one barrier of the cluster.  (As two launches
// with the partial sums in memory: 6.9 us for one token at rank 16, 2560 -> 9728, against 4.4.)

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "cr_device.cuh"
#include "cr_internal.h"
#include "lora_device.cuh"

namespace cr {
namespace {

constexpr int kMostCluster = 16;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 8;   // ranks of U on their way from the start

__device__ __forceinline__ void st_shared_cluster_f1(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

__global__ void __launch_bounds__(kThreads, 3)
    lora_rows_kernel(const uint16_t* __restrict__ X, int64_t ldx, const int32_t* __restrict__ adapter,
                     const uint16_t* __restrict__ down, const uint16_t* __restrict__ up,
                     const float* __restrict__ scale, const uint16_t* base, int64_t ldb, uint16_t* Y, int64_t ldy,
                     uint16_t* __restrict__ Vout, int N, int K, int rank, int L, int ctas) {
  __shared__ float part[kMostCluster][kMaxRank];
  __shared__ float v[kMaxRank];
  const int c = static_cast<int>(cluster_ctarank());
  const int64_t m = blockIdx.x / ctas;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int a = row_adapter(adapter, m, L);  // the same in the whole cluster
  // this CTA's columns of Y, eight a thread and pass
  const int per_n = (N / 8 + ctas - 1) / ctas;
  const int n_end = 8 * min((c + 1) * per_n, N / 8);
  int n = 8 * (c * per_n + threadIdx.x);
  const uint16_t* brow = base ? base + m * ldb : nullptr;
  if (a < 0) {
    for (; n < n_end; n += 8 * kThreads)
      *reinterpret_cast<uint4*>(Y + m * ldy + n) =
          brow ? *reinterpret_cast<const uint4*>(brow + n) : make_uint4(0, 0, 0, 0);
    if (Vout && c == 0 && threadIdx.x < rank) Vout[m * rank + threadIdx.x] = 0;
    return;
  }
  cluster_arrive();
  const uint16_t* u = up + static_cast<int64_t>(a) * rank * N;
  uint4 ahead[kAhead], b = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    ahead[j] = make_uint4(0, 0, 0, 0);
    if (n < n_end && j < rank) ahead[j] = ldg_here_u4(u + static_cast<int64_t>(j) * N + n);
  }
  if (n < n_end && brow) b = ld_here_u4(brow + n);

  // partial sums over this CTA's columns of X: ranks warp, warp + 8, ... for each warp
  const int per_k = (K / 8 + ctas - 1) / ctas;
  const int k_end = 8 * min((c + 1) * per_k, K / 8);
  const uint16_t* x = X + m * ldx;
  const uint16_t* w = down + static_cast<int64_t>(a) * rank * K;
  float acc[kMaxRank / kWarps] = {};
  for (int k = 8 * (c * per_k + lane); k < k_end; k += 256) {
    float xv[8];
    widen8(ldg16(x + k), xv);
#pragma unroll
    for (int i = 0; i < kMaxRank / kWarps; ++i) {
      const int j = warp + kWarps * i;
      if (j < rank) {
        float wv[8];
        widen8(ldg16(w + static_cast<int64_t>(j) * K + k), wv);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i] = fmaf(xv[e], wv[e], acc[i]);
      }
    }
  }
  cluster_wait();  // every CTA of the cluster has started: its shared memory may be written to
#pragma unroll
  for (int i = 0; i < kMaxRank / kWarps; ++i) {
    const int j = warp + kWarps * i;
    if (j < rank) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      if (lane < ctas) st_shared_cluster_f1(mapa_shared(smem_u32(&part[c][j]), lane), acc[i]);
    }
  }
  __syncwarp();
  cluster_sync();
  if (threadIdx.x < rank) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kMostCluster; ++i)
      if (i < ctas) t += part[i][threadIdx.x];
    if (Vout && c == 0) Vout[m * rank + threadIdx.x] = bf16_bits(t);
    v[threadIdx.x] = t * __ldg(scale + a);
  }
  __syncthreads();
  for (bool first = true; n < n_end; n += 8 * kThreads, first = false) {
    float y[8] = {};
    if (first) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (j < rank) {
          float uv[8];
          widen8(ahead[j], uv);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = fmaf(v[j], uv[e], y[e]);
        }
      }
    } else if (brow) {
      b = *reinterpret_cast<const uint4*>(brow + n);
    }
#pragma unroll 8
    for (int j = first ? kAhead : 0; j < rank; ++j) {
      float uv[8];
      widen8(ldg16(u + static_cast<int64_t>(j) * N + n), uv);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(v[j], uv[e], y[e]);
    }
    float bv[8];
    widen8(b, bv);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += bv[e];
    *reinterpret_cast<uint4*>(Y + m * ldy + n) = narrow8(y);
  }
}

std::atomic<bool> g_attr_done[64];

}  // namespace

int launch_lora_rows(const uint16_t* X, int64_t ldx, const int32_t* adapter, const uint16_t* down, const uint16_t* up,
                     const float* scale, const uint16_t* base, int64_t ldb, uint16_t* Y, int64_t ldy, uint16_t* Vout,
                     int M, int N, int K, int rank, int L, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CR_ERR_CUDA;
  if (!g_attr_done[dev].load()) {
    if (cudaFuncSetAttribute(lora_rows_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return CR_ERR_CUDA;
    g_attr_done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  // fewer CTAs a row where more rows share the machine
  const int ctas = M <= 8 ? 16 : M <= 24 ? 8 : 4;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(M * ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_rows_kernel, X, ldx, adapter, down, up, scale, base, ldb, Y, ldy, Vout, N, K,
                            rank, L, ctas) == cudaSuccess
             ? CR_OK
             : CR_ERR_CUDA;
}

}  // namespace cr
