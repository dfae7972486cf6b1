// lora_rows.cu -- low-rank adapters beside a projection for few rows (single tokens of many requests), on the
// CUDA cores, one launch:
//
//   V[m, j] = sum_k X[m, k] A[a][j, k]
//   Y[m, n] = base[m, n] + s[a] sum_j V[m, j] U[a][j, n]
//
// with a = adapter[m]; rows whose adapter lies outside the pool have V = 0 and Y = base.
//
// A row has a cluster of 16 CTAs (fewer when there are more rows).  Each multiplies its part of the row by the
// rank rows of A and sends the partial sums to all the others, which add them in order; then each makes its part
// of the columns.  What costs time here is latency: a token's factors are a few hundred KB.  So each warp has
// four loads on their way whatever the rank (its tasks are pairs of a rank and 256 columns, not ranks), the
// ranks of a column are shared out between the threads that columns leave idle, their first U and the base are
// on their way before the first product, and the only other wait is one barrier of the cluster.  One token of
// rank 16, 2560 -> 9728, takes 4.2 us, 64 tokens of 48 adapters, of which they name 33, 7.1 a call (16 MB: 2.3 TB/s;
// the index, two dependent rounds of loads and the cluster's exchange, not bandwidth).  Asking L2 for the rest of U before the first product took
// longer.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "cr_device.cuh"
#include "cr_internal.h"
#include "f16_device.cuh"
#include "grid_sync.cuh"
#include "lora_device.cuh"

namespace cr {
namespace {

constexpr int kMostCluster = 16;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 1;     // ranks of U that a thread has on their way from the start
constexpr int kTasks = 4;     // loads of A that a warp has on their way
// More of either, or of U in the second product, does not fit 64 registers a thread, two CTAs an SM, and costs more
// in spills than it hides: 64 rows of 48 adapters take 7.5 us a call so, 8.5 with two ranks ahead, 8.4 with eight
// tasks, 10.9 with four and eight; one row 4.0 on the device, with eight tasks 4.7 (all before the index was asked for
// once a CTA).
constexpr int kMostPasses = CR_MAX_K / 256 / 4;  // 256 columns at a time: of a CTA in a cluster of 4 (2: half the K)

__device__ __forceinline__ void st_shared_cluster_f1(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

__global__ void __launch_bounds__(kThreads, 2)
    lora_rows_kernel(const uint16_t* __restrict__ X, int64_t ldx, const int32_t* __restrict__ adapter,
                     const uint16_t* __restrict__ down, const uint16_t* __restrict__ up,
                     const float* __restrict__ scale, const uint16_t* base, int64_t ldb, uint16_t* Y, int64_t ldy,
                     float* __restrict__ V32, uint16_t* __restrict__ Vout, int N, int K, int rank, int L, int ctas,
                     int* __restrict__ status) {
  __shared__ float part[kMostCluster][kMaxRank];
  // sums of the tasks [pass][rank]; later partial results [rank group][column piece][8]
  __shared__ __align__(16) float scratch[kMostPasses * kMaxRank];
  __shared__ float v[kMaxRank];
  griddep_wait();  // for what the stream ran before; past L1 from here on: that may have left older values there
  if (threadIdx.x == 0) {
    griddep_launch_dependents();
    if (status && blockIdx.x == 0) *status = CR_OK;
  }
  const int c = static_cast<int>(cluster_ctarank());
  const int64_t m = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The adapter, the same in the whole cluster.  One thread asks for it: past L1 each warp's load is a request of its
  // own, and those of all CTAs meet in the same few bytes of L2 (calls in a chain, each warp | one thread: 64 rows 8.2 |
  // 7.8 us; one row, where the barrier is all that counts, 4.0 | 4.2).
  __shared__ int own;
  if (tid == 0) own = row_adapter(adapter, m, L);
  __syncthreads();
  const int a = own;
  // this CTA's columns of Y in pieces of eight, and their ranks in groups where there are threads to spare
  const int per_n = (N / 8 + ctas - 1) / ctas;
  const int p0 = c * per_n;
  const int pieces = min(per_n, N / 8 - p0);  // (none, or fewer than none, for the last CTAs of a short row)
  const int groups = per_n > kThreads / 2 ? 1 : min(kThreads / per_n, 16);
  const int group = groups > 1 ? tid / per_n : 0, piece = groups > 1 ? tid - group * per_n : tid;
  const bool mine = piece < pieces && group < groups;
  const uint16_t* brow = base ? base + m * ldb : nullptr;
  if (a < 0) {
    for (int p = tid; p < pieces; p += kThreads)
      *reinterpret_cast<uint4*>(Y + m * ldy + 8 * (p0 + p)) =
          brow ? ldcg_here_u4(brow + 8 * (p0 + p)) : make_uint4(0, 0, 0, 0);
    if (V32 && c == 0 && tid < rank) V32[m * rank + tid] = 0.f;
    if (Vout && c == 0 && tid < rank) Vout[m * rank + tid] = 0;
    return;
  }
  cluster_arrive();
  const float sc = tid < rank ? ldcg_here_f1(scale + a) : 0.f;
  const uint16_t* u = up + static_cast<int64_t>(a) * rank * N + 8 * p0;
  uint4 ahead[kAhead], b = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int j = group + groups * i;
    ahead[i] = make_uint4(0, 0, 0, 0);
    if (mine && j < rank) ahead[i] = ldcg_here_u4(u + static_cast<int64_t>(j) * N + 8 * piece);
  }
  if (mine && group == 0 && brow) b = ldcg_here_u4(brow + 8 * (p0 + piece));

  // partial sums over this CTA's columns of X: task t is rank t % rank over 256 columns
  const int per_k = (K / 8 + ctas - 1) / ctas;
  const int q0 = c * per_k, q_end = min(q0 + per_k, K / 8);
  const int passes = (per_k + 31) / 32;
  const uint16_t* x = X + m * ldx;
  const uint16_t* w = down + static_cast<int64_t>(a) * rank * K;
  for (int t0 = kTasks * warp; t0 < rank * passes; t0 += kTasks * kWarps) {
    uint4 xq[kTasks / 4], wq[kTasks];  // four tasks in a row are of one pass: ranks come in fours
#pragma unroll
    for (int i = 0; i < kTasks; i += 4) {
      const int t = t0 + i, pass = t / rank, j = t - pass * rank;
      const int q = q0 + 32 * pass + lane;
      const bool in = q < q_end && t < rank * passes;
      const uint16_t* src = w + static_cast<int64_t>(j) * K + 8 * q;
      xq[i / 4] = in ? ldcg_here_u4(x + 8 * q) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) wq[i + e] = in ? ldcg_here_u4(src + static_cast<int64_t>(e) * K) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kTasks; ++i) {
      float xv[8], wv[8], s = 0.f;
      widen8(xq[i / 4], xv);
      widen8(wq[i], wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(xv[e], wv[e], s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0 && t0 + i < rank * passes) scratch[t0 + i] = s;
    }
  }
  __syncthreads();
  cluster_wait();  // every CTA of the cluster has started: its shared memory may be written to
  for (int i = tid; i < rank * ctas; i += kThreads) {
    const int to = i / rank, j = i - to * rank;
    float s = 0.f;
    for (int p = 0; p < passes; ++p) s += scratch[p * rank + j];
    st_shared_cluster_f1(mapa_shared(smem_u32(&part[c][j]), to), s);
  }
  __syncwarp();
  cluster_sync();
  if (tid < rank) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kMostCluster; ++i)
      if (i < ctas) t += part[i][tid];
    if (V32 && c == 0) V32[m * rank + tid] = t;
    if (Vout && c == 0) Vout[m * rank + tid] = bf16_bits(t);
    v[tid] = t * sc;
  }
  __syncthreads();
  for (int p = piece, first = 1; p < pieces && group < groups; p += kThreads, first = 0) {
    float y[8] = {};
    if (first) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = group + groups * i;
        if (j < rank) {
          float uv[8];
          widen8(ahead[i], uv);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = fmaf(v[j], uv[e], y[e]);
        }
      }
    } else if (brow) {
      b = ldcg_here_u4(brow + 8 * (p0 + p));
    }
#pragma unroll 4
    for (int j = group + (first ? groups * kAhead : 0); j < rank; j += groups) {
      float uv[8];
      widen8(ldcg_here_u4(u + static_cast<int64_t>(j) * N + 8 * p), uv);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(v[j], uv[e], y[e]);
    }
    if (groups == 1) {
      float bv[8];
      widen8(b, bv);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] += bv[e];
      *reinterpret_cast<uint4*>(Y + m * ldy + 8 * (p0 + p)) = narrow8(y);
    } else {  // (one pass: a thread for each piece and group)
      float4* d = reinterpret_cast<float4*>(scratch) + 2 * (group * per_n + p);
      d[0] = make_float4(y[0], y[1], y[2], y[3]);
      d[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
  }
  if (groups == 1) return;
  __syncthreads();
  if (mine && group == 0) {
    float y[8];
    widen8(b, y);
    for (int g = 0; g < groups; ++g) {
      const float4* d = reinterpret_cast<const float4*>(scratch) + 2 * (g * per_n + piece);
      const float4 f0 = d[0], f1 = d[1];
      y[0] += f0.x; y[1] += f0.y; y[2] += f0.z; y[3] += f0.w;
      y[4] += f1.x; y[5] += f1.y; y[6] += f1.z; y[7] += f1.w;
    }
    *reinterpret_cast<uint4*>(Y + m * ldy + 8 * (p0 + piece)) = narrow8(y);
  }
}

std::atomic<bool> g_attr_done[64];

}  // namespace

// By microseconds, fitted to both forms' times for 260 calls of 1 to 1400 rows, 256 to 10240 columns, ranks 4 to
// 128 and pools of 1 to 48 adapters: the choice costs 0.4 % over the better form on average and 52 % at worst.
// The row form costs 3.8, a row's CTAs a fiftieth, and each row's own factors come at 8.6 TB/s (L2).  The batch
// form costs 8.3, its first adapter's factors at 0.35 TB/s, the rows' values, and for every further adapter that
// may occur among a tile's rows 0.45 and its factors at 1.4 TB/s.
//   960 rows, rank 16, 1488 -> 1272, 43 adapters:   rows 33, batch 13
//   336 rows, rank 4, 584 -> 416, 7 adapters:       rows 10, batch 9
//   34 rows, rank 64, 4112 -> 5400, one adapter:    rows 14, batch 9 (the worst choice)
// The workspace's size goes by the same rule and its call knows of no indices, so a pool of several counts as that also
// for calls without indices, whose rows all use the first adapter.
bool use_lora_rows(int M, int N, int K, int rank, int L) {
  if (M > 1024) return false;
  const double columns = static_cast<double>(K) + N, factors = 2.0 * rank * columns;
  const int most = L < M ? (L < 128 ? L : 128) : (M < 128 ? M : 128);
  const double rows = 3.8 + M / 50.0 + M * factors / 8.6e6;
  const double batch = 8.3 + factors / 3.5e5 + M * columns / 1.7e6 + (most - 1) * (0.45 + factors / 1.4e6);
  return rows < batch;
}

int launch_lora_rows(const uint16_t* X, int64_t ldx, const int32_t* adapter, const uint16_t* down, const uint16_t* up,
                     const float* scale, const uint16_t* base, int64_t ldb, uint16_t* Y, int64_t ldy, float* V,
                     uint16_t* Vout, int M, int N, int K, int rank, int L, int* status, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CR_ERR_CUDA;
  if (!g_attr_done[dev].load()) {
    if (cudaFuncSetAttribute(lora_rows_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return CR_ERR_CUDA;
    g_attr_done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  // fewer CTAs a row where more rows share the machine; two only where their passes fit
  const int ctas = M <= 4 ? 16 : M <= 8 ? 8 : M <= 64 || K > CR_MAX_K / 2 ? 4 : 2;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(M * ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, lora_rows_kernel, X, ldx, adapter, down, up, scale, base, ldb, Y, ldy, V, Vout, N, K,
                            rank, L, ctas, status) == cudaSuccess
             ? CR_OK
             : CR_ERR_CUDA;
}

}  // namespace cr
