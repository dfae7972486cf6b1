// gemm_bf16.cu -- bf16 x bf16 GEMM on a CTA pair (tcgen05 cta_group::2), for the packed layer's input
// gradient: Y[m, k] = sum_n A[m, n] W[n, k], float32 accumulators, one rounding to bf16.
//
// A (the output gradient) lies along the sum ("K-major"); W [N, K] is read as it is stored, its rows
// across the sum, as an MN-major operand: no transposed copy of the weights is made.
//
// * A pair of CTAs (a cluster of 2) computes a 256 x 256 output tile (M = 256, N = 256, K = 16 a
//   instruction); each CTA loads 128 rows of A and 128 columns of W.
// * A stage holds 64 steps of the sum: one 128-row box of A (128-byte rows) and two boxes of 64 rows x
//   64 columns of W, 32 KB for each CTA, six stages.  Both CTAs' loads of a stage complete on the
//   leader's full barrier.  No multicast.
// * The tensor cores bound it (two 16 KB operands for 4 x 131 cycles of MMA a stage); accumulators are
//   double-buffered (2 x 256 TMEM columns) so that the epilogue runs beside the next tile's product.
//   8192 x 12288 x 3072 takes 452-476 us at full clocks (1.30-1.37 PFLOP/s, tensor pipe 82 % active) and about 530
//   in a long loop, where power lowers them.
// * The sum's tail past N and rows and columns past the matrices are zeros that TMA fills in.
//
// Roles (192 threads per CTA): warp 0 TMEM allocation and, in the leader CTA, the MMA issuer; warp 1 TMA
// producer; warps 2-5 epilogue (TMEM -> bf16 -> swizzled staging -> TMA stores).  Every wait is bounded;
// on expiry the CTA records CR_ERR_TIMEOUT in the device status word and winds down.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "cr_device.cuh"
#include "cr_internal.h"
#include "f16_device.cuh"
#include "lora_device.cuh"
#include "lost_wait.cuh"

namespace cr {
namespace {

constexpr int CM = 128;            // A rows per CTA (pair: 256)
constexpr int PN = 256;            // output columns per pair tile
constexpr int CN = PN / 2;         // W columns per CTA
constexpr int BK = 64;             // steps of the sum per stage
constexpr int STAGES = 6;
constexpr int A_S = CM * BK * 2;   // 16 KB
constexpr int B_GROUP = 64 * BK * 2;  // one box: 64 columns x BK rows of W, 8 KB
constexpr int B_S = 2 * B_GROUP;   // 16 KB
constexpr int STAGE = A_S + B_S;
constexpr int OFF_RING = 0;
constexpr int OFF_STAGE = OFF_RING + STAGES * STAGE;  // epilogue output staging
constexpr int STAGE_BYTES = 32 * 64 * 2;              // 32 rows x 64 bf16 columns
constexpr int OFF_BAR = OFF_STAGE + 4 * 2 * STAGE_BYTES;
constexpr int NUM_BARS = 2 * STAGES + 4;
constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
constexpr int SMEM_BYTES = OFF_MISC + 16;
constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;
constexpr int NUM_THREADS = 192;
constexpr int TMEM_COLS = 512;
constexpr int ACC_COLS = PN;
constexpr int EMPTY_ACC_ARRIVALS = 2 * 4;  // 4 epilogue warps x 2 CTAs
constexpr uint32_t IDESC = idesc_bf16(2 * CM, PN, false, true);

static_assert(2 * ACC_COLS <= TMEM_COLS, "TMEM budget");
static_assert(STAGE_BYTES % 1024 == 0 && OFF_STAGE % 1024 == 0, "swizzle atoms need 1024-byte alignment");
static_assert(SMEM_ALLOC <= 232448, "shared memory budget");

struct Smem {
  uint8_t* base;
  __device__ uint8_t* a(int s) const { return base + OFF_RING + s * STAGE; }
  __device__ uint8_t* b(int s) const { return base + OFF_RING + s * STAGE + A_S; }
  __device__ uint8_t* stage(int q, int buf) const { return base + OFF_STAGE + (2 * q + buf) * STAGE_BYTES; }
  __device__ uint32_t bar(int i) const { return smem_u32(base + OFF_BAR + 8 * i); }
  __device__ uint32_t full(int s) const { return bar(s); }
  __device__ uint32_t empty(int s) const { return bar(STAGES + s); }
  __device__ uint32_t tmem_full(int b) const { return bar(2 * STAGES + b); }
  __device__ uint32_t tmem_empty(int b) const { return bar(2 * STAGES + 2 + b); }
  __device__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(base + OFF_MISC); }
  __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(base + OFF_MISC + 4); }
};

__device__ __forceinline__ void fail(const Smem& sm, int* status) {
  record_timeout(status);
  *sm.abort_flag() = 1;
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    gemm_bf16_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                          const __grid_constant__ CUtensorMap tmap_y, int M, int N, int K, int* __restrict__ status) {
  extern __shared__ uint8_t smem_raw[];
  Smem sm;
  sm.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0 = leader (issues the MMAs), 1 = peer
  const int pair = static_cast<int>(cluster_id_x());
  const int npairs = static_cast<int>(num_clusters_x());
  const int num_m = (M + 2 * CM - 1) / (2 * CM);
  const int num_n = (K + PN - 1) / PN;
  const int num_tiles = num_m * num_n;
  const int nk = (N + BK - 1) / BK;
  const int my_tiles = pair < num_tiles ? (num_tiles - pair + npairs - 1) / npairs : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(sm.full(s), 1);   // the leader producer's arrive (+ both CTAs' bytes)
      mbar_init(sm.empty(s), 1);  // the MMA commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sm.tmem_full(b), 1);
      mbar_init(sm.tmem_empty(b), EMPTY_ACC_ARRIVALS);
    }
    *sm.abort_flag() = 0;
    fence_mbar_init();
  }
  if (warp == 1 && lane == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_w);
    prefetch_tmap(&tmap_y);
  }
  if (warp == 0) {
    tmem_alloc_pair(smem_u32(sm.tmem_slot()), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrive or load completion
  tc_fence_after();
  const uint32_t tmem_base = *sm.tmem_slot();
  volatile int* abort = sm.abort_flag();

  auto tile_of = [&](int local) { return pair + local * npairs; };

  if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer (leader CTA, one thread)
    if (rank == 0 && elect_one()) {
      bool ok = true;
      bool committed = false;
      uint32_t last_bar = 0, last_par = 0;
      int s = 0;
      uint32_t ph = 0;
      bool next_full = my_tiles > 0 && mbar_test(sm.full(0), 0);
      for (int t = 0; ok && t < my_tiles; ++t) {
        const int b = t & 1;
        if (!mbar_wait(sm.tmem_empty(b), static_cast<uint32_t>(((t >> 1) & 1) ^ 1), abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * ACC_COLS);
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait_from(sm.full(s), ph, next_full, abort)) { ok = false; break; }
          tc_fence_after();
          const uint64_t da = sw128_kmajor_desc(smem_u32(sm.a(s)));
          const uint64_t db = sw128_mnmajor_desc(smem_u32(sm.b(s)), B_GROUP);
          // 16 steps of the sum: 32 bytes along A's rows, 16 rows (2048 bytes) of W
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            umma_f16_pair_ss(d_tmem, da + 2u * kk, db + 128u * kk, IDESC, (kb | kk) ? 1u : 0u);
          umma_commit_pair_mc(sm.empty(s), 0x3);
          last_bar = sm.empty(s);
          last_par = ph;
          committed = true;
          if (++s == STAGES) { s = 0; ph ^= 1u; }
          // test the next stage while these MMAs run
          next_full = mbar_test(sm.full(s), ph);
        }
        if (!ok) break;
        umma_commit_pair_mc(sm.tmem_full(b), 0x3);
      }
      if (!ok) {
        fail(sm, status);
        if (committed) {
          volatile int never = 0;
          mbar_wait(last_bar, last_par, &never);  // the MMAs issued so far have finished reading
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      bool ok = true;
      const uint32_t full_leader0 = mapa_shared(sm.full(0), 0);
      int f = 0, s = 0;
      uint32_t ph = 0;  // phase parity of stage s's current use
      for (int t = 0; ok && t < my_tiles; ++t) {
        const int tile = tile_of(t);
        const int m0 = (tile / num_n) * 2 * CM + CM * static_cast<int>(rank);
        const int c0 = (tile % num_n) * PN + CN * static_cast<int>(rank);
        for (int x = 0; x < nk * BK; x += BK) {
          if (f >= STAGES && !mbar_wait(sm.empty(s), ph ^ 1u, abort)) { ok = false; break; }
          // the leader's full barrier counts both CTAs' bytes of this stage
          if (rank == 0) mbar_arrive_expect_tx(sm.full(s), 2 * STAGE);
          const uint32_t fb = full_leader0 + 8u * static_cast<uint32_t>(s);
          tma_load_2d_pair(smem_u32(sm.a(s)), &tmap_a, x, m0, fb);
          tma_load_2d_pair(smem_u32(sm.b(s)), &tmap_w, c0, x, fb);
          tma_load_2d_pair(smem_u32(sm.b(s)) + B_GROUP, &tmap_w, c0 + 64, x, fb);
          ++f;
          if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
      }
      if (!ok) {
        fail(sm, status);
        // Loads already issued must land before the CTA exits.  Their completion is counted on the
        // leader's barriers, which the peer cannot wait on, so each CTA gives them a bounded grace
        // period instead (a tile load takes microseconds).
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2-5)
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const uint32_t empty_leader = mapa_shared(sm.tmem_empty(0), 0);
    bool ok = true;
    int nstore = 0;  // chunks stored by this warp: their staging buffers alternate
    for (int t = 0; ok && t < my_tiles; ++t) {
      const int b = t & 1;
      const int tile = tile_of(t);
      const int m0 = (tile / num_n) * 2 * CM + CM * static_cast<int>(rank);
      const int c0 = (tile % num_n) * PN;
      if (!mbar_wait_warp(sm.tmem_full(b), static_cast<uint32_t>((t >> 1) & 1), abort)) { ok = false; break; }
      tc_fence_after();
#pragma unroll 1
      for (int ch = 0; ch < PN / 64; ++ch) {
        if (c0 + ch * 64 >= K || m0 + 32 * q >= M) break;  // nothing of this chunk lies inside Y
        uint32_t r[2][32];
        const uint32_t src = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(b * ACC_COLS + ch * 64);
        tmem_ld32(src, r[0]);
        tmem_ld32(src + 32, r[1]);
        tmem_ld_wait();
        // one row of 64 bf16 a lane -> staging, 16-byte pieces in the 128-byte TMA swizzle's places
        uint8_t* stg = sm.stage(q, nstore++ & 1);
        if (lane == 0) bulk_wait_group_read<1>();  // the store that used this buffer has read it
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t* v = &r[j >> 2][8 * (j & 3)];
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) pk[e] = pack_bf16(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmap_y, c0 + ch * 64, m0 + 32 * q, smem_u32(stg));
          bulk_commit_group();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(empty_leader + 8u * b);
    }
    if (lane == 0) bulk_wait_group<0>();  // every output tile has been written
    if (!ok) fail(sm, status);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer no longer arrives on our barriers and the pair's MMAs are done
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// Pairs the device holds at once, asked once for each device (0: not asked yet).
std::atomic<int> g_max_pairs[64];

}  // namespace

int launch_gemm_bf16(const void* A, int64_t lda, const void* W, void* Y, int64_t ldy, int M, int N, int K, int* status,
                     int num_sms, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CR_ERR_CUDA;
  CUtensorMap ta, tw, ty;
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const auto l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  if (!make_tmap_2d(&ta, bf, A, M, N, static_cast<uint64_t>(lda) * 2, BK, CM, sw, l2) ||
      !make_tmap_2d(&tw, bf, W, N, K, static_cast<uint64_t>(K) * 2, 64, BK, sw, l2) ||
      !make_tmap_2d(&ty, bf, Y, M, K, static_cast<uint64_t>(ldy) * 2, 64, 32, sw, CU_TENSOR_MAP_L2_PROMOTION_NONE))
    return CR_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_ALLOC;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int most = g_max_pairs[dev].load();
  if (!most) {
    if (cudaFuncSetAttribute(gemm_bf16_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ALLOC) !=
        cudaSuccess)
      return CR_ERR_CUDA;
    cfg.gridDim = dim3(2 * (num_sms / 2), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&most, gemm_bf16_pair_kernel, &cfg) != cudaSuccess || most < 1) {
      cudaGetLastError();
      most = num_sms / 2;
    }
    g_max_pairs[dev].store(most);
  }
  const int64_t tiles = (static_cast<int64_t>(M) + 2 * CM - 1) / (2 * CM) * ((K + PN - 1) / PN);
  cfg.gridDim = dim3(2 * static_cast<unsigned>(tiles < most ? tiles : most), 1, 1);
  return cudaLaunchKernelEx(&cfg, gemm_bf16_pair_kernel, ta, tw, ty, M, N, K, status) == cudaSuccess ? CR_OK
                                                                                                     : CR_ERR_CUDA;
}

cudaError_t gemm_bf16_lost_wait(cudaStream_t stream, bool* found) { return take_lost_wait(stream, found); }

}  // namespace cr
