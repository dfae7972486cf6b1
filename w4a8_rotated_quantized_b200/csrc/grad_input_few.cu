// grad_input_few.cu -- the W4A4 layer's input gradient for few tokens, straight from the packed weights:
//
//   P[m, k] = sum_n (s_w[n] dY[m, n]) q[n, k],   dX[m, :] = bf16( P[m, :] H_group )
//
// The rotation is linear, so it can run on the M rows of the result instead of the N rows of the weights; for
// few tokens that leaves the packed weights, half a byte each, as all that has to be read.  (Unpacking them to
// bf16 first writes and reads four times their bytes: 36 us of GPU time for 130 tokens, 9728 x 2560.)
//
// * A CTA takes 256 columns of the weights, up to 256 tokens and a part of the sum over n, 64 rows of the weights
//   at a time: the packed codes arrive by TMA, become bf16 (exact) and are the product's M side as they lie
//   (MN-major); s_w dY, rounded to bf16, is its N side.  Two sets of eight warps prepare alternate tiles of codes.
// * s_w dY is made once, by a small kernel before: made in each CTA it cost as much as the codes (128 tokens,
//   9728 x 2560: 23 us against 15).  This one starts beside it and waits for it before the first N side's load.
// * float32 sums in TMEM; the parts of the sum go to the workspace and a third kernel adds them in order,
//   rotates and rounds once.  (Joined by a cluster through distributed shared memory instead, without the third
//   kernel, 130 tokens of 9728 x 2560 took 31 us instead of 24: few clusters fit, and the sums' way is no shorter.)
//
// What bounds it: not the packed weights' bytes (of 24 us for 130 tokens of 9728 x 2560 their 12.5 MB are two) and not
// the codes' way through the ALUs (13 instructions for 8: 1.3 million of a warp's, 1.4 us over 114 SMs), but waiting.
// Token blocks of more than 128 rows leave room for two tiles of codes, 16 KB, on their way to an SM, one for each set
// of warps; with few tiles a CTA, setting up and the parts' way to the third kernel come on top.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "cr_device.cuh"
#include "cr_internal.h"
#include "f16_device.cuh"
#include "grid_sync.cuh"
#include "lora_device.cuh"
#include "lost_wait.cuh"

namespace cr {
namespace {

#include "act_device.cuh"
#include "unit_device.cuh"

constexpr int GN = 64;             // weight rows of a tile
constexpr int GC = 256;            // columns of a CTA
constexpr int kBox = GN * 128;     // 64 rows x 64 bf16 columns
constexpr int kZTile = 4 * kBox;
constexpr int kRawTile = GN * GC / 2;
constexpr int kSet = 8;            // warps of a set
constexpr int kWarps = 2 * kSet;
constexpr int kThreads = 32 * (kWarps + 3);  // then the MMA's warp and those that load the codes and the N side
constexpr int kMostTokens = 256;   // of a block
constexpr int kSmemMax = 232448 - 1024;

struct Plan {
  int blocks, rp, raws, stage, stages, off_raw, off_bar, smem, cols;  // rp: rows of a token block
};
inline __host__ __device__ Plan plan(int M) {
  Plan p;
  p.blocks = (M + kMostTokens - 1) / kMostTokens;
  p.rp = ((M + p.blocks - 1) / p.blocks + 15) & ~15;
  p.stage = kZTile + p.rp * 128;
  // an even number of raw tiles, so that each set of warps meets its slots round by round
  p.raws = p.stage <= 48 * 1024 ? 4 : 2;
  p.stages = (kSmemMax - 256 - p.raws * kRawTile) / p.stage;
  if (p.stages > 4) p.stages = 4;
  p.off_raw = p.stages * p.stage;
  p.off_bar = p.off_raw + p.raws * kRawTile;
  p.smem = p.off_bar + 256;
  const int c = 2 * p.rp;  // two halves of the columns
  p.cols = c <= 32 ? 32 : c <= 64 ? 64 : c <= 128 ? 128 : c <= 256 ? 256 : 512;
  return p;
}

// Eight nibbles -> bf16, exactly: biased by 8 they are put into the mantissa of 128, less 136.
__device__ __forceinline__ uint4 nibbles_to_bf16(uint32_t w) {
  const uint32_t v = w >> 4;
  const __nv_bfloat162 m = __floats2bfloat162_rn(136.f, 136.f);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = (__byte_perm(w, v, 0x4400 + 0x1111 * i) & 0x000F000Fu) ^ 0x43084308u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t), m);
    o[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A producer whose wait ran out: copies on their way land before the block ends.
__device__ __forceinline__ void give_up(volatile int* abort, int* status) {
  record_timeout(status);
  *abort = 1;
  const uint64_t t = globaltimer_ns();
  while (globaltimer_ns() - t < 1000000ull) __nanosleep(1000);
}

// The N side: bf16(s_w dY), rows of zeros behind the last token.  Rounding it once is off by at most 2^-8 of each
// term, what the GEMM's form pays for bf16 weights (here those are exact); with the rests as a second part of the
// sum 130 tokens of 9728 x 2560 took 27 us instead of 24.
__global__ void __launch_bounds__(256)
    grad_input_operand_kernel(const uint16_t* __restrict__ dY, int64_t lddy, const float* __restrict__ w_scale,
                              uint16_t* __restrict__ V, int M, int N, int* __restrict__ status) {
  griddep_wait();  // for what the stream ran before
  griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = CR_OK;
  const int n = (blockIdx.x * 256 + threadIdx.x) * 8, m = blockIdx.y;
  if (n >= N) return;
  float v[8] = {};
  if (m < M) {
    widen8(ldcg_here_u4(dY + m * lddy + n), v);
    float s[8];
    if ((reinterpret_cast<uintptr_t>(w_scale) & 15) == 0) {  // (one sector for each thread instead of eight loads)
      const float4 s0 = ldcg_here_f4(w_scale + n), s1 = ldcg_here_f4(w_scale + n + 4);
      s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
      s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = ldcg_here_f1(w_scale + n + e);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= s[e];
  }
  *reinterpret_cast<uint4*>(V + static_cast<int64_t>(m) * N + n) = narrow8(v);
}

__global__ void __launch_bounds__(kThreads, 1)
    grad_input_few_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_v,
                          float* __restrict__ P, int M, int N, int K, int splits, int* __restrict__ status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Plan p = plan(M);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int colblocks = K / GC;
  const int c0 = (blockIdx.x % colblocks) * GC;
  const int block = blockIdx.x / colblocks % p.blocks;
  const int split = blockIdx.x / colblocks / p.blocks;
  const int m0 = block * p.rp;
  const int tiles = (N + GN - 1) / GN;
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / splits);
  const int nt = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / splits) - t0;
  const uint32_t bars = smem_u32(base + p.off_bar);
  auto raw_full = [&](int s) { return bars + 8u * s; };
  auto raw_empty = [&](int s) { return bars + 32u + 8u * s; };
  auto ready = [&](int s) { return bars + 64u + 8u * s; };
  auto empty = [&](int s) { return bars + 96u + 8u * s; };
  auto v_full = [&](int s) { return bars + 128u + 8u * s; };
  const uint32_t acc_full = bars + 160u;
  uint32_t* slot = reinterpret_cast<uint32_t*>(base + p.off_bar + 168);
  volatile int* abort = reinterpret_cast<volatile int*>(base + p.off_bar + 172);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), kSet);
      mbar_init(ready(s), kSet);
      mbar_init(empty(s), 1);
      mbar_init(v_full(s), 1);
    }
    mbar_init(acc_full, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarps + 1 && lane == 0) {
    prefetch_tmap(&tmap_w);
    prefetch_tmap(&tmap_v);
  }
  if (warp == kWarps) {
    tmem_alloc(smem_u32(slot), p.cols);
    tmem_relinquish();
    if (lane == 0) griddep_launch_dependents();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- MMA issuer (one thread)
    if (elect_one()) {
      bool ok = true;
      uint32_t ph = 0, last_bar = 0, last_ph = 0;
      int s = 0, i = 0;
      const uint32_t idesc = idesc_bf16(128, p.rp, true, false);
      for (; i < nt; ++i) {
        if (!mbar_sleep(v_full(s), ph, abort) || !mbar_sleep(ready(s), ph, abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t z = smem_u32(base + s * p.stage);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint64_t dz = sw128_mnmajor_desc(z + half * 2 * kBox, kBox);
          const uint64_t dv = sw128_kmajor_desc(z + kZTile);
#pragma unroll
          for (int kk = 0; kk < GN / 16; ++kk)
            umma_f16_ss(tmem + static_cast<uint32_t>(half * p.rp), dz + 128u * kk, dv + 2u * kk, idesc,
                        (i || kk) ? 1u : 0u);
        }
        umma_commit(empty(s));
        last_bar = empty(s);
        last_ph = ph;
        if (++s == p.stages) { s = 0; ph ^= 1u; }
      }
      if (ok) umma_commit(acc_full);
      if (!ok) {
        record_timeout(status);
        *abort = 1;
        volatile int never = 0;
        if (i > 0) mbar_sleep(last_bar, last_ph, &never);
      }
    }
  } else if (warp == kWarps + 1) {
    // ---------------------------------------------------------------- TMA: packed codes
    if (lane == 0) {
      bool ok = true;
      int s = 0;
      uint32_t ph = 1;
      for (int i = 0; i < nt; ++i) {
        if (!mbar_sleep(raw_empty(s), ph, abort)) { ok = false; break; }
        mbar_arrive_expect_tx(raw_full(s), kRawTile);
        tma_load_2d(smem_u32(base + p.off_raw + s * kRawTile), &tmap_w, c0 / 2, (t0 + i) * GN, raw_full(s));
        if (++s == p.raws) { s = 0; ph ^= 1u; }
      }
      if (!ok) give_up(abort, status);
    }
  } else if (warp == kWarps + 2) {
    // ---------------------------------------------------------------- TMA: N side, once it has been made
    if (lane == 0) {
      griddep_wait();
      bool ok = true;
      int s = 0;
      uint32_t ph = 1;
      for (int i = 0; i < nt; ++i) {
        if (!mbar_sleep(empty(s), ph, abort)) { ok = false; break; }
        mbar_arrive_expect_tx(v_full(s), p.rp * 128);
        tma_load_2d(smem_u32(base + s * p.stage + kZTile), &tmap_v, (t0 + i) * GN, m0, v_full(s));
        if (++s == p.stages) { s = 0; ph ^= 1u; }
      }
      if (!ok) give_up(abort, status);
    }
  } else {
    // ---------------------------------------------------------------- operands
    const int set = warp / kSet, sw = warp % kSet;
    bool ok = true;
    int s = set, rs = set;
    uint32_t ph = 1, rph = 0;
    for (int i = set; i < nt; i += 2) {
      uint8_t* z = base + s * p.stage;
      if (!mbar_sleep_warp(empty(s), ph, abort)) { ok = false; break; }
      if (!mbar_sleep_warp(raw_full(rs), rph, abort)) { ok = false; break; }
      const uint8_t* raw = base + p.off_raw + rs * kRawTile;
#pragma unroll
      for (int k = 0; k < GN / kSet; ++k) {  // a row of the tile for each warp
        const int r = kSet * k + sw;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(raw + r * (GC / 2) + 4 * lane);
        *reinterpret_cast<uint4*>(z + (lane >> 3) * kBox + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) = nibbles_to_bf16(w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ready(s));
        mbar_arrive(raw_empty(rs));
      }
      if ((s += 2) >= p.stages) { s -= p.stages; ph ^= 1u; }
      if ((rs += 2) >= p.raws) { rs -= p.raws; rph ^= 1u; }
    }
    // ---------------------------------------------------------------- epilogue: column 128 half + 32 q + lane
    const int q = warp & 3, half = (warp >> 2) & 1, part = warp >> 3;  // every other 16 tokens
    const int c = c0 + 128 * half + 32 * q + lane;
    float* out = P + (static_cast<int64_t>(split) * M + m0) * K + c;
    if (ok && nt > 0) ok = mbar_sleep_warp(acc_full, 0, abort);
    if (ok) {
      tc_fence_after();
#pragma unroll 1
      for (int j = 16 * part; j < p.rp; j += 32) {
        uint32_t r[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(half * p.rp + j), r);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (m0 + j + e < M) out[static_cast<int64_t>(j + e) * K] = __uint_as_float(r[e]);
      }
    } else {
      record_timeout(status);
      *abort = 1;
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, p.cols);
  }
}

// The parts of the sum joined, rotated (values and lane mapping of act_device.cuh: 4 lanes for each 256 values, 8
// slices a block) and rounded.
template <int kDig>
__global__ void __launch_bounds__(32 * kJoinWarps)
    grad_input_finish_kernel(const float* __restrict__ P, int parts, int64_t stride, uint16_t* __restrict__ dX,
                             int64_t lddx, int64_t units, int upr) {
  griddep_wait();  // launched as a dependent of the product's kernel
  __shared__ JoinSums sums;
  const int lane = threadIdx.x & 31, k0 = lane >> 2, l = lane & 3;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + k0;
  const bool in = u < units;
  float4 v[16];
  auto at = [&](int k) { return 32 * ((k >> 1) ^ k0) + 8 * l + 4 * (k & 1); };
  if (!join_parts(P + u * 256, parts, stride, in, at, sums, v)) return;
  Pairs V;
#pragma unroll
  for (int k = 0; k < 16; ++k) put4(V, k, v[k]);
  fwht256_mapped<kDig>(V);
  if (in)
    store_unit_bf16(V, k0, 1.f / static_cast<float>(1 << kDig), dX + u / upr * lddx + (u % upr) * 256);
}

std::atomic<bool> g_attr_done[64];

bool set_attrs() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (g_attr_done[dev].load()) return true;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (cudaFuncSetAttribute(grad_input_few_kernel, attr, kSmemMax + 1024) != cudaSuccess) return false;
  g_attr_done[dev].store(true);
  return true;
}

}  // namespace

// Unpacking the weights for the bf16 GEMM costs by their number, this form by the tokens for each of them.  Fitted
// to both forms' times for 310 calls of 1 to 1600 tokens and 128 to 12288 rows and columns: the choice costs 1.2 %
// over the faster form on average and 59 % at worst (us, this form first):
//   112 tokens, 7936 x 11200 (K x N): 40 | 118        238 tokens, 5376 x 520:  21 | 12
//   308 tokens, 4608 x 6368:          41 | 58         435 tokens, 7680 x 4416: 52 | 52
//   621 tokens, 768 x 7888:           33 | 52 (the worst choice)
bool use_grad_input_few(int M, int N, int K) { return M <= 600 && static_cast<int64_t>(N) * K > 100000 + 34000LL * M; }

int grad_input_few_splits(int M, int N, int K, int num_sms) {
  const int tiles = (N + GN - 1) / GN;
  const int ctas = K / GC * plan(M).blocks;
  // rounds of CTAs, each with its tiles and about six tiles' worth of setting up and writing out
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int s = 1; s <= 16 && s <= (tiles + 1) / 2; ++s) {
    const int64_t cost = static_cast<int64_t>((ctas * s + num_sms - 1) / num_sms) * ((tiles + s - 1) / s + 6);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

size_t grad_input_few_operand_rows(int M) {
  const Plan p = plan(M);
  return static_cast<size_t>(p.blocks) * p.rp;
}

int launch_grad_input_few(const uint16_t* dY, int64_t lddy, const uint8_t* Wq, const float* w_scale, uint16_t* V,
                          float* P, uint16_t* dX, int64_t lddx, int M, int N, int K, int group, int splits, int* status,
                          cudaStream_t stream) {
  const Plan p = plan(M);
  CUtensorMap tw, tv;
  if (!set_attrs() ||
      !make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, Wq, N, K / 2, K / 2, GC / 2, GN, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !make_tmap_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, V, grad_input_few_operand_rows(M), N,
                    static_cast<uint64_t>(N) * 2, 64, p.rp, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return CR_ERR_CUDA;
  const dim3 ogrid((N / 8 + 255) / 256, p.blocks * p.rp);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = ogrid;
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, grad_input_operand_kernel, dY, lddy, w_scale, V, M, N, status) != cudaSuccess)
    return CR_ERR_CUDA;
  cfg.gridDim = dim3(static_cast<unsigned>(K / GC * p.blocks * splits), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = p.smem + 1024;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, grad_input_few_kernel, tw, tv, P, M, N, K, splits, status) != cudaSuccess)
    return CR_ERR_CUDA;
  const int64_t units = static_cast<int64_t>(M) * (K / 256), stride = static_cast<int64_t>(M) * K;
  const unsigned blocks = static_cast<unsigned>((units + 7) / 8);
  auto fin = group == 16   ? grad_input_finish_kernel<2>
             : group == 64 ? grad_input_finish_kernel<3>
             : group == 256 ? grad_input_finish_kernel<4>
                            : grad_input_finish_kernel<5>;
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(32 * kJoinWarps, 1, 1);
  cfg.dynamicSmemBytes = 0;
  const float* sums = P;
  return cudaLaunchKernelEx(&cfg, fin, sums, splits, stride, dX, lddx, units, K / 256) == cudaSuccess ? CR_OK
                                                                                                      : CR_ERR_CUDA;
}

cudaError_t grad_input_few_lost_wait(cudaStream_t stream, bool* found) { return take_lost_wait(stream, found); }

}  // namespace cr
