// ckpt_mma.cu -- 8-bit activation checkpoints: for each row and slice of 256 columns y = x H256, one float32
// scale s = max(amax|y| / 127, 2^-100) and codes c = rne(y / s); back, x^ = bf16((c s) H256).  A scale for each
// slice of each row costs 1/64 byte a value and keeps a loud token's or another slice's range out of it.
//
// Both directions move 3 bytes a value and are bound by that, but only if the rotation costs next to nothing.
// As a butterfly on the CUDA cores (shuffles and 11 two-wide operations for every two values) it took 54 us to
// save and 66 us to load 8192 x 12288, where the bytes take 46.  Here it runs on the tensor cores, as a product
// with the 256 x 256 matrix of +-1, exact in its operands and with the same float32 sums, and takes 51 and 58 us:
//
// * save: bf16 rows times bf16 +-1.  Four blocks of 64 columns come by TMA and are multiplied as they arrive:
//   H256 = H4 (x) H64, so block i contributes +-(x_i H64) to each of the four result blocks; two results at a
//   time (N = 128) need only [H64, H64], [-H64, H64] and [H64, -H64] in shared memory (48 KB).
// * load: the codes as they are, kind::i8, times int8 +-1 (64 KB): the sums are exact integers, and the scale is
//   applied once to each.
//
// Tiles of 128 rows x 256 columns, persistent CTAs, accumulators double-buffered in TMEM; a thread of the
// epilogue has half a row of a slice, so amax needs one exchange between two threads and no shuffles.  Few rows
// are a matter of starting: 130 x 2560 takes 9.9 us for both calls, each kernel setting itself up (operand of H,
// TMEM, barriers) beside the end of the one before; 16.4 without that.
//
// The code is rne(y r), r = fl(1 / s), in one fma: the reciprocal's rounding moves a code only where y / s lies
// within 2^-24 of itself from a border, less than y's own float32 sums do.

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

constexpr int TM = 128;            // rows of a tile
constexpr int TC = 256;            // columns of a tile: one slice
constexpr int kBox = TM * 128;     // 128 rows x 128 bytes
constexpr int kThreads = 320;      // warp 0 MMA, warp 1 TMA, warps 2-9 epilogue (half a row's slice a thread)
constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100: below it 1/s would leave float32's range

constexpr int kSaveStages = 6;                 // boxes of 64 columns on their way
constexpr int kSaveOffRing = 3 * kBox;         // after the three operands of H64
constexpr int kSaveOffOut = kSaveOffRing + kSaveStages * kBox;
constexpr int kSaveOffRed = kSaveOffOut + 4 * kBox;  // two boxes of codes for each half
constexpr int kSaveOffBar = kSaveOffRed + 2 * 2 * TM * 4;
constexpr int kSaveSmem = kSaveOffBar + 256;
constexpr int kLoadStages = 4;                 // boxes of 128 codes a row
constexpr int kLoadOffRing = TC * TC;          // after H256 as bytes
constexpr int kLoadOffOut = kLoadOffRing + kLoadStages * kBox;
constexpr int kLoadOffBar = kLoadOffOut + 6 * kBox;  // three boxes of values for each half
constexpr int kLoadSmem = kLoadOffBar + 256;
static_assert(kSaveSmem + 1024 <= 232448 && kLoadSmem + 1024 <= 232448, "shared memory budget");

// Signs of row n of the unnormalised Hadamard matrix over the 16 columns 16 c .. 16 c + 15, a set bit for -1: a
// column's sign turns with every base-4 digit in which it agrees with the row.
__device__ __forceinline__ uint32_t h_signs16(int n, int c, bool four_digits) {
  uint32_t m = (1u << (n & 3)) * 0x1111u ^ 0xFu << (4 * ((n >> 2) & 3));
  if (((n >> 4) & 3) == (c & 3)) m ^= 0xFFFFu;
  if (four_digits && (n >> 6) == (c >> 2)) m ^= 0xFFFFu;
  return m;
}

// The largest magnitude of three; NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

struct Bars {
  uint32_t b;
  __device__ uint32_t full(int s) const { return b + 8u * s; }
  __device__ uint32_t empty(int s) const { return b + 64u + 8u * s; }
  __device__ uint32_t acc_full(int i) const { return b + 128u + 8u * i; }
  __device__ uint32_t acc_empty(int i) const { return b + 144u + 8u * i; }
};

// Barriers, by the TMA's thread: it asks for its first boxes at once, before the rest of the block is set up.
__device__ __forceinline__ void init_bars(const Bars& bars, volatile int* abort, int stages) {
  for (int s = 0; s < stages; ++s) {
    mbar_init(bars.full(s), 1);
    mbar_init(bars.empty(s), 1);
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init(bars.acc_full(i), 1);
    mbar_init(bars.acc_empty(i), 8);
  }
  *abort = 0;
  fence_mbar_init();
  fence_proxy_async_smem();
}

// What the stream ran before, TMEM, and the block's meeting; returns the TMEM base.
__device__ __forceinline__ uint32_t start(uint8_t* misc) {
  uint32_t* slot = reinterpret_cast<uint32_t*>(misc);
  griddep_wait();
  if (threadIdx.x < 32) {
    tmem_alloc(smem_u32(slot), 512);
    tmem_relinquish();
  }
  fence_proxy_async_smem();  // the operand of H, written before this
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return *slot;
}

__device__ __forceinline__ void finish(uint32_t tmem) {
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A wait that ran out: no status word here, so the values say it (NaN scales, NaN rows); copies on their way
// land before the block ends.
__device__ __forceinline__ void gave_up(volatile int* abort) {
  record_timeout(nullptr);
  *abort = 1;
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
}

__global__ void __launch_bounds__(kThreads, 1)
    ckpt_save_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_c,
                     float* __restrict__ scales, int M, int slices) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Bars bars{smem_u32(base + kSaveOffBar)};
  uint8_t* misc = base + kSaveOffBar + 160;
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 4);
  const int64_t tiles = (static_cast<int64_t>(M) + TM - 1) / TM * slices;

  auto load = [&](int64_t t, int i, int s) {
    mbar_arrive_expect_tx(bars.full(s), kBox);
    tma_load_2d(smem_u32(base + kSaveOffRing + s * kBox), &tmap_x, static_cast<int>(t % slices) * TC + 64 * i,
                static_cast<int>(t / slices) * TM, bars.full(s));
  };
  if (warp == 1 && lane == 0) {
    init_bars(bars, abort, kSaveStages);
    griddep_wait();  // for what the stream ran before
    for (int i = 0; i < 4; ++i) load(blockIdx.x, i, i);  // (there is no block without a tile)
  }
  // [H64, H64], [-H64, H64], [H64, -H64]: 128 rows of 64 values, 16-byte pieces in the 128-byte swizzle's places
  for (int e = threadIdx.x; e < 3 * TM * 8; e += kThreads) {
    const int v = e >> 10, n = (e >> 3) & 127, piece = e & 7;
    const bool flip = (v == 1 && n < 64) || (v == 2 && n >= 64);
    const uint32_t m = (h_signs16(n & 63, piece >> 1, false) >> (8 * (piece & 1))) ^ (flip ? 0xFFu : 0u);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 0x3F803F80u | (m >> (2 * i) & 1) << 15 | (m >> (2 * i + 1) & 1) << 31;
    *reinterpret_cast<uint4*>(base + v * kBox + n * 128 + ((piece ^ (n & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const uint32_t tmem = start(misc);
  if (threadIdx.x == 0) griddep_launch_dependents();

  if (warp == 0) {
    // ---------------------------------------------------------------- MMA issuer (one thread)
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_bf16(TM, 128, false, false);
      int s = 0, b = 0;
      uint32_t ph = 0, bph = 1;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        if (!mbar_sleep(bars.acc_empty(b), bph, abort)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!mbar_sleep(bars.full(s), ph, abort)) { ok = false; break; }
          tc_fence_after();
          const uint64_t dx = sw128_kmajor_desc(smem_u32(base + kSaveOffRing + s * kBox));
#pragma unroll
          for (int jp = 0; jp < 2; ++jp) {
            // results 2 jp and 2 jp + 1 take block i with the signs of H4's row i
            const uint64_t dh = sw128_kmajor_desc(smem_u32(base + ((i >> 1) == jp ? 1 + (i & 1) : 0) * kBox));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_ss(tmem + static_cast<uint32_t>(256 * b + 128 * jp), dx + 2u * kk, dh + 2u * kk, idesc,
                          (i | kk) ? 1u : 0u);
          }
          umma_commit(bars.empty(s));
          if (++s == kSaveStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        umma_commit(bars.acc_full(b));
        b ^= 1;
        if (b == 0) bph ^= 1u;
      }
      if (!ok) gave_up(abort);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      int s = 4;  // the first tile is on its way
      uint32_t ph = 1;
      bool ok = true;
      for (int64_t t = static_cast<int64_t>(blockIdx.x) + gridDim.x; ok && t < tiles; t += gridDim.x) {
        for (int i = 0; i < 4; ++i) {
          if (s == kSaveStages) { s = 0; ph ^= 1u; }
          if (!mbar_sleep(bars.empty(s), ph, abort)) { ok = false; break; }
          load(t, i, s++);
        }
      }
      if (!ok) gave_up(abort);
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 2) >> 2, row = 32 * q + lane;
    const bool storer = (warp == 2 || warp == 6) && lane == 0;  // of this half's box of codes
    float* red = reinterpret_cast<float*>(base + kSaveOffRed);
    int b = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
      const int64_t m0 = t / slices * TM;
      const int slice = static_cast<int>(t % slices);
      if (ok) ok = mbar_sleep_warp(bars.acc_full(b), ph, abort);
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(256 * b + 128 * half);
      float top = ok ? 0.f : __uint_as_float(0x7FC00000u);
#pragma unroll 1
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t r[2][32];
        tmem_ld32(src + 64 * ch, r[0]);
        tmem_ld32(src + 64 * ch + 32, r[1]);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) top = max_abs3(top, __uint_as_float(r[0][e]), __uint_as_float(r[1][e]));
      }
      float* both = red + b * 2 * TM;  // (two buffers: the other half may be a tile behind in its reading)
      both[half * TM + row] = top;
      uint8_t* box = base + kSaveOffOut + (2 * half + b) * kBox;
      if (storer) bulk_wait_group_read<1>();  // the box's codes of two tiles ago have left
      named_bar_sync(1, 256);
      top = max_abs3(top, both[(half ^ 1) * TM + row], 0.f);
      const bool finite = top <= 3.402823466e38f;
      // the values are 16 times the rotated ones; 1/16 is exact
      const float s16 = fmaxf(__fdiv_rn(top, 127.f), 16.f * kMinScale);
      if (half == 0 && m0 + row < M)
        scales[(m0 + row) * slices + slice] = finite ? s16 * 0.0625f : __uint_as_float(0x7FC00000u);
      const float rs = __frcp_rn(s16);
      const float2 r2 = make_float2(rs, rs), magic2 = make_float2(12582912.0f, 12582912.0f);
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t r[32];
        tmem_ld32(src + 32 * ch, r);
        tmem_ld_wait();
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // the code is the low byte of the sum with 1.5 * 2^23
          const float2 lo = __ffma2_rn(make_float2(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1])), r2, magic2);
          const float2 hi = __ffma2_rn(make_float2(__uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3])), r2, magic2);
          w[e] = __byte_perm(__byte_perm(__float_as_uint(lo.x), __float_as_uint(lo.y), 0x0040),
                             __byte_perm(__float_as_uint(hi.x), __float_as_uint(hi.y), 0x0040), 0x5410);
          if (!finite) w[e] = 0;
        }
#pragma unroll
        for (int p = 0; p < 2; ++p)
          *reinterpret_cast<uint4*>(box + row * 128 + (((2 * ch + p) ^ (row & 7)) << 4)) =
              make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
      }
      tc_fence_before();
      fence_proxy_async_smem();
      named_bar_sync(2 + half, 128);
      if (lane == 0) mbar_arrive(bars.acc_empty(b));
      if (storer) {
        tma_store_2d(&tmap_c, slice * TC + 128 * half, static_cast<int32_t>(m0), smem_u32(box));
        bulk_commit_group();
      }
      b ^= 1;
      if (b == 0) ph ^= 1u;
    }
    if (storer) bulk_wait_group<0>();
  }
  finish(tmem);
}

__global__ void __launch_bounds__(kThreads, 1)
    ckpt_load_kernel(const __grid_constant__ CUtensorMap tmap_c, const __grid_constant__ CUtensorMap tmap_x,
                     const float* __restrict__ scales, int M, int slices) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Bars bars{smem_u32(base + kLoadOffBar)};
  uint8_t* misc = base + kLoadOffBar + 160;
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 4);
  const int64_t tiles = (static_cast<int64_t>(M) + TM - 1) / TM * slices;

  auto load = [&](int64_t t, int kb, int s) {
    mbar_arrive_expect_tx(bars.full(s), kBox);
    tma_load_2d(smem_u32(base + kLoadOffRing + s * kBox), &tmap_c, static_cast<int>(t % slices) * TC + 128 * kb,
                static_cast<int>(t / slices) * TM, bars.full(s));
  };
  if (warp == 1 && lane == 0) {
    init_bars(bars, abort, kLoadStages);
    griddep_wait();  // for what the stream ran before
    for (int i = 0; i < 2; ++i) load(blockIdx.x, i, i);  // (there is no block without a tile)
  }
  // H256 as bytes: for each 128 of the sum, 256 rows of 128 bytes
  for (int e = threadIdx.x; e < 2 * TC * 8; e += kThreads) {
    const int kb = e >> 11, n = (e >> 3) & 255, piece = e & 7;
    const uint32_t m = h_signs16(n, 8 * kb + piece, true);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // four bits, one to the lowest place of each byte; 1 -> 0xFF, 0 -> 0x01
      w[i] = ((m >> (4 * i) & 15u) * 0x00204081u & 0x01010101u) * 0xFEu + 0x01010101u;
    *reinterpret_cast<uint4*>(base + kb * 2 * kBox + n * 128 + ((piece ^ (n & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const uint32_t tmem = start(misc);
  if (threadIdx.x == 0) griddep_launch_dependents();

  if (warp == 0) {
    // ---------------------------------------------------------------- MMA issuer (one thread)
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_i8(TM, TC);
      int s = 0, b = 0;
      uint32_t ph = 0, bph = 1;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        if (!mbar_sleep(bars.acc_empty(b), bph, abort)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          if (!mbar_sleep(bars.full(s), ph, abort)) { ok = false; break; }
          tc_fence_after();
          const uint64_t dc = sw128_kmajor_desc(smem_u32(base + kLoadOffRing + s * kBox));
          const uint64_t dh = sw128_kmajor_desc(smem_u32(base + kb * 2 * kBox));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_i8_ss(tmem + static_cast<uint32_t>(256 * b), dc + 2u * kk, dh + 2u * kk, idesc, (kb | kk) ? 1u : 0u);
          umma_commit(bars.empty(s));
          if (++s == kLoadStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        umma_commit(bars.acc_full(b));
        b ^= 1;
        if (b == 0) bph ^= 1u;
      }
      if (!ok) gave_up(abort);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      int s = 2;  // the first tile is on its way
      uint32_t ph = 1;
      bool ok = true;
      for (int64_t t = static_cast<int64_t>(blockIdx.x) + gridDim.x; ok && t < tiles; t += gridDim.x) {
        for (int kb = 0; kb < 2; ++kb) {
          if (s == kLoadStages) { s = 0; ph ^= 1u; }
          if (!mbar_sleep(bars.empty(s), ph, abort)) { ok = false; break; }
          load(t, kb, s++);
        }
      }
      if (!ok) gave_up(abort);
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 2) >> 2, row = 32 * q + lane;
    const bool storer = (warp == 2 || warp == 6) && lane == 0;  // of this half's two boxes of values
    int b = 0, o = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
      const int64_t m0 = t / slices * TM;
      const int slice = static_cast<int>(t % slices);
      float s = m0 + row < M ? ldcg_here_f1(scales + (m0 + row) * slices + slice) * 0.0625f : 0.f;
      if (ok) ok = mbar_sleep_warp(bars.acc_full(b), ph, abort);
      if (!ok) s = __uint_as_float(0x7FC00000u);
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(256 * b + 128 * half);
      const float2 s2 = make_float2(s, s), magic2 = make_float2(-12582912.0f, -12582912.0f);
#pragma unroll 1
      for (int bx = 0; bx < 2; ++bx) {  // 64 columns, one of the half's three boxes in turn
        uint8_t* box = base + kLoadOffOut + (3 * half + o) * kBox;
        uint32_t r[2][32];
        tmem_ld32(src + 64 * bx, r[0]);
        tmem_ld32(src + 64 * bx + 32, r[1]);
        tmem_ld_wait();
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // integers up to 2^15: added to the bits of 1.5 * 2^23 they read as that plus themselves
            const uint32_t* v = &r[p >> 2][8 * (p & 3) + 2 * e];
            const float2 f = __fadd2_rn(
                make_float2(__uint_as_float(v[0] + 0x4B400000u), __uint_as_float(v[1] + 0x4B400000u)), magic2);
            const float2 x = __fmul2_rn(f, s2);
            w[e] = pack_bf16(x.x, x.y);
          }
          *reinterpret_cast<uint4*>(box + row * 128 + ((p ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        if (bx == 1) tc_fence_before();
        if (storer) bulk_wait_group_read<1>();  // the next box's values of three boxes ago have left
        named_bar_sync(2 + half, 128);
        if (storer) {
          tma_store_2d(&tmap_x, slice * TC + 128 * half + 64 * bx, static_cast<int32_t>(m0), smem_u32(box));
          bulk_commit_group();
        }
        if (++o == 3) o = 0;
      }
      if (lane == 0) mbar_arrive(bars.acc_empty(b));
      b ^= 1;
      if (b == 0) ph ^= 1u;
    }
    if (storer) bulk_wait_group<0>();
  }
  finish(tmem);
}

std::atomic<bool> g_attr_done[64];

bool set_attrs() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (g_attr_done[dev].load()) return true;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (cudaFuncSetAttribute(ckpt_save_kernel, attr, kSaveSmem + 1024) != cudaSuccess ||
      cudaFuncSetAttribute(ckpt_load_kernel, attr, kLoadSmem + 1024) != cudaSuccess)
    return false;
  g_attr_done[dev].store(true);
  return true;
}

unsigned blocks(int M, int K, int num_sms) {
  const int64_t tiles = (static_cast<int64_t>(M) + TM - 1) / TM * (K / TC);
  return static_cast<unsigned>(tiles < num_sms ? tiles : num_sms);
}

// A launch as a programmatic dependent of what the stream ran before: the block sets itself up beside its end.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  Launch(unsigned grid, int smem, cudaStream_t stream) {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem + 1024;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
};

bool codes_map(CUtensorMap* map, const void* codes, int M, int K) {
  return make_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, M, K, K, 128, TM, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
bool values_map(CUtensorMap* map, const void* X, int M, int K, int64_t ldx) {
  return make_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, M, K, static_cast<uint64_t>(ldx) * 2, 64, TM,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

}  // namespace

int launch_ckpt_save(const uint16_t* X, int M, int K, int64_t ldx, int8_t* codes, float* scales, int num_sms,
                     cudaStream_t stream) {
  CUtensorMap tx, tc;
  if (!set_attrs() || !values_map(&tx, X, M, K, ldx) || !codes_map(&tc, codes, M, K)) return CR_ERR_CUDA;
  Launch l(blocks(M, K, num_sms), kSaveSmem, stream);
  return cudaLaunchKernelEx(&l.cfg, ckpt_save_kernel, tx, tc, scales, M, K / TC) == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

int launch_ckpt_load(const int8_t* codes, const float* scales, int M, int K, uint16_t* X, int64_t ldx, int num_sms,
                     cudaStream_t stream) {
  CUtensorMap tx, tc;
  if (!set_attrs() || !values_map(&tx, X, M, K, ldx) || !codes_map(&tc, codes, M, K)) return CR_ERR_CUDA;
  Launch l(blocks(M, K, num_sms), kLoadSmem, stream);
  return cudaLaunchKernelEx(&l.cfg, ckpt_load_kernel, tc, tx, scales, M, K / TC) == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

cudaError_t ckpt_lost_wait(cudaStream_t stream, bool* found) { return take_lost_wait(stream, found); }

}  // namespace cr
