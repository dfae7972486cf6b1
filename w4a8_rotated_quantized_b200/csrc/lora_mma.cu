// lora_mma.cu -- low-rank adapters beside a projection on the tensor cores (tcgen05 kind::f16, float32
// accumulators in TMEM): the three products of forward and backward, for batches of tokens.
//
//   v:    V[m, j]    = sum_k X[m, k] A[a][j, k]                      (also dV from dY and U)
//   y:    Y[m, n]    = base[m, n] + s[a] sum_j V[m, j] U[a][j, n]    (also dX from dV and A)
//   grad: G[a][j, c] = s[a] sum_{m of a} V[m, j] Z[m, c]             (d_up from dY; d_down from X or its codes)
//
// With ranks up to 128 each product does 2 r flops for every activation value it moves, so all three are
// bound by memory; the tensor cores keep the arithmetic out of the way, and the tiles are laid out so that
// every activation is read once, by TMA, with the next tiles already on their way.
//
// Rows name their adapters in any order.  A tile of tokens takes the list of the adapters that occur in it:
// v multiplies by all of them at once (up to 256 rank rows side by side) and keeps each row's own columns;
// y runs one short product for each and writes only the rows that named it; grad takes the tiles in which
// its adapter occurs and clears the other rows in both operands.  No row's or adapter's values can reach
// another's result that way, non-finite ones included.
//
// V stays float32 between the products.  As an operand it is split into two bf16 values (the rounded value
// and the rounded rest: 16 bits of mantissa), so the one rounding that counts is the output's own.
//
// Every wait is bounded; on expiry a CTA records CR_ERR_TIMEOUT in the device status word and winds down.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

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

constexpr int TM = 128;             // tokens of a v or y tile
constexpr int KB = 64;              // bf16 values of a 128-byte swizzle row
constexpr int kSmemMax = 232448 - 1024;  // the base is aligned up to 1024
constexpr int kBarBytes = 256;      // mbarriers and the TMEM slot
constexpr int kListBytes = 2 * TM * 4;   // a tile's row adapters and the list of distinct ones

inline __host__ __device__ int round16(int r) { return (r + 15) & ~15; }
inline __host__ __device__ int tmem_cols_for(int c) { return c <= 32 ? 32 : c <= 64 ? 64 : c <= 128 ? 128 : c <= 256 ? 256 : 512; }

__device__ __forceinline__ uint8_t* align_smem(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ void fail(volatile int* abort, int* status) {
  record_timeout(status);
  *abort = 1;
}

// TMA loads of this CTA that nobody waits for any more must land before it exits.
__device__ __forceinline__ void grace() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
}

// The adapters of the tile's 128 rows into ids[] (-1: none, rows past M too) and the distinct ones, in order
// of first appearance, into list[]; returns how many.  Warps 2-5 do it, a thread for each row; `threads`
// threads call it (these and others) and meet at barrier 3.
__device__ __forceinline__ int tile_adapters(const int32_t* __restrict__ adapter, int64_t m0, int M, int L, int* ids,
                                             int* list, int* counts, int threads) {
  const int t = static_cast<int>(threadIdx.x) - 64, warp = t >> 5, lane = t & 31;
  const bool mine = t >= 0 && t < TM;
  if (mine) ids[t] = m0 + t < M ? row_adapter(adapter, m0 + t, L) : -1;
  if (!adapter) {
    if (t == 0) list[0] = 0;
    named_bar_sync(3, threads);
    return 1;
  }
  named_bar_sync(3, threads);
  bool first = false;
  uint32_t firsts = 0;
  if (mine) {
    const int a = ids[t];
    const uint32_t same = __match_any_sync(0xffffffffu, a);
    first = a >= 0 && __ffs(same) - 1 == lane;
    // against the rows of the warps before, four at a time
#pragma unroll 4
    for (int i = 0; i < 32 * warp; i += 4) {
      const int4 o = *reinterpret_cast<const int4*>(ids + i);
      first = first && o.x != a && o.y != a && o.z != a && o.w != a;
    }
    firsts = __ballot_sync(0xffffffffu, first);
    if (lane == 0) counts[warp] = __popc(firsts);
  }
  named_bar_sync(3, threads);
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < TM / 32; ++w) {
    before += w < warp ? counts[w] : 0;
    all += counts[w];
  }
  if (first) list[before + __popc(firsts & ((1u << lane) - 1))] = ids[t];
  named_bar_sync(3, threads);
  return all;
}

// ---------------------------------------------------------------------------------------------------
// v: 128 tokens x (up to 256 / rank adapters side by side); the sum over k split over a cluster's CTAs,
// whose partial sums go to the CTA that adds up their row, in rank order, through distributed shared memory.
// By itself it takes 12 to 13 us for 4096 x 3072 at rank 64 and 15 to 16 us for 8192 x 3072 at rank 32 (2.0 and 3.3
// TB/s): X comes in about 5 and 9 of them, the rest is starting and the exchange.  Of the kernels after it little runs
// beside it: with rings that fill an SM's shared memory, here and in y, a CTA of y starts where one of v has ended or
// none ran.  (As one kernel with y, V passed round a cluster, the two took 28.4 us where the two kernels of that time
// took 26.6 for 4096 tokens, and 20.5 against 15.5 for 130.)
// ---------------------------------------------------------------------------------------------------

struct VPlan {
  int rp, cap, ring, part_ld, off_part, off_list, off_bar, smem, cols;
};
constexpr int kVStages = 8;  // at most
inline __host__ __device__ VPlan v_plan(int rank, int L) {
  VPlan p;
  p.rp = round16(rank);
  p.cap = 256 / p.rp;
  if (p.cap > L) p.cap = L;
  p.part_ld = p.rp + 4;  // rows 4 banks apart: eight rows' 16-byte pieces lie side by side
  const int part = TM * p.part_ld * 4;
  // the ring takes what is left, up to eight of the largest stages; a tile with few adapters cuts it into
  // more and smaller ones
  const int stage = TM * 128 + p.cap * p.rp * 128;
  int room = (kSmemMax - part - kListBytes - kBarBytes) & ~1023;
  p.ring = room < kVStages * stage ? room : kVStages * stage;
  p.off_part = p.ring;
  p.off_list = p.off_part + part;
  p.off_bar = p.off_list + kListBytes;
  p.smem = p.off_bar + kBarBytes;
  p.cols = tmem_cols_for(p.cap * p.rp + 16);  // the epilogue reads 32 columns at a time
  return p;
}

constexpr int kVMostSplits = 16;  // CTAs of a cluster (over 8: asked for as not portable)
constexpr int kVThreads = 192;  // warp 0 MMA, warp 1 TMA, warps 2-5 epilogue

__global__ void __launch_bounds__(kVThreads, 1)
    lora_v_mma_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_a,
                      const int32_t* __restrict__ adapter, float* __restrict__ V, uint16_t* __restrict__ Vout, int M,
                      int K, int rank, int L, int splits, int* __restrict__ status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = align_smem(smem_raw);
  const VPlan p = v_plan(rank, L);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = static_cast<int>(cluster_ctarank());
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / splits) * TM;
  float* part = reinterpret_cast<float*>(base + p.off_part);
  int* ids = reinterpret_cast<int*>(base + p.off_list);
  int* list = ids + TM;
  auto full = [&](int s) { return smem_u32(base + p.off_bar) + 8u * s; };
  auto empty = [&](int s) { return smem_u32(base + p.off_bar) + 64u + 8u * s; };
  const uint32_t acc_full = smem_u32(base + p.off_bar) + 128u, acc_empty = acc_full + 8u;
  uint32_t* slot = reinterpret_cast<uint32_t*>(base + p.off_bar + 144);
  volatile int* abort = reinterpret_cast<volatile int*>(base + p.off_bar + 148);
  int* counts = reinterpret_cast<int*>(base + p.off_bar + 160);

  const int nkb = (K + KB - 1) / KB;
  const int kb0 = static_cast<int>(static_cast<int64_t>(nkb) * split / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(nkb) * (split + 1) / splits);
  // `c` adapters' rows of A beside the block of X
  auto load = [&](int stage, int s, int kb, const int* which, int c) {
    const uint32_t dst = smem_u32(base + s * stage);
    mbar_arrive_expect_tx(full(s), static_cast<uint32_t>(TM + c * p.rp) * 128u);
    tma_load_2d(dst, &tmap_x, kb * KB, static_cast<int32_t>(m0), full(s));
    for (int i = 0; i < c; ++i)
      tma_load_3d(dst + TM * 128 + i * p.rp * 128, &tmap_a, kb * KB, 0, which ? which[i] : 0, full(s));
  };

  cluster_arrive();  // this CTA has started: its shared memory may be written to
  int asked = 0;     // loads on their way before the block is set up
  if (warp == 1 && lane == 0) {
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 4);
    *abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    griddep_wait();
    if (!adapter) {  // nothing to look up first
      const int stage = (TM + p.rp) * 128;
      const int stages = p.ring / stage < kVStages ? p.ring / stage : kVStages;
      for (; asked < stages && kb0 + asked < kb1; ++asked) load(stage, asked, kb0 + asked, nullptr, 1);
    } else {
      prefetch_tmap(&tmap_x);
      prefetch_tmap(&tmap_a);
    }
  }
  griddep_wait();  // for what the stream ran before
  if (warp == 0) {
    tmem_alloc(smem_u32(slot), p.cols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    griddep_launch_dependents();  // the y kernel may set itself up beside this one
    if (blockIdx.x == 0) *status = CR_OK;
  }
  const int nd = tile_adapters(adapter, m0, M, L, ids, list, counts, kVThreads);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_wait();
  const uint32_t tmem = *slot;

  const int stage = (TM + (nd < p.cap ? nd : p.cap) * p.rp) * 128;
  const int stages = p.ring / stage < kVStages ? p.ring / stage : kVStages;
  const int rows = TM / splits;  // that this CTA adds up

  if (warp == 0) {
    // ---------------------------------------------------------------- MMA issuer (one thread)
    if (elect_one()) {
      bool ok = true, committed = false;
      uint32_t ph = 0, last_bar = 0, last_ph = 0;
      int s = 0, pass = 0;
      for (int d0 = 0; ok && d0 < nd; d0 += p.cap, ++pass) {
        const int c = nd - d0 < p.cap ? nd - d0 : p.cap;
        const uint32_t idesc = idesc_bf16(TM, c * p.rp, false, false);
        if (pass && !mbar_sleep(acc_empty, (pass - 1) & 1, abort)) { ok = false; break; }
        tc_fence_after();
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_sleep(full(s), ph, abort)) { ok = false; break; }
          tc_fence_after();
          const uint64_t da = sw128_kmajor_desc(smem_u32(base + s * stage));
          const uint64_t db = sw128_kmajor_desc(smem_u32(base + s * stage + TM * 128));
#pragma unroll
          for (int kk = 0; kk < KB / 16; ++kk)
            umma_f16_ss(tmem, da + 2u * kk, db + 2u * kk, idesc, (kb != kb0 || kk) ? 1u : 0u);
          umma_commit(empty(s));
          last_bar = empty(s);
          last_ph = ph;
          committed = true;
          if (++s == stages) { s = 0; ph ^= 1u; }
        }
        if (ok) umma_commit(acc_full);
      }
      if (!ok) {
        fail(abort, status);
        volatile int never = 0;
        if (committed) mbar_sleep(last_bar, last_ph, &never);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      bool ok = true;
      int s = 0, f = 0;
      uint32_t ph = 0;
      for (int d0 = 0; ok && d0 < nd; d0 += p.cap) {
        const int c = nd - d0 < p.cap ? nd - d0 : p.cap;
        for (int kb = kb0; kb < kb1; ++kb, ++f) {
          if (f >= stages && !mbar_sleep(empty(s), ph ^ 1u, abort)) { ok = false; break; }
          if (f >= asked) load(stage, s, kb, list + d0, c);
          if (++s == stages) { s = 0; ph ^= 1u; }
        }
      }
      if (!ok) {
        fail(abort, status);
        grace();
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue: own columns of each row
    const int q = warp & 3;
    const int row = 32 * q + lane;
    const int mine = ids[row];
    // this split's place for the row, in the CTA that adds up the row
    const uint32_t out = mapa_shared(smem_u32(part) + 4u * ((split * rows + row % rows) * p.part_ld), row / rows);
    if (mine < 0)
      for (int j = 0; j < p.rp; j += 4) st_shared_cluster_f4(out + 4u * j, 0.f, 0.f, 0.f, 0.f);
    bool ok = true;
    int pass = 0;
    for (int d0 = 0; ok && d0 < nd; d0 += p.cap, ++pass) {
      const int c = nd - d0 < p.cap ? nd - d0 : p.cap;
      if (!mbar_sleep_warp(acc_full, pass & 1, abort)) { ok = false; break; }
      tc_fence_after();
      for (int i = 0; i < c; ++i) {
        const bool hit = mine == list[d0 + i];
        if (!__any_sync(0xffffffffu, hit)) continue;
#pragma unroll 1
        for (int j = 0; j < p.rp; j += 32) {
          uint32_t r[32];  // (past the last 16 ranks: columns that nobody keeps)
          tmem_ld32(tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(i * p.rp + j), r);
          tmem_ld_wait();
          if (hit) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if (e < 16 || j + 16 < p.rp)
                st_shared_cluster_f4(out + 4u * (j + e), __uint_as_float(r[e]), __uint_as_float(r[e + 1]),
                                     __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
    }
    if (!ok) fail(abort, status);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every split's partial sums have arrived
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, p.cols);
  }
  // this CTA's rows: the splits' sums added in order
  const int groups = rank >> 2;
  const int mine = M - m0 - split * rows < rows ? static_cast<int>(M - m0 - split * rows) : rows;  // up to the last row
#pragma unroll 4
  for (int i = threadIdx.x; i < mine * groups; i += kVThreads) {
    const int r = i / groups, j = 4 * (i - r * groups);
    const int64_t m = m0 + split * rows + r;
    const float* src = part + r * p.part_ld + j;
    float4 t = *reinterpret_cast<const float4*>(src);
    for (int c = 1; c < splits; ++c) {
      const float4 u = *reinterpret_cast<const float4*>(src + c * rows * p.part_ld);
      t.x += u.x;
      t.y += u.y;
      t.z += u.z;
      t.w += u.w;
    }
    *reinterpret_cast<float4*>(V + m * rank + j) = t;
    if (Vout) *reinterpret_cast<uint2*>(Vout + m * rank + j) = make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
  }
}

// ---------------------------------------------------------------------------------------------------
// y: 128 tokens x 128 columns a tile.  The tile's base arrives by TMA in the buffer that its result leaves
// from.  V of the 128 rows, scaled and split into bf16 pairs, stays in TMEM as the product's A operand for
// all column tiles: read from shared memory it would cost as many bytes there as U does, and at rank 128
// those bytes, not memory's, set the pace (134 us against 110 us for 8192 x 12288).
// Column tiles are dealt out over the CTAs token tile by token tile; where that does not come out even a CTA goes on
// to the next token tile, with that one's V.
// By itself the kernel takes 72 us for 8192 -> 12288 at rank 32 (402 MB of base and result: 5.6 TB/s); at rank 128
// with four adapters memory waits for the products of the tiles that hold two adapters' rows (97 us: 4.1 TB/s).
// ---------------------------------------------------------------------------------------------------

constexpr int TN = 128;
constexpr int kYTile = TM * TN * 2;  // 32 KB: two boxes of 64 columns x 128 rows
constexpr int kAcc = 3;              // accumulators
constexpr int kVCol = kAcc * TN;     // TMEM: the accumulators, then V's rounded values, then the rests
struct YPlan {
  int rp, nb, nu, u, off_y, off_list, off_bar, smem;
};
inline __host__ __device__ YPlan y_plan(int rank) {
  YPlan p;
  p.rp = round16(rank);
  p.u = p.rp * 256;  // two boxes of 64 columns x rank rows
  p.nu = p.rp <= 64 ? 4 : 3;
  p.off_y = p.nu * p.u;
  p.nb = (kSmemMax - p.off_y - kListBytes - kBarBytes) / kYTile;
  if (p.nb > 5) p.nb = 5;
  p.off_list = p.off_y + p.nb * kYTile;
  p.off_bar = p.off_list + kListBytes;
  p.smem = p.off_bar + kBarBytes;
  return p;
}
// warp 0 MMA, warps 1 and 10 TMA (base, U), warps 2-9 V and epilogue (64 columns each four)
constexpr int kYMmaThreads = 352;

__global__ void __launch_bounds__(kYMmaThreads, 1)
    lora_y_mma_kernel(const __grid_constant__ CUtensorMap tmap_u, const __grid_constant__ CUtensorMap tmap_base,
                      const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ CUtensorMap tmap_v,
                      const float* __restrict__ V, const int32_t* __restrict__ adapter, const float* __restrict__ scale, int has_base,
                      int M, int N, int rank, int L, int parts, int* __restrict__ status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = align_smem(smem_raw);
  const YPlan p = y_plan(rank);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's share of the tiles: one of `parts` of a token tile, or (0) an even one of all, token tile by token tile
  const int tiles = (N + TN - 1) / TN;
  int mt, t0, left;  // `left` tiles from column tile t0 of token tile mt on
  if (parts) {
    const int part = blockIdx.x % parts, each = tiles / parts, more = tiles % parts;
    mt = blockIdx.x / parts;
    t0 = part * each + min(part, more);
    left = each + (part < more);
  } else {
    const int64_t all = (static_cast<int64_t>(M) + TM - 1) / TM * tiles;
    const int64_t begin = all * blockIdx.x / gridDim.x;
    mt = static_cast<int>(begin / tiles);
    t0 = static_cast<int>(begin % tiles);
    left = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x - begin);
  }
  int* ids = reinterpret_cast<int*>(base + p.off_list);
  int* list = ids + TM;
  const uint32_t bars = smem_u32(base + p.off_bar);
  auto y_full = [&](int s) { return bars + 8u * s; };
  auto y_empty = [&](int s) { return bars + 40u + 8u * s; };
  auto u_full = [&](int s) { return bars + 80u + 8u * s; };
  auto u_empty = [&](int s) { return bars + 112u + 8u * s; };
  auto acc_full = [&](int b) { return bars + 144u + 8u * b; };
  auto acc_empty = [&](int b) { return bars + 168u + 8u * b; };
  const uint32_t v_ready = bars + 192u;
  uint32_t* slot = reinterpret_cast<uint32_t*>(base + p.off_bar + 200);
  volatile int* abort = reinterpret_cast<volatile int*>(base + p.off_bar + 204);
  int* counts = reinterpret_cast<int*>(base + p.off_bar + 208);
  const uint32_t v_in = bars + 224u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.nb; ++s) {
      mbar_init(y_full(s), 1);
      mbar_init(y_empty(s), 2);
    }
    for (int s = 0; s < p.nu; ++s) {
      mbar_init(u_full(s), 1);
      mbar_init(u_empty(s), 1);
    }
    for (int b = 0; b < kAcc; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 8);
    }
    mbar_init(v_ready, 256);
    mbar_init(v_in, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1 && lane == 0) {
    prefetch_tmap(&tmap_u);
    if (has_base) prefetch_tmap(&tmap_base);
    prefetch_tmap(&tmap_y);
    prefetch_tmap(&tmap_v);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(slot), 512);
    tmem_relinquish();
    if (lane == 0) griddep_launch_dependents();  // what follows may set itself up beside this kernel
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  // where the rings stand: next slots and their phases; tiles and products so far (the latter while it matters)
  int tiles_done = 0, products = 0, y_first = 0, u_first = 0, b_first = 0;
  uint32_t y_phase = 0, u_phase = 0, b_phase = 0, vs = 0;  // vs: times that V was made
  for (; left > 0; ++mt, t0 = 0) {
    const int64_t m0 = static_cast<int64_t>(mt) * TM;
    const int t1 = left < tiles - t0 ? t0 + left : tiles;
    left -= t1 - t0;
    const int nd = tile_adapters(adapter, m0, M, L, ids, list, counts, kYMmaThreads);
    // V of a tile comes by TMA at more than 32 ranks, by way of the buffers that the base reaches last, 32 ranks of
    // the rows at a time: each thread loading its row is 32 half-used sectors a load (us a call by TMA | by threads:
    // rank 128, 8192 x 12288 113 | 117, rank 64, 4096 x 3072 23.2 | 24.4, rank 8 backward, 777 x 512 15.5 | 14.4)
    const bool v_tma = rank > 32;
    auto v_box = [&](int i) { return base + p.off_y + (y_first + 2 + (i >> 1)) % p.nb * kYTile + (i & 1) * (kYTile / 2); };

    if (warp == 0) {
      // ---------------------------------------------------------------- MMA issuer (one thread)
      if (elect_one()) {
        bool ok = nd == 0 || mbar_sleep(v_ready, vs & 1, abort);
        tc_fence_after();
        bool committed = false;
        uint32_t last_bar = 0, last_ph = 0, ph = u_phase;
        int s = u_first, b = b_first;  // the product's U stage and accumulator
        uint32_t bph = b_phase ^ 1u;   // its accumulator is free: the phase before the first counts as completed
        const uint32_t idesc = idesc_bf16(TM, TN, false, true);
        for (int t = t0; ok && t < t1; ++t) {
          for (int i = 0; i < nd; ++i) {
            if (!mbar_sleep(acc_empty(b), bph, abort)) { ok = false; break; }
            if (!mbar_sleep(u_full(s), ph, abort)) { ok = false; break; }
            tc_fence_after();
            const uint64_t du = sw128_mnmajor_desc(smem_u32(base + s * p.u), p.rp * 128);
#pragma unroll
            for (int h = 0; h < 2; ++h)  // V's rounded values, then the rests
#pragma unroll
              for (int kk = 0; kk < kMaxRank / 16; ++kk)
                if (kk < p.rp / 16)
                  umma_f16_ts(tmem + static_cast<uint32_t>(b * TN),
                              tmem + static_cast<uint32_t>(kVCol + h * (p.rp / 2) + 8 * kk), du + 128u * kk, idesc,
                              (h | kk) ? 1u : 0u);
            umma_commit(u_empty(s));
            umma_commit(acc_full(b));
            last_bar = u_empty(s);
            last_ph = ph;
            committed = true;
            if (++s == p.nu) { s = 0; ph ^= 1u; }
            if (++b == kAcc) { b = 0; bph ^= 1u; }
          }
        }
        if (!ok) {
          fail(abort, status);
          volatile int never = 0;
          if (committed) mbar_sleep(last_bar, last_ph, &never);
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- TMA: base tiles
      if (lane == 0) {
        bool ok = true;
        int y = y_first;
        uint32_t yph = y_phase;
        auto load_v = [&] {
          griddep_wait();  // it comes from the kernel before this one
          const int boxes = (rank + 31) / 32;
          mbar_arrive_expect_tx(v_in, static_cast<uint32_t>(boxes) * (kYTile / 2));
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(smem_u32(v_box(i)), &tmap_v, 32 * i, static_cast<int32_t>(m0), v_in);
        };
        for (int t = t0; t < t1; ++t) {
          // two tiles, then V's turn: behind the whole ring's loads it would take microseconds to arrive (4096 x
          // 3072 -> 3072 at rank 64: 28.7 us a call with the ring first, 26.6 so)
          if (t - t0 == 2 && nd > 0) {
            if (v_tma) load_v();
            if (!mbar_sleep(v_ready, vs & 1, abort)) { ok = false; break; }
          }
          if (tiles_done + t - t0 >= p.nb && !mbar_sleep(y_empty(y), yph ^ 1u, abort)) { ok = false; break; }
          const uint32_t dst = smem_u32(base + p.off_y + y * kYTile);
          if (has_base) {
            mbar_arrive_expect_tx(y_full(y), kYTile);
            tma_load_2d(dst, &tmap_base, t * TN, static_cast<int32_t>(m0), y_full(y));
            tma_load_2d(dst + kYTile / 2, &tmap_base, t * TN + 64, static_cast<int32_t>(m0), y_full(y));
          } else {
            mbar_arrive(y_full(y));
          }
          if (++y == p.nb) { y = 0; yph ^= 1u; }
        }
        if (ok && v_tma && t1 - t0 <= 2 && nd > 0) load_v();
        if (!ok) {
          fail(abort, status);
          grace();
        }
      }
    } else if (warp == 10) {
      // ---------------------------------------------------------------- TMA: U tiles
      if (lane == 0) {
        bool ok = true;
        int s = u_first, f = products;
        uint32_t ph = u_phase;
        for (int t = t0; ok && t < t1; ++t) {
          for (int i = 0; i < nd; ++i, ++f) {
            if (f >= p.nu && !mbar_sleep(u_empty(s), ph ^ 1u, abort)) { ok = false; break; }
            const uint32_t ud = smem_u32(base + s * p.u);
            mbar_arrive_expect_tx(u_full(s), p.u);
            tma_load_3d(ud, &tmap_u, t * TN, 0, list[i], u_full(s));
            tma_load_3d(ud + p.u / 2, &tmap_u, t * TN + 64, 0, list[i], u_full(s));
            if (++s == p.nu) { s = 0; ph ^= 1u; }
          }
        }
        if (!ok) {
          fail(abort, status);
          grace();
        }
      }
    } else {
      // ---------------------------------------------------------------- V, then the epilogue
      const int q = warp & 3, half = (warp - 2) >> 2, row = 32 * q + lane;
      griddep_wait();  // V comes from the kernel before this one
      const int mine = ids[row];
      bool ok = nd == 0 || !v_tma || mbar_sleep_warp(v_in, vs & 1, abort);
      if (ok && nd > 0) {
        // this warp's rows, every other 16 ranks
        const float sc = mine >= 0 ? ldcg_here_f1(scale + mine) : 0.f;
        auto put = [&](int g, const float4 (&f)[4]) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float t = 16 * g + 4 * k < rank ? sc : 0.f;  // (an infinite scale makes NaN of the zeros past the rank)
            split_bf16(f[k].x * t, f[k].y * t, hi[2 * k], lo[2 * k]);
            split_bf16(f[k].z * t, f[k].w * t, hi[2 * k + 1], lo[2 * k + 1]);
          }
          const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(kVCol + 8 * g);
          tmem_st8(at, hi);
          tmem_st8(at + static_cast<uint32_t>(p.rp / 2), lo);
        };
        if (v_tma) {
          for (int g = half; g < p.rp / 16; g += 2) {
            const uint8_t* src = v_box(g >> 1) + row * 128;
            float4 f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              f[k] = *reinterpret_cast<const float4*>(src + (((4 * (g & 1) + k) ^ (row & 7)) << 4));
              if (mine < 0) f[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            put(g, f);
          }
          fence_proxy_async_smem();  // the base's next tiles come where V was
        } else if (half < p.rp / 16) {
          const float* src = V + (m0 + row) * rank + 16 * half;
          float4 f[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mine >= 0 && 16 * half + 4 * k < rank) f[k] = ldcg_here_f4(src + 4 * k);
          }
          put(half, f);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(v_ready);
      }
      const bool storer = (warp == 2 || warp == 6) && lane == 0;  // of this half's 64 columns
      int y = y_first, b = b_first;
      uint32_t yph = y_phase, bph = b_phase;
      for (int t = t0; ok && t < t1; ++t) {
        uint8_t* box = base + p.off_y + y * kYTile + half * (kYTile / 2);
        uint8_t* tile = box + row * 128;
        if (!mbar_sleep_warp(y_full(y), yph, abort)) { ok = false; break; }
        if (!has_base && mine < 0) {  // no adapter, no base: zeros
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(tile + (c << 4)) = make_uint4(0, 0, 0, 0);
        }
        for (int i = 0; i < nd; ++i) {
          if (!mbar_sleep_warp(acc_full(b), bph, abort)) { ok = false; break; }
          tc_fence_after();
          const bool hit = mine == list[i];
          if (__any_sync(0xffffffffu, hit)) {
            uint32_t r[2][32];
            const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(b * TN + 64 * half);
            tmem_ld32(src, r[0]);
            tmem_ld32(src + 32, r[1]);
            tmem_ld_wait();
            if (hit) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                uint4* at = reinterpret_cast<uint4*>(tile + ((c ^ (row & 7)) << 4));
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r[c >> 2][8 * (c & 3) + e]);
                if (has_base) {
                  float bv[8];
                  widen8(*at, bv);
#pragma unroll
                  for (int e = 0; e < 8; ++e) v[e] += bv[e];
                }
                *at = narrow8(v);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty(b));
          if (++b == kAcc) { b = 0; bph ^= 1u; }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        named_bar_sync(1 + half, 128);
        if (storer) {
          if (t * TN + 64 * half < N) tma_store_2d(&tmap_y, t * TN + 64 * half, static_cast<int32_t>(m0), smem_u32(box));
          bulk_commit_group();
          // the box before this one has left its buffer
          bulk_wait_group_read<1>();
          if (t > t0) mbar_arrive(y_empty(y ? y - 1 : p.nb - 1));
        }
        if (++y == p.nb) { y = 0; yph ^= 1u; }
      }
      if (storer && left > 0) {
        bulk_wait_group_read<0>();
        if (ok) mbar_arrive(y_empty(y ? y - 1 : p.nb - 1));
      } else if (storer) {
        bulk_wait_group<0>();
      }
      if (!ok) fail(abort, status);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();  // the tile's list and V have been read
    tc_fence_after();
    if (left == 0 || *abort) break;
    const int n = t1 - t0;
    auto advance = [](int& slot, uint32_t& phase, int by, int slots) {
      slot += by;
      phase ^= slot / slots & 1;
      slot %= slots;
    };
    advance(y_first, y_phase, n, p.nb);
    advance(u_first, u_phase, nd * n, p.nu);
    advance(b_first, b_phase, nd * n, kAcc);
    tiles_done += n;
    products = min(products + nd * n, p.nu);
    vs += nd > 0;
  }

  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------------------------
// grad: 256 columns of Z against all ranks of one adapter, summed over tiles of 64 tokens.  Z's columns are
// the product's M side and V its N side, both as they lie in memory (MN-major).  One launch runs both
// gradients' products (d_down and d_up); token tiles are split over CTAs and the partial sums joined by the
// finish kernel.  Two sets of eight warps make the operands of alternate tiles (V split into pairs; codes
// widened to bf16): a set's chain of loads, conversions, stores and signals is longer than a tile's time, and
// each set's next V is on its way in registers meanwhile.  V's rounded values and rests lie side by side as
// twice as many columns of one product, which costs the same up to 64 columns: the MMAs' issue bounds those.
// A gradient that is not split is rounded here, one against codes after its rotation in shared memory: for few
// tokens the partial sums' way through memory and a kernel more cost as much as the product (1 token, 14 adapters
// of rank 64, 1024 -> 4296: 32 us a backward pass with them, 21 without).
// By itself it takes 17.6 us for 4096 x (3072 + 3072) at rank 64 (52 MB: 3.0 TB/s; start, first tiles and sums are
// half of it) and 54 us for 8192 x (12288 codes + 3072 bf16) at rank 32 (154 MB: 2.8 TB/s), bound by shared memory:
// of 1145 cycles for a tile of codes about 900 are its bytes' (16 KB in and out, 32 KB as bf16 in and out, V).
// ---------------------------------------------------------------------------------------------------

constexpr int GM = 64;           // tokens of a tile
constexpr int GC = 256;          // columns of a CTA
constexpr int kZBox = GM * 128;  // 64 tokens x 64 columns, 8 KB
constexpr int kZTile = 4 * kZBox;
constexpr int kRawTile = GM * GC;   // the tile's codes, 16 KB
constexpr int kMaxGradTiles = 512;  // token tiles of one CTA (64-bit row masks in shared memory)
struct GPlan {
  int rp, vcols, stage, stages, off_raw, off_mask, off_bar, smem, cols;
};
constexpr int kSumsLd = GC + 4;  // floats between the ranks' sums: eight ranks' fours, 32 columns apart, side by side
constexpr int kRaws = 4;  // tiles of codes on their way; even, so that each set meets its slots round by round
inline __host__ __device__ GPlan g_plan(int rank, bool codes, bool v16) {
  GPlan p;
  p.rp = round16(rank);
  p.vcols = v16 ? p.rp : 2 * p.rp;
  p.stage = kZTile + (p.vcols + 63) / 64 * GM * 128;
  const int raw = codes ? kRaws * kRawTile : 0;
  p.stages = (kSmemMax - kMaxGradTiles * 8 - kBarBytes - raw) / p.stage;
  if (p.stages > 4) p.stages = 4;
  p.off_raw = p.stages * p.stage;
  p.off_mask = p.off_raw + raw;
  p.off_bar = p.off_mask + kMaxGradTiles * 8;
  p.smem = p.off_bar + kBarBytes;
  p.cols = tmem_cols_for(2 * p.vcols);
  return p;
}
constexpr int kGSet = 8;                  // warps of a set
constexpr int kGWarps = 2 * kGSet;        // make the operands and, at the end, write the sums
constexpr int kGThreads = 32 * (kGWarps + 2);  // then the MMA's and TMA's warps

// Four signed bytes -> bf16 pairs of 2^-6 times them, exactly: a byte's bits alone are a bf16 value of 2^-133
// times the byte (subnormal up to 127, the first binade from 128 on), so with the sign bit turned one fma by
// 2^127 and less 2 gives (byte + 128 - 128) 2^-6.  Half the integer operations of putting it into a mantissa.
__device__ __forceinline__ uint2 bytes_to_bf16(uint32_t w) {
  const uint32_t u = w ^ 0x80808080u, big = 0x7F007F00u, two = 0xC000C000u;  // bf16 pairs of 2^127 and -2
  uint2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t x = __byte_perm(u, 0u, h ? 0x4342 : 0x4140);
    const __nv_bfloat162 d =
        __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&big),
                *reinterpret_cast<const __nv_bfloat162*>(&two));
    (h ? o.y : o.x) = *reinterpret_cast<const uint32_t*>(&d);
  }
  return o;
}

// kV16: V is bf16 (exact as it is: one product); else float32, as pairs.  kN: groups of four ranks of a tile's
// V that each thread takes, at most.  `block` of this product's blocks.
template <bool kCodes, bool kV16, int kN>
__device__ __forceinline__ void grad_body(const CUtensorMap& tmap_z, const float* __restrict__ code_scale,
                                          const void* __restrict__ V, const int32_t* __restrict__ adapter,
                                          const float* __restrict__ scale, float* __restrict__ G,
                                          uint16_t* __restrict__ grad, int M, int C, int rank,
                                          int L, int splits, int block, int* __restrict__ status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = align_smem(smem_raw);
  const GPlan p = g_plan(rank, kCodes, kV16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int colblocks = (C + GC - 1) / GC;
  const int c0 = (block % colblocks) * GC;
  const int a = block / colblocks % L;
  const int split = block / colblocks / L;
  const int tiles = static_cast<int>((static_cast<int64_t>(M) + GM - 1) / GM);
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / splits);
  const int nt = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / splits) - t0;
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(base + p.off_mask);
  const uint32_t bars = smem_u32(base + p.off_bar);
  auto z_full = [&](int s) { return bars + 8u * s; };         // TMA: the tile's Z or codes
  auto raw_empty = [&](int s) { return bars + 32u + 8u * s; };  // codes: converted
  auto ready = [&](int s) { return bars + 64u + 8u * s; };    // operands complete
  auto empty = [&](int s) { return bars + 96u + 8u * s; };    // MMA has read them
  const uint32_t acc_full = bars + 128u;
  uint32_t* slot = reinterpret_cast<uint32_t*>(base + p.off_bar + 136);
  volatile int* abort = reinterpret_cast<volatile int*>(base + p.off_bar + 140);

  const bool plain = !adapter && a == 0;  // every row of every tile
  const int ring = kCodes ? kRaws : p.stages;
  auto load = [&](int s, int i) {
    const int y = (t0 + i) * GM;
    if constexpr (kCodes) {
      mbar_arrive_expect_tx(z_full(s), kRawTile);
      tma_load_2d(smem_u32(base + p.off_raw + s * kRawTile), &tmap_z, c0, y, z_full(s));
    } else {
      const uint32_t z = smem_u32(base + s * p.stage);
      mbar_arrive_expect_tx(z_full(s), kZTile);
#pragma unroll
      for (int b = 0; b < 4; ++b) tma_load_2d(z + b * kZBox, &tmap_z, c0 + 64 * b, y, z_full(s));
    }
  };
  int asked = 0;  // tiles on their way before the block is set up: without indices none has to be looked up
  if (warp == kGWarps + 1 && lane == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(z_full(s), 1);
      mbar_init(raw_empty(s), kGSet);
      mbar_init(ready(s), kGSet);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full, 1);
    *abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    if (plain)
      for (; asked < ring && asked < nt; ++asked) load(asked, asked);
    else
      prefetch_tmap(&tmap_z);
  }
  if (warp == kGWarps) {
    tmem_alloc(smem_u32(slot), p.cols);
    tmem_relinquish();
    if (lane == 0) griddep_launch_dependents();
  }
  // the rows of this CTA's token tiles that name its adapter
  for (int t = warp; !plain && t < nt; t += kGThreads / 32) {
    const int64_t m = static_cast<int64_t>(t0 + t) * GM + lane;
    const uint32_t lo = __ballot_sync(0xffffffffu, m < M && row_adapter(adapter, m, L) == a);
    const uint32_t hi = __ballot_sync(0xffffffffu, m + 32 < M && row_adapter(adapter, m + 32, L) == a);
    if (lane == 0) mask[t] = static_cast<unsigned long long>(hi) << 32 | lo;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  // first tile at or after i with such a row, nt if none
  auto next_tile = [&](int i) {
    if (!plain)
      while (i < nt && mask[i] == 0) ++i;
    return i;
  };

  if (warp == kGWarps) {
    // ---------------------------------------------------------------- MMA issuer (one thread)
    if (elect_one()) {
      bool ok = true, committed = false;
      uint32_t ph = 0, last_bar = 0, last_ph = 0;
      int s = 0;
      const uint32_t idesc = idesc_bf16(128, p.vcols, true, true);
      for (int i = next_tile(0); i < nt; i = next_tile(i + 1)) {
        if (!mbar_sleep(ready(s), ph, abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t z = smem_u32(base + s * p.stage);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint64_t dz = sw128_mnmajor_desc(z + half * 2 * kZBox, kZBox);
          const uint64_t dv = sw128_mnmajor_desc(z + kZTile, GM * 128);
#pragma unroll
          for (int kk = 0; kk < GM / 16; ++kk)
            umma_f16_ss(tmem + static_cast<uint32_t>(half * p.vcols), dz + 128u * kk, dv + 128u * kk, idesc,
                        (committed || kk) ? 1u : 0u);
        }
        umma_commit(empty(s));
        last_bar = empty(s);
        last_ph = ph;
        committed = true;
        if (++s == p.stages) { s = 0; ph ^= 1u; }
      }
      if (ok) umma_commit(acc_full);
      if (!ok) {
        fail(abort, status);
        volatile int never = 0;
        if (committed) mbar_sleep(last_bar, last_ph, &never);
      }
    }
  } else if (warp == kGWarps + 1) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      bool ok = true;
      int s = 0, f = 0;
      uint32_t ph = 0;
      for (int i = next_tile(0); i < nt; i = next_tile(i + 1), ++f) {
        if (f >= ring && !mbar_sleep(kCodes ? raw_empty(s) : empty(s), ph ^ 1u, abort)) { ok = false; break; }
        if (f >= asked) load(s, i);
        if (++s == ring) { s = 0; ph ^= 1u; }
      }
      if (!ok) {
        fail(abort, status);
        grace();
      }
    }
  } else {
    // ---------------------------------------------------------------- operands
    const int set = warp / kGSet, sw = warp % kGSet;
    const int tid = threadIdx.x - set * 32 * kGSet;
    // places of a thread's fours in the V operand, as values (its row in the bits above 15) and as rests;
    // offsets from the tile's V.  A four past the tile's rows goes nowhere.
    int at[kN], rest[kV16 ? 1 : kN], from[kN];
    auto place = [](int r, int c) { return (c >> 6) * GM * 128 + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4) + (c & 4) * 2; };
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int per = p.rp >> 2, e = tid + 32 * kGSet * k;
      const int r = e / per, j = 4 * (e - r * per);
      at[k] = r < GM ? place(r, j) + (r << 16) : -1;
      if constexpr (!kV16) rest[k] = place(r, p.rp + j);
      from[k] = r < GM && j < rank ? r * rank + j : -1;
    }
    struct Ahead {
      float4 v[kN];  // bf16: bits in x, y
      float cs[kCodes ? kN : 1];
    };
    const uint32_t* mask32 = reinterpret_cast<const uint32_t*>(mask);
    auto fetch = [&](int i, Ahead& x) {
      if (i >= nt) return;
      const int64_t m0 = static_cast<int64_t>(t0 + i) * GM;
      const int rows = M - m0 < GM ? static_cast<int>(M - m0) : GM;
      const uint8_t* v = static_cast<const uint8_t*>(V) + m0 * rank * (kV16 ? 2 : 4);
      const float* cs = kCodes ? code_scale + m0 * (C >> 8) + (c0 >> 8) : nullptr;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        x.v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (kCodes) x.cs[k] = 0.f;
        const int r = at[k] >> 16;
        if (from[k] >= 0 && (plain ? r < rows : (mask32[2 * i + (r >> 5)] >> (r & 31) & 1) != 0)) {
          if constexpr (kV16) {
            const uint2 w = ldcg_here_u2(v + from[k] * 2);
            x.v[k].x = __uint_as_float(w.x);
            x.v[k].y = __uint_as_float(w.y);
          } else {
            x.v[k] = ldcg_here_f4(reinterpret_cast<const float*>(v) + from[k]);
            if constexpr (kCodes) x.cs[k] = ldcg_here_f1(cs + r * (C >> 8));
          }
        }
      }
    };
    bool ok = true;
    // the set's tiles are every other one: its stage of each ring, with the rounds that it has gone
    int s = set, rs = set, f = set;
    uint32_t ph = 0, rph = 0;
    auto make = [&](int i, Ahead& x) {
      uint8_t* z = base + s * p.stage;
      // The MMA has read the stage's last tile.  With an odd number of stages that tile was the other set's, so
      // this also says that it had landed: a wait on z_full goes by parity and must not be two rounds behind.
      if (f >= p.stages && !mbar_sleep_warp(empty(s), ph ^ 1u, abort)) return false;
      if constexpr (kCodes) {
        // codes are finite: those of other adapters' rows meet zeros of V
        if (!mbar_sleep_warp(z_full(rs), rph, abort)) return false;
        const uint8_t* raw = base + p.off_raw + rs * kRawTile;
#pragma unroll
        for (int k = 0; k < GM / kGSet; ++k) {  // a row of the tile for each warp
          const int r = kGSet * k + sw;
          const uint2 w = *reinterpret_cast<const uint2*>(raw + r * GC + 8 * lane);
          const uint2 lo = bytes_to_bf16(w.x), hi = bytes_to_bf16(w.y);
          *reinterpret_cast<uint4*>(z + (lane >> 3) * kZBox + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) =
              make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
      } else {
        if (!mbar_sleep_warp(z_full(s), ph, abort)) return false;
        const unsigned long long rows = plain ? ~0ull : mask[i];  // (rows past M are zeros already)
        if (~rows) {
#pragma unroll 1
          for (int k = 0; k < GM / kGSet; ++k) {
            const int r = kGSet * k + sw;
            if (!(rows >> r & 1))
              *reinterpret_cast<uint4*>(z + (lane >> 3) * kZBox + r * 128 + ((lane & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        if (at[k] < 0) continue;
        uint8_t* d = z + kZTile + (at[k] & 0xFFFF);
        float4 v = x.v[k];
        if constexpr (kV16) {
          *reinterpret_cast<uint2*>(d) = make_uint2(__float_as_uint(v.x), __float_as_uint(v.y));
        } else {
          if constexpr (kCodes) {
            v.x *= x.cs[k];  // 0 for both in a row that is not the adapter's
            v.y *= x.cs[k];
            v.z *= x.cs[k];
            v.w *= x.cs[k];
          }
          uint32_t hi[2], lo[2];
          split_bf16(v.x, v.y, hi[0], lo[0]);
          split_bf16(v.z, v.w, hi[1], lo[1]);
          *reinterpret_cast<uint2*>(d) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(z + kZTile + rest[k]) = make_uint2(lo[0], lo[1]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ready(s));
        if (kCodes) mbar_arrive(raw_empty(rs));
      }
      f += 2;
      if ((s += 2) >= p.stages) { s -= p.stages; ph ^= 1u; }
      if (kCodes && (rs += 2) >= kRaws) { rs -= kRaws; rph ^= 1u; }
      return true;
    };
    // dV comes from the kernel before (Z and a bf16 V do not, and may be read beside it)
    if constexpr (!kV16) griddep_wait();
    Ahead x;
    const int first = next_tile(0);
    int i = set ? next_tile(first + 1) : first;
    fetch(i, x);
    while (i < nt) {
      if (!(ok = make(i, x))) break;
      i = next_tile(next_tile(i + 1) + 1);
      fetch(i, x);
    }
    // ---------------------------------------------------------------- epilogue: column 128 half + 32 q + lane
    if constexpr (kV16) griddep_wait();  // this kernel's end is to mean the ones before have ended, too
    const int q = warp & 3, half = (warp >> 2) & 1, part = warp >> 3;  // every other 16 ranks
    const int c = c0 + 128 * half + 32 * q + lane;
    const float sc = ldcg_here_f1(scale + a) * (kCodes ? 64.f : 1.f);  // codes come as 2^-6 of themselves
    const bool whole = splits == 1;  // no other part: rounded here
    float* out = G + (static_cast<int64_t>(split) * L + a) * rank * C + c;
    uint16_t* rows16 = grad + static_cast<int64_t>(a) * rank * C + c0;
    float* sums = reinterpret_cast<float*>(base);  // [rank, kSumsLd], where the operands were
    if (first < nt) {
      if (ok && mbar_sleep_warp(acc_full, 0, abort)) {
        tc_fence_after();
#pragma unroll 1
        for (int j = 16 * part; j < p.rp; j += 32) {
          uint32_t r[16], l[16];
          const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(half * p.vcols + j);
          tmem_ld16(src, r);
          if constexpr (!kV16) tmem_ld16(src + static_cast<uint32_t>(p.rp), l);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float t = __uint_as_float(r[e]);
            if constexpr (!kV16) t += __uint_as_float(l[e]);
            if (j + e < rank) {
              if (whole) sums[(j + e) * kSumsLd + c - c0] = sc * t;
              else if (c < C) out[static_cast<int64_t>(j + e) * C] = sc * t;
            }
          }
        }
      } else {
        ok = false;
      }
      if (whole) {
        named_bar_sync(1, 32 * kGWarps);
        if constexpr (kCodes) {  // taken against codes: rotated back, a rank's 256 columns by four lanes
          const int u = 8 * warp + (lane >> 2), k0 = lane >> 2, l = lane & 3;
          Pairs P;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (u < rank)
              f = *reinterpret_cast<const float4*>(sums + u * kSumsLd + 32 * ((k >> 1) ^ k0) + 8 * l + 4 * (k & 1));
            put4(P, k, f);
          }
          fwht256_mapped<4>(P);
          if (u < rank) store_unit_bf16(P, k0, 0.0625f, rows16 + static_cast<int64_t>(u) * C);
        } else if (c0 + 8 * lane < C) {
          for (int j = warp; j < rank; j += kGWarps) {
            float v[8];
            const float4 f0 = *reinterpret_cast<const float4*>(sums + j * kSumsLd + 8 * lane);
            const float4 f1 = *reinterpret_cast<const float4*>(sums + j * kSumsLd + 8 * lane + 4);
            v[0] = f0.x; v[1] = f0.y; v[2] = f0.z; v[3] = f0.w;
            v[4] = f1.x; v[5] = f1.y; v[6] = f1.z; v[7] = f1.w;
            *reinterpret_cast<uint4*>(rows16 + static_cast<int64_t>(j) * C + 8 * lane) = narrow8(v);
          }
        }
      }
    } else if (whole) {
      if (c0 + 8 * lane < C)
        for (int j = warp; j < rank; j += kGWarps)
          *reinterpret_cast<uint4*>(rows16 + static_cast<int64_t>(j) * C + 8 * lane) = make_uint4(0, 0, 0, 0);
    } else if (c < C) {
      for (int j = part; j < rank; j += 2) out[static_cast<int64_t>(j) * C] = 0.f;
    }
    if (!ok) fail(abort, status);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kGWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, p.cols);
  }
}

template <bool kCodes, int kN>
__global__ void __launch_bounds__(kGThreads, 1)
    lora_grad_mma_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_dy,
                         const float* __restrict__ code_scale, const float* __restrict__ dV,
                         const uint16_t* __restrict__ V, const int32_t* __restrict__ adapter,
                         const float* __restrict__ scale, float* __restrict__ Gdown, float* __restrict__ Gup,
                         uint16_t* __restrict__ d_down, uint16_t* __restrict__ d_up, int M, int K, int N, int rank, int L, int splits_down, int splits_up, int down_blocks,
                         int* __restrict__ status) {
  if (static_cast<int>(blockIdx.x) < down_blocks)
    grad_body<kCodes, false, kN>(tmap_x, code_scale, dV, adapter, scale, Gdown, d_down, M, K, rank, L, splits_down,
                                blockIdx.x, status);
  else
    grad_body<false, true, kN>(tmap_dy, nullptr, V, adapter, scale, Gup, d_up, M, N, rank, L, splits_up,
                               blockIdx.x - down_blocks, status);
}

std::atomic<bool> g_attr_done[64];

bool set_attrs() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (g_attr_done[dev].load()) return true;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const int most = kSmemMax + 1024;
  if (cudaFuncSetAttribute(lora_v_mma_kernel, attr, most) != cudaSuccess ||
      cudaFuncSetAttribute(lora_v_mma_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      cudaFuncSetAttribute(lora_y_mma_kernel, attr, most) != cudaSuccess ||
      cudaFuncSetAttribute(lora_grad_mma_kernel<false, 1>, attr, most) != cudaSuccess ||
      cudaFuncSetAttribute(lora_grad_mma_kernel<false, 2>, attr, most) != cudaSuccess ||
      cudaFuncSetAttribute(lora_grad_mma_kernel<false, 4>, attr, most) != cudaSuccess ||
      cudaFuncSetAttribute(lora_grad_mma_kernel<false, 8>, attr, most) != cudaSuccess ||
      cudaFuncSetAttribute(lora_grad_mma_kernel<true, 1>, attr, most) != cudaSuccess ||
      cudaFuncSetAttribute(lora_grad_mma_kernel<true, 2>, attr, most) != cudaSuccess ||
      cudaFuncSetAttribute(lora_grad_mma_kernel<true, 4>, attr, most) != cudaSuccess ||
      cudaFuncSetAttribute(lora_grad_mma_kernel<true, 8>, attr, most) != cudaSuccess)
    return false;
  g_attr_done[dev].store(true);
  return true;
}

const auto kBf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
const auto kSw128 = CU_TENSOR_MAP_SWIZZLE_128B;
const auto kL2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;

}  // namespace

int launch_lora_v_mma(const uint16_t* X, int64_t ldx, const int32_t* adapter, const uint16_t* down, float* V,
                      uint16_t* Vout, int M, int K, int rank, int L, int* status, int num_sms, cudaStream_t stream) {
  if (!set_attrs()) return CR_ERR_CUDA;
  const VPlan p = v_plan(rank, L);
  CUtensorMap tx, ta;
  if (!make_tmap_2d(&tx, kBf, X, M, K, static_cast<uint64_t>(ldx) * 2, KB, TM, kSw128, kL2) ||
      !make_tmap_3d(&ta, kBf, down, L, rank, K, static_cast<uint64_t>(K) * 2, KB, p.rp, kSw128, kL2))
    return CR_ERR_CUDA;
  const int64_t tiles = (static_cast<int64_t>(M) + TM - 1) / TM;
  const int nkb = (K + KB - 1) / KB;
  int splits = 1;
  while (splits < kVMostSplits && tiles * splits * 2 <= num_sms && nkb >= 4 * splits) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits), 1, 1);
  cfg.blockDim = dim3(kVThreads, 1, 1);
  cfg.dynamicSmemBytes = p.smem + 1024;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, lora_v_mma_kernel, tx, ta, adapter, V, Vout, M, K, rank, L, splits, status) ==
                 cudaSuccess
             ? CR_OK
             : CR_ERR_CUDA;
}

int launch_lora_y_mma(const float* V, const int32_t* adapter, const uint16_t* up, const float* scale,
                      const uint16_t* base, int64_t ldb, uint16_t* Y, int64_t ldy, int M, int N, int rank, int L,
                      int* status, int num_sms, cudaStream_t stream) {
  if (!set_attrs()) return CR_ERR_CUDA;
  const YPlan p = y_plan(rank);
  CUtensorMap tu, tb, ty, tv;
  memset(&tb, 0, sizeof(tb));
  if (!make_tmap_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, V, M, rank, static_cast<uint64_t>(rank) * 4, 32, TM, kSw128, kL2) ||
      !make_tmap_3d(&tu, kBf, up, L, rank, N, static_cast<uint64_t>(N) * 2, 64, p.rp, kSw128, kL2) ||
      !make_tmap_2d(&ty, kBf, Y, M, N, static_cast<uint64_t>(ldy) * 2, 64, TM, kSw128, CU_TENSOR_MAP_L2_PROMOTION_NONE) ||
      (base && !make_tmap_2d(&tb, kBf, base, M, N, static_cast<uint64_t>(ldb) * 2, 64, TM, kSw128, kL2)))
    return CR_ERR_CUDA;
  const int64_t tiles_m = (static_cast<int64_t>(M) + TM - 1) / TM;
  const int tiles_n = (N + TN - 1) / TN;
  // the same number of column parts of every token tile, or all tiles dealt out evenly: by rounds of (column tiles +
  // about two tiles' worth of prologue for each token tile that a CTA meets).  Dealing evenly also evens out tiles of
  // several adapters; of one it has to gain more than a tenth.  us a call, evenly | in parts: 5000 x 8192, rank 32,
  // one adapter 38.5 | 36.3, four 48.9 | 49.9; 9500 x 2504, rank 64, one 30.3 | 32.8, four 34.7 | 36.4; 8192 x 12288,
  // rank 128, one 85 | 82, four 104 | 108
  int parts = 1;
  int64_t best_cost = INT64_MAX;
  for (int s = 1; s <= tiles_n && s <= 4 * num_sms; ++s) {
    const int64_t cost = (tiles_m * s + num_sms - 1) / num_sms * ((tiles_n + s - 1) / s + 2);
    if (cost < best_cost) {
      best_cost = cost;
      parts = s;
    }
  }
  const int64_t share = (tiles_m * tiles_n + num_sms - 1) / num_sms;
  int64_t even = 10 * (share + 2 * ((share + tiles_n - 1) / tiles_n + 1));
  if (!adapter || L == 1) even += even / 10;
  if (even < 10 * best_cost) parts = 0;
  const int64_t ctas = parts ? tiles_m * parts : num_sms;
  // a programmatic dependent of the v kernel: it starts, loads base and U while that one ends, and waits for
  // it on the device before it reads V
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kYMmaThreads, 1, 1);
  cfg.dynamicSmemBytes = p.smem + 1024;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_y_mma_kernel, tu, tb, ty, tv, V, adapter, scale, static_cast<int>(base != nullptr), M,
                            N, rank, L, parts, status) == cudaSuccess
             ? CR_OK
             : CR_ERR_CUDA;
}

// Token splits of the two gradient products, down's and up's.  In units of one bf16 tile's time on an SM (about
// a third of a microsecond; a tile of codes takes about 1.5): each CTA has its tiles and about eight tiles'
// worth of setting up and writing out; if either is split a kernel more costs about ten, and the partial sums go to
// memory and back (about 0.8 MB a unit).  Up's splits follow from down's so that both kinds of CTA take as long.
void lora_grad_splits(int M, int K, int N, int rank, int L, bool codes, int num_sms, int* down, int* up) {
  const int64_t cd = static_cast<int64_t>((K + GC - 1) / GC) * L, cu = static_cast<int64_t>((N + GC - 1) / GC) * L;
  const int tiles = static_cast<int>((static_cast<int64_t>(M) + GM - 1) / GM);
  const int least = tiles > kMaxGradTiles ? (tiles + kMaxGradTiles - 1) / kMaxGradTiles : 1;
  int64_t best = INT64_MAX;
  *down = *up = least;
  for (int sd = least; sd <= least + 15 && sd <= (tiles > least ? tiles : least); ++sd) {
    const int64_t td = ((tiles + sd - 1) / sd + 8) * (codes ? 6 : 4);  // quarters of a unit
    int64_t room = td / 4 - 8;
    if (room < 1) room = 1;
    int64_t su = (tiles + room - 1) / room;
    if (su < least) su = least;
    if (su > least + 15) su = least + 15;
    const int64_t tu = ((tiles + su - 1) / su + 8) * 4;
    const int64_t most = td > tu ? td : tu, ctas = cd * sd + cu * su;
    // one round: the longest CTA; more: the work spread over the SMs and half of a CTA left over
    const int64_t time = ctas <= num_sms ? most : (cd * sd * td + cu * su * tu) / num_sms + most / 2;
    const int64_t parts = sd > 1 || su > 1 ? 40 + (sd * K + su * N) * static_cast<int64_t>(L) * rank / 50000 : 0;
    const int64_t cost = time + parts;
    if (cost < best) {
      best = cost;
      *down = sd;
      *up = static_cast<int>(su);
    }
  }
}

int launch_lora_grad_mma(const void* X, int64_t ldx, const float* code_scale, const void* dY, int64_t lddy,
                         const float* dV, const uint16_t* V, const int32_t* adapter, const float* scale, float* Gdown,
                         float* Gup, uint16_t* d_down, uint16_t* d_up, int M, int K, int N, int rank, int L,
                         int splits_down, int splits_up, int* status, cudaStream_t stream) {
  if (!set_attrs()) return CR_ERR_CUDA;
  const bool codes = code_scale != nullptr;
  CUtensorMap tx, ty;
  memset(&tx, 0, sizeof(tx));
  memset(&ty, 0, sizeof(ty));
  if (d_down && !(codes ? make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, X, M, K, K, GC, GM, CU_TENSOR_MAP_SWIZZLE_NONE, kL2)
                       : make_tmap_2d(&tx, kBf, X, M, K, static_cast<uint64_t>(ldx) * 2, 64, GM, kSw128, kL2)))
    return CR_ERR_CUDA;
  if (d_up && !make_tmap_2d(&ty, kBf, dY, M, N, static_cast<uint64_t>(lddy) * 2, 64, GM, kSw128, kL2)) return CR_ERR_CUDA;
  const int64_t down = d_down ? static_cast<int64_t>((K + GC - 1) / GC) * L * splits_down : 0;
  const int64_t up = d_up ? static_cast<int64_t>((N + GC - 1) / GC) * L * splits_up : 0;
  if (down + up > INT32_MAX) return CR_ERR_UNSUPPORTED_SHAPE;
  const int s0 = g_plan(rank, codes, false).smem, s1 = g_plan(rank, false, true).smem;
  const int smem = (s0 > s1 ? s0 : s1) + 1024;
  // a thread's share of a tile's V: 64 rows of 16 ranks make one group of four for each thread of a set
  auto kern = rank <= 16   ? (codes ? lora_grad_mma_kernel<true, 1> : lora_grad_mma_kernel<false, 1>)
              : rank <= 32 ? (codes ? lora_grad_mma_kernel<true, 2> : lora_grad_mma_kernel<false, 2>)
              : rank <= 64 ? (codes ? lora_grad_mma_kernel<true, 4> : lora_grad_mma_kernel<false, 4>)
                           : (codes ? lora_grad_mma_kernel<true, 8> : lora_grad_mma_kernel<false, 8>);
  // a programmatic dependent of the kernel before it on the stream
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(down + up), 1, 1);
  cfg.blockDim = dim3(kGThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tx, ty, code_scale, dV, V, adapter, scale, Gdown, Gup, d_down, d_up, M, K, N,
                            rank, L, splits_down, splits_up, static_cast<int>(down), status) == cudaSuccess
             ? CR_OK
             : CR_ERR_CUDA;
}

cudaError_t lora_lost_wait(cudaStream_t stream, bool* found) { return take_lost_wait(stream, found); }

}  // namespace cr
