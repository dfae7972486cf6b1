// grad_values.cu -- streaming kernels of the backward pass around the rotation:
//
// * packed INT4 weights as bf16 values, w^[n, :] = s_w[n] (q[n, :] H_g), for the input gradient's product.
// * adapter gradients: partial sums of the product kernels added in order, rotated back where they were
//   taken against checkpoint codes (sum_m v[m] x^[m] = (sum_m v[m] s[m] c[m]) H256: the transform runs
//   on the r rows of the result instead of the M rows of the checkpoint), and rounded to bf16.
//
// The transform is 8 two-wide adds and fmas for a value pair and 4 digits.  Unpacking 12288 x 3072 weights takes
// 26 us: the 94 MB alone would take 14, the rest is the issue of unpacking, transform and rounding (59 % of the
// slots).  Joining the parts of two gradients of rank 64 and 3072 columns takes about 5 us, one round trip to L2
// after another.  Lane mapping and transform: act_device.cuh, 4 lanes for each 256 values, 8 slices a warp.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cr_device.cuh"
#include "cr_internal.h"
#include "grid_sync.cuh"
#include "lora_device.cuh"

namespace cr {
namespace {

#include "act_device.cuh"
#include "unit_device.cuh"

constexpr int kWarps = 4;

// The warp's first slice and this lane's: slices are numbered row by row, `upr` to a row.
__device__ __forceinline__ int64_t lane_unit() {
  return (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * 8 + ((threadIdx.x & 31) >> 2);
}

// Eight biased values in the low bytes (of x: elements 0-3, of y: 4-7) as floats less `bias`: a byte put into
// the mantissa of 2^23 reads as 2^23 plus it.  (The conversion instructions run at a sixteenth of this rate.)
__device__ __forceinline__ void bytes_to_floats(uint2 q, float bias, float2 (&v)[4]) {
  const float2 b2 = make_float2(-8388608.f - bias, -8388608.f - bias);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = e < 2 ? q.x : q.y;
    v[e] = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + 2 * (e & 1))),
                            __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441 + 2 * (e & 1)))), b2);
  }
}

// The eight values of slot k into the pairs.
__device__ __forceinline__ void put8(Pairs& P, int k, const float2 (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2& a = P.w[8 * (k & 3) + 2 * e];
    float2& b = P.w[8 * (k & 3) + 2 * e + 1];
    if (k < 4) {
      a.x = v[e].x;
      b.x = v[e].y;
    } else {
      a.y = v[e].x;
      b.y = v[e].y;
    }
  }
}

// Packed INT4 weights to bf16 values in the unrotated basis.  Rounding the weights once to bf16 lets the
// product run on bf16 operands; each is off by at most 2^-8 of itself, the same half step that rounding
// the result costs.
template <int kDig>
__global__ void __launch_bounds__(32 * kWarps)
    weight_values_kernel(const uint8_t* __restrict__ Wq, const float* __restrict__ w_scale, uint16_t* __restrict__ W,
                         int64_t units, int upr, int* __restrict__ status) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = CR_OK;
  const int64_t u = lane_unit();
  const int k0 = (threadIdx.x & 31) >> 2, l = threadIdx.x & 3;
  Pairs P;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t w = u < units ? __ldg(reinterpret_cast<const uint32_t*>(Wq + u * 128 + 16 * (k ^ k0) + 4 * l)) : 0u;
    // nibbles to bytes, biased by 8: even elements, odd elements, then in order
    const uint32_t ev = (w & 0x0F0F0F0Fu) ^ 0x08080808u, od = ((w >> 4) & 0x0F0F0F0Fu) ^ 0x08080808u;
    float2 v[4];
    bytes_to_floats(make_uint2(__byte_perm(ev, od, 0x5140), __byte_perm(ev, od, 0x7362)), 8.f, v);
    put8(P, k, v);
  }
  fwht256_mapped<kDig>(P);
  if (u >= units) return;
  const float s = __ldg(w_scale + u / upr) * (1.f / static_cast<float>(1 << kDig));
  store_unit_bf16(P, k0, s, W + u * 256);
}

// The gradients' partial sums joined and rounded, a block of four warps for what one can hold.  The first
// `rot_blocks` blocks take eight slices of 256 values of the rotated d_down, the rest 256 values each of what is
// left: d_down unrotated, then d_up.
__global__ void __launch_bounds__(32 * kJoinWarps)
    lora_grad_finish_kernel(const float* __restrict__ Gdown, const float* __restrict__ Gup, int parts_down, int parts_up,
                            int64_t n_down, int64_t n_up, uint16_t* __restrict__ d_down, uint16_t* __restrict__ d_up,
                            int rot_blocks, int down_blocks) {
  griddep_wait();  // launched as a dependent of the products' kernel
  __shared__ JoinSums sums;
  const int lane = threadIdx.x & 31, block = static_cast<int>(blockIdx.x);
  if (block < rot_blocks) {
    const int64_t u = static_cast<int64_t>(block) * 8 + (lane >> 2);
    const int k0 = lane >> 2, l = lane & 3;
    const bool in = u < n_down >> 8;
    float4 v[16];
    auto at = [&](int k) { return 32 * ((k >> 1) ^ k0) + 8 * l + 4 * (k & 1); };
    if (!join_parts(Gdown + u * 256, parts_down, n_down, in, at, sums, v)) return;
    Pairs P;
#pragma unroll
    for (int k = 0; k < 16; ++k) put4(P, k, v[k]);
    fwht256_mapped<4>(P);
    if (in) store_unit_bf16(P, k0, 0.0625f, d_down + u * 256);
    return;
  }
  const bool down = block - rot_blocks < down_blocks;
  const int64_t i = static_cast<int64_t>(block - rot_blocks - (down ? 0 : down_blocks)) * 256 + 8 * lane;
  const int64_t n = down ? n_down : n_up;
  float4 f[2];
  if (!join_parts((down ? Gdown : Gup) + i, down ? parts_down : parts_up, n, i < n, [](int k) { return 4 * k; }, sums, f))
    return;
  if (i >= n) return;
  const float v[8] = {f[0].x, f[0].y, f[0].z, f[0].w, f[1].x, f[1].y, f[1].z, f[1].w};
  *reinterpret_cast<uint4*>((down ? d_down : d_up) + i) = narrow8(v);
}

unsigned unit_blocks(int64_t units) { return static_cast<unsigned>((units + 8 * kWarps - 1) / (8 * kWarps)); }

}  // namespace

cudaError_t launch_weight_values(const uint8_t* Wq, const float* w_scale, uint16_t* W, int N, int K, int group,
                                 int* status, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(N) * (K / 256);
  const unsigned g = unit_blocks(units);
  const int upr = K / 256, t = 32 * kWarps;
  if (group == 16) weight_values_kernel<2><<<g, t, 0, stream>>>(Wq, w_scale, W, units, upr, status);
  else if (group == 64) weight_values_kernel<3><<<g, t, 0, stream>>>(Wq, w_scale, W, units, upr, status);
  else if (group == 256) weight_values_kernel<4><<<g, t, 0, stream>>>(Wq, w_scale, W, units, upr, status);
  else weight_values_kernel<5><<<g, t, 0, stream>>>(Wq, w_scale, W, units, upr, status);
  return cudaGetLastError();
}

cudaError_t launch_lora_grad_finish(const float* Gdown, const float* Gup, int parts_down, int parts_up, int64_t rows, int K, int N,
                                    uint16_t* d_down, uint16_t* d_up, bool rotate, cudaStream_t stream) {
  const int64_t n_down = d_down ? rows * K : 0, n_up = d_up ? rows * N : 0;
  const unsigned rot = rotate ? static_cast<unsigned>((n_down / 256 + 7) / 8) : 0;
  const unsigned down = rotate ? 0 : static_cast<unsigned>((n_down + 255) / 256);
  const unsigned blocks = rot + down + static_cast<unsigned>((n_up + 255) / 256);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(32 * kJoinWarps, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_grad_finish_kernel, Gdown, Gup, parts_down, parts_up, n_down, n_up, d_down, d_up,
                            static_cast<int>(rot), static_cast<int>(down));
}

}  // namespace cr
