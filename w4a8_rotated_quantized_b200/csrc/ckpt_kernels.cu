// ckpt_kernels.cu -- streaming kernels around the rotation that go from or to codes:
//
// * 8-bit activation checkpoints: for each row and slice of 256 columns y = x H256, one float32 scale
//   s = max(amax|y| / 127, 2^-100) and codes c = rne(y / s); back, x^ = (c s) H256.  A scale for each
//   slice of each row costs 1/64 byte a value and keeps a loud channel's or a loud token's range away
//   from the others (the rotation spreads a loud channel over its own slice only).
// * packed INT4 weights as bf16 values, w^[n, :] = s_w[n] (q[n, :] H_g), for the input gradient's product.
// * adapter gradients: partial sums of the product kernels added in order, rotated back where they were
//   taken against checkpoint codes (sum_m v[m] x^[m] = (sum_m v[m] s[m] c[m]) H256: the transform runs
//   on the r rows of the result instead of the M rows of the checkpoint), and rounded to bf16.
//
// All of them move bytes: the transform is 8 two-wide adds and fmas for a value pair and 4 digits, far
// below what the memory takes.  Lane mapping and transform: act_device.cuh, 4 lanes for each 256 values,
// 8 slices a warp.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cr_device.cuh"
#include "cr_internal.h"
#include "lora_device.cuh"

namespace cr {
namespace {

#include "act_device.cuh"

constexpr int kWarps = 4;
constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100: below it 1/s would leave float32's range

// The warp's first slice and this lane's: slices are numbered row by row, `upr` to a row.
__device__ __forceinline__ int64_t lane_unit() {
  return (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * 8 + ((threadIdx.x & 31) >> 2);
}

__global__ void __launch_bounds__(32 * kWarps)
    ckpt_save_kernel(const uint16_t* __restrict__ X, int64_t ldx, int8_t* __restrict__ codes,
                     float* __restrict__ scales, int64_t units, int upr) {
  const int64_t u = lane_unit();
  const int k0 = (threadIdx.x & 31) >> 2;
  Raw raw;
  if (u < units) {
    const int64_t row = u / upr;
    load_unit_mapped(X + row * ldx + (u - row * upr) * 256, k0, raw);
  } else {
    zero_raw(raw);
  }
  Pairs P;
  widen_pairs(raw, P);
  fwht256_mapped<4>(P);
  // the largest magnitude by bit pattern, so that a NaN or infinity wins and marks the slice
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    top = max(top, max(__float_as_uint(P.w[i].x) & 0x7FFFFFFFu, __float_as_uint(P.w[i].y) & 0x7FFFFFFFu));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (u >= units) return;
  const bool finite = top < 0x7F800000u;
  // the values are 16 times the rotated ones; 1/16 is exact
  const float s16 = fmaxf(__fdiv_rn(__uint_as_float(top), 127.f), 16.f * kMinScale);
  if ((threadIdx.x & 3) == 0) scales[u] = finite ? s16 * 0.0625f : __uint_as_float(0x7FC00000u);
  if (!finite) {
#pragma unroll
    for (int i = 0; i < 32; ++i) P.w[i] = make_float2(0.f, 0.f);
  }
  const float s = finite ? s16 : 1.f;
  const float r = __frcp_rn(s);
  codes_to_unit_global<kFmtByte8>(P, k0, make_float2(r, r), make_float2(-s, -s),
                                  reinterpret_cast<uint8_t*>(codes) + u * 256);
}

// Pairs of the lane's 64 values of a slice to bf16, times `f`: piece p = k ^ k0 at elements 32p + 8l.
__device__ __forceinline__ void store_unit_bf16(const Pairs& P, int k0, float f, uint16_t* __restrict__ unit) {
  const int l = threadIdx.x & 3;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f * (k < 4 ? P.w[8 * (k & 3) + e].x : P.w[8 * (k & 3) + e].y);
    *reinterpret_cast<uint4*>(unit + 32 * (k ^ k0) + 8 * l) = narrow8(v);
  }
}

__global__ void __launch_bounds__(32 * kWarps)
    ckpt_load_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scales, uint16_t* __restrict__ X,
                     int64_t ldx, int64_t units, int upr) {
  const int64_t u = lane_unit();
  const int k0 = (threadIdx.x & 31) >> 2, l = threadIdx.x & 3;
  uint2 q[8];
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    q[k] = u < units ? __ldg(reinterpret_cast<const uint2*>(codes + u * 256 + 32 * (k ^ k0) + 8 * l)) : make_uint2(0, 0);
  if (u < units) s = __ldg(scales + u);
  Pairs P;
#pragma unroll
  for (int k = 0; k < 8; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = e < 4 ? q[k].x : q[k].y;
      const float v = static_cast<float>(static_cast<int8_t>(w >> (8 * (e & 3))));
      if (k < 4) P.w[8 * (k & 3) + e].x = v; else P.w[8 * (k & 3) + e].y = v;
    }
  fwht256_mapped<4>(P);  // integers up to 256 * 127: exact
  if (u >= units) return;
  const int64_t row = u / upr;
  store_unit_bf16(P, k0, s * 0.0625f, X + row * ldx + (u - row * upr) * 256);
}

// Packed INT4 weights to bf16 values in the unrotated basis.  Rounding the weights once to bf16 lets the
// product run on bf16 operands; each is off by at most 2^-9 of itself, the same half step that rounding
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
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = static_cast<float>(static_cast<int32_t>(w << (28 - 4 * e)) >> 28);
      if (k < 4) P.w[8 * (k & 3) + e].x = v; else P.w[8 * (k & 3) + e].y = v;
    }
  }
  fwht256_mapped<kDig>(P);
  if (u >= units) return;
  const float s = __ldg(w_scale + u / upr) * (1.f / static_cast<float>(1 << kDig));
  store_unit_bf16(P, k0, s, W + u * 256);
}

// Eight values of the partial sums, added in order.
__device__ __forceinline__ void add_parts(const float* __restrict__ src, int parts, int64_t stride, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float4 f0 = __ldg(reinterpret_cast<const float4*>(src + p * stride));
    const float4 f1 = __ldg(reinterpret_cast<const float4*>(src + p * stride + 4));
    v[0] += f0.x; v[1] += f0.y; v[2] += f0.z; v[3] += f0.w;
    v[4] += f1.x; v[5] += f1.y; v[6] += f1.z; v[7] += f1.w;
  }
}

// The gradients' partial sums joined and rounded.  The first `rot_blocks` blocks take slices of 256 values
// of the rotated d_down, the rest eight values a thread of what is left: d_down unrotated, then d_up.
__global__ void __launch_bounds__(32 * kWarps)
    lora_grad_finish_kernel(const float* __restrict__ Gdown, const float* __restrict__ Gup, int parts_down, int parts_up, int64_t n_down,
                            int64_t n_up, uint16_t* __restrict__ d_down, uint16_t* __restrict__ d_up, int rot_blocks) {
  if (static_cast<int>(blockIdx.x) < rot_blocks) {
    const int64_t u = lane_unit();
    const int k0 = (threadIdx.x & 31) >> 2, l = threadIdx.x & 3;
    const bool in = u < n_down >> 8;
    Pairs P;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float v[8];
      add_parts(Gdown + u * 256 + 32 * (k ^ k0) + 8 * l, in ? parts_down : 0, n_down, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (k < 4) P.w[8 * (k & 3) + e].x = v[e]; else P.w[8 * (k & 3) + e].y = v[e];
      }
    }
    fwht256_mapped<4>(P);
    if (in) store_unit_bf16(P, k0, 0.0625f, d_down + u * 256);
    return;
  }
  int64_t i = (static_cast<int64_t>(blockIdx.x - rot_blocks) * 32 * kWarps + threadIdx.x) * 8;
  float v[8];
  if (!rot_blocks) {
    if (i < n_down) {
      add_parts(Gdown + i, parts_down, n_down, v);
      *reinterpret_cast<uint4*>(d_down + i) = narrow8(v);
      return;
    }
    i -= n_down;
  }
  if (i >= n_up) return;
  add_parts(Gup + i, parts_up, n_up, v);
  *reinterpret_cast<uint4*>(d_up + i) = narrow8(v);
}

unsigned unit_blocks(int64_t units) { return static_cast<unsigned>((units + 8 * kWarps - 1) / (8 * kWarps)); }

}  // namespace

cudaError_t launch_ckpt_save(const uint16_t* X, int M, int K, int64_t ldx, int8_t* codes, float* scales,
                             cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(M) * (K / 256);
  ckpt_save_kernel<<<unit_blocks(units), 32 * kWarps, 0, stream>>>(X, ldx, codes, scales, units, K / 256);
  return cudaGetLastError();
}

cudaError_t launch_ckpt_load(const int8_t* codes, const float* scales, int M, int K, uint16_t* X, int64_t ldx,
                             cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(M) * (K / 256);
  ckpt_load_kernel<<<unit_blocks(units), 32 * kWarps, 0, stream>>>(codes, scales, X, ldx, units, K / 256);
  return cudaGetLastError();
}

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
  const unsigned rot = rotate && d_down ? unit_blocks(n_down / 256) : 0;
  const int64_t plain = (rot ? 0 : n_down) + n_up;
  const unsigned blocks = rot + static_cast<unsigned>((plain + 256 * kWarps - 1) / (256 * kWarps));
  lora_grad_finish_kernel<<<blocks, 32 * kWarps, 0, stream>>>(Gdown, Gup, parts_down, parts_up, n_down, n_up, d_down, d_up,
                                                              static_cast<int>(rot));
  return cudaGetLastError();
}

}  // namespace cr
