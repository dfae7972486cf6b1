// unit_device.cuh -- slices of 256 values by act_device.cuh's lane mapping (4 lanes for each, 8 a warp): from
// floats into pairs, partial sums joined, and from pairs to bf16.  Included inside an anonymous namespace of cr, after act_device.cuh
// and lora_device.cuh.
#pragma once

// The lane's 16 fours of a slice, four k of them at elements 32 ((k >> 1) ^ k0) + 8 l + 4 (k & 1), into the pairs.
__device__ __forceinline__ void put4(Pairs& P, int k, float4 f) {
  const float e[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float2& pair = P.w[8 * ((k >> 1) & 3) + 4 * (k & 1) + c];
    if (k < 8) pair.x = e[c]; else pair.y = e[c];
  }
}

// Pairs of the lane's 64 values of a slice to bf16, times `f`: piece p = k ^ k0 at elements 32p + 8l.
__device__ __forceinline__ void store_unit_bf16(const Pairs& P, int k0, float f, uint16_t* __restrict__ unit) {
  const int l = threadIdx.x & 3;
  const float2 f2 = make_float2(f, f);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 t = __fmul2_rn(P.w[8 * k + e], f2);
      lo[e] = t.x;
      hi[e] = t.y;
    }
    *reinterpret_cast<uint4*>(unit + 32 * (k ^ k0) + 8 * l) = narrow8(lo);
    *reinterpret_cast<uint4*>(unit + 32 * ((k + 4) ^ k0) + 8 * l) = narrow8(hi);
  }
}

__device__ __forceinline__ void add4(float4& a, float4 b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
}

constexpr int kJoinWarps = 4;  // of a block that joins partial sums
typedef float4 JoinSums[kJoinWarps - 1][16][32];

// kF fours of each thread's from `parts` parts, `stride` floats apart: four f at src + at(f).  Warp w adds parts w,
// w + 4, ..., in order, and the first warp the four sums: as many loads on their way as four warps can have, since
// each is a round trip to L2.  Returns whether this thread has the result.
template <int kF, typename At>
__device__ __forceinline__ bool join_parts(const float* __restrict__ src, int parts, int64_t stride, bool in, At at,
                                           JoinSums& sums, float4 (&v)[kF]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int f = 0; f < kF; ++f) v[f] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = warp; p < (in ? parts : 0); p += kJoinWarps) {
#pragma unroll
    for (int f = 0; f < kF; ++f) add4(v[f], ldcg_here_f4(src + p * stride + at(f)));
  }
  if (warp > 0) {
#pragma unroll
    for (int f = 0; f < kF; ++f) sums[warp - 1][f][lane] = v[f];
  }
  __syncthreads();
  if (warp > 0) return false;
#pragma unroll
  for (int f = 0; f < kF; ++f)
#pragma unroll
    for (int w = 0; w < kJoinWarps - 1; ++w) add4(v[f], sums[w][f][lane]);
  return true;
}
