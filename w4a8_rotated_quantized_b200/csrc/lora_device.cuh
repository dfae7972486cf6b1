// lora_device.cuh -- small device helpers of the adapter kernels: bf16 conversions of eight values and
// the adapter of a row.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace cr {

__device__ __forceinline__ uint16_t bf16_bits(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// Eight bf16 values as floats: the bit patterns 16 bits up.
__device__ __forceinline__ void widen8(uint4 q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    v[2 * h] = __uint_as_float(w[h] << 16);
    v[2 * h + 1] = __uint_as_float(w[h] & 0xFFFF0000u);
  }
}

// Two floats -> packed bf16 (round to nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// Loads of what a kernel may have written that this one started beside, indices and scales included.  Past L1,
// which may hold older values: a read-only load (ld.global.nc) asks that nobody writes while the kernel runs, and this
// kernel runs before the writer has ended.  Volatile, so that they stay where they are written: behind
// griddepcontrol.wait, and before their first use, to which the compiler would sink them and undo a prefetch into
// registers.
__device__ __forceinline__ float4 ldcg_here_f4(const float* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldcg_here_u2(const void* p) {
  uint2 v;
  asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ldcg_here_u4(const void* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float ldcg_here_f1(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int ldcg_here_s32(const int32_t* p) {
  int v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// Two floats as bf16 pairs: the rounded values in `hi`, what they leave, rounded, in `lo`.  `hi` stays finite: what
// would round to an infinity there, infinities themselves included, is held at the largest bf16 value and leaves the
// rest to `lo`, or else the rest would be inf - inf.  So an infinity times a factor other than zero is an infinity of
// the product's sign, as it is without the split.  A NaN's rest is NaN, which the sum keeps.
__device__ __forceinline__ float hold_bf16(float a) {
  float d;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(__uint_as_float(0x7F7F0000u)));
  return d;
}
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(hold_bf16(a), hold_bf16(b));
  lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}

// Row m's adapter, -1 where it has none (an index outside the pool); without indices every row has the first.
__device__ __forceinline__ int row_adapter(const int32_t* adapter, int64_t m, int L) {
  if (!adapter) return 0;
  const int a = ldcg_here_s32(adapter + m);
  return static_cast<unsigned>(a) < static_cast<unsigned>(L) ? a : -1;
}

}  // namespace cr
