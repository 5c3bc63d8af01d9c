// fp32 products on the tensor cores: tf32 with every factor in two parts.
#pragma once

#include "common.cuh"

namespace dfl {

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const bf16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y));
}
// D += A B: 16 x 8 of A, row g or g + 8 and element c or c + 4 of lane 4 g + c; 8 x 8 of B, its element c or c + 4 and column g.
__device__ __forceinline__ void mma_tf32(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The two parts of K's and V's values: hi is cut, not rounded, so that the
// largest finite value stays finite; what tf32 drops of lo is 2^-21 of x.
__device__ __forceinline__ void cut2(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// Of Q's and P's: hi rounded, so that lo has a bit less to hold. -0 is (-0, 0). (A
// value within 2^-12 of the largest finite one becomes infinite; P is at most 1.)
__device__ __forceinline__ void round2(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

}  // namespace dfl
