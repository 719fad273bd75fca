// Device helpers shared by the kernels that came after device_util.cuh's: packed fp32
// arithmetic, tcgen05 products with A in tensor memory, the exponent of V scales, and bf16
// queries taken to f16.
#pragma once

#include <cstdint>

#include "device_util.cuh"


namespace vas {

// D[tmem] (+)= A[tmem] * B[smem]: A's rows are the lanes, two 16-bit elements of the
// contraction dimension a column (16 of them: 8 columns a product); issued by one thread.
__device__ __forceinline__ void umma_ts_lh(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                           uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}


// Two fp32 operations in one instruction, and a maximum of three.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}


// Exponent e of a set of V scales, one or more a lane as their largest magnitude x: they
// lie below 2^(e + 7).  The whole warp.  Between -60 and 60, so that the sums of weights
// relative to 2^e stay within fp32; scales that are not finite count as the largest.
__device__ __forceinline__ float v_exponent(float x) {
  const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7fffffffu);
  return (float)max(-60, min(60, (int)(top >> 23) - 126 - 7));
}

// Largest magnitude of eight bf16 values.
__device__ __forceinline__ float absmax_bf16x8(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo_f32(w[i])), fabsf(bf16_hi_f32(w[i]))));
  return m;
}
// Eight bf16 values times mul (a power of two), as f16 (exact unless below the f16
// normal range).
__device__ __forceinline__ uint4 bf16x8_to_f16x8(uint4 v, float mul) {
  uint4 r;
  r.x = pack_f16x2(bf16_lo_f32(v.x) * mul, bf16_hi_f32(v.x) * mul);
  r.y = pack_f16x2(bf16_lo_f32(v.y) * mul, bf16_hi_f32(v.y) * mul);
  r.z = pack_f16x2(bf16_lo_f32(v.z) * mul, bf16_hi_f32(v.z) * mul);
  r.w = pack_f16x2(bf16_lo_f32(v.w) * mul, bf16_hi_f32(v.w) * mul);
  return r;
}

}  // namespace vas
