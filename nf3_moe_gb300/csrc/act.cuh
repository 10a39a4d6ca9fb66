// Pairs of 16-bit activation values and fp32, in one instruction each way.
#pragma once
#include "common.cuh"

namespace hmoe {

// Two packed 16-bit values as fp32 (exact), and back in one conversion
// instruction (the same rounding as f32x2_to_act).
template <int ACT>
__device__ __forceinline__ float2 act_x2_to_f32(uint32_t w) {
  if constexpr (ACT == ACT_F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <int ACT>
__device__ __forceinline__ uint32_t f32_to_act_x2(float a, float b) {
  uint32_t d;
  if constexpr (ACT == ACT_F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}

}  // namespace hmoe
