// Two fp32 operations in one instruction (sm_100 family), each rounded as its
// scalar form.
#pragma once

#include "common.cuh"

namespace moe_f32x2 {

MOE_DEVICE unsigned long long bits(const float2& a) {
  return *reinterpret_cast<const unsigned long long*>(&a);
}
MOE_DEVICE float2 floats(unsigned long long d) { return *reinterpret_cast<float2*>(&d); }

MOE_DEVICE float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return floats(d);
}
MOE_DEVICE float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return floats(d);
}
MOE_DEVICE float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return floats(d);
}
MOE_DEVICE float2 pair(float a) { return make_float2(a, a); }

}  // namespace moe_f32x2
