// Rows of activations as e4m3 codes with a scale per column group, and back.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe_e4m3 {

MOE_DEVICE uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

MOE_DEVICE uint32_t amax8(const float* f) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(f[q]) & 0x7fffffffu);
  return m;
}

// Eight e4m3 codes of f / sc (0 where the whole group is zero).  The quotients
// are IEEE's: with r = RN(1 / sc) and q = RN(f r), RN(q + r (f - q sc)) is the
// correctly rounded quotient (Markstein's theorem) while nothing leaves the
// normal range, which scales within 2^+-80 see to -- |f / sc| is at most 448.
// Three operations per value where the division takes about ten.
MOE_DEVICE uint2 codes8(const float* f, float sc) {
  if (sc == 0.f) return make_uint2(0u, 0u);
  float q[8];
  if (sc > 0x1p-80f && sc < 0x1p80f) {
    const float r = __frcp_rn(sc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q0 = f[i] * r;
      q[i] = fmaf(fmaf(-q0, sc, f[i]), r, q0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(f[i], sc);
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w[h] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[4 * h], q[4 * h + 1]), __NV_SATFINITE,
                                              __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[4 * h + 2], q[4 * h + 3]),
                                              __NV_SATFINITE, __NV_E4M3)
               << 16;
  return make_uint2(w[0], w[1]);
}

// 16 codes times their scale, each product rounded to bf16.
MOE_DEVICE void decode16(const uint4& q, float sc, uint4* out) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
    o[i] = pack_bf16x2(f.x * sc, f.y * sc);
  }
  out[0] = make_uint4(o[0], o[1], o[2], o[3]);
  out[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// Eight codes as pairs of fp32 (e4m3 is exact in fp16, and that in fp32).
MOE_DEVICE void codes4(const uint2& q, float2* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((i < 2 ? q.x : q.y) >> (16 * (i & 1))), __NV_E4M3);
    f[i] = __half22float2(*reinterpret_cast<const __half2*>(&hr));
  }
}

}  // namespace moe_e4m3
