// Rows of activations as e4m3 codes with an fp32 scale per row and 128 columns (the
// W8A8 activation format), and codes back to bf16 rows.
//
//   pack:   s = max |v| / 448 over the group, code = e4m3(v / s)
//   unpack: v = bf16(code * s)
//
// Both are bound by memory (3 bytes a value and a scale per 128) once the work per
// value is small enough and enough loads are in flight.  Pack gives a group to four
// lanes, four 16-byte vectors each: the scale and its reciprocal are then made once per
// 32 values, the maximum takes two shuffles.  T = 8191, H = 7168: 40 us with a group per
// half warp and a vector per lane (157 instructions per vector), 33 us with a group per
// four lanes, 26.5 us with two of them (29 with three).  Unpack takes 8 codes a lane and
// time, so that a warp's stores are whole lines (16 codes a lane: 20 us at T = 16384,
// H = 2048, so 16.5).
// Measured on one GB300 (copy rate 6797 GB/s): pack T = 8191, H = 7168 26.5 us, 99 % of
// the copy rate; unpack T = 16384, H = 2048 16.5 us, 91 %; T = 1 1.4 us.
#include "common.cuh"
#include "e4m3.cuh"
#include "f32x2.cuh"
#include "internal.h"

namespace {

using namespace moe_e4m3;
using namespace moe_f32x2;

constexpr int kThreads = 256;
constexpr int kVec = 4;              // vectors of a group per lane (pack), vectors per thread (unpack)
constexpr int kTeams = kThreads / 4;  // pack
constexpr int kGroups = 2;            // pack: of a team

// The largest magnitude of 8 bf16 per half, as bits (a NaN is above every number).
MOE_DEVICE uint32_t amax_bf16x8(const uint4& v) {
  const uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
}

// codes8 of 8 bf16, two values at a time; r = RN(1 / sc), sc within 2^+-80.
MOE_DEVICE uint2 codes_bf16x8(const uint4& v, float sc, float r) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(bf16_lo(u[i]), bf16_hi(u[i]));
    const float2 q0 = mul2(f, pair(r));
    const float2 q = fma2(fma2(q0, pair(-sc), f), pair(r), q0);
    c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Four lanes per group of 16 vectors; G groups in a row (the last may hold fewer vectors).
// A team takes two groups, a block's teams apart, all loads first.
__global__ void __launch_bounds__(kThreads)
pack_q8_kernel(const uint4* __restrict__ x, long long T, int H8, int G, uint2* __restrict__ q,
               float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  const long long first = (long long)blockIdx.x * (kTeams * kGroups);
  const long long r0 = first / G;
  const uint32_t at = (uint32_t)(first % G) + (threadIdx.x >> 2);
  uint4 v[kGroups][kVec];
#pragma unroll
  for (int b = 0; b < kGroups; ++b) {
    const uint32_t a = at + b * kTeams;
    const long long row = r0 + a / (uint32_t)G;
    const int c0 = (int)(a % (uint32_t)G) * 16 + (threadIdx.x & 3);
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      v[b][j] = row < T && c0 + 4 * j < H8 ? __ldg(x + (size_t)row * H8 + c0 + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int b = 0; b < kGroups; ++b) {
    const uint32_t a = at + b * kTeams;
    const long long row = r0 + a / (uint32_t)G;
    const int g = (int)(a % (uint32_t)G), c0 = g * 16 + (threadIdx.x & 3);
    const size_t base = (size_t)row * H8 + c0;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) m = __vmaxu2(m, amax_bf16x8(v[b][j]));
    m = max(m >> 16, m & 0xffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (row >= T) continue;
    const float sc = __fdiv_rn(__uint_as_float(m << 16), 448.f);
    if ((threadIdx.x & 3) == 0) scale[row * G + g] = sc;
    if (sc > 0x1p-80f && sc < 0x1p80f) {
      const float r = __frcp_rn(sc);
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (c0 + 4 * j < H8) q[base + 4 * j] = codes_bf16x8(v[b][j], sc, r);
    } else {  // zeros, and scales near the range's ends
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        float f[8];
        bf16x8_to_f32(v[b][j], f);
        if (c0 + 4 * j < H8) q[base + 4 * j] = codes8(f, sc);
      }
    }
  }
}

// 8 codes per vector, W of them in a row; a block's vectors follow one another.
__global__ void __launch_bounds__(kThreads)
unpack_q8_kernel(const uint2* __restrict__ q, const float* __restrict__ scale, long long T, int W,
                 uint4* __restrict__ x) {
  pdl_wait();
  pdl_trigger();
  const int groups = (W + 15) >> 4;
  const long long first = (long long)blockIdx.x * (kThreads * kVec);
  const long long r0 = first / W;
  const uint32_t c0 = (uint32_t)(first % W) + threadIdx.x;
  q += first + threadIdx.x;
  x += first + threadIdx.x;
  const long long left = T * W - first - threadIdx.x;
  uint2 v[kVec];
  float s[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    if (j * kThreads >= left) continue;
    const uint32_t c = c0 + j * kThreads;
    v[j] = __ldg(q + j * kThreads);
    s[j] = __ldg(scale + (r0 + c / (uint32_t)W) * groups + ((c % (uint32_t)W) >> 4));
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    if (j * kThreads >= left) continue;
    float2 f[4];
    codes4(v[j], f);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = mul2(f[i], pair(s[j]));
      o[i] = pack_bf16x2(f[i].x, f[i].y);
    }
    x[j * kThreads] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

unsigned blocks_of(long long n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace

cudaError_t launch_pack_q8(const void* x, int T, int H, void* xq, float* scale, cudaStream_t stream) {
  const int G = (H + 127) / 128;
  return moe_launch(pack_q8_kernel, dim3(blocks_of((long long)T * G, kTeams * kGroups)), dim3(kThreads), 0,
                    stream, 1, static_cast<const uint4*>(x), (long long)T, H / 8, G,
                    static_cast<uint2*>(xq), scale);
}

cudaError_t launch_unpack_q8(const void* xq, const float* scale, int T, int H, void* x,
                             cudaStream_t stream) {
  const int W = H / 8;
  return moe_launch(unpack_q8_kernel, dim3(blocks_of((long long)T * W, kThreads * kVec)),
                    dim3(kThreads), 0, stream, 1, static_cast<const uint2*>(xq), scale, (long long)T, W,
                    static_cast<uint4*>(x));
}
