// Rows of activations as e4m3 codes with an fp32 scale per row and 128 columns (the
// W8A8 activation format), and codes back to bf16 rows.
//
//   pack:   s = max |v| / 448 over the group, code = e4m3(v / s)
//   unpack: v = bf16(code * s)
//
// Both are bound by memory: 3 bytes a value and a scale per 128.  Pack gives a group
// to half a warp, a 16-byte vector per lane, so the maximum is four shuffles; a
// thread has several vectors in flight.
#include "common.cuh"
#include "e4m3.cuh"
#include "internal.h"

namespace {

using namespace moe_e4m3;

constexpr int kThreads = 256;
constexpr int kVec = 4;  // vectors per thread: a block's loads are all in flight at once

// Slots of a row: its vectors, up to whole groups of 16.
__global__ void __launch_bounds__(kThreads)
pack_q8_kernel(const uint4* __restrict__ x, long long T, int H8, uint2* __restrict__ q,
               float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  const int W = (H8 + 15) & ~15;
  const long long first = (long long)blockIdx.x * (kThreads * kVec);
  const long long r0 = first / W;
  const int c0 = (int)(first % W) + threadIdx.x;
  uint4 v[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = c0 + j * kThreads, c = i % W;
    const long long r = r0 + i / W;
    v[j] = r < T && c < H8 ? __ldg(x + r * H8 + c) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = c0 + j * kThreads, c = i % W;
    const long long r = r0 + i / W;
    float f[8];
    bf16x8_to_f32(v[j], f);
    uint32_t m = amax8(f);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float sc = __fdiv_rn(__uint_as_float(m), 448.f);
    if (r >= T || c >= H8) continue;
    q[r * H8 + c] = codes8(f, sc);
    if ((c & 15) == 0) scale[r * (W >> 4) + (c >> 4)] = sc;
  }
}

// 16 codes per vector.
__global__ void __launch_bounds__(kThreads)
unpack_q8_kernel(const uint4* __restrict__ q, const float* __restrict__ scale, long long T, int W,
                 uint4* __restrict__ x) {
  pdl_wait();
  pdl_trigger();
  const int groups = (W + 7) >> 3;
  const long long first = (long long)blockIdx.x * (kThreads * kVec);
  const long long r0 = first / W;
  const int c0 = (int)(first % W) + threadIdx.x;
  uint4 v[kVec];
  float s[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = c0 + j * kThreads;
    const long long r = r0 + i / W;
    if (r >= T) continue;
    v[j] = __ldg(q + r * W + i % W);
    s[j] = __ldg(scale + r * groups + ((i % W) >> 3));
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int i = c0 + j * kThreads;
    const long long r = r0 + i / W;
    if (r < T) decode16(v[j], s[j], x + (r * W + i % W) * 2);
  }
}

unsigned blocks_of(long long slots) {
  return (unsigned)((slots + kThreads * kVec - 1) / (kThreads * kVec));
}

}  // namespace

cudaError_t launch_pack_q8(const void* x, int T, int H, void* xq, float* scale, cudaStream_t stream) {
  const int H8 = H / 8;
  return moe_launch(pack_q8_kernel, dim3(blocks_of((long long)T * ((H8 + 15) & ~15))), dim3(kThreads), 0,
                    stream, 1, static_cast<const uint4*>(x), (long long)T, H8, static_cast<uint2*>(xq),
                    scale);
}

cudaError_t launch_unpack_q8(const void* xq, const float* scale, int T, int H, void* x,
                             cudaStream_t stream) {
  return moe_launch(unpack_q8_kernel, dim3(blocks_of((long long)T * (H / 16))), dim3(kThreads), 0, stream,
                    1, static_cast<const uint4*>(xq), scale, (long long)T, H / 16,
                    static_cast<uint4*>(x));
}
