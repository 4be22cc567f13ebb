// Gradient of the weighted unpermute / combine
//   out[t] = sum_k w[t,k] * y[row(t,k)] + g[t] * sh[t]
// With d = dout[t]:
//   dy[row(t,k)] = w[t,k] * d        dw[t,k] = <d, y[row(t,k)]>
//   dsh[t]       = g[t] * d          dg[t]   = <d, sh[t]>
// One pass: a block holds d in registers (VPT 16-byte vectors per thread) and
// walks the token's rows in groups of KB, each row read and its gradient
// written once; the dot products of a group are reduced together.  Few tokens
// spread their groups over gridDim.y blocks.  Bound by memory.  No atomics:
// every row belongs to one (t, k).
// Measured on one GB300: T = 8192, K = 10, H = 2048 with the shared expert 116 us,
// 99 % of the copy rate (164 us with each row's loads behind the last row's
// stores); T = 509, K = 4, H = 2880 5.6 us; T = 1, K = 8, H = 2048 3.0 us (4.7 as
// one block).
#include "common.cuh"
#include "internal.h"

namespace {

constexpr int kMaxWarps = 32;

MOE_DEVICE float dot8(const uint4& v, const float* d, float s) {
  float f[8];
  bf16x8_to_f32(v, f);
#pragma unroll
  for (int q = 0; q < 8; ++q) s = fmaf(f[q], d[q], s);
  return s;
}

MOE_DEVICE uint4 scaled8(const float* d, float w) {
  return make_uint4(pack_bf16x2(w * d[0], w * d[1]), pack_bf16x2(w * d[2], w * d[3]),
                    pack_bf16x2(w * d[4], w * d[5]), pack_bf16x2(w * d[6], w * d[7]));
}

// Row index K of the walk stands for the shared expert's row.  y and dy (and
// the shared pair) are not __restrict__: they may be the same buffer.
template <int VPT, int KB>
__global__ void __launch_bounds__(512)
unpermute_backward_kernel(const uint4* __restrict__ dout, const uint4* y,
                          const int32_t* __restrict__ flat_to_row,
                          const float* __restrict__ weights, int T, int K, int H8,
                          const uint4* shared_y, const float* __restrict__ shared_gate, uint4* dy,
                          float* __restrict__ d_weights, uint4* d_shared_y,
                          float* __restrict__ d_shared_gate) {
  __shared__ float red[2][KB][kMaxWarps];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x;
  const int nw = blockDim.x >> 5;
  const long long R = (long long)T * K;
  float d[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = threadIdx.x + blockDim.x * j;
    bf16x8_to_f32(c < H8 ? __ldg(dout + (size_t)t * H8 + c) : make_uint4(0u, 0u, 0u, 0u), d[j]);
  }
  // unsigned: K may be the largest int, and a step of the grid passes it
  const unsigned n = (unsigned)K + (d_shared_y || d_shared_gate ? 1 : 0);
  int slot = 0;
  for (unsigned k0 = blockIdx.y * KB; k0 < n; k0 += gridDim.y * KB, slot ^= 1) {
    float acc[KB];
    long long row[KB];
    float wk[KB];
    bool shared[KB];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const unsigned k = k0 + i;
      shared[i] = k == (unsigned)K && k < n;
      row[i] = -1;
      wk[i] = 0.f;
      if (k < (unsigned)K && flat_to_row) {
        const long long r = __ldg(flat_to_row + (size_t)t * K + k);
        row[i] = r < R ? r : -1;
        if (dy) wk[i] = __ldg(weights + (size_t)t * K + k);
      } else if (shared[i]) {
        row[i] = t;
        if (d_shared_y) wk[i] = __ldg(shared_gate + t);
      }
      acc[i] = 0.f;
    }
    // every vector of the group in flight before the first one is used
    uint4 v[KB][VPT];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const uint4* src = shared[i] ? shared_y : y;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + blockDim.x * j;
        v[i][j] = src && row[i] >= 0 && c < H8 ? src[(size_t)row[i] * H8 + c]
                                               : make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      uint4* dst = shared[i] ? d_shared_y : dy;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + blockDim.x * j;
        acc[i] = dot8(v[i][j], d[j], acc[i]);
        if (dst && row[i] >= 0 && c < H8) dst[(size_t)row[i] * H8 + c] = scaled8(d[j], wk[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      if (row[i] < 0) acc[i] = 0.f;  // a dropped replica, whatever dout holds
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      if (lane_id() == 0) red[slot][i][warp_id()] = acc[i];
    }
    __syncthreads();
    if (threadIdx.x < KB && k0 + threadIdx.x < n) {
      const unsigned k = k0 + threadIdx.x;
      float s = 0.f;
      for (int w = 0; w < nw; ++w) s += red[slot][threadIdx.x][w];
      if (k < (unsigned)K) {
        if (d_weights) d_weights[(size_t)t * K + k] = s;
      } else if (d_shared_gate) {
        d_shared_gate[t] = s;
      }
    }
  }
}

}  // namespace

cudaError_t launch_unpermute_backward(const void* dout, const void* y, const int32_t* flat_to_row,
                                      const float* weights, int T, int K, int H,
                                      const void* shared_y, const float* shared_gate, void* dy,
                                      float* d_weights, void* d_shared_y, float* d_shared_gate,
                                      cudaStream_t stream) {
  const int H8 = H / 8;
  const int vpt = H8 <= 2048 ? moe_row_vectors(H8) : 8;  // 512 threads at most
  const int threads = moe_cdiv(H8, 32 * vpt) * 32;
  const int kb = vpt <= 4 ? 4 : 2;
  auto k = vpt == 1   ? unpermute_backward_kernel<1, 4>
           : vpt == 2 ? unpermute_backward_kernel<2, 4>
           : vpt == 3 ? unpermute_backward_kernel<3, 4>
           : vpt == 4 ? unpermute_backward_kernel<4, 4>
                      : unpermute_backward_kernel<8, 2>;
  const int groups = moe_cdiv((long long)K + (d_shared_y || d_shared_gate ? 1 : 0), kb);
  constexpr int kMaxY = 65535;  // of a grid
  const int split = T >= 2 * 152 ? 1 : groups < kMaxY ? groups : kMaxY;
  // inputs that no requested output needs are not read
  return moe_launch(k, dim3(T, split), dim3(threads), 0, stream, 1, static_cast<const uint4*>(dout),
                    static_cast<const uint4*>(d_weights ? y : nullptr),
                    dy || d_weights ? flat_to_row : nullptr, weights, T, K, H8,
                    static_cast<const uint4*>(d_shared_gate ? shared_y : nullptr), shared_gate,
                    static_cast<uint4*>(dy), d_weights, static_cast<uint4*>(d_shared_y),
                    d_shared_gate);
}
