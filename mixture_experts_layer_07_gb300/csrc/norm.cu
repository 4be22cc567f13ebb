// N: root-mean-square norm with the residual's addition, an optional e4m3 copy
// of its output, and its gradient.
//
//   h = x + residual               (fp32; stored once, rounded to bf16)
//   s = 1 / sqrt(mean_j h_j^2 + eps)
//   y_j = h_j * s * w_j            (rounded to bf16), from the unrounded h
//   yq  = e4m3(y / scale), scale = amax(group) / 448, from the unrounded y
//
// Backward, with n = h * s (h as stored, s as kept by the forward pass):
//   dx_j = s * (dy_j w_j - n_j * mean_i(dy_i w_i n_i)) + dh_j
//   dw_j = sum_t dy_tj n_tj
//
// Both are bound by memory: a row is read once, held in registers between the
// row's reduction and its use, and written once.  A row is shared by `tpr`
// threads (a multiple of the warp), each owning the 16-byte vectors
// tid + tpr*j, j < VPT; a 128-column scale group is then the 16 vectors of half
// a warp, so its maximum needs four shuffles.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace {

constexpr int kMaxWarps = 16;

// Sum over the row's threads.  `slot` alternates between calls so that one
// barrier per row is enough; rows of one warp need none.
MOE_DEVICE float row_sum(float v, int tpr, float (*red)[kMaxWarps], int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr == 32) return v;
  const int nw = tpr >> 5;  // a row of several warps is the whole block
  if (lane_id() == 0) red[slot][warp_id()] = v;
  __syncthreads();
  float s = lane_id() < nw ? red[slot][lane_id()] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return __shfl_sync(0xffffffffu, s, 0);
}

// largest magnitude as its bit pattern (a NaN is larger than every number, so
// it reaches the scale instead of being lost)
MOE_DEVICE uint32_t row_amax(uint32_t v, int tpr, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (tpr == 32) return v;
  if (lane_id() == 0) red[warp_id()] = v;
  __syncthreads();
  const int nw = tpr >> 5;
  return __reduce_max_sync(0xffffffffu, lane_id() < nw ? red[lane_id()] : 0u);
}

template <bool W32>
MOE_DEVICE void load_weight8(const void* w, int vec, float* f) {
  if constexpr (W32) {
    const float4* p = reinterpret_cast<const float4*>(w) + 2 * (size_t)vec;
    const float4 a = __ldg(p), b = __ldg(p + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(w) + vec), f);
  }
}

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

enum { kQNone = 0, kQGroup = 1, kQRow = 2 };

// One row per group of tpr threads; blockDim.x / tpr rows per block (one row
// where it takes several warps).
// x, residual, h and y are not __restrict__: h may be x or residual, y may be x.
template <int VPT, int MAXT, int Q, bool W32>
__global__ void __launch_bounds__(MAXT)
add_rmsnorm_kernel(const uint4* x, const uint4* residual, const void* __restrict__ w, long long T,
                   int H8, float inv_h, float eps, int tpr, uint4* h_out, uint4* y,
                   float* __restrict__ rstd, uint2* __restrict__ yq, float* __restrict__ yscale) {
  __shared__ float red[2][kMaxWarps];
  __shared__ uint32_t redm[kMaxWarps];
  pdl_wait();
  pdl_trigger();
  const int rpb = blockDim.x / tpr;
  const long long t = (long long)blockIdx.x * rpb + threadIdx.x / tpr;
  if (t >= T) return;  // whole warps only, and only where a row is one warp
  const int lt = threadIdx.x % tpr;
  const size_t base = (size_t)t * H8;
  uint4 a[VPT], b[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = lt + tpr * j;
    const bool in = c < H8;
    a[j] = in ? x[base + c] : make_uint4(0u, 0u, 0u, 0u);
    b[j] = in && residual ? residual[base + c] : make_uint4(0u, 0u, 0u, 0u);
  }
  float h[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float r[8];
    bf16x8_to_f32(a[j], h[j]);
    bf16x8_to_f32(b[j], r);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      h[j][q] += r[q];
      ss = fmaf(h[j][q], h[j][q], ss);
    }
    const int c = lt + tpr * j;
    if (h_out && c < H8) h_out[base + c] = pack8(h[j]);
  }
  const float s = __frsqrt_rn(fmaf(row_sum(ss, tpr, red, 0), inv_h, eps));
  if (rstd && lt == 0) rstd[t] = s;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = lt + tpr * j;
    if (c < H8) {
      float wf[8];
      load_weight8<W32>(w, c, wf);
#pragma unroll
      for (int q = 0; q < 8; ++q) h[j][q] = h[j][q] * s * wf[q];
      if (y) y[base + c] = pack8(h[j]);
    }
    if constexpr (Q == kQGroup) {
      // columns past H take no part (they hold 0, or NaN in a NaN row)
      uint32_t g = c < H8 ? amax8(h[j]) : 0u;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
      const float sc = __fdiv_rn(__uint_as_float(g), 448.f);
      if (c < H8) {
        yq[base + c] = codes8(h[j], sc);
        if ((c & 15) == 0) yscale[(size_t)t * ((H8 + 15) >> 4) + (c >> 4)] = sc;
      }
    } else if constexpr (Q == kQRow) {
      if (c < H8) m = max(m, amax8(h[j]));
    }
  }
  if constexpr (Q == kQRow) {
    const float sc = __fdiv_rn(__uint_as_float(row_amax(m, tpr, redm)), 448.f);
    if (lt == 0) yscale[t] = sc;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = lt + tpr * j;
      if (c < H8) yq[base + c] = codes8(h[j], sc);
    }
  }
}

// Persistent over row groups of rpb rows, one row per tpr threads.  A thread
// keeps its columns' weight gradient in registers; its vectors of the next
// S - 1 groups are on their way into a ring in shared memory that only the
// thread itself reads, so the copies need no barrier -- one barrier per group,
// for the rows' dot products, is all.  At the end the block's rows are added
// and one fp32 partial row is written.
template <int VPT, int S, int BPS, bool W32>
__global__ void __launch_bounds__(512, BPS)
rmsnorm_backward_kernel(const uint4* dy, const uint4* dh, const uint4* __restrict__ h,
                        const float* __restrict__ rstd, const void* __restrict__ w, int T, int H8,
                        float inv_h, int tpr, uint4* dx, float* __restrict__ part) {
  extern __shared__ uint4 ring[];  // [S][3][VPT][blockDim.x]
  __shared__ float red[2][kMaxWarps];
  const int nt = blockDim.x;
  const int rpb = nt / tpr, rs = threadIdx.x / tpr, lt = threadIdx.x % tpr;
  const int wpr = tpr >> 5;
  const int groups = (T + rpb - 1) / rpb;
  pdl_wait();
  pdl_trigger();
  auto slot_of = [&](int st, int arr, int j) { return ring + ((st * 3 + arr) * VPT + j) * nt + threadIdx.x; };
  auto issue = [&](int g, int st) {
    if (g < groups) {
      const long long t = (long long)g * rpb + rs;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = lt + tpr * j;
        const bool in = c < H8 && t < T;
        const size_t o = in ? (size_t)t * H8 + c : 0;
        moe_ptx::cp_async_16(moe_ptx::smem_u32(slot_of(st, 0, j)), dy + o, in ? 16 : 0);
        moe_ptx::cp_async_16(moe_ptx::smem_u32(slot_of(st, 1, j)), h + o, in ? 16 : 0);
        if (dh) moe_ptx::cp_async_16(moe_ptx::smem_u32(slot_of(st, 2, j)), dh + o, in ? 16 : 0);
      }
    }
    moe_ptx::cp_async_commit();
  };
  auto row_rstd = [&](int g) {
    const long long t = (long long)g * rpb + rs;
    return g < groups && t < T ? __ldg(rstd + t) : 0.f;
  };
  constexpr bool kKeepW = VPT <= 1;  // the weight stays in registers where they suffice
  float dw[VPT][8], wk[kKeepW ? VPT : 1][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
#pragma unroll
    for (int q = 0; q < 8; ++q) dw[j][q] = 0.f;
    if constexpr (kKeepW) {
      if (lt + tpr * j < H8) load_weight8<W32>(w, lt + tpr * j, wk[j]);
      else
#pragma unroll
        for (int q = 0; q < 8; ++q) wk[j][q] = 0.f;
    }
  }
  int g = blockIdx.x;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(g + i * gridDim.x, i);
  float s = row_rstd(g);
  for (int it = 0; g < groups; ++it, g += gridDim.x) {
    issue(g + (S - 1) * gridDim.x, (it + S - 1) % S);
    const float s_next = row_rstd(g + gridDim.x);
    moe_ptx::cp_async_wait<S - 1>();
    const int st = it % S;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (lt + tpr * j >= H8) continue;
      float gf[8], hf[8], wf[8];
      bf16x8_to_f32(*slot_of(st, 0, j), gf);
      bf16x8_to_f32(*slot_of(st, 1, j), hf);
      if constexpr (!kKeepW) load_weight8<W32>(w, lt + tpr * j, wf);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float n = hf[q] * s;
        dw[j][q] = fmaf(gf[q], n, dw[j][q]);
        dot = fmaf(gf[q] * (kKeepW ? wk[kKeepW ? j : 0][q] : wf[q]), n, dot);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (wpr > 1) {
      if (lane_id() == 0) red[it & 1][warp_id()] = dot;
      __syncthreads();
      dot = lane_id() < wpr ? red[it & 1][rs * wpr + lane_id()] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      dot = __shfl_sync(0xffffffffu, dot, 0);
    }
    const float c1 = dot * inv_h * s;
    const long long t = (long long)g * rpb + rs;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = lt + tpr * j;
      if (c >= H8 || t >= T) continue;
      float gf[8], hf[8], wf[8], ef[8], o[8];
      bf16x8_to_f32(*slot_of(st, 0, j), gf);
      bf16x8_to_f32(*slot_of(st, 1, j), hf);
      bf16x8_to_f32(dh ? *slot_of(st, 2, j) : make_uint4(0u, 0u, 0u, 0u), ef);
      if constexpr (!kKeepW) load_weight8<W32>(w, c, wf);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        o[q] = fmaf(s, fmaf(-hf[q], c1, gf[q] * (kKeepW ? wk[kKeepW ? j : 0][q] : wf[q])), ef[q]);
      dx[(size_t)t * H8 + c] = pack8(o);
    }
    s = s_next;
  }
  float4* p = reinterpret_cast<float4*>(part) + (size_t)blockIdx.x * H8 * 2;
  if (rpb == 1) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = lt + tpr * j;
      if (c >= H8) continue;
      p[2 * c] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
      p[2 * c + 1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
    return;
  }
  moe_ptx::cp_async_wait<0>();
  __syncthreads();  // the ring takes the rows' sums: [rpb][H8 * 2] float4
  float4* sums = reinterpret_cast<float4*>(ring);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = lt + tpr * j;
    if (c >= H8) continue;
    sums[(rs * H8 + c) * 2] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
    sums[(rs * H8 + c) * 2 + 1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < H8 * 2; i += nt) {
    float4 v = sums[i];
    for (int r = 1; r < rpb; ++r) {
      const float4 x = sums[r * H8 * 2 + i];
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    p[i] = v;
  }
}

// dw[c] = sum over the partial rows, in a fixed order: 32 columns per block,
// warp r takes rows r, r + 32, ..., then the warps' sums are added in order.
__global__ void __launch_bounds__(1024)
column_sum_kernel(const float* __restrict__ part, int rows, int H, float* __restrict__ out) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * 32 + lane_id();
  float s = 0.f;
  if (c < H)
    for (int r = warp_id(); r < rows; r += 32) s += __ldg(part + (size_t)r * H + c);
  red[warp_id()][lane_id()] = s;
  __syncthreads();
  if (warp_id() == 0 && c < H) {
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) v += red[r][lane_id()];
    out[c] = v;
  }
}

struct RowShape {
  int vpt, tpr, rpb;
};

// Up to four vectors per thread while that takes at most 256 threads (H <=
// 8192), eight above (512 threads at H = 32768).  Rows of one warp go eight to
// a block.
RowShape row_shape(int H8) {
  RowShape r;
  r.vpt = H8 <= 32 ? 1 : H8 <= 64 ? 2 : H8 <= 1024 ? 4 : 8;
  r.tpr = moe_cdiv(H8, 32 * r.vpt) * 32;
  r.rpb = r.tpr == 32 ? 8 : 1;
  return r;
}

// Backward: as few vectors per thread as 512 threads allow, as many rows per
// block as fill them (fewer where the rows are too few to go round the SMs).
// The SM count is fixed, not asked of the device: the scratch size must not
// depend on which device is current.
constexpr int kGridSms = 152;
struct BackShape {
  int vpt, tpr, rpb, grid;
};
BackShape back_shape(int T, int H8) {
  BackShape r;
  r.vpt = H8 <= 512 ? 1 : H8 <= 1024 ? 2 : H8 <= 2048 ? 4 : 8;
  r.tpr = moe_cdiv(H8, 32 * r.vpt) * 32;
  const int bps = r.vpt <= 2 ? 2 : 1;
  int rpb = 512 / r.tpr;
  const int share = moe_cdiv(T, bps * kGridSms);
  if (rpb > share) rpb = share;
  r.rpb = rpb < 1 ? 1 : rpb;
  const int groups = moe_cdiv(T, r.rpb);
  r.grid = groups < bps * kGridSms ? groups : bps * kGridSms;
  return r;
}

struct NormArgs {
  const void *x, *residual, *w;
  long long T;
  int H;
  float eps;
  void *h, *y;
  float* rstd;
  void* yq;
  float* yscale;
};

template <int VPT, int MAXT, int Q>
cudaError_t run_norm(bool w32, const RowShape& r, const NormArgs& a, cudaStream_t stream) {
  auto k = w32 ? add_rmsnorm_kernel<VPT, MAXT, Q, true> : add_rmsnorm_kernel<VPT, MAXT, Q, false>;
  return moe_launch(k, dim3((unsigned)((a.T + r.rpb - 1) / r.rpb)), dim3(r.tpr * r.rpb), 0, stream,
                    1, static_cast<const uint4*>(a.x), static_cast<const uint4*>(a.residual), a.w,
                    a.T, a.H / 8, 1.f / (float)a.H, a.eps, r.tpr, static_cast<uint4*>(a.h),
                    static_cast<uint4*>(a.y), a.rstd, static_cast<uint2*>(a.yq), a.yscale);
}

template <int VPT, int MAXT>
cudaError_t run_norm_q(int q, bool w32, const RowShape& r, const NormArgs& a, cudaStream_t s) {
  return q == kQGroup ? run_norm<VPT, MAXT, kQGroup>(w32, r, a, s)
         : q == kQRow ? run_norm<VPT, MAXT, kQRow>(w32, r, a, s)
                      : run_norm<VPT, MAXT, kQNone>(w32, r, a, s);
}

template <int VPT, int S, int BPS>
cudaError_t run_backward(bool w32, const BackShape& r, const void* dy, const void* dh,
                         const void* h, const float* rstd, const void* w, int T, int H, void* dx,
                         float* part, cudaStream_t stream) {
  auto k = w32 ? rmsnorm_backward_kernel<VPT, S, BPS, true> : rmsnorm_backward_kernel<VPT, S, BPS, false>;
  const int threads = r.tpr * r.rpb;
  // the ring, or the rows' sums at the end
  size_t smem = (size_t)S * 3 * VPT * threads * 16;
  const size_t sums = r.rpb > 1 ? (size_t)r.rpb * H * 4 : 0;
  if (smem < sums) smem = sums;
  static std::atomic<unsigned long long> set[2];
  cudaError_t e = moe_raise_smem(k, (size_t)S * 3 * VPT * 512 * 16, set[w32]);
  if (e != cudaSuccess) return e;
  return moe_launch(k, dim3(r.grid), dim3(threads), smem, stream, 1,
                    static_cast<const uint4*>(dy), static_cast<const uint4*>(dh),
                    static_cast<const uint4*>(h), rstd, w, T, H / 8, 1.f / (float)H, r.tpr,
                    static_cast<uint4*>(dx), part);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void* x, const void* residual, const void* w, bool w32, int T,
                               int H, float eps, void* h, void* y, float* rstd, void* yq,
                               float* yscale, int q_group, cudaStream_t stream) {
  const RowShape r = row_shape(H / 8);
  const int q = !yq ? kQNone : q_group ? kQGroup : kQRow;
  const NormArgs a{x, residual, w, T, H, eps, h, y, rstd, yq, yscale};
  switch (r.vpt) {
    case 1: return run_norm_q<1, 256>(q, w32, r, a, stream);
    case 2: return run_norm_q<2, 256>(q, w32, r, a, stream);
    case 4: return run_norm_q<4, 256>(q, w32, r, a, stream);
    default: return run_norm_q<8, 512>(q, w32, r, a, stream);
  }
}

size_t add_rmsnorm_backward_scratch_bytes(int T, int H) {
  const int rows = T > 0 ? back_shape(T, H / 8).grid : 1;
  return moe_align_up((size_t)rows * H * sizeof(float), 256);
}

cudaError_t launch_add_rmsnorm_backward(const void* dy, const void* dh, const void* h,
                                        const float* rstd, const void* w, bool w32, int T, int H,
                                        void* dx, float* dweight, void* scratch,
                                        cudaStream_t stream) {
  float* part = static_cast<float*>(scratch);
  int rows = 0;
  if (T > 0) {
    const BackShape r = back_shape(T, H / 8);
    rows = r.grid;
    cudaError_t e;
    switch (r.vpt) {  // stages: what about 200 KB of shared memory per SM hold
      case 1: e = run_backward<1, 4, 2>(w32, r, dy, dh, h, rstd, w, T, H, dx, part, stream); break;
      case 2: e = run_backward<2, 2, 2>(w32, r, dy, dh, h, rstd, w, T, H, dx, part, stream); break;
      case 4: e = run_backward<4, 2, 1>(w32, r, dy, dh, h, rstd, w, T, H, dx, part, stream); break;
      default: e = run_backward<8, 1, 1>(w32, r, dy, dh, h, rstd, w, T, H, dx, part, stream);
    }
    if (e != cudaSuccess) return e;
  }
  return moe_launch(column_sum_kernel, dim3(moe_cdiv(H, 32)), dim3(1024), 0, stream, 1,
                    (const float*)part, rows, H, dweight);
}
