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
// Measured on one GB300 (copy rate 6696 GB/s): T = 8191, H = 7168 with residual
// and a scale per row 79.7 us, 99 % of the copy rate; T = 4096, H = 2880 with a
// scale per 128 columns 20.8 us (77 %, 1.7 us of it the launch); T = 1, H = 2048
// 1.7 us.  Backward T = 8192, H = 7168 75.6 us (93 %).
#include "common.cuh"
#include "e4m3.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace {

using namespace moe_e4m3;
using namespace moe_f32x2;

constexpr int kMaxWarps = 32;

// Sum of v over the row, in an order that depends on H alone, not on how the
// row is spread over threads (nor so on the batch): first the 32 vectors of a
// chunk, lanes 16 apart, 8 apart and so on, then the chunks likewise, chunk i at
// lane i % 32.  A warp's VPT chunks are halved as the distance is -- a lane hands
// over what its partner goes on with -- so four take six exchanges, not twenty.
template <int VPT>
MOE_DEVICE float row_sum(const float (&v)[VPT], int tpr, float* red) {
  const int lane = lane_id();
  float s = v[0];
  int mine = 0;  // the chunk whose sum this lane ends up with
  if constexpr (VPT == 1) {
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    s += __shfl_xor_sync(0xffffffffu, s, 8);
  } else if constexpr (VPT == 2) {
    mine = lane >> 4;
    s = mine ? v[1] : v[0];
    s += __shfl_xor_sync(0xffffffffu, mine ? v[0] : v[1], 16);
    s += __shfl_xor_sync(0xffffffffu, s, 8);
  } else {
    const float v3 = VPT == 4 ? v[VPT - 1] : 0.f;
    const bool hi = lane & 16, odd = lane & 8;
    float a = hi ? v[2] : v[0], b = hi ? v3 : v[1];
    a += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
    b += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v3, 16);
    s = odd ? b : a;
    s += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
    mine = 2 * (lane >> 4) + (lane >> 3 & 1);  // 0, 1, 2, 3 from lanes 0, 8, 16, 24
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (tpr == 32) {  // the chunks' sum as the butterfly below makes it
    if constexpr (VPT > 1) s += __shfl_xor_sync(0xffffffffu, s, 16);
    if constexpr (VPT > 2) s += __shfl_xor_sync(0xffffffffu, s, 8);
    return s;
  }
  const int nw = tpr >> 5;  // a row of several warps is the whole block
  constexpr int kEach = VPT == 1 ? 32 : VPT == 2 ? 16 : 8;  // lanes per chunk
  if (lane % kEach == 0 && mine < VPT) red[warp_id() + nw * mine] = s;
  __syncthreads();
  const int n = nw * VPT;
  s = lane < n ? red[lane] : 0.f;
  if (n > 32) {
#pragma unroll
    for (int i = 32; i < 4 * kMaxWarps; i += 32) s += lane + i < n ? red[lane + i] : 0.f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
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

enum { kQNone = 0, kQGroup = 1, kQRow = 2 };

// One row per group of tpr threads; blockDim.x / tpr rows per block (one row
// where it takes several warps).
// x, residual, h and y are not __restrict__: h may be x or residual, y may be x.
template <int VPT, int Q, bool W32>
__global__ void __launch_bounds__(1024)
add_rmsnorm_kernel(const uint4* x, const uint4* residual, const void* __restrict__ w, long long T,
                   int H8, float inv_h, float eps, int tpr, uint4* h_out, uint4* y,
                   float* __restrict__ rstd, uint2* __restrict__ yq, float* __restrict__ yscale) {
  __shared__ float red[4 * kMaxWarps];
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
  float ss[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float r[8];
    ss[j] = 0.f;
    bf16x8_to_f32(a[j], h[j]);
    bf16x8_to_f32(b[j], r);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      h[j][q] += r[q];
      ss[j] = fmaf(h[j][q], h[j][q], ss[j]);
    }
    const int c = lt + tpr * j;
    if (h_out && c < H8) h_out[base + c] = pack8(h[j]);
  }
  const float s = __frsqrt_rn(fmaf(row_sum(ss, tpr, red), inv_h, eps));
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

MOE_DEVICE void unpack4(const uint4& v, float2* f) {
  f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
  f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
  f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z));
  f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
}
template <bool W32>
MOE_DEVICE void weight4(const void* w, int vec, float2* f) {
  if constexpr (W32) {
    const float4* p = reinterpret_cast<const float4*>(w) + 2 * (size_t)vec;
    const float4 a = __ldg(p), b = __ldg(p + 1);
    f[0] = make_float2(a.x, a.y); f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y); f[3] = make_float2(b.z, b.w);
  } else {
    unpack4(__ldg(reinterpret_cast<const uint4*>(w) + vec), f);
  }
}

// Persistent over row groups of rpb rows, one row per tpr threads.  A thread
// keeps its columns' weight gradient in registers.  Its vectors of the next
// row groups are on their way into a ring of S stages in shared memory that
// only the thread itself reads, so the copies need no barrier; the rows' dot
// products take one barrier per group.  With LAG, a group's dx is computed one
// group late, behind the next group's sums, so that no warp waits at the
// barrier with nothing to do.  At the end the block's rows are added and one
// fp32 partial row is written.  (T = 8192, H = 7168: rows loaded into registers
// when their turn comes 88 us; ring of two stages, two vectors per thread 86;
// four stages, one vector, LAG 78; running offsets 76.)
// HQ: h lies as e4m3 codes with a scale per row and 16 vectors.  An even lane copies the
// codes of its vector and of its neighbour's, the scales stay in registers, loaded a group
// ahead (T = 8192, H = 7168 92 us with a copy of codes and scale per lane, 84 us so: 73 % of
// the copy rate; the schedulers issue on 69 % of the cycles, 300 instructions per vector,
// and two vectors per thread, half the instructions around them, leave too few warps: 91 us).
template <int VPT, int S, int MAXT, int BPS, bool LAG, bool W32, bool HQ>
__global__ void __launch_bounds__(MAXT, BPS)
rmsnorm_backward_kernel(const uint4* dy, const uint4* dh, const void* __restrict__ h,
                        const float* __restrict__ hscale, const float* __restrict__ rstd, const void* __restrict__ w, int T, int H8,
                        float inv_h, int tpr, uint4* dx, float* __restrict__ part) {
  constexpr int kAhead = LAG ? S - 2 : S - 1;  // groups in flight behind the current one
  extern __shared__ uint4 ring[];              // [S][3][VPT][blockDim.x]
  __shared__ float red[2][MAXT / 32];
  const int nt = blockDim.x;
  const int rpb = nt / tpr, rs = threadIdx.x / tpr, lt = threadIdx.x % tpr;
  const int wpr = tpr >> 5;
  const int groups = (T - 1) / rpb + 1;  // T > 0; T + rpb may pass the largest int
  pdl_wait();
  pdl_trigger();
  // vector j of array arr (dy, h, dh) in stage st
  const int arrs = VPT * nt;
  auto slot_of = [&](int st, int arr, int j) { return ring + (st * 3 + arr) * arrs + j * nt + threadIdx.x; };
  // this thread's first vector of the group that is issued, and of the one that
  // is finished; groups lie `step` apart
  const int step = gridDim.x;
  const size_t hop = (size_t)step * rpb * H8;
  const uint32_t rows = (uint32_t)step * rpb;
  uint32_t t_issue = blockIdx.x * rpb + rs, t_done = t_issue;  // rows; past T: nothing to do
  size_t o_issue = (size_t)t_issue * H8 + lt, o_done = o_issue;
  auto issue = [&](int st) {
    if (t_issue < (uint32_t)T) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (lt + tpr * j >= H8) continue;
        const size_t o = o_issue + tpr * j;
        moe_ptx::cp_async_16(moe_ptx::smem_u32(slot_of(st, 0, j)), dy + o, 16);
        if constexpr (HQ) {
          if ((threadIdx.x & 1) == 0)
            moe_ptx::cp_async_16(moe_ptx::smem_u32(slot_of(st, 1, j)), static_cast<const uint2*>(h) + o, 16);
        } else {
          moe_ptx::cp_async_16(moe_ptx::smem_u32(slot_of(st, 1, j)), static_cast<const uint4*>(h) + o, 16);
        }
        if (dh) moe_ptx::cp_async_16(moe_ptx::smem_u32(slot_of(st, 2, j)), dh + o, 16);
      }
    }
    moe_ptx::cp_async_commit();
    t_issue += rows;
    o_issue += hop;
  };
  // h of vector j in stage st; HQ: its codes (they lie in the even lane's slot), whose scale
  // goes into the factor that h is multiplied with
  auto load_h = [&](int st, int j, float2* f) {
    if constexpr (HQ)
      codes4(*(reinterpret_cast<const uint2*>(slot_of(st, 1, j) - (threadIdx.x & 1)) + (threadIdx.x & 1)), f);
    else
      unpack4(*slot_of(st, 1, j), f);
  };
  struct Scales {
    float v[HQ ? VPT : 1];
  };
  auto row_scales = [&](uint32_t t) {
    Scales r;
    if constexpr (HQ) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        r.v[j] = t < (uint32_t)T && lt + tpr * j < H8
                     ? __ldg(hscale + (size_t)t * ((H8 + 15) >> 4) + ((lt + tpr * j) >> 4))
                     : 0.f;
    }
    return r;
  };
  auto row_rstd = [&](uint32_t t) { return t < (uint32_t)T ? __ldg(rstd + t) : 0.f; };
  constexpr bool kKeepW = VPT == 1;  // the weight stays in registers where they suffice
  float2 dw[VPT][4], wk[4];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) dw[j][q] = pair(0.f);
  if (kKeepW && lt < H8) weight4<W32>(w, lt, wk);

  // dx of the next group to finish, whose rows lie in stage st and whose dot
  // products in red[slot]
  auto finish = [&](int st, int slot, float s, float dot, const Scales& sc) {
    if (wpr > 1) {
      dot = lane_id() < wpr ? red[slot][rs * wpr + lane_id()] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    const float c1 = -(dot * inv_h) * s;  // dx = s (dy w + h c1) + dh
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (lt + tpr * j >= H8 || t_done >= (uint32_t)T) continue;
      float2 gf[4], hf[4], wf[4], ef[4], o[4];
      unpack4(*slot_of(st, 0, j), gf);
      load_h(st, j, hf);
      const float2 hc = pair(HQ ? c1 * sc.v[HQ ? j : 0] : c1);
      unpack4(dh ? *slot_of(st, 2, j) : make_uint4(0u, 0u, 0u, 0u), ef);
      if constexpr (!kKeepW) weight4<W32>(w, lt + tpr * j, wf);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = fma2(pair(s), fma2(hf[q], hc, mul2(gf[q], kKeepW ? wk[q] : wf[q])), ef[q]);
      dx[o_done + tpr * j] = make_uint4(pack_bf16x2(o[0].x, o[0].y), pack_bf16x2(o[1].x, o[1].y),
                                        pack_bf16x2(o[2].x, o[2].y), pack_bf16x2(o[3].x, o[3].y));
    }
    t_done += rows;
    o_done += hop;
  };

  uint32_t t = t_issue;  // the current group's row
#pragma unroll
  for (int i = 0; i < kAhead; ++i) issue(i);
  float s = row_rstd(t), s_prev = 0.f, dot_prev = 0.f;
  Scales sc = row_scales(t), sc_prev = sc;
  int it = 0;
  for (int g = blockIdx.x; g < groups; ++it, g += step) {
    if constexpr (HQ) __syncwarp();  // the neighbour is done with the stage that is filled next
    issue((it + kAhead) % S);
    const float s_next = row_rstd(t + rows);
    const Scales sc_next = row_scales(t + rows);
    moe_ptx::cp_async_wait<kAhead>();
    if constexpr (HQ) __syncwarp();  // the neighbour's copy too
    const int st = it % S;
    float2 dot2 = pair(0.f);
    if (t < (uint32_t)T) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (lt + tpr * j >= H8) continue;
        float2 gf[4], hf[4], wf[4];
        unpack4(*slot_of(st, 0, j), gf);
        load_h(st, j, hf);
        const float2 hs = pair(HQ ? s * sc.v[HQ ? j : 0] : s);
        if constexpr (!kKeepW) weight4<W32>(w, lt + tpr * j, wf);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 n = mul2(hf[q], hs);
          dw[j][q] = fma2(gf[q], n, dw[j][q]);
          dot2 = fma2(mul2(gf[q], kKeepW ? wk[q] : wf[q]), n, dot2);
        }
      }
    }
    float dot = dot2.x + dot2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (wpr > 1 && lane_id() == 0) red[it & 1][warp_id()] = dot;
    if (LAG && it > 0) finish((it - 1) % S, (it - 1) & 1, s_prev, dot_prev, sc_prev);
    if (wpr > 1) __syncthreads();
    if (!LAG) finish(st, it & 1, s, dot, sc);
    s_prev = s;
    dot_prev = dot;
    s = s_next;
    sc_prev = sc;
    sc = sc_next;
    t += rows;
  }
  if (LAG && it > 0) finish((it - 1) % S, (it - 1) & 1, s_prev, dot_prev, sc_prev);

  float4* p = reinterpret_cast<float4*>(part) + (size_t)blockIdx.x * H8 * 2;
  // one row per block: its sums are the block's; else they meet in the ring,
  // as [rpb][H8 * 2] float4
  float4* sums = rpb == 1 ? p : reinterpret_cast<float4*>(ring) + (size_t)rs * H8 * 2;
  if (rpb > 1) {
    moe_ptx::cp_async_wait<0>();
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = lt + tpr * j;
    if (c >= H8) continue;
    sums[c * 2] = make_float4(dw[j][0].x, dw[j][0].y, dw[j][1].x, dw[j][1].y);
    sums[c * 2 + 1] = make_float4(dw[j][2].x, dw[j][2].y, dw[j][3].x, dw[j][3].y);
  }
  if (rpb == 1) return;
  __syncthreads();
  sums = reinterpret_cast<float4*>(ring);
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
  if (c < H) {
#pragma unroll 8
    for (int r = warp_id(); r < rows; r += 32) s += __ldg(part + (size_t)r * H + c);
  }
  red[warp_id()][lane_id()] = s;
  __syncthreads();
  if (warp_id() == 0 && c < H) {
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) v += red[r][lane_id()];
    out[c] = v;
  }
}

// Forward.  Where the rows are too few to fill the SMs the call is one row's
// latency, and as many threads as a row can feed shorten it (T = 1, H = 2048 2.4
// -> 1.7 us against the four vectors per thread that large batches take; T =
// 8191, H = 7168 79.8 -> 99.5 us the other way).  Rows of one warp go eight to a
// block.
constexpr int kGridSms = 152;
struct RowShape {
  int vpt, tpr, rpb;
};
RowShape row_shape(long long T, int H8) {
  RowShape r;
  r.vpt = T >= 2 * kGridSms ? moe_row_vectors(H8) : H8 <= 1024 ? 1 : H8 <= 2048 ? 2 : 4;
  r.tpr = moe_cdiv(H8, 32 * r.vpt) * 32;
  r.rpb = r.tpr == 32 ? 8 : 1;
  return r;
}

// Backward: one vector per thread up to 1024 threads (H <= 8192), several
// beyond; two blocks of up to 512 threads per SM where a row fits one (H <=
// 4096), else one block.  As many rows per block as fill the threads, fewer
// where the rows are too few to go round.  The SM count is fixed, not asked of the device:
// the scratch size must not depend on which device is current.
struct BackShape {
  int vpt, tpr, rpb, grid;
};
BackShape back_shape(int T, int H8) {
  BackShape r;
  r.vpt = H8 <= 1024 ? 1 : H8 <= 2048 ? 4 : 8;
  r.tpr = moe_cdiv(H8, 32 * r.vpt) * 32;
  const int slots = kGridSms * (H8 <= 512 ? 2 : 1);
  const int share = moe_cdiv(T, slots);
  const int fit = (H8 <= 512 || r.vpt > 1 ? 512 : 1024) / r.tpr;
  r.rpb = share < fit ? share : fit;
  const int groups = moe_cdiv(T, r.rpb);
  r.grid = groups < slots ? groups : slots;
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

template <int VPT, int Q>
cudaError_t run_norm(bool w32, const RowShape& r, const NormArgs& a, cudaStream_t stream) {
  auto k = w32 ? add_rmsnorm_kernel<VPT, Q, true> : add_rmsnorm_kernel<VPT, Q, false>;
  return moe_launch(k, dim3((unsigned)((a.T + r.rpb - 1) / r.rpb)), dim3(r.tpr * r.rpb), 0, stream,
                    1, static_cast<const uint4*>(a.x), static_cast<const uint4*>(a.residual), a.w,
                    a.T, a.H / 8, 1.f / (float)a.H, a.eps, r.tpr, static_cast<uint4*>(a.h),
                    static_cast<uint4*>(a.y), a.rstd, static_cast<uint2*>(a.yq), a.yscale);
}

template <int VPT>
cudaError_t run_norm_q(int q, bool w32, const RowShape& r, const NormArgs& a, cudaStream_t s) {
  return q == kQGroup ? run_norm<VPT, kQGroup>(w32, r, a, s)
         : q == kQRow ? run_norm<VPT, kQRow>(w32, r, a, s)
                      : run_norm<VPT, kQNone>(w32, r, a, s);
}

struct BackArgs {
  const void *dy, *dh, *h;
  const float* hscale;  // h as codes, or NULL
  const float* rstd;
  const void* w;
  int T, H;
  void* dx;
  float* part;
};

template <int VPT, int S, int MAXT, int BPS, bool LAG, bool HQ>
cudaError_t run_backward(bool w32, const BackShape& r, const BackArgs& a, cudaStream_t stream) {
  auto k = w32 ? rmsnorm_backward_kernel<VPT, S, MAXT, BPS, LAG, true, HQ>
               : rmsnorm_backward_kernel<VPT, S, MAXT, BPS, LAG, false, HQ>;
  constexpr size_t kPerThread = (size_t)S * 3 * VPT * 16;  // >= 32 VPT: the rows' sums fit
  static std::atomic<unsigned long long> set[2];
  cudaError_t e = moe_raise_smem(k, kPerThread * MAXT, set[w32]);
  if (e != cudaSuccess) return e;
  const int threads = r.tpr * r.rpb;
  return moe_launch(k, dim3(r.grid), dim3(threads), kPerThread * threads, stream, 1,
                    static_cast<const uint4*>(a.dy), static_cast<const uint4*>(a.dh), a.h, a.hscale,
                    a.rstd, a.w, a.T, a.H / 8, 1.f / (float)a.H, r.tpr, static_cast<uint4*>(a.dx),
                    a.part);
}

template <bool HQ>
cudaError_t run_backward_of(bool w32, const BackShape& r, const BackArgs& a, cudaStream_t s) {
  switch (r.vpt) {  // 196 KB of ring per SM each
    case 1:
      return a.H <= 4096 ? run_backward<1, 4, 512, 2, true, HQ>(w32, r, a, s)
                         : run_backward<1, 4, 1024, 1, true, HQ>(w32, r, a, s);
    case 4: return run_backward<4, 2, 512, 1, false, HQ>(w32, r, a, s);
    default: return run_backward<8, 1, 512, 1, false, HQ>(w32, r, a, s);
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void* x, const void* residual, const void* w, bool w32, int T,
                               int H, float eps, void* h, void* y, float* rstd, void* yq,
                               float* yscale, int q_group, cudaStream_t stream) {
  const RowShape r = row_shape(T, H / 8);
  const int q = !yq ? kQNone : q_group ? kQGroup : kQRow;
  const NormArgs a{x, residual, w, T, H, eps, h, y, rstd, yq, yscale};
  switch (r.vpt) {
    case 1: return run_norm_q<1>(q, w32, r, a, stream);
    case 2: return run_norm_q<2>(q, w32, r, a, stream);
    case 3: return run_norm_q<3>(q, w32, r, a, stream);
    default: return run_norm_q<4>(q, w32, r, a, stream);
  }
}

size_t add_rmsnorm_backward_scratch_bytes(int T, int H) {
  const int rows = T > 0 ? back_shape(T, H / 8).grid : 1;
  return moe_align_up((size_t)rows * H * sizeof(float), 256);
}

cudaError_t launch_add_rmsnorm_backward(const void* dy, const void* dh, const void* h,
                                        const float* hscale, const float* rstd, const void* w,
                                        bool w32, int T, int H, void* dx, float* dweight,
                                        void* scratch, cudaStream_t stream) {
  float* part = static_cast<float*>(scratch);
  int rows = 0;
  if (T > 0) {
    const BackShape r = back_shape(T, H / 8);
    rows = r.grid;
    const BackArgs a{dy, dh, h, hscale, rstd, w, T, H, dx, part};
    const cudaError_t e =
        hscale ? run_backward_of<true>(w32, r, a, stream) : run_backward_of<false>(w32, r, a, stream);
    if (e != cudaSuccess) return e;
  }
  return moe_launch(column_sum_kernel, dim3(moe_cdiv(H, 32)), dim3(1024), 0, stream, 1,
                    (const float*)part, rows, H, dweight);
}
