// L: per-expert counts, load-balance loss and router z-loss of a batch, and
// the gradient of both -- with that of the routing weights and of the shared
// gate -- with respect to the router's logits.
//
// Tokens come as n_seq sequences of L = T / n_seq; a token mask leaves padding
// out.  With n_s the kept tokens of sequence s, S+ the sequences that keep
// any, N their sum, c_se the replicas of kept tokens sent to expert e:
//   p_te  = softmax(l_t)_e                      (mode 0)
//         = sigmoid(l_te) / sum_i sigmoid(l_ti) (mode 1)
//   f_se  = E c_se / (K n_s),  P_se = sum_t p_te / n_s
//   balance = (1/S+) sum_s sum_e f_se P_se     z = (1/N) sum_t lse_t^2
// A row whose E logits are all -inf has p = 0 and lse = 0.
//
// The counts carry no gradient, so with a_e = g_bal f_se / (n_s S+) a kept
// token's row is
//   dl_e = p_e (a_e - sum_i a_i p_i) [* (1 - sigmoid(l_e)) in mode 1]
//        + 2 g_z lse softmax(l)_e / N
// and its selected columns add w_k (g_k - sum_j w_j g_j / scale) [* (1 -
// sigmoid) in mode 1]: mode 0 is softmax over the selected logits (scale 1),
// mode 1 is scale * sigmoid / sum of the selected sigmoids.
//
// Memory bounds both where the batch is large: each row of logits is read once
// into registers (a group of LPR lanes per row, NPL columns per lane, the next
// row on its way) and used for every sum.  Measured on one GB300: losses T = 8 x
// 4096, E = 512, 41 % kept 13.5 us; losses and gradient T = 4 x 2048, E = 896,
// sigmoid, 39 % kept 23.4 us; T = 65536, E = 512 losses 29 us (71 % of the copy
// rate; 8.5 us of it are the launch, the first rows and the hand-over between
// blocks, the marginal rate is the copy's), gradient 54 us (76 %), of the routing
// weights alone 26 us (83 %).  Small batches are bound by latency, T = 2048,
// E = 128 losses 4.35 us; few experts by a token's fixed work, T = 2^20, E = 8
// losses 26 us (24 %), gradient 53 us (26 %).
// Determinism: a block's probability sums are fp32 in a fixed order; across
// blocks they are added as 64-bit fixed point, so the order does not matter.  A
// step is 2^-(61 - ceil(log2 L)), 2^-49 at L = 4096: half of one per block is the
// error, and a block's sum below that counts as 0.
#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"

namespace {

using namespace moe_f32x2;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kNegInf = -__builtin_huge_valf();

// all zero between calls
struct Scratch {
  unsigned long long* psum;  // [n_seq][E] fixed-point sums
  int32_t* cnt;              // [n_seq][E]
  unsigned long long* head;  // [n_seq]: blocks done << 48 | blocks with a NaN << 32 | kept tokens
  unsigned long long* done;  // sequences done
  float* zpart;              // [blocks] sums of lse^2
  float* bal_seq;            // [n_seq]
  float* z_seq;              // [n_seq]
};

template <int LPR>
MOE_DEVICE float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LPR>
MOE_DEVICE float group_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

constexpr float kLog2E = 1.4426950408889634f;

// Hardware 2^x (relative error about 2^-22; results below 2^-126 are 0) and
// 1 / x (about 2^-23).  As e^l, with the argument l log2(e) rounded to fp32, the
// error grows by about 2 |l| 2^-24; no reduction of the argument is spent on it,
// for at l = -30 that is 4e-6 of a value e^-30 of the row's largest.
MOE_DEVICE float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
MOE_DEVICE float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + e^-l): e^-l past the largest float makes it 0
MOE_DEVICE float sigmoid_fast(float l) { return rcp(1.f + ex2(-l * kLog2E)); }

// The rows' code is straight-line: the kernels are short, and instructions
// fetched for the first time cost more than those that a rare case would save.

// The lane's sum of e^(v[i] - m), which STORE leaves in v.
template <bool STORE, int NPL>
MOE_DEVICE float exp_row(float (&v)[NPL], float m) {
  float2 s = pair(0.f);
#pragma unroll
  for (int i = 0; i < NPL; i += 2) {
    const float2 x = mul2(add2(make_float2(v[i], v[i + 1]), pair(-m)), pair(kLog2E));
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    s = add2(s, e);
    if constexpr (STORE) {
      v[i] = e.x;
      v[i + 1] = e.y;
    }
  }
  return s.x + s.y;
}

// The row's maximum, 0 where that is -inf (no expert is left).
template <int LPR, int NPL>
MOE_DEVICE float row_max(const float (&v)[NPL]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < NPL; ++i) m = fmaxf(m, v[i]);
  m = group_max<LPR>(m);
  return m == kNegInf ? 0.f : m;
}

// What mode 1 adds to the logits of a row with maximum m: nothing, or where m
// lies below -60 what brings it there.  sigmoid(l) is e^l to 26 digits then, so
// the shift is a common factor of the row's sigmoids, which cancels in a ratio
// and keeps them from vanishing.
MOE_DEVICE float row_shift(float m) { return m < -60.f ? -(m + 60.f) : 0.f; }

// Mode 1: u[i] <- sigmoid(v[i] + row_shift).  Returns the lane's sum.
template <int NPL>
MOE_DEVICE float sigmoid_row(const float (&v)[NPL], float m, float (&u)[NPL]) {
  const float2 d = pair(row_shift(m));
  float2 s = pair(0.f);
#pragma unroll
  for (int i = 0; i < NPL; i += 2) {
    const float2 x = mul2(add2(make_float2(v[i], v[i + 1]), d), pair(-kLog2E));
    const float2 t = add2(make_float2(ex2(x.x), ex2(x.y)), pair(1.f));
    u[i] = rcp(t.x);
    u[i + 1] = rcp(t.y);
    s = add2(s, make_float2(u[i], u[i + 1]));
  }
  return s.x + s.y;
}

// Mode 1, gradient: x[i] <- u (1 - u) with u = sigmoid(v[i] + row_shift); adds u
// to s and a[column] u to dot.  1 - u is e^-l u for l > 0, never a difference of
// nearly equal numbers: where the balance loss alone reaches a column, its whole
// gradient has this factor (as 1.f - u it is off by up to 0.5 % at l = 12 and is 0
// past 17; here e^-l is at hand, so it takes no further special function).
template <int LPR, int NPL, bool FULL>
MOE_DEVICE void sigmoid_slope_row(const float (&v)[NPL], float m, const float* a, int E, int lig,
                                  float (&x)[NPL], float& s, float& dot) {
  const float2 d = pair(row_shift(m));
  float2 sum = pair(0.f);
#pragma unroll
  for (int i = 0; i < NPL; i += 2) {
    const float2 n = mul2(add2(make_float2(v[i], v[i + 1]), d), pair(-kLog2E));
    const float2 e = make_float2(ex2(n.x), ex2(n.y));
    const float2 t = add2(e, pair(1.f));
    const float2 u = make_float2(rcp(t.x), rcp(t.y));
    sum = add2(sum, u);
    if (FULL || lig + LPR * i < E) dot = fmaf(a[lig + LPR * i], u.x, dot);
    if (FULL || lig + LPR * (i + 1) < E) dot = fmaf(a[lig + LPR * (i + 1)], u.y, dot);
    const float2 eu = mul2(e, u);
    x[i] = u.x * (n.x < 0.f ? eu.x : 1.f - u.x);
    x[i + 1] = u.y * (n.y < 0.f ? eu.y : 1.f - u.y);
  }
  s += sum.x + sum.y;
}

// 1 / s, 0 for an empty row's sum
MOE_DEVICE float inverse(float s) { return s == 0.f ? 0.f : rcp(s); }

// A row's columns lig + LPR*i, -inf past E and where the row is not `on`.
// FULL: E == LPR * NPL, no column is missing.
template <int LPR, int NPL, bool FULL>
MOE_DEVICE void load_row(const float* __restrict__ row, int E, int lig, bool on, float (&v)[NPL]) {
  if (on) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      v[i] = FULL || lig + LPR * i < E ? __ldg(row + lig + LPR * i) : kNegInf;
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = kNegInf;
  }
}

MOE_DEVICE unsigned long long add_acq_rel(unsigned long long* p, unsigned long long v) {
  unsigned long long old;
  asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], %2;" : "=l"(old) : "l"(p), "l"(v) : "memory");
  return old;
}

// Sums of a pair over the block; `red` is free again after the next barrier.
template <typename A, typename B>
struct Pair {
  A a;
  B b;
};
template <typename A, typename B>
MOE_DEVICE void block_sums(Pair<A, B>* red, A& a, B& b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (lane_id() == 0) red[warp_id()] = {a, b};
  __syncthreads();
  a = red[0].a;
  b = red[0].b;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    a += red[w].a;
    b += red[w].b;
  }
}

// Blocks per SM that the registers of a row pair (this row and the next one,
// loaded ahead) allow; the grid is that many per SM.  The gradient holds a
// third row, and with few lanes per row several replicas per lane.
constexpr int blocks_per_sm(int npl) { return npl <= 8 ? 4 : npl <= 16 ? 3 : 2; }
constexpr int back_blocks_per_sm(int lpr, int npl) {
  return npl <= 4 ? 4 : npl <= 8 && lpr == 32 ? 4 : npl <= 16 ? 3 : 2;
}

// ---------------------------------------------------------------- forward
// Block b takes every chunks-th pass of kStep rows of sequence b / chunks, from
// pass b % chunks on, so that padding at a sequence's end is spread over its
// blocks.  The last block of a sequence to finish turns its sums into outputs,
// and the last sequence's block the sequences' losses into the batch's.  A
// sequence of one block, and a batch of one sequence, skip the hand-over
// through global memory.
template <int LPR, int NPL, int MODE, bool FULL>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(NPL))
balance_kernel(const float* __restrict__ logits, int ld, const int32_t* __restrict__ ids,
               const uint8_t* __restrict__ mask, int L, int E, int K, int n_seq, int chunks,
               int shift, Scratch sc, int32_t* __restrict__ counts,
               float* __restrict__ mean_prob, int32_t* __restrict__ valid,
               float* __restrict__ losses, int32_t* __restrict__ dev_status) {
  constexpr int RPW = 32 / LPR;
  constexpr int KPL = NPL < 32 / LPR ? NPL : 32 / LPR;  // replicas per lane, K <= min(E, 32)
  constexpr int kStep = kWarps * RPW;
  extern __shared__ float smem[];
  float* psm = smem;                                              // [kWarps][E]
  int32_t* hist = reinterpret_cast<int32_t*>(smem + kWarps * E);  // [E]
  __shared__ Pair<float, int> fired[kWarps];
  __shared__ Pair<float, float> ffred[kWarps];
  __shared__ Pair<int, int> iired[kWarps];
  __shared__ int bad, last;
  __shared__ unsigned long long total_s;
  const int seq = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int stride = chunks * kStep;
  const size_t t0 = (size_t)seq * L;
  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  auto some = [&](int j) { return j == 0 || LPR * j < K; };  // the warp has a replica LPR*j + ...
  const int lig = lane % LPR, sub = lane / LPR;
  for (int e = tid; e < E; e += kThreads) hist[e] = 0;
  if (tid == 0) bad = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();

  // this row, the next one's logits and ids and the one after's mask are in
  // flight
  const uint8_t* mrow = mask ? mask + t0 : nullptr;
  auto kept_row = [&](int r) { return r < L && (!mrow || __ldg(mrow + r)); };
  auto load = [&](int r, bool on, float(&v)[NPL], int(&id)[KPL]) {
    load_row<LPR, NPL, FULL>(logits + (t0 + r) * ld, E, lig, on, v);
#pragma unroll
    for (int j = 0; j < KPL; ++j)
      if (some(j)) id[j] = on && lig + LPR * j < K ? __ldg(ids + (t0 + r) * K + lig + LPR * j) : 0;
  };
  const int rw = chunk * kStep + warp * RPW;
  int r = rw + sub;
  bool on = kept_row(r), on1 = kept_row(r + stride);

  float acc[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) acc[i] = 0.f;
  float z = 0.f, keep_m = 0.f, keep_s = 0.f;
  int kept = 0, it = 0;
  bool nan = false;
  // the logarithms of LPR rows at a time, one per lane of the row's group
  auto add_z = [&]() {
    const float lse = keep_s == 0.f ? 0.f : keep_m + logf(keep_s);
    z = fmaf(lse, lse, z);
    keep_s = 0.f;
  };
  float v[NPL];
  int id[KPL];
  load(r, on, v, id);
#pragma unroll 1
  for (int rb = rw; rb < L; rb += stride) {
    float nx[NPL];
    int idn[KPL];
    load(r + stride, on1, nx, idn);
    const bool on2 = kept_row(r + 2 * stride);
    if (__any_sync(0xffffffffu, on)) {  // else the warp's rows are padding
      const float m = row_max<LPR, NPL>(v);
      float s, inv;
      if constexpr (MODE == MOE_SCORE_SOFTMAX_RENORM) {
        s = group_sum<LPR>(exp_row<true>(v, m));
        inv = inverse(s);
      } else {
        s = group_sum<LPR>(exp_row<false>(v, m));
        inv = inverse(group_sum<LPR>(sigmoid_row(v, m, v)));
      }
      // a row left out is all -inf and adds zeros
#pragma unroll
      for (int i = 0; i < NPL; i += 2) {
        const float2 x = fma2(make_float2(v[i], v[i + 1]), pair(inv), make_float2(acc[i], acc[i + 1]));
        acc[i] = x.x;
        acc[i + 1] = x.y;
      }
      if (on) {
        if (lig == it % LPR) {
          keep_m = m;
          keep_s = s;
          ++kept;
        }
        nan |= !(inv == inv);
#pragma unroll
        for (int j = 0; j < KPL; ++j)
          if (some(j) && lig + LPR * j < K) {
            if ((unsigned)id[j] < (unsigned)E) atomicAdd(&hist[id[j]], 1);
            else moe_set_status(dev_status, MOE_DEV_BAD_EXPERT_ID);
          }
      }
    }
    if (++it % LPR == 0) add_z();
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = nx[i];
#pragma unroll
    for (int j = 0; j < KPL; ++j) id[j] = idn[j];
    on = on1;
    on1 = on2;
    r += stride;
  }
  add_z();
  // the warp's rows, then the block's warps in order
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    float s = acc[i];
#pragma unroll
    for (int o = 16; o >= LPR; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int c = lig + LPR * i;
    if (sub == 0 && (FULL || c < E)) psm[warp * E + c] = s;
  }
  if (nan) bad = 1;
  int nv = kept;
  block_sums(fired, z, nv);  // its barrier also publishes psm, hist and bad
  bool poisoned = bad;
  auto block_prob = [&](int e) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += psm[w * E + e];
    return s;
  };

  unsigned long long* head = sc.head + seq;
  if (chunks > 1) {
    const float fix = __int_as_float((shift + 127) << 23);  // 2^shift
    for (int e = tid; e < E; e += kThreads) {
      const float s = block_prob(e);
      if (s > 0.f)
        atomicAdd(sc.psum + (size_t)seq * E + e, (unsigned long long)__float2ll_rn(s * fix));
      if (hist[e]) atomicAdd(sc.cnt + (size_t)seq * E + e, hist[e]);
    }
    if (tid == 0) sc.zpart[blockIdx.x] = z;
    __syncthreads();
    if (tid == 0) {  // one thread's release and acquire order the block's work, by the barriers
      const unsigned long long mine =
          1ull << 48 | (unsigned long long)poisoned << 32 | (unsigned)nv;
      total_s = add_acq_rel(head, mine) + mine;
    }
    __syncthreads();
    if (total_s >> 48 != (unsigned)chunks) return;
    nv = (int)(uint32_t)total_s;
    poisoned = (total_s >> 32 & 0xffff) != 0;
  }

  // last block of the sequence: its outputs and its share of the losses
  const float poison = poisoned ? __int_as_float(0x7fffffff) : 0.f;
  const float inv_n = nv ? 1.f / (float)nv : 0.f;
  float part = 0.f;
  if (chunks > 1) {
    constexpr int kPer = (LPR * NPL + kThreads - 1) / kThreads;  // experts per thread
    constexpr int kZ = 3;                                        // blocks per thread, as a rule
    unsigned long long ps[kPer];
    int c[kPer];
    float zp[kZ];
    float* zrow = sc.zpart + (size_t)seq * chunks;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid + i * kThreads;
      const size_t o = (size_t)seq * E + e;
      ps[i] = e < E ? __ldcg(sc.psum + o) : 0ull;
      c[i] = e < E ? __ldcg(sc.cnt + o) : 0;
    }
#pragma unroll
    for (int i = 0; i < kZ; ++i) zp[i] = tid + i * kThreads < chunks ? __ldcg(zrow + tid + i * kThreads) : 0.f;
    const float unfix = __int_as_float((127 - shift) << 23);  // 2^-shift
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid + i * kThreads;
      if (e >= E) continue;
      const size_t o = (size_t)seq * E + e;
      const float p = __ull2float_rn(ps[i]) * unfix * inv_n;
      counts[o] = c[i];
      mean_prob[o] = p + poison;
      part = fmaf((float)c[i], p, part);
      sc.cnt[o] = 0;
      sc.psum[o] = 0;
    }
    z = 0.f;
#pragma unroll
    for (int i = 0; i < kZ; ++i) z += zp[i];
    for (int i = tid + kZ * kThreads; i < chunks; i += kThreads) z += __ldcg(zrow + i);
    for (int i = tid; i < chunks; i += kThreads) zrow[i] = 0.f;
  } else {
    for (int e = tid; e < E; e += kThreads) {
      const size_t o = (size_t)seq * E + e;
      const float p = block_prob(e) * inv_n;
      counts[o] = hist[e];
      mean_prob[o] = p + poison;
      part = fmaf((float)hist[e], p, part);
    }
  }
  if (chunks == 1 && tid != 0) z = 0.f;  // the block's sum already
  block_sums(ffred, part, z);
  const float bal = part * ((float)E / (float)K) * inv_n + poison;
  if (n_seq == 1) {
    if (tid == 0) {
      losses[0] = bal;
      losses[1] = z * inv_n;
      valid[0] = valid[1] = nv;
      valid[2] = nv > 0;
      if (chunks > 1) *head = 0;
    }
    return;
  }
  if (tid == 0) {
    sc.bal_seq[seq] = bal;
    sc.z_seq[seq] = z;
    valid[seq] = nv;
    if (chunks > 1) *head = 0;
    last = add_acq_rel(sc.done, 1ull) == (unsigned long long)(n_seq - 1);
  }
  __syncthreads();
  if (!last) return;

  // last sequence of all: the two losses
  float b = 0.f, zz = 0.f;
  int total = 0, full = 0;
  for (int s = tid; s < n_seq; s += kThreads) {
    const int n = __ldcg(valid + s);
    b += __ldcg(sc.bal_seq + s);
    zz += __ldcg(sc.z_seq + s);
    total += n;
    full += n > 0;
    sc.bal_seq[s] = sc.z_seq[s] = 0.f;
  }
  __syncthreads();
  block_sums(ffred, b, zz);
  block_sums(iired, total, full);
  if (tid == 0) {
    losses[0] = full > 0 ? b / (float)full : 0.f;
    losses[1] = total > 0 ? zz / (float)total : 0.f;
    valid[n_seq] = total;
    valid[n_seq + 1] = full;
    *sc.done = 0;
  }
}

// T = 0: nothing kept
__global__ void balance_empty_kernel(int E, int n_seq, int32_t* __restrict__ counts,
                                     float* __restrict__ mean_prob, int32_t* __restrict__ valid,
                                     float* __restrict__ losses) {
  pdl_wait();
  pdl_trigger();
  const long long n = (long long)n_seq * E, all = max(n, n_seq + 2ll);
  const long long step = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += step) {
    if (i < n) {
      counts[i] = 0;
      mean_prob[i] = 0.f;
    }
    if (i < n_seq + 2ll) valid[i] = 0;
    if (i < 2) losses[i] = 0.f;
  }
}

// ---------------------------------------------------------------- backward
// Row stride of the per-row buffers in shared memory: the rows of a warp fall
// into different banks.
__host__ __device__ constexpr int buf_stride(int E, int lpr) { return (E + 31) / 32 * 32 + lpr; }

// AUX: with the losses' gradient (reads the whole row of logits).
template <int LPR, int NPL, int MODE, bool AUX, bool FULL>
__global__ void __launch_bounds__(kThreads, back_blocks_per_sm(LPR, NPL))
route_backward_kernel(RouteBackwardArgs a, int L, int chunks) {
  constexpr int RPW = 32 / LPR;
  constexpr int KPL = NPL < 32 / LPR ? NPL : 32 / LPR;  // replicas per lane, K <= min(E, 32)
  constexpr int kStep = kWarps * RPW;
  constexpr bool kSigmoid = MODE != MOE_SCORE_SOFTMAX_RENORM;
  constexpr bool kEarly = kSigmoid && AUX && KPL == 1;  // the selected logit loaded ahead of its use
  extern __shared__ float smem[];
  const int E = a.E, K = a.K;
  const int warp = warp_id(), lane = lane_id();
  const int lig = lane % LPR, sub = lane / LPR;
  const bool routing = a.d_weights != nullptr;
  auto some = [&](int j) { return j == 0 || LPR * j < K; };
  // a_e of this sequence (AUX), then the row's routing gradient, zero between rows
  float* buf = smem + (AUX ? E : 0) + (size_t)(warp * RPW + sub) * buf_stride(E, LPR);
  const int seq = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int stride = chunks * kStep;
  const size_t t0 = (size_t)seq * L;
  if (routing)
    for (int c = lig; c < E; c += LPR) buf[c] = 0.f;
  pdl_wait();
  pdl_trigger();

  const uint8_t* mrow = a.mask ? a.mask + t0 : nullptr;
  auto kept_row = [&](int r) { return r < L && (!mrow || __ldg(mrow + r)); };
  const int rw = chunk * kStep + warp * RPW;
  int r = rw + sub;
  bool on = kept_row(r), on1 = kept_row(r + stride);
  float v[NPL];
  if constexpr (AUX) load_row<LPR, NPL, FULL>(a.logits + (t0 + r) * a.ld, E, lig, on, v);

  float gz = 0.f;
  if constexpr (AUX) {
    const int nv = __ldg(a.valid + seq), total = __ldg(a.valid + a.n_seq),
              full = __ldg(a.valid + a.n_seq + 1);
    gz = total > 0 ? 2.f * __ldg(a.grad_losses + 1) / (float)total : 0.f;
    const float k = nv > 0 ? __ldg(a.grad_losses) * (float)E / ((float)K * (float)nv) /
                                 ((float)nv * (float)full)
                           : 0.f;
    for (int e = threadIdx.x; e < E; e += kThreads)
      smem[e] = k * (float)__ldg(a.counts + (size_t)seq * E + e);
  }
  const float inv_scale = !kSigmoid ? 1.f : a.scale != 0.f ? 1.f / a.scale : 0.f;
  __syncthreads();

#pragma unroll 1
  for (int rb = rw; rb < L; rb += stride) {
    float nx[NPL];
    if constexpr (AUX)
      load_row<LPR, NPL, FULL>(a.logits + (t0 + r + stride) * a.ld, E, lig, on1, nx);
    const bool on2 = kept_row(r + 2 * stride);
    const size_t t = t0 + r;
    const bool in = r < L;
    float* out = a.dlogits + t * a.ld_d;
    if (!__any_sync(0xffffffffu, on)) {  // the warp's rows are padding
      if (in) {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (FULL || lig + LPR * i < E) out[lig + LPR * i] = 0.f;
        if (a.d_shared_gate && lig == 0) out[E] = 0.f;
      }
    } else {
    int id[KPL];
    float wk[KPL], gk[KPL], lk = 0.f;
    if (routing) {
#pragma unroll
      for (int j = 0; j < KPL; ++j) {
        if (!some(j)) continue;
        const int k = lig + LPR * j;
        const bool have = on && k < K;
        id[j] = have ? __ldg(a.ids + t * K + k) : -1;
        wk[j] = have ? __ldg(a.weights + t * K + k) : 0.f;
        gk[j] = have ? __ldg(a.d_weights + t * K + k) : 0.f;
      }
    }
    // mode 0: e^(v - max); mode 1: u (1 - u) of the shifted sigmoids u
    float x[NPL];
    float m = 0.f, lse = 0.f, inv = 0.f, inv_exp = 0.f, dot = 0.f;
    if constexpr (AUX) {
      m = row_max<LPR, NPL>(v);
      if constexpr (!kSigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) x[i] = v[i];
      }
      if (!kSigmoid || gz != 0.f) {
        const float s = group_sum<LPR>(kSigmoid ? exp_row<false>(v, m) : exp_row<true>(x, m));
        lse = s == 0.f ? 0.f : m + logf(s);
        inv_exp = inverse(s);
      }
      if constexpr (kSigmoid) {
        float s = 0.f;
        sigmoid_slope_row<LPR, NPL, FULL>(v, m, smem, E, lig, x, s, dot);
        inv = inverse(group_sum<LPR>(s));
      } else {
        inv = inv_exp;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (FULL || lig + LPR * i < E) dot = fmaf(smem[lig + LPR * i], x[i], dot);
      }
      if constexpr (kEarly)
        if (routing && (unsigned)id[0] < (unsigned)E) lk = __ldg(a.logits + t * a.ld + id[0]);
      dot = group_sum<LPR>(dot) * inv;
    }
    if (routing) {
      float wg = 0.f;
      bool lost = false;
      int* tag = reinterpret_cast<int*>(buf);
#pragma unroll
      for (int j = 0; j < KPL; ++j) {
        if (!some(j)) continue;
        if (on && lig + LPR * j < K && (unsigned)id[j] >= (unsigned)E) {
          moe_set_status(a.dev_status, MOE_DEV_BAD_EXPERT_ID);
          id[j] = -1;
        }
        wg = fmaf(wk[j], gk[j], wg);
        if (id[j] >= 0) tag[id[j]] = lig + LPR * j + 1;
      }
      wg = group_sum<LPR>(wg) * inv_scale;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < KPL; ++j) {
        if (!some(j)) continue;
        gk[j] = wk[j] * (gk[j] - wg);
        if (id[j] < 0) continue;
        lost |= tag[id[j]] != lig + LPR * j + 1;
        // 1 - sigmoid of a selected expert: small as a rule, so not as a difference
        if constexpr (kSigmoid) gk[j] *= sigmoid_fast(-(kEarly ? lk : __ldg(a.logits + t * a.ld + id[j])));
      }
      // top-K gives distinct ids: every replica found its own tag and the
      // values go out together; a repeated id adds up in k order instead
      if (!__any_sync(0xffffffffu, lost)) {
#pragma unroll
        for (int j = 0; j < KPL; ++j)
          if (some(j) && id[j] >= 0) buf[id[j]] = gk[j];
      } else {
#pragma unroll
        for (int j = 0; j < KPL; ++j)
          if (some(j) && id[j] >= 0) buf[id[j]] = 0.f;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < KPL; ++j)
          for (int o = 0; o < LPR && LPR * j + o < K; ++o) {
            if (lig == o && id[j] >= 0) buf[id[j]] += gk[j];
            __syncwarp();
          }
      }
      __syncwarp();
    }
    // mode 0: p (a - dot) = x (a inv - dot inv), and the z-loss's p zl joins it;
    // mode 1: p (a - dot) (1 - u) likewise
    const float zl = gz != 0.f ? gz * lse : 0.f;
    const float shift = kSigmoid ? -dot * inv : (zl - dot) * inv;
    const float zq = zl * inv_exp;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int c = lig + LPR * i;
      if (!FULL && c >= E) continue;
      float d = routing ? buf[c] : 0.f;
      if constexpr (AUX && !kSigmoid) {
        d = fmaf(x[i], fmaf(smem[c], inv, shift), d);
      } else if constexpr (AUX) {
        d = fmaf(x[i], fmaf(smem[c], inv, shift), d);
        if (gz != 0.f) d = fmaf(zq, ex2((v[i] - m) * kLog2E), d);
      }
      if (RPW == 1 || in) out[c] = RPW == 1 || on ? d : 0.f;
    }
    if (routing) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < KPL; ++j)
        if (some(j) && id[j] >= 0) buf[id[j]] = 0.f;
      __syncwarp();
    }
    if (a.d_shared_gate && in && lig == 0) {
      float g = 0.f;
      if (on) {
        const float l = __ldg(a.logits + t * a.ld + E);
        const float ea = expf(-fabsf(l));
        const float q = 1.f / (1.f + ea);
        g = __ldg(a.d_shared_gate + t) * (ea * q * q);
      }
      out[E] = g;
    }
    }
    if constexpr (AUX) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) v[i] = nx[i];
    }
    on = on1;
    on1 = on2;
    r += stride;
  }
}

// ---------------------------------------------------------------- shapes
// Calls f<LPR, NPL, FULL> for E: lanes per row and columns per lane, so that a
// row never takes more lanes than it can feed and a lane never more than 32
// columns.  E = 896 has its own tier, as in the top-K.  For 64 < E <= 128 the
// losses run faster with 8 lanes (T = 2^18, E = 128: 30 us, 35 with 16) and the
// gradient, which holds more rows in registers, with 16 (59 us, 68 with 8).
#define MOE_TIER(f, E, LPR, NPL, ...)                                        \
  if ((E) <= LPR * NPL)                                                      \
    return (E) == LPR * NPL ? f<LPR, NPL, true>(__VA_ARGS__) : f<LPR, NPL, false>(__VA_ARGS__);
#define MOE_BY_SHAPE(f, E, LPR128, LPR256, ...)    \
  MOE_TIER(f, E, 4, 4, __VA_ARGS__)                \
  MOE_TIER(f, E, 8, 4, __VA_ARGS__)                \
  MOE_TIER(f, E, 8, 8, __VA_ARGS__)                \
  MOE_TIER(f, E, LPR128, 128 / LPR128, __VA_ARGS__) \
  MOE_TIER(f, E, LPR256, 256 / LPR256, __VA_ARGS__) \
  MOE_TIER(f, E, 32, 16, __VA_ARGS__)              \
  MOE_TIER(f, E, 32, 28, __VA_ARGS__)              \
  return (E) == 1024 ? f<32, 32, true>(__VA_ARGS__) : f<32, 32, false>(__VA_ARGS__);

// `blocks` per SM over all sequences, at least one pass of the block's warps
// each; a fixed SM count, so that the scratch size does not depend on which
// device is current.  (Losses: one wave.  Their blocks add to the same E sums,
// so twice as many cost T = 32768, E = 512 18.6 -> 22.5 us; a third as many of 24
// warps gained nothing there and lost 3 us on padded batches.)
constexpr int kGridSms = 152;
int chunks_of(int L, int n_seq, int lpr, int blocks) {
  const int passes = moe_cdiv(L, kWarps * (32 / lpr));
  const int wave = blocks * kGridSms / n_seq;
  return passes < wave ? passes : wave > 0 ? wave : 1;
}

Scratch scratch_of(void* p, int E, int n_seq, int blocks, size_t* bytes) {
  char* b = static_cast<char*>(p);
  size_t off = 0;
  auto take = [&](size_t n) {
    char* r = b + off;
    off = moe_align_up(off + n, 256);
    return r;
  };
  Scratch s;
  const size_t se = (size_t)n_seq * E;
  s.psum = reinterpret_cast<unsigned long long*>(take(se * 8));
  s.cnt = reinterpret_cast<int32_t*>(take(se * 4));
  s.head = reinterpret_cast<unsigned long long*>(take((size_t)n_seq * 8));
  s.done = reinterpret_cast<unsigned long long*>(take(8));
  s.zpart = reinterpret_cast<float*>(take((size_t)blocks * 4));
  s.bal_seq = reinterpret_cast<float*>(take((size_t)n_seq * 4));
  s.z_seq = reinterpret_cast<float*>(take((size_t)n_seq * 4));
  if (bytes) *bytes = off;
  return s;
}

struct BalanceArgs {
  const float* logits;
  int ld;
  const int32_t* ids;
  const uint8_t* mask;
  int T, E, K, n_seq, mode;
  void* scratch;
  int32_t* counts;
  float* mean_prob;
  int32_t* valid;
  float* losses;
  int32_t* dev_status;
};

template <int LPR, int NPL, bool FULL>
cudaError_t run_balance(const BalanceArgs& a, cudaStream_t stream) {
  const int L = a.T / a.n_seq;
  const int chunks = chunks_of(L, a.n_seq, LPR, blocks_per_sm(NPL));
  const Scratch s = scratch_of(a.scratch, a.E, a.n_seq, a.n_seq * chunks, nullptr);
  // L probabilities of at most 1 sum to at most 2^bits, so 2^61 in fixed point
  int bits = 0;
  while (bits < 31 && (1ll << bits) < L) ++bits;
  const size_t smem = (size_t)(kWarps + 1) * a.E * 4;
  auto k = a.mode == MOE_SCORE_SOFTMAX_RENORM
               ? balance_kernel<LPR, NPL, MOE_SCORE_SOFTMAX_RENORM, FULL>
               : balance_kernel<LPR, NPL, MOE_SCORE_SIGMOID_BIAS_SCALED, FULL>;
  return moe_launch(k, dim3(a.n_seq * chunks), dim3(kThreads), smem, stream, 1, a.logits, a.ld,
                    a.ids, a.mask, L, a.E, a.K, a.n_seq, chunks, 61 - bits, s, a.counts,
                    a.mean_prob, a.valid, a.losses, a.dev_status);
}

template <int LPR, int NPL, bool FULL>
int chunks_of_shape(int L, int n_seq) {
  return chunks_of(L, n_seq, LPR, blocks_per_sm(NPL));
}
int loss_chunks(int L, int n_seq, int E) { MOE_BY_SHAPE(chunks_of_shape, E, 8, 16, L, n_seq) }

template <int LPR, int NPL, bool FULL>
cudaError_t run_route_backward(const RouteBackwardArgs& a, cudaStream_t stream) {
  const int L = a.T / a.n_seq;
  const bool aux = a.grad_losses != nullptr;
  // without the losses a row is a few loads and many stores, which three waves
  // of blocks overlap (weights alone, T = 32768: E = 512 17.6 -> 14.3 us, E = 896
  // 27.2 -> 22.9; with the losses one wave is better, 29.1 against 30.4)
  const int chunks = chunks_of(L, a.n_seq, LPR, (aux ? 1 : 3) * back_blocks_per_sm(LPR, NPL));
  const size_t smem =
      4 * ((aux ? a.E : 0) +
           (a.d_weights ? (size_t)kWarps * (32 / LPR) * buf_stride(a.E, LPR) : 0));
  constexpr int S0 = MOE_SCORE_SOFTMAX_RENORM, S1 = MOE_SCORE_SIGMOID_BIAS_SCALED;
  auto k = a.mode == S0 ? (aux ? route_backward_kernel<LPR, NPL, S0, true, FULL>
                               : route_backward_kernel<LPR, NPL, S0, false, false>)
                        : (aux ? route_backward_kernel<LPR, NPL, S1, true, FULL>
                               : route_backward_kernel<LPR, NPL, S1, false, false>);
  return moe_launch(k, dim3(a.n_seq * chunks), dim3(kThreads), smem, stream, 1, a, L, chunks);
}

}  // namespace

size_t balance_loss_scratch_bytes(int T, int E, int n_seq) {
  const int chunks = T > 0 ? loss_chunks(T / n_seq, n_seq, E) : 1;
  size_t bytes = 0;
  scratch_of(nullptr, E, n_seq, n_seq * chunks, &bytes);
  return bytes;
}

cudaError_t launch_balance_loss(const float* logits, int ld, const int32_t* ids,
                                const uint8_t* mask, int T, int E, int K, int n_seq, int mode,
                                int32_t* counts, float* mean_prob, int32_t* valid, float* losses,
                                void* scratch, int32_t* dev_status, cudaStream_t stream) {
  if (T == 0) {
    const long long n = (long long)n_seq * E;
    const int grid = (int)((n + 255) / 256 < 1024 ? (n + 255) / 256 : 1024);
    return moe_launch(balance_empty_kernel, dim3(grid), dim3(256), 0, stream, 1, E, n_seq, counts,
                      mean_prob, valid, losses);
  }
  const BalanceArgs a{logits, ld,      ids,    mask,      T,     E,      K,         n_seq,
                      mode,   scratch, counts, mean_prob, valid, losses, dev_status};
  MOE_BY_SHAPE(run_balance, E, 8, 16, a, stream)
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t stream) {
  MOE_BY_SHAPE(run_route_backward, a.E, 16, 32, a, stream)
}
