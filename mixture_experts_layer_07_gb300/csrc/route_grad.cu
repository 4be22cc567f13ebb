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
// Memory bounds both: each row of logits is read once into registers (a group
// of LPR lanes per row, NPL columns per lane) and used for every sum.
// Determinism: a block's probability sums are fp32 in a fixed order; across
// blocks they are added as 64-bit fixed point, so the order does not matter.
#include "common.cuh"
#include "internal.h"

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kNegInf = -__builtin_huge_valf();

// all zero between calls
struct Scratch {
  unsigned long long* psum;  // [n_seq][E] fixed-point sums
  int32_t* cnt;              // [n_seq][E]
  uint32_t* head;            // [n_seq][4]: kept tokens, any NaN, blocks done, unused
  uint32_t* done;            // sequences done
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

// What a row's logits turn into (-inf past E): its probabilities, log-sum-exp
// (0 for a row of -inf) and sum of exponentials relative to the maximum.
template <int NPL>
struct Row {
  float p[NPL];
  float lse, sum;
};

// sigmoid(l) * exp(c), c = max(0, -row maximum): the common factor cancels in
// p and keeps rows of very negative logits from vanishing
MOE_DEVICE float scaled_sigmoid(float l, float c) {
  const float a = __expf(-fabsf(l));
  return (l > 0.f ? 1.f : expf(l + c)) / (1.f + a);  // l > 0 makes c 0
}

// 1 - sigmoid(l)
MOE_DEVICE float sigmoid_tail(float l) {
  const float a = __expf(-fabsf(l));
  return (l > 0.f ? a : 1.f) / (1.f + a);
}

template <int LPR, int NPL, int MODE>
MOE_DEVICE void row_probs(const float (&v)[NPL], Row<NPL>& r) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < NPL; ++i) m = fmaxf(m, v[i]);
  m = group_max<LPR>(m);
  if (m == kNegInf) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    r.p[i] = expf(v[i] - m);
    s += r.p[i];
  }
  s = group_sum<LPR>(s);
  r.sum = s;
  r.lse = s == 0.f ? 0.f : m + logf(s);
  if constexpr (MODE == MOE_SCORE_SOFTMAX_RENORM) {
    const float inv = s == 0.f ? 0.f : 1.f / s;
#pragma unroll
    for (int i = 0; i < NPL; ++i) r.p[i] *= inv;
  } else {
    const float c = fmaxf(0.f, -m);
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      r.p[i] = scaled_sigmoid(v[i], c);
      q += r.p[i];
    }
    q = group_sum<LPR>(q);
    const float inv = q == 0.f ? 0.f : 1.f / q;
#pragma unroll
    for (int i = 0; i < NPL; ++i) r.p[i] *= inv;
  }
}

template <int LPR, int NPL>
MOE_DEVICE void load_row(const float* __restrict__ row, int E, int lig, bool on, float (&v)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int c = lig + LPR * i;
    v[i] = on && c < E ? __ldg(row + c) : kNegInf;
  }
}

// ---------------------------------------------------------------- forward
// Block b takes chunk b % chunks of sequence b / chunks.
template <int LPR, int NPL, int MODE>
__global__ void __launch_bounds__(kThreads)
balance_kernel(const float* __restrict__ logits, int ld, const int32_t* __restrict__ ids,
               const uint8_t* __restrict__ mask, int L, int E, int K, int n_seq, int chunks,
               int rows_per_block, int shift, Scratch sc, int32_t* __restrict__ counts,
               float* __restrict__ mean_prob, int32_t* __restrict__ valid,
               float* __restrict__ losses, int32_t* __restrict__ dev_status) {
  constexpr int RPW = 32 / LPR;
  extern __shared__ float smem[];
  float* psm = smem;                                              // [kWarps][E]
  int32_t* hist = reinterpret_cast<int32_t*>(smem + kWarps * E);  // [E]
  __shared__ float zred[kWarps];
  __shared__ int nred[kWarps];
  __shared__ int bad, last;
  __shared__ double dred[2][kWarps];
  pdl_wait();
  pdl_trigger();
  const int seq = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int r0 = chunk * rows_per_block;
  const int r1 = min(L, r0 + rows_per_block);
  const size_t t0 = (size_t)seq * L;
  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int lig = lane % LPR, sub = lane / LPR;
  for (int e = tid; e < E; e += kThreads) hist[e] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();

  for (int i = tid; i < (r1 - r0) * K; i += kThreads) {
    const size_t t = t0 + r0 + i / K;
    if (mask && !__ldg(mask + t)) continue;
    const int id = __ldg(ids + (t0 + r0) * K + i);
    if ((unsigned)id < (unsigned)E) atomicAdd(&hist[id], 1);
    else moe_set_status(dev_status, MOE_DEV_BAD_EXPERT_ID);
  }

  float acc[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) acc[i] = 0.f;
  float z = 0.f;
  int kept = 0;
  bool nan = false;
  for (int rb = r0 + warp * RPW; rb < r1; rb += kWarps * RPW) {
    const int r = rb + sub;
    const size_t t = t0 + r;
    const bool on = r < r1 && (!mask || __ldg(mask + t));
    float v[NPL];
    load_row<LPR, NPL>(logits + t * ld, E, lig, on, v);
    Row<NPL> w;
    row_probs<LPR, NPL, MODE>(v, w);
    if (on) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) acc[i] += w.p[i];
      if (lig == 0) {
        z = fmaf(w.lse, w.lse, z);
        ++kept;
      }
      nan |= !(w.p[0] == w.p[0]);
    }
  }
  // the warp's rows, then the block's warps in order
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    float s = acc[i];
#pragma unroll
    for (int o = 16; o >= LPR; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int c = lig + LPR * i;
    if (sub == 0 && c < E) psm[warp * E + c] = s;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    kept += __shfl_xor_sync(0xffffffffu, kept, o);
  }
  if (lane == 0) {
    zred[warp] = z;
    nred[warp] = kept;
  }
  if (nan) bad = 1;
  __syncthreads();
  const float fix = __int_as_float((shift + 127) << 23);  // 2^shift
  for (int e = tid; e < E; e += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += psm[w * E + e];
    if (s > 0.f)
      atomicAdd(sc.psum + (size_t)seq * E + e, (unsigned long long)__float2ll_rn(s * fix));
    if (hist[e]) atomicAdd(sc.cnt + (size_t)seq * E + e, hist[e]);
  }
  uint32_t* head = sc.head + (size_t)seq * 4;
  if (tid == 0) {
    float s = 0.f;
    int n = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      s += zred[w];
      n += nred[w];
    }
    sc.zpart[blockIdx.x] = s;
    atomicAdd(head, (uint32_t)n);
    if (bad) atomicOr(head + 1, 1u);
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(head + 2, 1u) == (uint32_t)(chunks - 1);
  __syncthreads();
  if (!last) return;

  // last block of the sequence: its outputs and its share of the losses
  __threadfence();
  const int nv = (int)__ldcg(head);
  const float poison = __ldcg(head + 1) ? __int_as_float(0x7fffffff) : 0.f;
  const double scale = nv ? ldexp(1.0, -shift) / (double)nv : 0.0;
  const double fs = nv ? (double)E / ((double)K * (double)nv) : 0.0;
  double part = 0.0;
  for (int e = tid; e < E; e += kThreads) {
    const size_t o = (size_t)seq * E + e;
    const int c = __ldcg(sc.cnt + o);
    const double p = (double)__ldcg(sc.psum + o) * scale;
    counts[o] = c;
    mean_prob[o] = (float)p + poison;
    part += fs * (double)c * p;
    sc.cnt[o] = 0;
    sc.psum[o] = 0;
  }
  double zs = 0.0;
  for (int i = tid; i < chunks; i += kThreads) {
    float* zp = sc.zpart + (size_t)seq * chunks + i;
    zs += (double)__ldcg(zp);
    *zp = 0.f;
  }
  auto block_sum2 = [&](double a, double b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    __syncthreads();
    if (lane == 0) {
      dred[0][warp] = a;
      dred[1][warp] = b;
    }
    __syncthreads();
    a = b = 0.0;
    for (int w = 0; w < kWarps; ++w) {
      a += dred[0][w];
      b += dred[1][w];
    }
    return make_double2(a, b);
  };
  const double2 bz = block_sum2(part, zs);
  if (tid == 0) {
    sc.bal_seq[seq] = (float)bz.x + poison;
    sc.z_seq[seq] = (float)bz.y;
    valid[seq] = nv;
    head[0] = head[1] = head[2] = 0;
    __threadfence();
    last = atomicAdd(sc.done, 1u) == (uint32_t)(n_seq - 1);
  }
  __syncthreads();
  if (!last) return;

  // last sequence of all: the two losses
  __threadfence();
  double b = 0.0, zz = 0.0;
  int total = 0, full = 0;
  for (int s = tid; s < n_seq; s += kThreads) {
    const int n = __ldcg(valid + s);
    b += (double)__ldcg(sc.bal_seq + s);
    zz += (double)__ldcg(sc.z_seq + s);
    total += n;
    full += n > 0;
    sc.bal_seq[s] = sc.z_seq[s] = 0.f;
  }
  const double2 lz = block_sum2(b, zz);
  const double2 nf = block_sum2((double)total, (double)full);
  if (tid == 0) {
    losses[0] = nf.y > 0.0 ? (float)(lz.x / nf.y) : 0.f;
    losses[1] = nf.x > 0.0 ? (float)(lz.y / nf.x) : 0.f;
    valid[n_seq] = (int)nf.x;
    valid[n_seq + 1] = (int)nf.y;
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
    if (i < n_seq + 2) valid[i] = 0;
    if (i < 2) losses[i] = 0.f;
  }
}

// ---------------------------------------------------------------- backward
template <int LPR, int NPL, int MODE, bool AUX>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(RouteBackwardArgs a, int L, int chunks, int rows_per_block) {
  constexpr int RPW = 32 / LPR;
  constexpr int KPL = 32 / LPR;  // replicas of a token per lane, K <= 32
  extern __shared__ float smem[];
  pdl_wait();
  pdl_trigger();
  const int E = a.E, K = a.K;
  const int warp = warp_id(), lane = lane_id();
  const int lig = lane % LPR, sub = lane / LPR;
  float* buf = smem + (size_t)(warp * RPW + sub) * E;  // the row's routing gradient; zero between rows
  const int seq = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int r0 = chunk * rows_per_block;
  const int r1 = min(L, r0 + rows_per_block);
  const size_t t0 = (size_t)seq * L;
  if (a.d_weights)
    for (int c = lig; c < E; c += LPR) buf[c] = 0.f;

  float f[NPL];
  float gz = 0.f;
  if constexpr (AUX) {
    const int nv = __ldg(a.valid + seq), total = __ldg(a.valid + a.n_seq),
              full = __ldg(a.valid + a.n_seq + 1);
    const float gb = __ldg(a.grad_losses);
    gz = total > 0 ? 2.f * __ldg(a.grad_losses + 1) / (float)total : 0.f;
    const float k = nv > 0 ? gb * (float)E / ((float)K * (float)nv) / ((float)nv * (float)full) : 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int c = lig + LPR * i;
      f[i] = c < E ? k * (float)__ldg(a.counts + (size_t)seq * E + c) : 0.f;
    }
  }
  const float inv_scale = MODE == MOE_SCORE_SOFTMAX_RENORM ? 1.f : a.scale != 0.f ? 1.f / a.scale : 0.f;
  __syncwarp();

  for (int rb = r0 + warp * RPW; rb < r1; rb += kWarps * RPW) {
    const int r = rb + sub;
    const size_t t = t0 + r;
    const bool in = r < r1;
    const bool on = in && (!a.mask || __ldg(a.mask + t));
    float d[NPL];
    if constexpr (AUX) {
      float v[NPL];
      load_row<LPR, NPL>(a.logits + t * a.ld, E, lig, on, v);
      Row<NPL> w;
      row_probs<LPR, NPL, MODE>(v, w);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) dot = fmaf(f[i], w.p[i], dot);
      dot = group_sum<LPR>(dot);
      const float zl = gz * w.lse;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        float g = w.p[i] * (f[i] - dot);
        if constexpr (MODE == MOE_SCORE_SOFTMAX_RENORM) {
          if (gz != 0.f) g = fmaf(zl, w.p[i], g);
        } else {
          g *= sigmoid_tail(v[i]);
          if (gz != 0.f && w.sum != 0.f) g = fmaf(zl, expf(v[i] - w.lse), g);
        }
        d[i] = g;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i) d[i] = 0.f;
    }
    if (a.d_weights) {
      int id[KPL];
      float wk[KPL], gk[KPL];
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < KPL; ++j) {
        const int k = lig + LPR * j;
        const bool have = on && k < K;
        id[j] = have ? __ldg(a.ids + t * K + k) : -1;
        wk[j] = have ? __ldg(a.weights + t * K + k) : 0.f;
        gk[j] = have ? __ldg(a.d_weights + t * K + k) : 0.f;
        if (have && (unsigned)id[j] >= (unsigned)E) {
          moe_set_status(a.dev_status, MOE_DEV_BAD_EXPERT_ID);
          id[j] = -1;
        }
        dot = fmaf(wk[j], gk[j], dot);
      }
      dot = group_sum<LPR>(dot) * inv_scale;
#pragma unroll
      for (int j = 0; j < KPL; ++j) {
        gk[j] = wk[j] * (gk[j] - dot);
        if constexpr (MODE != MOE_SCORE_SOFTMAX_RENORM) {
          if (id[j] >= 0) gk[j] *= sigmoid_tail(__ldg(a.logits + t * a.ld + id[j]));
        }
        // one replica after the other: a repeated id adds up, in k order
        for (int o = 0; o < LPR && LPR * j + o < K; ++o) {
          if (lig == o && id[j] >= 0) buf[id[j]] += gk[j];
          __syncwarp();
        }
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int c = lig + LPR * i;
        if (c < E) {
          d[i] += buf[c];
          buf[c] = 0.f;
        }
      }
      __syncwarp();
    }
    if (in) {
      float* o = a.dlogits + t * a.ld_d;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int c = lig + LPR * i;
        if (c < E) o[c] = on ? d[i] : 0.f;
      }
      if (a.d_shared_gate && lig == 0) {
        float g = 0.f;
        if (on) {
          const float l = __ldg(a.logits + t * a.ld + E);
          const float ea = expf(-fabsf(l));
          const float q = 1.f / (1.f + ea);
          g = __ldg(a.d_shared_gate + t) * (ea * q * q);
        }
        o[E] = g;
      }
    }
  }
}

// ---------------------------------------------------------------- shapes
struct Chunks {
  int chunks, rows;
};

// about four blocks per SM over all sequences, at least one pass of the
// block's warps each; a fixed SM count, so that the scratch size does not
// depend on which device is current
constexpr int kGridSms = 152;
Chunks chunks_of(int L, int n_seq, int rows_per_pass) {
  const int most = moe_cdiv(4 * kGridSms, n_seq);
  int rows = moe_cdiv(L, most);
  rows = moe_cdiv(rows, rows_per_pass) * rows_per_pass;
  Chunks c;
  c.rows = rows;
  c.chunks = moe_cdiv(L, rows);
  return c;
}

int rows_per_pass(int E) { return kWarps * (E <= 128 ? 4 : E <= 256 ? 2 : 1); }

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
  s.head = reinterpret_cast<uint32_t*>(take((size_t)n_seq * 16));
  s.done = reinterpret_cast<uint32_t*>(take(4));
  s.zpart = reinterpret_cast<float*>(take((size_t)blocks * 4));
  s.bal_seq = reinterpret_cast<float*>(take((size_t)n_seq * 4));
  s.z_seq = reinterpret_cast<float*>(take((size_t)n_seq * 4));
  if (bytes) *bytes = off;
  return s;
}

template <int LPR, int NPL, int MODE>
cudaError_t run_balance(const float* logits, int ld, const int32_t* ids, const uint8_t* mask, int T,
                        int E, int K, int n_seq, void* scratch, int32_t* counts, float* mean_prob,
                        int32_t* valid, float* losses, int32_t* dev_status, cudaStream_t stream) {
  const int L = T / n_seq;
  const Chunks c = chunks_of(L, n_seq, rows_per_pass(E));
  const Scratch s = scratch_of(scratch, E, n_seq, n_seq * c.chunks, nullptr);
  // L probabilities of at most 1 sum to at most 2^bits, so 2^61 in fixed point
  int bits = 0;
  while (bits < 31 && (1ll << bits) < L) ++bits;
  const size_t smem = (size_t)(kWarps + 1) * E * 4;
  return moe_launch(balance_kernel<LPR, NPL, MODE>, dim3(n_seq * c.chunks), dim3(kThreads), smem,
                    stream, 1, logits, ld, ids, mask, L, E, K, n_seq, c.chunks, c.rows, 61 - bits,
                    s, counts, mean_prob, valid, losses, dev_status);
}

template <int LPR, int NPL>
cudaError_t run_route_backward(const RouteBackwardArgs& a, cudaStream_t stream) {
  const int L = a.T / a.n_seq;
  const Chunks c = chunks_of(L, a.n_seq, rows_per_pass(a.E));
  const size_t smem = a.d_weights ? (size_t)kWarps * (32 / LPR) * a.E * 4 : 0;
  const bool aux = a.grad_losses != nullptr;
  auto k = a.mode == MOE_SCORE_SOFTMAX_RENORM
               ? (aux ? route_backward_kernel<LPR, NPL, MOE_SCORE_SOFTMAX_RENORM, true>
                      : route_backward_kernel<LPR, NPL, MOE_SCORE_SOFTMAX_RENORM, false>)
               : (aux ? route_backward_kernel<LPR, NPL, MOE_SCORE_SIGMOID_BIAS_SCALED, true>
                      : route_backward_kernel<LPR, NPL, MOE_SCORE_SIGMOID_BIAS_SCALED, false>);
  return moe_launch(k, dim3(a.n_seq * c.chunks), dim3(kThreads), smem, stream, 1, a, L, c.chunks,
                    c.rows);
}

}  // namespace

size_t balance_loss_scratch_bytes(int T, int E, int n_seq) {
  const int L = T / n_seq;
  const int chunks = L > 0 ? chunks_of(L, n_seq, rows_per_pass(E)).chunks : 1;
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
#define MOE_BALANCE(LPR, NPL)                                                                      \
  return mode == MOE_SCORE_SOFTMAX_RENORM                                                          \
             ? run_balance<LPR, NPL, MOE_SCORE_SOFTMAX_RENORM>(logits, ld, ids, mask, T, E, K,     \
                                                               n_seq, scratch, counts, mean_prob,  \
                                                               valid, losses, dev_status, stream)  \
             : run_balance<LPR, NPL, MOE_SCORE_SIGMOID_BIAS_SCALED>(                               \
                   logits, ld, ids, mask, T, E, K, n_seq, scratch, counts, mean_prob, valid,       \
                   losses, dev_status, stream)
  if (E <= 32) MOE_BALANCE(8, 4);
  if (E <= 64) MOE_BALANCE(8, 8);
  if (E <= 128) MOE_BALANCE(8, 16);
  if (E <= 256) MOE_BALANCE(16, 16);
  if (E <= 512) MOE_BALANCE(32, 16);
  if (E <= 896) MOE_BALANCE(32, 28);
  MOE_BALANCE(32, 32);
#undef MOE_BALANCE
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t stream) {
  if (a.E <= 32) return run_route_backward<8, 4>(a, stream);
  if (a.E <= 64) return run_route_backward<8, 8>(a, stream);
  if (a.E <= 128) return run_route_backward<8, 16>(a, stream);
  if (a.E <= 256) return run_route_backward<16, 16>(a, stream);
  if (a.E <= 512) return run_route_backward<32, 16>(a, stream);
  if (a.E <= 896) return run_route_backward<32, 28>(a, stream);
  return run_route_backward<32, 32>(a, stream);
}
