// Gradient of sort by expert, SwiGLU experts and weighted return.
//
// Forward, for replica r = (t, k) of token t on expert e:
//   g = x_t W1^T, u = x_t W3^T, act = g s u with s = sigmoid(g), out_t = sum_k w_r act W2^T
// Backward, with a = dout_t W2 (one row of I values):
//   d_w_r = <a, act>
//   dg = w a u s (1 + g (1 - s)),  du = w a g s
//   dx_t = sum_k (dg W1 + du W3) (+ dx_add_t)
//   dW1 = sum_r dg^T x, dW3 = sum_r du^T x, dW2 = sum_r dout^T (w act)
// g and u are computed again, so the forward pass keeps the tokens and the routing
// alone, and <a, act> in place of <dout, y> makes the experts' output rows unneeded.
//
// Launches:
//   rows    the experts' rows of x (bf16, or e4m3 codes decoded to bf16) and of dout,
//           each expert's starting at a whole 128-row tile, zeros up to a whole 64 rows
//   part 0  per tile and 128 columns of I: a, g, u in TMEM; writes dg, du, w act
//           (bf16) and the columns' share of <a, act>
//   part 2  per expert: its three matrices' gradients, K = its rows (zeros behind them)
//   part 1  per tile and 256 columns of H: dg W1 + du W3 in fp32, over x's and dout's rows
//   finish  per token: the K rows' sum, and the shares of <a, act> added in order
// The products are one kernel: 128 x 256 tiles (tcgen05, 1 CTA per SM, persistent),
// a ring of 64-deep stages filled by TMA, accumulators in TMEM double buffered so that
// the epilogue of a unit runs under the next one's products.  Operands that the sums
// run across the rows of (W2 in a; W1, W3 in dx; both in the matrices' gradients) are
// read MN-major, as they lie.
//
// Roundings: dg, du and w act to bf16 (the tensor cores' operands), the outputs once.
// Everything else is fp32.  No atomics: sums have an order that the sizes and the
// routing fix.
#include <cuda.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"
#include "tmap.h"

namespace {

using namespace moe_e4m3;
using namespace moe_ptx;

constexpr uint64_t kWaitNs = 2000000000ull;  // every wait gives up after 2 s
constexpr int kMaxE = 1024;

// What `rows` writes for the later launches, at the start of the scratch.
struct Plan {
  int32_t tiles;
  int32_t pad[63];
  int32_t row0[kMaxE];   // an expert's first row in the padded order (a multiple of 128)
  int32_t count[kMaxE];  // its rows
};

// Where things lie in the scratch.
struct Layout {
  long long Rp;  // padded rows: at most R + 127 per expert that has any
  size_t tile, place, weight, share, rows, act, total;
  int shares;
};
Layout layout_of(long long R, int H, int E, int I) {
  Layout l;
  const long long most = R + 127 * (R < E ? R : E);
  l.Rp = most < 128 ? 128 : most / 128 * 128;
  l.shares = 2 * moe_cdiv(I, 128);
  size_t off = sizeof(Plan);
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = moe_align_up(off + bytes, 1024);
    return o;
  };
  l.tile = take((size_t)(l.Rp / 128) * 8);
  l.place = take((size_t)R * 4);
  l.weight = take((size_t)l.Rp * 4);
  l.share = take((size_t)l.shares * l.Rp * 4);
  l.rows = take((size_t)l.Rp * H * 4);  // x's rows, dout's rows; then dx's in fp32
  l.act = take((size_t)l.Rp * I * 6);   // dg, du, w act
  l.total = moe_align_up(off, 256);
  return l;
}

// ---------------------------------------------------------------- rows
struct RowArgs {
  const uint4 *x, *dout;
  const uint4* xq;       // e4m3 codes and their scales, in place of x
  const float* xs;
  const int32_t *offsets, *row_to_flat;
  const float* weights;
  int R, H, E, K;
  Plan* plan;
  int2* tile;
  int32_t* place;
  float* weight;
  uint4 *xp, *dp;
};

// offsets as far as they can be used: not falling, within [0, R]
MOE_DEVICE int usable(int v, int least, int R) { return max(least, min(v, R)); }

template <bool Q>
__global__ void __launch_bounds__(256)
rows_kernel(const RowArgs a) {
  __shared__ int first[kMaxE + 1];  // of an expert in the sorted order
  __shared__ int at[kMaxE + 1];     // in the padded order
  pdl_wait();
  pdl_trigger();
  const int E = a.E;
  for (int e = threadIdx.x; e <= E; e += blockDim.x) first[e] = __ldg(a.offsets + e);
  __syncthreads();
  if (threadIdx.x < 32) {
    // a lane's experts: running maximum, then the tiles' running sum
    const int per = (E + 32) / 32, lo = min(lane_id() * per, E + 1), hi = min(lo + per, E + 1);
    int m = 0;
    for (int e = lo; e < hi; ++e) m = first[e] = usable(first[e], m, a.R);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, m, o);
      if (lane_id() >= o) m = max(m, v);
    }
    int before = __shfl_up_sync(0xffffffffu, m, 1);
    if (lane_id() == 0) before = 0;
    for (int e = lo; e < hi; ++e) first[e] = max(first[e], before);
    __syncwarp();
    int s = 0;
    for (int e = lo; e < min(hi, E); ++e) s += (first[e + 1] - first[e] + 127) & ~127;
    int sum = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane_id() >= o) sum += v;
    }
    s = sum - s;
    for (int e = lo; e < hi; ++e) {
      at[e] = s;
      if (e < E) s += (first[e + 1] - first[e] + 127) & ~127;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.plan->tiles = at[E] / 128;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      const int n = first[e + 1] - first[e];
      a.plan->row0[e] = at[e];
      a.plan->count[e] = n;
      for (int j = 0; j < n; j += 128) a.tile[(at[e] + j) / 128] = make_int2(e, min(128, n - j));
    }
  }
  // a warp takes half of a padded row's copies: x's or dout's
  const int H8 = a.H / 8, lane = lane_id();
  const int warps = gridDim.x * (blockDim.x / 32);
  const long long jobs = 2ll * at[E];
  for (long long j = blockIdx.x * (blockDim.x / 32) + warp_id(); j < jobs; j += warps) {
    const int p = (int)(j >> 1);
    const bool of_x = (j & 1) == 0;
    int e = 0;  // the last expert that starts at or before p
    for (int lo = 0, hi = E; lo < hi;) {
      const int mid = (lo + hi) >> 1;
      if (at[mid + 1] <= p) lo = mid + 1; else hi = mid;
      e = lo;
    }
    const int i = p - at[e], n = first[e + 1] - first[e];
    if (i >= ((n + 63) & ~63)) continue;  // no sum reaches these rows
    int flat = -1;
    if (i < n) {
      const int row = first[e] + i;
      flat = __ldg(a.row_to_flat + row);
      if (of_x && lane == 0) a.place[row] = p;
      if (flat >= a.R) flat = -1;
    }
    if (of_x && lane == 0) a.weight[p] = flat >= 0 ? __ldg(a.weights + flat) : 0.f;
    uint4* to = (of_x ? a.xp : a.dp) + (size_t)p * H8;
    if (flat < 0) {
      for (int c = lane; c < H8; c += 32) to[c] = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    const size_t t = flat / a.K;
    if (Q && of_x) {
      const uint4* from = a.xq + t * (H8 / 2);
      const float* sc = a.xs + t * moe_cdiv(a.H, 128);
#pragma unroll 4
      for (int c = lane; c < H8 / 2; c += 32) decode16(__ldg(from + c), __ldg(sc + (c >> 3)), to + 2 * c);
    } else {
      const uint4* from = (of_x ? a.x : a.dout) + t * H8;
#pragma unroll 8
      for (int c = lane; c < H8; c += 32) to[c] = __ldg(from + c);
    }
  }
}

// ---------------------------------------------------------------- products
enum { kAct = 0, kDx = 1, kDw = 2 };  // the launches' parts

constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kABytes = kBM * kBK * 2, kPanel = 64 * kBK * 2;  // a panel: 64 of M or N, 64 of K
constexpr int kStageBytes = kABytes + kBN * kBK * 2;
constexpr int kStages = 4;
constexpr int kEpiWarps = 8;  // two per TMEM lane quarter, splitting the columns
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kBoxBytes = 32 * 128;  // an epilogue warp's staging: 32 rows of 128 bytes
constexpr int kNumBars = 2 * kStages + 2 + 3 + 1;
constexpr size_t kSmemBytes =
    1024 + (size_t)kStages * kStageBytes + kEpiWarps * kBoxBytes + kNumBars * 8 + 16;
static_assert(kSmemBytes <= 232448, "227 KB of shared memory per CTA");

struct GradArgs {
  const Plan* plan;
  const int2* tile;
  const float* weight;
  float* share;
  long long Rp;
  int H, I, E;
  int accumulate;
  int32_t* dev_status;
};
// A and B of the parts' products and what they store.
//   kAct: dout's and x's rows | W1, W3, W2 | dg and du, w act
//   kDx:  dg and du           | W1, W3     | dx's rows
//   kDw:  dg and du, dout's   | x's, w act | dW1, dW3, dW2
struct Maps {
  CUtensorMap a0, a1, b0, b1, b2, o0, o1, o2;
};

// one unit of work: a tile of one expert
struct Unit {
  int e, row, m;      // expert, first padded row, rows in use
  int m0, n0, n;      // the output tile's first row and column, its columns
  int part, steps;    // which product; 64-deep steps of K
};

template <int MODE>
MOE_DEVICE Unit unit_of(const GradArgs& a, long long w) {
  Unit u;
  if constexpr (MODE == kDw) {
    const int nI = moe_cdiv(a.I, kBM), nH = moe_cdiv(a.H, kBM);
    const int wI = moe_cdiv(a.I, kBN), wH = moe_cdiv(a.H, kBN);
    const int up = nI * wH, per = 2 * up + nH * wI;  // dW1 and dW3 [I, H], dW2 [H, I]
    u.e = (int)(w / per);
    int r = (int)(w % per);
    u.part = r < up ? 0 : r < 2 * up ? 1 : 2;
    r -= u.part * up;
    const int wide = u.part == 2 ? wI : wH;
    u.m0 = r / wide * kBM;
    u.n0 = r % wide * kBN;
    u.n = min(kBN, (u.part == 2 ? a.I : a.H) - u.n0);
    u.row = __ldg(&a.plan->row0[u.e]);
    u.m = __ldg(&a.plan->count[u.e]);
    u.steps = (u.m + kBK - 1) / kBK;
  } else {
    const int cols = MODE == kAct ? moe_cdiv(a.I, 128) : moe_cdiv(a.H, kBN);
    const int t = (int)(w / cols);
    const int2 it = __ldg(a.tile + t);
    u.e = it.x;
    u.m = it.y;
    u.row = t * 128;
    u.part = 0;
    u.m0 = 0;
    u.n0 = (int)(w % cols) * (MODE == kAct ? 128 : kBN);
    u.n = MODE == kAct ? 128 : min(kBN, a.H - u.n0);
    u.steps = 2 * moe_cdiv(MODE == kAct ? a.H : a.I, kBK);
  }
  return u;
}
template <int MODE>
MOE_DEVICE long long units_of(const GradArgs& a) {
  if constexpr (MODE == kDw)
    return (long long)a.E * (2 * moe_cdiv(a.I, kBM) * moe_cdiv(a.H, kBN) +
                             moe_cdiv(a.H, kBM) * moe_cdiv(a.I, kBN));
  return (long long)__ldg(&a.plan->tiles) * (MODE == kAct ? moe_cdiv(a.I, 128) : moe_cdiv(a.H, kBN));
}

// A warp's 32 rows x 128 bytes from registers to the tensor: lane's row, as eight
// 16-byte pieces, through the warp's staging box.
MOE_DEVICE void box_wait(int lane) {
  if (lane == 0) bulk_wait_read();  // the last store has read the box
  __syncwarp();
}
MOE_DEVICE void box_piece(uint8_t* box, int lane, int i, const uint4& v) {
  *reinterpret_cast<uint4*>(box + lane * 128 + ((i ^ (lane & 7)) << 4)) = v;
}
MOE_DEVICE void box_store(const CUtensorMap* map, const uint8_t* box, int lane, int c0, int c1, int c2,
                          bool add) {
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (add) tma_reduce_add_3d(map, smem_u32(box), c0, c1, c2);
    else tma_store_3d(map, smem_u32(box), c0, c1, c2);
    bulk_commit();
  }
}

// F32: the matrices' gradients in fp32 (kDw), else bf16
template <int MODE, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
products_kernel(const __grid_constant__ Maps maps, const GradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  uint8_t* boxes = smem + (size_t)kStages * kStageBytes;
  uint8_t* bar_area = boxes + kEpiWarps * kBoxBytes;
  const uint32_t bar0 = smem_u32(bar_area);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto acc_full = [&](uint32_t i) { return bar0 + 8u * (2 * kStages + i); };
  // kAct: the two sets of a, and the one of g and u; else the two accumulators
  auto acc_empty = [&](uint32_t i) { return bar0 + 8u * (2 * kStages + 2 + i); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 5);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(acc_full(i), 1);
    for (int i = 0; i < 3; ++i) mbar_init(acc_empty(i), 32 * kEpiWarps);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  auto fail = [&]() {
    moe_set_status(a.dev_status, MOE_DEV_WAIT_TIMEOUT);
    *abort_flag = 1;
  };
  const long long total = units_of<MODE>(a);
  const int nkH = moe_cdiv(a.H, kBK), nkI = moe_cdiv(a.I, kBK);

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      for (long long w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const Unit u = unit_of<MODE>(a, w);
        const int panels = (u.n + 63) / 64;
        for (int s = 0; s < u.steps; ++s) {
          if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, kWaitNs)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t A = sbase + stage * kStageBytes, B = A + kABytes, bar = full_bar(stage);
          if constexpr (MODE == kAct) {
            if (s < nkH) {  // a = dout W2: W2 [H, I] lies MN-major
              mbar_arrive_expect_tx(bar, kABytes + 2 * kPanel);
              tma_load_3d(A, &maps.a0, bar, s * kBK, u.row, 0);
              for (int p = 0; p < 2; ++p)
                tma_load_3d(B + p * kPanel, &maps.b2, bar, u.n0 + 64 * p, s * kBK, u.e);
            } else {        // g | u
              const int k = (s - nkH) * kBK;
              mbar_arrive_expect_tx(bar, kStageBytes);
              tma_load_3d(A, &maps.a1, bar, k, u.row, 0);
              tma_load_3d(B, &maps.b0, bar, k, u.n0, u.e);
              tma_load_3d(B + kBM * kBK * 2, &maps.b1, bar, k, u.n0, u.e);
            }
          } else if constexpr (MODE == kDx) {
            const int part = s >= nkI, k = (s - part * nkI) * kBK;
            mbar_arrive_expect_tx(bar, kABytes + panels * kPanel);
            tma_load_3d(A, &maps.a0, bar, k, u.row, part);
            for (int p = 0; p < panels; ++p)
              tma_load_3d(B + p * kPanel, part ? &maps.b1 : &maps.b0, bar, u.n0 + 64 * p, k, u.e);
          } else {
            const int row = u.row + s * kBK;
            mbar_arrive_expect_tx(bar, kABytes + panels * kPanel);
            for (int p = 0; p < 2; ++p) {
              if (u.part == 2) tma_load_3d(A + p * kPanel, &maps.a1, bar, u.m0 + 64 * p, row, 0);
              else tma_load_3d(A + p * kPanel, &maps.a0, bar, u.m0 + 64 * p, row, u.part);
            }
            for (int p = 0; p < panels; ++p)
              tma_load_3d(B + p * kPanel, u.part == 2 ? &maps.b1 : &maps.b0, bar, u.n0 + 64 * p, row, 0);
          }
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      // every copy this thread started has landed before the CTA moves on
      for (int s = 0; s < kStages; ++s)
        if (armed & (1u << s))
          if (!mbar_wait_bounded(full_bar(s), (armed_parity >> s) & 1u, nullptr, kWaitNs)) fail();
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer
      int stage = 0;
      uint32_t phase = 0, n = 0;
      bool ok = true, issued = false;
      auto step = [&](uint32_t d, int N, bool mnA, bool mnB, bool first) {
        if (!mbar_wait_bounded(full_bar(stage), phase, abort_flag, kWaitNs)) {
          fail();
          return false;
        }
        tc_fence_after();
        const uint32_t A = sbase + stage * kStageBytes, B = A + kABytes;
        const uint32_t id = idesc_bf16_f32(kBM, N) | (mnA ? kIdescMnA : 0u) | (mnB ? kIdescMnB : 0u);
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)
          tc_mma_f16(d, mnA ? sdesc_mn_sw128(A + k * 2048, kPanel) : sdesc_k128_sw128(A + k * 32),
                     mnB ? sdesc_mn_sw128(B + k * 2048, kPanel) : sdesc_k128_sw128(B + k * 32), id,
                     !first || k > 0);
        issued = true;
        tc_commit(empty_bar(stage));
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
        return true;
      };
      auto free_acc = [&](uint32_t i, uint32_t use) {  // before the use-th time accumulator i is written
        if (!mbar_wait_bounded(acc_empty(i), (use & 1u) ^ 1u, abort_flag, kWaitNs)) {
          fail();
          return false;
        }
        tc_fence_after();
        return true;
      };
      for (long long w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const Unit u = unit_of<MODE>(a, w);
        if (u.steps == 0) continue;
        if constexpr (MODE == kAct) {
          ok = free_acc(n & 1u, n >> 1);
          for (int s = 0; s < nkH && ok; ++s) ok = step(tmem + 128 * (n & 1u), 128, false, true, s == 0);
          ok = ok && free_acc(2, n);
          for (int s = 0; s < nkH && ok; ++s) ok = step(tmem + 256, 256, false, false, s == 0);
        } else {
          ok = free_acc(n & 1u, n >> 1);
          for (int s = 0; s < u.steps && ok; ++s)
            ok = step(tmem + 256 * (n & 1u), u.n, MODE == kDw, true, s == 0);
        }
        if (!ok) break;
        tc_commit(acc_full(n & 1u));
        ++n;
      }
      if (issued) {
        // all MMAs of this thread complete before TMEM is released
        tc_commit(drain_bar);
        if (!mbar_wait_bounded(drain_bar, 0, nullptr, kWaitNs)) fail();
      }
    }
  } else {
    // ---------------- epilogue: lane quarter = warp % 4, half of the columns each
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    uint8_t* box = boxes + (warp - 2) * kBoxBytes;
    uint32_t n = 0;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
      const Unit u = unit_of<MODE>(a, w);
      const int r0 = quarter * 32;  // the warp's first row of the tile
      if (MODE == kDw && u.steps == 0) {
        // an expert without rows: zeros, or nothing to add
        const int rows = u.part == 2 ? a.H : a.I;
        if (a.accumulate || u.m0 + r0 >= rows) continue;
        box_wait(lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) box_piece(box, lane, i, make_uint4(0u, 0u, 0u, 0u));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          for (int c = half * 128; c < min(u.n, half * 128 + 128); c += F32 ? 32 : 64)
            tma_store_3d(u.part == 0 ? &maps.o0 : u.part == 1 ? &maps.o1 : &maps.o2, smem_u32(box),
                         u.n0 + c, u.m0 + r0, u.e);
          bulk_commit();
        }
        __syncwarp();
        continue;
      }
      if (!mbar_wait_bounded(acc_full(n & 1u), (n >> 1) & 1u, abort_flag, kWaitNs)) {
        fail();
        break;
      }
      tc_fence_after();
      if constexpr (MODE == kAct) {
        const int row = u.row + r0 + lane;
        const bool in = r0 + lane < u.m;
        const float wr = in ? __ldg(a.weight + row) : 0.f;
        uint32_t pg[32], pu[32], pa[32];
        float share = 0.f;
        const uint32_t ta = t_lane + 128 * (n & 1u) + 64 * half, tg = t_lane + 256 + 64 * half;
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
          uint32_t va[16], vg[16], vu[16];
          tc_ld_32x32b_x16(ta + c, va);
          tc_ld_32x32b_x16(tg + c, vg);
          tc_ld_32x32b_x16(tg + 128 + c, vu);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float dg[2], du[2], act[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float av = __uint_as_float(va[j + q]), g = __uint_as_float(vg[j + q]);
              const float uv = __uint_as_float(vu[j + q]);
              const float s = __fdividef(1.f, 1.f + __expf(-g));
              const float gs = g * s, aw = av * wr;
              share = fmaf(av, gs * uv, share);
              dg[q] = aw * uv * (s + gs * (1.f - s));
              du[q] = aw * gs;
              act[q] = wr * gs * uv;
            }
            const int i = (c + j) / 2;
            pg[i] = in ? pack_bf16x2(dg[0], dg[1]) : 0u;  // the sums over rows go on to 64
            pu[i] = in ? pack_bf16x2(du[0], du[1]) : 0u;
            pa[i] = in ? pack_bf16x2(act[0], act[1]) : 0u;
          }
        }
        tc_fence_before();
        mbar_arrive(acc_empty(n & 1u));
        mbar_arrive(acc_empty(2));
        const int c0 = u.n0 + 64 * half;
        if (in) a.share[(size_t)(c0 / 64) * a.Rp + row] = share;
        if (c0 < a.I) {
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t(&v)[32] = k == 0 ? pg : k == 1 ? pu : pa;
            box_wait(lane);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              box_piece(box, lane, i, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
            box_store(k == 2 ? &maps.o1 : &maps.o0, box, lane, c0, u.row + r0, k == 1, false);
          }
        }
      } else {
        constexpr bool kF = MODE == kDx || F32;  // 32 columns of a row per 128 bytes, or 64
        const uint32_t t0 = t_lane + 256 * (n & 1u);
        const int rows = MODE == kDx ? 128 : u.part == 2 ? a.H : a.I;
        const CUtensorMap* map = u.part == 0 ? &maps.o0 : u.part == 1 ? &maps.o1 : &maps.o2;
        const int c1 = min(u.n, half * 128 + 128);
        if (u.m0 + r0 < rows) {
          for (int c = half * 128; c < c1; c += kF ? 32 : 64) {
            uint32_t v[kF ? 32 : 64];
#pragma unroll
            for (int i = 0; i < (kF ? 32 : 64); i += 16)
              tc_ld_32x32b_x16(t0 + c + i, *reinterpret_cast<uint32_t(*)[16]>(v + i));
            tc_wait_ld();
            box_wait(lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if constexpr (kF) {
                box_piece(box, lane, i, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
              } else {
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  o[q] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * q]), __uint_as_float(v[8 * i + 2 * q + 1]));
                box_piece(box, lane, i, make_uint4(o[0], o[1], o[2], o[3]));
              }
            }
            if constexpr (MODE == kDx) box_store(map, box, lane, u.n0 + c, u.row + r0, 0, false);
            else box_store(map, box, lane, u.n0 + c, u.m0 + r0, u.e, a.accumulate);
          }
        }
        tc_fence_before();
        mbar_arrive(acc_empty(n & 1u));
      }
      ++n;
    }
    if (lane == 0) bulk_wait();  // the stores are done before the CTA is
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- finish
struct FinishArgs {
  const float4* rows;  // [Rp][H]
  const float* share;  // [shares][Rp]
  const int32_t *place, *flat_to_row, *offsets;
  const uint4* add;
  uint4* dx;
  float* d_weights;
  long long Rp;
  int T, K, H, E, shares;
};

// The padded row of replica f: -1 where it was dropped.
MOE_DEVICE int padded_row(const FinishArgs& a, long long f) {
  const int r = __ldg(a.flat_to_row + f);
  if (r < 0 || r >= a.T * a.K || r >= __ldg(a.offsets + a.E)) return -1;
  const int p = __ldg(a.place + r);
  return p >= 0 && p < a.Rp ? p : -1;  // offsets that start above 0 leave places unset
}

// A warp takes 256 columns of a token; behind those, 32 replicas' weights.
__global__ void __launch_bounds__(256)
finish_kernel(const FinishArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = lane_id(), H8 = a.H / 8, K = a.K;
  const int chunks = a.dx ? moe_cdiv(H8, 32) : 0;
  const long long w = (long long)blockIdx.x * 8 + warp_id();
  const long long tokens = (long long)a.T * chunks, R = (long long)a.T * K;
  if (w < tokens) {
    const long long t = w / chunks;
    const int c = (int)(w % chunks) * 32 + lane;
    const int p = lane < K ? padded_row(a, t * K + lane) : -1;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
      const int q = __shfl_sync(0xffffffffu, p, k);
      if (q < 0 || c >= H8) continue;
      const float4* v = a.rows + ((size_t)q * H8 + c) * 2;
      const float4 x = __ldg(v), y = __ldg(v + 1);
      s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
      s[4] += y.x; s[5] += y.y; s[6] += y.z; s[7] += y.w;
    }
    if (c >= H8) return;
    const size_t o = (size_t)t * H8 + c;
    if (a.add) {
      float f[8];
      bf16x8_to_f32(a.add[o], f);  // may be dx itself
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += f[q];
    }
    a.dx[o] = make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]),
                         pack_bf16x2(s[6], s[7]));
    return;
  }
  const long long f = (w - tokens) * 32 + lane;
  if (!a.d_weights || f >= R) return;
  const int p = padded_row(a, f);
  float s = 0.f;
  if (p >= 0) {
#pragma unroll 8
    for (int j = 0; j < a.shares; ++j) s += __ldg(a.share + (size_t)j * a.Rp + p);
  }
  a.d_weights[f] = s;
}

template <int MODE, bool F32>
cudaError_t run_products(const Maps& maps, const GradArgs& a, cudaStream_t stream) {
  static std::atomic<unsigned long long> set{0};
  const cudaError_t e = moe_raise_smem(products_kernel<MODE, F32>, kSmemBytes, set);
  if (e != cudaSuccess) return e;
  return moe_launch(products_kernel<MODE, F32>, dim3(moe_num_sms()), dim3(kThreads), kSmemBytes, stream,
                    1, maps, a);
}

}  // namespace

size_t experts_backward_scratch_bytes(int T, int H, int E, int K, int I) {
  return layout_of((long long)T * K, H, E, I).total;
}

cudaError_t launch_experts_backward(const ExpertsBackwardArgs& g, void* scratch, cudaStream_t stream) {
  using moe_tmap::bf16_map_3d;
  using moe_tmap::f32_map_3d;
  const int T = g.T, H = g.H, E = g.E, K = g.K, I = g.I, R = T * K;
  const Layout l = layout_of(R, H, E, I);
  char* s = static_cast<char*>(scratch);
  char* xp = s + l.rows;
  char* dp = xp + (size_t)l.Rp * H * 2;
  char* dgu = s + l.act;
  char* act = dgu + (size_t)l.Rp * I * 4;
  GradArgs a{reinterpret_cast<const Plan*>(s), reinterpret_cast<const int2*>(s + l.tile),
             reinterpret_cast<const float*>(s + l.weight), reinterpret_cast<float*>(s + l.share),
             l.Rp, H, I, E, g.accumulate, g.dev_status};

  RowArgs r{static_cast<const uint4*>(g.x), static_cast<const uint4*>(g.dout),
            static_cast<const uint4*>(g.xq), g.xq_scale, g.offsets, g.row_to_flat, g.weights, R, H, E, K,
            reinterpret_cast<Plan*>(s), reinterpret_cast<int2*>(s + l.tile),
            reinterpret_cast<int32_t*>(s + l.place), reinterpret_cast<float*>(s + l.weight),
            reinterpret_cast<uint4*>(xp), reinterpret_cast<uint4*>(dp)};
  const int blocks = (int)(l.Rp / 4 < 152 * 8 ? l.Rp / 4 : 152 * 8);
  cudaError_t e = moe_launch(g.xq ? rows_kernel<true> : rows_kernel<false>, dim3(blocks), dim3(256), 0,
                             stream, 1, r);
  if (e != cudaSuccess) return e;

  Maps m{};
  bool ok = bf16_map_3d(&m.a0, dp, H, l.Rp, 1, 64, 128) && bf16_map_3d(&m.a1, xp, H, l.Rp, 1, 64, 128) &&
            bf16_map_3d(&m.b0, g.w1, H, I, E, 64, 128) && bf16_map_3d(&m.b1, g.w3, H, I, E, 64, 128) &&
            bf16_map_3d(&m.b2, g.w2, I, H, E, 64, 64) && bf16_map_3d(&m.o0, dgu, I, l.Rp, 2, 64, 32) &&
            bf16_map_3d(&m.o1, act, I, l.Rp, 1, 64, 32);
  if (!ok) return cudaErrorInvalidValue;
  if (R > 0 && (e = run_products<kAct, false>(m, a, stream)) != cudaSuccess) return e;

  if (g.dw1) {
    m = Maps{};
    ok = bf16_map_3d(&m.a0, dgu, I, l.Rp, 2, 64, 64) && bf16_map_3d(&m.a1, dp, H, l.Rp, 1, 64, 64) &&
         bf16_map_3d(&m.b0, xp, H, l.Rp, 1, 64, 64) && bf16_map_3d(&m.b1, act, I, l.Rp, 1, 64, 64);
    auto out = [&](CUtensorMap* map, void* p, int n0, int n1) {
      return g.dw_f32 ? f32_map_3d(map, p, n0, n1, E, 32, 32) : bf16_map_3d(map, p, n0, n1, E, 64, 32);
    };
    ok = ok && out(&m.o0, g.dw1, H, I) && out(&m.o1, g.dw3, H, I) && out(&m.o2, g.dw2, I, H);
    if (!ok) return cudaErrorInvalidValue;
    e = g.dw_f32 ? run_products<kDw, true>(m, a, stream) : run_products<kDw, false>(m, a, stream);
    if (e != cudaSuccess) return e;
  }
  if (g.dx && R > 0) {
    m = Maps{};
    ok = bf16_map_3d(&m.a0, dgu, I, l.Rp, 2, 64, 128) && bf16_map_3d(&m.b0, g.w1, H, I, E, 64, 64) &&
         bf16_map_3d(&m.b1, g.w3, H, I, E, 64, 64) && f32_map_3d(&m.o0, xp, H, l.Rp, 1, 32, 32);
    if (!ok) return cudaErrorInvalidValue;
    if ((e = run_products<kDx, false>(m, a, stream)) != cudaSuccess) return e;
  }
  if (R == 0 || (!g.dx && !g.d_weights)) return cudaSuccess;
  FinishArgs f{reinterpret_cast<const float4*>(xp), a.share, r.place, g.flat_to_row, g.offsets,
               static_cast<const uint4*>(g.dx_add), static_cast<uint4*>(g.dx), g.d_weights, l.Rp, T, K, H,
               E, l.shares};
  const long long warps = (g.dx ? (long long)T * moe_cdiv(H / 8, 32) : 0) + (g.d_weights ? moe_cdiv(R, 32) : 0);
  return moe_launch(finish_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, stream, 1, f);
}
