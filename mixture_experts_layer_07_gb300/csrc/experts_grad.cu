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
//   rows    the experts' rows of x (bf16, or e4m3 codes decoded to bf16) and of dout in
//           the experts' order, zeros up to a whole 16 rows (the MMA's K)
//   part 0  per up to 128 rows and 256 columns of I: a, g, u; writes dg, du, w act (bf16)
//           and each 128 columns' share of <a, act>
//   part 1  per up to 256 rows and 256 columns of H: dg W1 + du W3 in fp32; and per expert
//           its three matrices' gradients, K = its rows
//   finish  per token: the K rows' sum, and the shares of <a, act> added in order
// The products are one kernel: 256 x N tiles by pairs of CTAs (tcgen05, cta_group::2, one
// CTA per SM, persistent), a ring of 64-deep stages filled by TMA, accumulators in TMEM.
// Part 0's tiles and those of dx have weight rows (features) as their 256 and tokens as N,
// so that an expert with few rows takes a narrow tile.  Operands that the sums run across
// the rows of (W2 in a; W1, W3 in dx; both in the matrices' gradients) are read MN-major,
// as they lie.  A pair, because each SM then loads half of B only: with single CTAs and
// 128 x 256 tiles the loads' 64 bytes per clock and SM were the bound (61 of them in part 0).
//
// Roundings: dg, du and w act to bf16 (the tensor cores' operands), the outputs once.
// Everything else is fp32.  The tensor cores cut what falls off an fp32 sum, which
// shortens it by about 1.7e-8 per K of 16.  a, g and u, whose errors d_weights shows (its
// fp32 is not behind a rounding to bf16), are therefore taken out of TMEM every 256 of K
// (the first 512 of a long one) and added in registers: d_weights is at most 9.2e-7 off 64
// bits whatever H is (H = 128 3.4e-7, 1024 6.6e-7, 1536 9.2e-7, 8192 7.2e-7), 9e-6 at
// H = 2880 in one go.  The sums of the matrices' gradients (K = an expert's rows) and of dx
// (K = 2 I) stay in TMEM: their operands' roundings to bf16 are far above what is cut there.
// fp32 gradients of an expert with 8192 rows end 8.6e-6 too short, with 32768 rows 3.4e-5;
// the operands' roundings put them 1.7e-3 off where the rows have no common direction, 3e-4
// at 32768 rows that have one.  No atomics: sums have an order that the sizes and the
// routing fix.
//
// Measured on one GB300 (copy rate 6797 GB/s, bf16 1947 TFLOP/s), per call in a graph of them:
//   T = 4096, H = I = 2880, E = 32, K = 4, from codes  1840 us, 1750 to 1885 with the clock,
//     which the power cap holds at 1560 to 1720 of 2070 MHz (2343 with single CTAs); the
//     tensor cores' 1116 us at full clock are the bound: part 0 is
//     held by its loads (83 bytes per clock and SM at full rate) and by what of its epilogue
//     the next unit's first products do not hide, part 1 by loads and stores on the same path
//   T = 2048, H = 2048, I = 768, E = 128, K = 8        710 us; memory: weights are read in
//     part 0 and, but for W2, again in part 1 (6.1 and 6.0 TB/s under the profiler)
//   T = 64, H = 2048, I = 512, E = 512, K = 10         1082 us, floor 948: the matrices'
//     gradients, mostly zeros or one row's, have to be written (fp32 1597 us, floor 1422;
//     added to fp32 2025, floor 1622)
//   T = 100, H = 256, I = 128, E = 8, K = 2            18 us: four dependent launches
#include <cuda.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"
#include "tmap.h"

namespace {

using namespace moe_e4m3;
using namespace moe_f32x2;
using namespace moe_ptx;

constexpr uint64_t kWaitNs = 2000000000ull;  // every wait gives up after 2 s
constexpr int kMaxE = 1024;

// Tokens of a tile, at most; a tile of the gradient of x is wider, as it has one
// accumulator where part 0 has three.
constexpr int kActTokens = 128, kDxTokens = 256;
// Part 0's tiles are halved, to 64 or 32 tokens, while all of its units still run at once:
// a unit then ends earlier, as its epilogue is by the token (T = 512, H = 1024, I = 512,
// E = 16, K = 4: 52.1 -> 50.7 us).  At most so many tiles more in the list.
constexpr int kMoreTiles = 512;

// What `rows` writes for the later launches, at the start of the scratch.
struct Plan {
  int32_t tiles[2];    // of part 0 and of part 1
  int32_t act_tokens;  // of a tile of part 0, at most
  int32_t pad[61];
  int2 rows[kMaxE];  // an expert's first row in the padded order (a multiple of 16), its rows
};
// The tiles of an expert follow one another; each names the expert, the first of its
// tiles, the expert's first row and its rows.
using Tile = int4;

// Where things lie in the scratch.
struct Layout {
  long long Rp;  // padded rows: at most R + 15 per expert that has any
  size_t tile[2], place, weight, share, rows, act, dx, total;
  int shares;
};
Layout layout_of(long long R, int H, int E, int I) {
  Layout l;
  const long long some = R < E ? R : E;  // experts with rows, at most
  const long long most = R + 15 * some;
  l.Rp = most < 16 ? 16 : most / 16 * 16;
  l.shares = 2 * moe_cdiv(I, 256);
  size_t off = sizeof(Plan);
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = moe_align_up(off + bytes, 1024);
    return o;
  };
  l.tile[0] = take((size_t)(R / kActTokens + some + 1 + kMoreTiles) * sizeof(Tile));
  l.tile[1] = take((size_t)(R / kDxTokens + some + 1) * sizeof(Tile));
  l.place = take((size_t)R * 4);
  l.weight = take((size_t)l.Rp * 4);
  l.share = take((size_t)l.shares * l.Rp * 4);
  l.rows = take((size_t)l.Rp * H * 4);  // x's rows, dout's rows
  l.act = take((size_t)l.Rp * I * 6);   // dg, du, w act
  l.dx = take((size_t)l.Rp * H * 4);    // dx's rows, fp32
  l.total = moe_align_up(off, 256);
  return l;
}

// ---------------------------------------------------------------- rows
struct RowArgs {
  const uint4 *x, *dout;
  const uint4* xq;       // e4m3 codes and their scales, in place of x
  const float* xs;
  const int32_t *offsets, *row_to_flat, *flat_to_row;
  const float* weights;
  int R, H, E, K;
  int at_once;  // part 0's tiles that run at once
  Plan* plan;
  Tile* tile[2];
  int32_t* place;  // of a replica: its padded row, -1 where it was dropped
  float* weight;   // of a padded row
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
  // Jobs of a warp: half of a row's copies each, x's or dout's, then the padding rows.  A job's
  // replica is loaded a job ahead, the first one beside the offsets.
  const int E = a.E, R = a.R;
  const int warps = gridDim.x * (blockDim.x / 32);
  const int first_job = blockIdx.x * (blockDim.x / 32) + warp_id();
  auto flat_of = [&](long long j) { return j < 2ll * R ? __ldg(a.row_to_flat + (j >> 1)) : -1; };
  int flat_next = flat_of(first_job);
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
    // sums over the experts before: padded rows, tiles of part 1, of part 0 by their size
    constexpr int kSums = 5;
    auto counts = [](int n, int (&c)[kSums]) {
      c[0] += (n + 15) & ~15;
      c[1] += moe_cdiv(n, kDxTokens);
#pragma unroll
      for (int i = 2; i < kSums; ++i) c[i] += moe_cdiv(n, kActTokens >> (i - 2));
    };
    int s[kSums] = {0, 0, 0, 0, 0}, all[kSums];
    for (int e = lo; e < min(hi, E); ++e) counts(first[e + 1] - first[e], s);
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      int sum = s[i];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane_id() >= o) sum += v;
      }
      all[i] = __shfl_sync(0xffffffffu, sum, 31);
      s[i] = sum - s[i];
    }
    const int most = min(a.at_once, kMoreTiles);
    const int half = all[4] <= most ? 2 : all[3] <= most ? 1 : 0;  // how often the tiles are halved
    for (int e = lo; e < hi; ++e) {
      at[e] = s[0];
      if (e == E) {
        if (blockIdx.x == 0) {
          a.plan->tiles[0] = half == 2 ? all[4] : half == 1 ? all[3] : all[2];
          a.plan->tiles[1] = all[1];
          a.plan->act_tokens = kActTokens >> half;
        }
        break;
      }
      const int n = first[e + 1] - first[e];
      if (blockIdx.x == 0) {
        const int t0 = half == 2 ? s[4] : half == 1 ? s[3] : s[2];
        a.plan->rows[e] = make_int2(s[0], n);
        for (int j = 0; j < moe_cdiv(n, kActTokens >> half); ++j) a.tile[0][t0 + j] = make_int4(e, t0, s[0], n);
        for (int j = 0; j < moe_cdiv(n, kDxTokens); ++j) a.tile[1][s[1] + j] = make_int4(e, s[1], s[0], n);
      }
      counts(n, s);
    }
  }
  __syncthreads();
  const int rows = first[E];
  for (int f = blockIdx.x * blockDim.x + threadIdx.x; f < R; f += gridDim.x * blockDim.x) {
    const int r = __ldg(a.flat_to_row + f);
    if (r < 0 || r >= rows) a.place[f] = -1;
  }
  const int H8 = a.H / 8, lane = lane_id();
  for (long long j = first_job; j < 2ll * R + 32 * E; j += warps) {
    const bool of_x = (j & 1) == 0;
    const int r = (int)(j >> 1);
    int flat = flat_next, p;
    flat_next = flat_of(j + warps);
    if (r < R) {
      if (r >= rows) continue;
      int e = 0;  // the last expert that starts at or before r
      for (int lo = 0, hi = E; lo < hi; e = lo) {
        const int mid = (lo + hi) >> 1;
        if (first[mid + 1] <= r) lo = mid + 1; else hi = mid;
      }
      if (r < first[e]) continue;  // offsets that do not start at 0
      p = at[e] + r - first[e];
      if (flat >= R) flat = -1;
      if (of_x && lane == 0) {
        if (flat >= 0) a.place[flat] = p;
        a.weight[p] = flat >= 0 ? __ldg(a.weights + flat) : 0.f;
      }
    } else {
      // up to 15 rows behind an expert's last one
      const int e = (r - R) >> 4;
      p = at[e] + first[e + 1] - first[e] + ((r - R) & 15);
      if (p >= at[e + 1]) continue;
      flat = -1;
      if (of_x && lane == 0) a.weight[p] = 0.f;
    }
    uint4* to = (of_x ? a.xp : a.dp) + (size_t)p * H8;
    if (flat < 0) {
      for (int c = lane; c < H8; c += 32) to[c] = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    const size_t t = flat / a.K;
    if (Q && of_x) {
      const uint4* from = a.xq + t * (H8 / 2);
      const float* sc = a.xs + t * moe_cdiv(a.H, 128);
      // four pieces' loads before the first is decoded (T = 1023, K = 4, H = 2880 20.5 -> 18.8 us)
      for (int c0 = 0; c0 < H8 / 2; c0 += 128) {
        uint4 q[4];
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + 32 * i + lane;
          if (c >= H8 / 2) continue;
          q[i] = __ldg(from + c);
          f[i] = __ldg(sc + (c >> 3));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + 32 * i + lane;
          if (c < H8 / 2) decode16(q[i], f[i], to + 2 * c);
        }
      }
    } else {
      const uint4* from = (of_x ? a.x : a.dout) + t * H8;
#pragma unroll 8
      for (int c = lane; c < H8; c += 32) to[c] = __ldg(from + c);
    }
  }
}

// ---------------------------------------------------------------- products
enum { kAct = 0, kBack = 1 };  // the launches' parts
enum { kW1 = 0, kW3 = 1, kW2 = 2, kX = 3 };  // what a unit of kBack is the gradient of

constexpr int kBM = 256, kBK = 64;       // a pair's tile rows; a stage's K
constexpr int kTile = 128 * kBK * 2;     // a CTA's 128 rows (or columns) of an operand, 64 deep
constexpr int kPanel = 64 * kBK * 2;     // MN-major: 64 of M or N
constexpr int kChunk = 4;                // kAct: stages between two additions in registers
// and before a unit's first one: as many again where K is long (T = 4096, H = 2880 1893 ->
// 1863 us, as the products run further ahead of the last unit's epilogue), which adds a
// third to the sums' error at H = 1536, less above; below it would be more
MOE_DEVICE int first_chunk(int stages) { return stages >= 24 ? 2 * kChunk : kChunk; }
constexpr int kEpiWarps = 8;             // two per TMEM lane quarter, splitting the columns
constexpr int kBoxBytes = 32 * 128;      // kBack: an epilogue warp's store, 32 rows of 128 bytes

template <int MODE>
struct Cfg {
  // kAct: W1, W3 (or W2) and half of 128 tokens; else A and half of 256 columns
  static constexpr int kStageBytes = MODE == kAct ? 2 * kTile + kTile / 2 : 2 * kTile;
  static constexpr int kB = MODE == kAct ? 2 * kTile : kTile;  // where B lies in a stage
  static constexpr int kStages = MODE == kBack ? 6 : 5;
  // kBack: a box per warp; kAct: two sets of the warps' column sums, the tokens' weights
  static constexpr int kEpiBytes = MODE == kBack ? kEpiWarps * kBoxBytes : kEpiWarps * 64 * 4 * 3;
  static constexpr int kNumBars = 2 * kStages + 3 + 3 + 1 + 2;
  static constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + kEpiBytes + kNumBars * 8 + 16;
  static_assert(kSmemBytes <= 232448, "227 KB of shared memory per CTA");
};
constexpr int kThreads = 128 + 32 * kEpiWarps;  // warp 0 TMA, warp 1 MMA, warps 4-11 epilogue

struct GradArgs {
  const Plan* plan;
  const Tile* tile[2];
  const float* weight;
  float* share;
  __nv_bfloat16 *dgu, *act;  // kAct's outputs: [2][Rp][I], [Rp][I]
  float* rows;               // kBack's: [Rp][H]
  long long Rp;
  int H, I, E;
  bool dx, dw, accumulate;   // what is wanted: the gradient of x, of the matrices
  int32_t* dev_status;
};
// The operands, and the matrices' gradients.
struct Maps {
  CUtensorMap w1, w3, w2, x, dout, dgu, act, d1, d3, d2;
};

// One unit of work of a pair: a tile of one expert.
struct Unit {
  int e, row, m;   // expert; the tile's first padded row and its tokens, or (matrices) the expert's
  int m0, n0, n;   // the tile's first row and column, its columns (a multiple of 16)
  int part;        // kBack: kW1, kW3, kW2 or kX
};

// The units w, w + step, ... of a pair; what a unit needs from memory is loaded while
// the one before it is worked on.
template <int MODE>
struct Walk {
  const GradArgs& a;
  int w, step, total, tokens, wI, wH;  // tokens: units of kAct, or of the gradient of x
  int most;                            // tokens of a tile, at most
  int4 raw;

  MOE_DEVICE Walk(const GradArgs& g, int first, int by) : a(g), w(first), step(by) {
    wI = moe_cdiv(a.I, kBM), wH = moe_cdiv(a.H, kBM);
    if constexpr (MODE == kAct) {
      most = __ldg(&a.plan->act_tokens);
      total = tokens = __ldg(&a.plan->tiles[0]) * wI;
    } else {
      most = kDxTokens;
      // The gradient of x first, whichever units are longer (2 I against the expert's rows): with
      // the matrices first T = 4096, H = I = 2880 1890 -> 1925 us, small batches 4 to 7 % more,
      // T = 64, E = 512 1102 -> 1081.  Units go to the pairs by a fixed stride, so shares are
      // uneven where kinds differ: T = 4096, I = 512, one expert has 128 units of K = 1024 and 48
      // of 4096 for 76 pairs, the longest share 6144 of K, the mean 4312.
      tokens = a.dx ? __ldg(&a.plan->tiles[1]) * wH : 0;
      total = tokens + (a.dw ? a.E * 3 * wI * wH : 0);
    }
    load();
  }
  MOE_DEVICE void load() {
    if (w >= total) return;
    if (MODE == kAct || w < tokens) {
      raw = __ldg(a.tile[MODE] + (uint32_t)w / (uint32_t)(MODE == kAct ? wI : wH));
    } else {
      const int e = (uint32_t)(w - tokens) / (uint32_t)(3 * wI * wH);
      const int2 r = __ldg(&a.plan->rows[e]);
      raw = make_int4(e, 0, r.x, r.y);
    }
  }
  MOE_DEVICE bool next(Unit& u) {
    if (w >= total) return false;
    u.e = raw.x;
    u.row = raw.z;
    u.m = raw.w;
    if (MODE == kAct || w < tokens) {
      // an expert's tiles of one block follow one another, so its weights are read once
      const int tiles = moe_cdiv(u.m, most);
      const int r = w - raw.y * (MODE == kAct ? wI : wH);
      const int t = r % tiles, n = (moe_cdiv(u.m, tiles) + 15) & ~15;
      u.part = kX;
      u.m0 = r / tiles * kBM;
      u.n0 = 0;
      u.row += t * n;
      u.m = min(n, u.m - t * n);
      u.n = (u.m + 15) & ~15;
    } else {
      // dW1, dW3 [I, H] and dW2 [H, I] have as many blocks each
      int r = w - tokens - u.e * 3 * wI * wH;
      u.part = r / (wI * wH);
      r -= u.part * wI * wH;
      const int wide = u.part == kW2 ? wI : wH;
      u.m0 = r / wide * kBM;
      u.n0 = r % wide * 256;
      u.n = min(256, (u.part == kW2 ? a.I : a.H) - u.n0);
    }
    w += step;
    load();
    return true;
  }
};

// A warp's 32 rows x 128 bytes from registers to the tensor: lane's row, as eight
// 16-byte pieces, through the warp's box.  The matrices' gradients are not read again
// here: L2 gives their lines up first, which keeps dx's rows for `finish` (T = 64, E = 512
// 1103 -> 1081 us, T = 2048, E = 128 714 -> 710).
MOE_DEVICE void box_wait(int lane) {
  if (lane == 0) bulk_wait_read<0>();  // the last store has read the box
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
    else tma_store_3d_hint(map, smem_u32(box), c0, c1, c2, l2_evict_first());
    bulk_commit();
  }
}

// Sums over the warp's lanes of 16 values each; lane 2 i ends up with the sum of value
// column(2 i).  A lane hands over the half that its partner goes on with.
MOE_DEVICE float lane_sums16(float (&v)[16], int lane) {
#pragma unroll
  for (int o = 16, n = 8; n > 0; o >>= 1, n >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float mine = up ? v[i + n] : v[i], other = up ? v[i] : v[i + n];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}
MOE_DEVICE int column_of(int lane) {
  return (lane >> 4 & 1) * 8 + (lane >> 3 & 1) * 4 + (lane >> 2 & 1) * 2 + (lane >> 1 & 1);
}

// Two tokens' values of this lane's feature -> two features' of one token: even lanes get
// the first token's, odd lanes the second's; `pick` is 0x5410 in even lanes, 0x3276 in odd.
MOE_DEVICE uint32_t turn_pair(float2 v, uint32_t pick) {
  const uint32_t mine = pack_bf16x2(v.x, v.y);
  return __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick);
}

// 1 / (1 + e^-g) from the hardware's 2^x and 1 / x (2^-22 relative each)
MOE_DEVICE float sigmoid(float g) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// F32: the matrices' gradients in fp32, else bf16
template <int MODE, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
products_kernel(const __grid_constant__ Maps maps, const GradArgs a) {
  using C = Cfg<MODE>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  uint8_t* epi = smem + (size_t)kStages * C::kStageBytes;
  uint8_t* bar_area = epi + C::kEpiBytes;
  const uint32_t bar0 = smem_u32(bar_area);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };  // the leader's counts for both
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  // accumulators -- kAct: 0, 1 the two of a, 2 that of g and u; else 0, 1.  empty: the leader's
  auto acc_full = [&](uint32_t i) { return bar0 + 8u * (2 * kStages + i); };
  auto acc_empty = [&](uint32_t i) { return bar0 + 8u * (2 * kStages + 3 + i); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 6);
  auto sums_bar = [&](int half) { return drain_bar + 8u * (1 + half); };  // kAct: the four warps' sums
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 8 * C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, warp_id(), 0), lane = lane_id();
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), 2 * kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    for (int i = 0; i < 2; ++i) mbar_init(sums_bar(i), 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && elect_one()) {
    for (const CUtensorMap* m : {&maps.w1, &maps.w3, &maps.x, &maps.dout}) prefetch_tmap(m);
    for (const CUtensorMap* m : {MODE == kAct ? &maps.w2 : &maps.dgu, MODE == kAct ? &maps.w2 : &maps.act})
      prefetch_tmap(m);
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(tmem_slot), 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  auto fail = [&]() {
    moe_set_status(a.dev_status, MOE_DEV_WAIT_TIMEOUT);
    *abort_flag = 1;
  };
  Walk<MODE> walk(a, blockIdx.x >> 1, gridDim.x >> 1);
  Unit u;
  const int nkH = moe_cdiv(a.H, kBK), nkI = moe_cdiv(a.I, kBK);

  if (warp < 4) {
    if constexpr (MODE == kAct) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      // ---------------- TMA producer (the warp as a whole): this CTA's rows of A, its half of B
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      const uint32_t lead = cluster_addr(bar0, 0);
      uint32_t st = 0, bar = 0;  // the stage being filled and its barrier, in the leader
      // the next free stage, `bytes` expected in each CTA; whether this lane fills it
      auto take = [&](int bytes) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, kWaitNs));
        if (!ok) {
          fail();
          return false;
        }
        st = sbase + stage * C::kStageBytes;
        bar = lead + 8u * stage;
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        const bool me = elect_one();
        if (me && rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * bytes);
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
        return me;
      };
      while (ok && walk.next(u)) {
        const int m0 = u.m0 + 128 * rank, half = u.n / 2;
        if constexpr (MODE == kAct) {
          const int row = u.row + half * rank;
          for (int k0 = 0, k1; k0 < nkH && ok; k0 = k1) {
            k1 = min(nkH, k0 ? k0 + kChunk : first_chunk(nkH));
            for (int k = k0; k < k1 && ok; ++k)  // a = dout W2: W2 [H, I] lies MN-major
              if (take(kTile + kTile / 2)) {
                tma_load2_3d(st, &maps.w2, bar, m0, k * kBK, u.e);
                tma_load2_3d(st + kPanel, &maps.w2, bar, m0 + 64, k * kBK, u.e);
                tma_load2_3d(st + C::kB, &maps.dout, bar, k * kBK, row, 0);
              }
            for (int k = k0; k < k1 && ok; ++k)  // g, u
              if (take(2 * kTile + kTile / 2)) {
                tma_load2_3d(st, &maps.w1, bar, k * kBK, m0, u.e);
                tma_load2_3d(st + kTile, &maps.w3, bar, k * kBK, m0, u.e);
                tma_load2_3d(st + C::kB, &maps.x, bar, k * kBK, row, 0);
              }
          }
        } else if (u.part == kX) {
          const int row = u.row + half * rank;
          const bool two = half > 64;
          for (int part = 0; part < 2; ++part)  // W1 and W3 [I, H]: MN-major
            for (int k = 0; k < nkI && ok; ++k)
              if (take(kTile + (two ? 2 : 1) * kPanel)) {
                const CUtensorMap* w = part ? &maps.w3 : &maps.w1;
                tma_load2_3d(st, w, bar, m0, k * kBK, u.e);
                tma_load2_3d(st + kPanel, w, bar, m0 + 64, k * kBK, u.e);
                tma_load2_3d(st + C::kB, &maps.dgu, bar, k * kBK, row, part);
                if (two) tma_load2_3d(st + C::kB + kPanel, &maps.dgu, bar, k * kBK, row + 64, part);
              }
        } else {
          const int n0 = u.n0 + half * rank, part = u.part == kW3;
          const bool two = half > 64;
          const CUtensorMap* ma = u.part == kW2 ? &maps.dout : &maps.dgu;
          const CUtensorMap* mb = u.part == kW2 ? &maps.act : &maps.x;
          for (int r = u.row; r < u.row + u.m && ok; r += kBK)
            if (take(kTile + (two ? 2 : 1) * kPanel)) {
              tma_load2_3d(st, ma, bar, m0, r, part);
              tma_load2_3d(st + kPanel, ma, bar, m0 + 64, r, part);
              tma_load2_3d(st + C::kB, mb, bar, n0, r, 0);
              if (two) tma_load2_3d(st + C::kB + kPanel, mb, bar, n0 + 64, r, 0);
            }
        }
        __syncwarp();
      }
      // every copy that was started has landed before the pair moves on
      if (rank == 0) {
        for (int s = 0; s < kStages; ++s)
          if (armed & (1u << s))
            if (!mbar_wait_bounded(full_bar(s), (armed_parity >> s) & 1u, nullptr, kWaitNs)) fail();
      }
      // and the stages' last commits have arrived: they are sent to both CTAs, and one still on
      // its way would find the shared memory of this SM's next CTA.  (The accumulators' are
      // waited for by the epilogues, and the drain is the leader's alone.)
      for (int s = 0; s < kStages && ok; ++s)
        if (armed & (1u << s)) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(s), (armed_parity >> s) & 1u, abort_flag, kWaitNs));
          if (!ok) fail();
        }
      if (rank == 1 && (!ok || *abort_flag)) {
        // given up: the copies count in the leader and the commits are its own, so they get
        // their time
        const uint64_t t0 = globaltimer_ns();
        for (int i = 0; i < (1 << 20) && globaltimer_ns() - t0 < 1000000; ++i) __nanosleep(1000);
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA issuer, for the pair (the warp as a whole, one lane issues)
      int stage = 0;
      uint32_t phase = 0, n = 0;
      bool ok = true, issued = false;
      const uint32_t one = sbase >> 4;
      // the next stage, once it is filled
      auto filled = [&]() {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(full_bar(stage), phase, abort_flag, kWaitNs));
        if (!ok) fail();
        tc_fence_after();
        return one + stage * (C::kStageBytes >> 4);
      };
      auto used = [&]() {
        if (elect_one()) tc_commit2(empty_bar(stage));
        issued = true;
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      };
      auto free_acc = [&](uint32_t i, uint32_t use) {  // before the use-th time accumulator i is written
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(acc_empty(i), (use & 1u) ^ 1u, abort_flag, kWaitNs));
        if (!ok) fail();
        tc_fence_after();
      };
      auto done = [&](uint32_t i) {
        if (elect_one()) tc_commit2(acc_full(i));
      };
      // descriptors of an operand at 0, and how far 16 of K lie apart (in 16 bytes)
      const uint64_t dk = sdesc_k128_sw128(0), dmn = sdesc_mn_sw128(0, kPanel);
      constexpr int kK = 32 >> 4, kMn = 2048 >> 4;
      while (ok && walk.next(u)) {
        const uint32_t id = idesc_bf16_f32(kBM, u.n);
        if constexpr (MODE == kAct) {
          for (int k0 = 0, k1; k0 < nkH && ok; k0 = k1, ++n) {
            k1 = min(nkH, k0 ? k0 + kChunk : first_chunk(nkH));
            free_acc(n & 1u, n >> 1);
            for (int k = k0; k < k1 && ok; ++k) {
              const uint32_t A = filled(), d = tmem + 128 * (n & 1u);
              if (!ok) break;
              if (elect_one()) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  tc_mma2_f16(d, dmn + A + q * kMn, dk + A + (C::kB >> 4) + q * kK, id | kIdescMnA, k > k0 || q > 0);
              }
              used();
            }
            if (!ok) break;
            done(n & 1u);
            free_acc(2, n);
            for (int k = k0; k < k1 && ok; ++k) {
              const uint32_t A = filled();
              if (!ok) break;
              if (elect_one()) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const uint64_t b = dk + A + (C::kB >> 4) + q * kK;
                  tc_mma2_f16(tmem + 256, dk + A + q * kK, b, id, k > k0 || q > 0);
                  tc_mma2_f16(tmem + 384, dk + A + (kTile >> 4) + q * kK, b, id, k > k0 || q > 0);
                }
              }
              used();
            }
            if (!ok) break;
            done(2);
          }
        } else {
          // x: all of I, twice; the matrices: the expert's rows, the last stage's as far as they go
          const bool of_x = u.part == kX;
          const int k16 = of_x ? 8 * nkI : (u.m + 15) / 16;
          if (k16 == 0) continue;
          const uint32_t d = tmem + 256 * (n & 1u), idb = id | kIdescMnA | (of_x ? 0u : kIdescMnB);
          const uint64_t db = of_x ? dk : dmn;
          const int kb = of_x ? kK : kMn;
          free_acc(n & 1u, n >> 1);
          for (int k = 0; k < k16 && ok; k += 4) {
            const uint32_t A = filled(), B = A + (C::kB >> 4);
            if (!ok) break;
            if (elect_one()) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (k + q < k16) tc_mma2_f16(d, dmn + A + q * kMn, db + B + q * kb, idb, k > 0 || q > 0);
            }
            used();
          }
          if (!ok) break;
          done(n & 1u);
          ++n;
        }
      }
      if (issued) {
        // all MMAs of this warp complete before TMEM is released
        if (elect_one()) tc_commit2(drain_bar, kLeader);
        if (!mbar_wait_bounded(drain_bar, 0, nullptr, kWaitNs)) fail();
      }
    }
  } else {
    // ---------------- epilogue: lane quarter = warp % 4, alternate columns for the two of a quarter
    if constexpr (MODE == kAct) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t n = 0;
    bool ok = true;
    auto wait_acc = [&](uint32_t i, uint32_t use) {
      if (!mbar_wait_bounded(acc_full(i), use & 1u, abort_flag, kWaitNs)) {
        fail();
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    };
    auto release_acc = [&](uint32_t i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(acc_empty(i), 0));
    };
    if constexpr (MODE == kAct) {
      float* sums = reinterpret_cast<float*>(epi);  // [2][warps][64]
      float* wts = sums + (2 * kEpiWarps + warp - 4) * 64;
      for (uint32_t unit = 0; ok && walk.next(u); ++unit) {
        // a thread's feature, and the warp's columns (tokens): 64 each of a quarter's two, half
        // of a narrow tile's (of wider ones too: T = 4096, I = 2880 1900 -> 1930 us)
        const int i = u.m0 + 128 * rank + 32 * quarter + lane;
        const int span = u.n > 64 ? 64 : (u.n / 2 + 15) & ~15, col0 = span * half;
        const int last = min(u.n, col0 + span);
        // its tokens' weights, where the whole warp reads them
        __syncwarp();
        for (int t = lane; t < 64; t += 32)
          wts[t] = col0 + t < min(last, u.m) ? __ldg(a.weight + u.row + col0 + t) : 0.f;
        __syncwarp();
        float va[64], vg[64], vu[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) va[c] = vg[c] = vu[c] = 0.f;
        for (int k0 = 0; k0 < nkH && ok; k0 = k0 ? k0 + kChunk : first_chunk(nkH), ++n) {
          auto add = [&](uint32_t t, float (&v)[64]) {
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
              if (col0 + c >= last) continue;
              uint32_t r[16];
              tc_ld_32x32b_x16(t_lane + t + col0 + c, r);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float2 x = add2(make_float2(v[c + j], v[c + j + 1]),
                                      make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])));
                v[c + j] = x.x;
                v[c + j + 1] = x.y;
              }
            }
          };
          wait_acc(n & 1u, n >> 1);
          if (!ok) break;
          add(128 * (n & 1u), va);
          release_acc(n & 1u);
          wait_acc(2, n);
          if (!ok) break;
          add(256, vg);
          add(384, vu);
          release_acc(2);
        }
        if (!ok) break;
        float* mine = sums + ((unit & 1) * kEpiWarps + warp - 4) * 64;
        // 32 tokens at a time; the registers move up, so that the code is there once
        const bool in = i < a.I;
        const uint32_t pick = lane & 1 ? 0x3276u : 0x5410u;
        const size_t pitch = (size_t)a.I;
        __nv_bfloat16* to = a.dgu + (size_t)(u.row + col0 + (lane & 1)) * pitch + (i & ~1);
        __nv_bfloat16* to_act = a.act + (to - a.dgu);
        const size_t to_du = (size_t)a.Rp * pitch;
#pragma unroll 1
        for (int c = 0; col0 + c < last; c += 32) {
          if (col0 + c + 32 > u.m) {  // rows behind the last one: zeros for the matrices' sums
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col0 + c + j >= u.m) va[j] = vg[j] = vu[j] = 0.f;
          }
#pragma unroll
          for (int h = 0; h < 32; h += 16) {
            if (col0 + c + h >= last) continue;
            float share[16];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 w = *reinterpret_cast<const float2*>(wts + c + h + j);
              const float2 av = make_float2(va[h + j], va[h + j + 1]);
              const float2 g = make_float2(vg[h + j], vg[h + j + 1]);
              const float2 uv = make_float2(vu[h + j], vu[h + j + 1]);
              const float2 s = make_float2(sigmoid(g.x), sigmoid(g.y));
              const float2 gs = mul2(g, s), aw = mul2(av, w), t = mul2(gs, uv);
              const float2 sh = mul2(av, t);
              share[j] = sh.x;
              share[j + 1] = sh.y;
              const float2 f = fma2(gs, fma2(s, pair(-1.f), pair(1.f)), s);  // s (1 + g (1 - s))
              const uint32_t dg = turn_pair(mul2(mul2(aw, uv), f), pick);
              const uint32_t du = turn_pair(mul2(aw, gs), pick);
              if (in) {
                *reinterpret_cast<uint32_t*>(to) = dg;
                *reinterpret_cast<uint32_t*>(to + to_du) = du;
              }
              if (a.dw) {
                const uint32_t act = turn_pair(mul2(w, t), pick);
                if (in) *reinterpret_cast<uint32_t*>(to_act) = act;
              }
              to += 2 * pitch;
              to_act += 2 * pitch;
            }
            const float s = lane_sums16(share, lane);
            if ((lane & 1) == 0) mine[c + h + column_of(lane)] = s;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            va[j] = va[j + 32];
            vg[j] = vg[j + 32];
            vu[j] = vu[j + 32];
          }
        }
        // the four warps of these columns
        __syncwarp();
        if (lane == 0) mbar_arrive(sums_bar(half));
        if (!mbar_wait_bounded(sums_bar(half), unit & 1u, abort_flag, kWaitNs)) {
          fail();
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int t = 16 * quarter + lane;
        if (lane < 16 && col0 + t < min(last, u.m)) {
          const float* s = sums + ((unit & 1) * kEpiWarps + 4 * half) * 64 + t;
          a.share[(size_t)(u.m0 / 128 + rank) * a.Rp + u.row + col0 + t] =
              (s[0] + s[64]) + (s[128] + s[192]);
        }
      }
    } else {
      uint8_t* box = epi + (warp - 4) * kBoxBytes;
      constexpr int kCols = F32 ? 32 : 64;  // of a box
      while (ok && walk.next(u)) {
        if (u.part == kX) {
          wait_acc(n & 1u, n >> 1);
          if (!ok) break;
          const int h = u.m0 + 128 * rank + 32 * quarter + lane;
          const uint32_t t0 = t_lane + 256 * (n & 1u);
          for (int c = 16 * half; c < u.m; c += 32) {
            uint32_t v[16];
            tc_ld_32x32b_x16(t0 + c, v);
            tc_wait_ld();
            float* to = a.rows + (size_t)(u.row + c) * a.H + h;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < u.m && h < a.H) to[(size_t)j * a.H] = __uint_as_float(v[j]);
          }
          release_acc(n & 1u);
          ++n;
          continue;
        }
        const int r0 = u.m0 + 128 * rank + 32 * quarter;  // the warp's first row of the matrix
        const bool in = r0 < (u.part == kW2 ? a.H : a.I);
        const CUtensorMap* map = u.part == kW1 ? &maps.d1 : u.part == kW3 ? &maps.d3 : &maps.d2;
        const int c1 = in ? min(u.n, half * 128 + 128) : 0;
        if (u.m == 0) {
          // an expert without rows: zeros, or nothing to add
          if (a.accumulate) continue;
          for (int c = half * 128; c < c1; c += kCols) {
            box_wait(lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) box_piece(box, lane, i, make_uint4(0u, 0u, 0u, 0u));
            box_store(map, box, lane, u.n0 + c, r0, u.e, false);
          }
          continue;
        }
        wait_acc(n & 1u, n >> 1);
        if (!ok) break;
        const uint32_t t0 = t_lane + 256 * (n & 1u) + 128 * half;
        if constexpr (F32) {
          for (int c = 128 * half; c < c1; c += kCols) {
            uint32_t v[32];
            tc_ld_32x32b_x32(t0 - 128 * half + c, v);
            tc_wait_ld();
            box_wait(lane);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              box_piece(box, lane, i, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
            box_store(map, box, lane, u.n0 + c, r0, u.e, a.accumulate);
          }
          release_acc(n & 1u);
        } else {
          // the second half's columns are read while the store takes the first's
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              uint32_t v[32];
              tc_ld_32x32b_x32(t0 + 64 * c + 32 * b, v);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                o[16 * b + j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            }
            if (c == 1) release_acc(n & 1u);
            if (128 * half + 64 * c >= c1) continue;
            box_wait(lane);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              box_piece(box, lane, i, make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
            box_store(map, box, lane, u.n0 + 128 * half + 64 * c, r0, u.e, false);
          }
        }
        ++n;
      }
      if (lane == 0) bulk_wait();  // the stores are done before the CTA is
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may still reach it
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem, 512);
}

// ---------------------------------------------------------------- finish
struct FinishArgs {
  const float4* rows;  // [Rp][H]
  const float* share;  // [shares][Rp]
  const int32_t* place;
  const uint4* add;
  uint4* dx;
  float* d_weights;
  long long Rp;
  int T, K, H, shares;
};

// The padded row of replica f: -1 where it was dropped (or where the maps contradict each
// other and its place was never written).
MOE_DEVICE int padded_row(const FinishArgs& a, long long f) {
  const int p = __ldg(a.place + f);
  return p >= 0 && p < a.Rp ? p : -1;
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
  const cudaError_t e = moe_raise_smem(products_kernel<MODE, F32>, Cfg<MODE>::kSmemBytes, set);
  if (e != cudaSuccess) return e;
  return moe_launch_clusters(products_kernel<MODE, F32>, dim3(moe_num_sms() & ~1), dim3(kThreads),
                             Cfg<MODE>::kSmemBytes, stream, dim3(2), maps, a);  // pairs lie along x
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
  GradArgs a{};
  a.plan = reinterpret_cast<const Plan*>(s);
  a.weight = reinterpret_cast<const float*>(s + l.weight);
  a.share = reinterpret_cast<float*>(s + l.share);
  a.dgu = reinterpret_cast<__nv_bfloat16*>(dgu);
  a.act = reinterpret_cast<__nv_bfloat16*>(act);
  a.rows = reinterpret_cast<float*>(s + l.dx);
  a.Rp = l.Rp; a.H = H; a.I = I; a.E = E;
  a.dx = g.dx != nullptr && R > 0;
  a.dw = g.dw1 != nullptr;
  a.accumulate = g.accumulate;
  a.dev_status = g.dev_status;

  RowArgs r{};
  r.x = static_cast<const uint4*>(g.x); r.dout = static_cast<const uint4*>(g.dout);
  r.xq = static_cast<const uint4*>(g.xq); r.xs = g.xq_scale;
  r.offsets = g.offsets; r.row_to_flat = g.row_to_flat; r.flat_to_row = g.flat_to_row;
  r.weights = g.weights;
  r.R = R; r.H = H; r.E = E; r.K = K;
  r.at_once = moe_num_sms() / 2 / moe_cdiv(I, kBM);
  r.plan = reinterpret_cast<Plan*>(s);
  for (int i = 0; i < 2; ++i) a.tile[i] = r.tile[i] = reinterpret_cast<Tile*>(s + l.tile[i]);
  r.place = reinterpret_cast<int32_t*>(s + l.place);
  r.weight = reinterpret_cast<float*>(s + l.weight);
  r.xp = reinterpret_cast<uint4*>(xp); r.dp = reinterpret_cast<uint4*>(dp);
  const int blocks = (int)(l.Rp / 4 < 152 * 8 ? l.Rp / 4 : 152 * 8);
  cudaError_t e = moe_launch(g.xq ? rows_kernel<true> : rows_kernel<false>, dim3(blocks), dim3(256), 0,
                             stream, 1, r);
  if (e != cudaSuccess) return e;

  Maps m{};
  bool ok = bf16_map_3d(&m.w1, g.w1, H, I, E, 64, 128) && bf16_map_3d(&m.w3, g.w3, H, I, E, 64, 128) &&
            bf16_map_3d(&m.w2, g.w2, I, H, E, 64, 64) && bf16_map_3d(&m.x, xp, H, l.Rp, 1, 64, 64) &&
            bf16_map_3d(&m.dout, dp, H, l.Rp, 1, 64, 64);
  if (!ok) return cudaErrorInvalidValue;
  if (R > 0 && (e = run_products<kAct, false>(m, a, stream)) != cudaSuccess) return e;

  if (a.dx || a.dw) {
    ok = bf16_map_3d(&m.w1, g.w1, H, I, E, 64, 64) && bf16_map_3d(&m.w3, g.w3, H, I, E, 64, 64) &&
         bf16_map_3d(&m.dgu, dgu, I, l.Rp, 2, 64, 64) && bf16_map_3d(&m.act, act, I, l.Rp, 1, 64, 64);
    auto out = [&](CUtensorMap* map, void* p, int n0, int n1) {
      return g.dw_f32 ? f32_map_3d(map, p, n0, n1, E, 32, 32) : bf16_map_3d(map, p, n0, n1, E, 64, 32);
    };
    if (a.dw) ok = ok && out(&m.d1, g.dw1, H, I) && out(&m.d3, g.dw3, H, I) && out(&m.d2, g.dw2, I, H);
    if (!ok) return cudaErrorInvalidValue;
    e = g.dw_f32 ? run_products<kBack, true>(m, a, stream) : run_products<kBack, false>(m, a, stream);
    if (e != cudaSuccess) return e;
  }
  if (R == 0 || (!g.dx && !g.d_weights)) return cudaSuccess;
  FinishArgs f{reinterpret_cast<const float4*>(a.rows), a.share, r.place,
               static_cast<const uint4*>(g.dx_add), static_cast<uint4*>(g.dx), g.d_weights, l.Rp, T, K, H,
               l.shares};
  const long long warps = (g.dx ? (long long)T * moe_cdiv(H / 8, 32) : 0) + (g.d_weights ? moe_cdiv(R, 32) : 0);
  return moe_launch(finish_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, stream, 1, f);
}
