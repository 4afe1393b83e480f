// Attention over one shared latent vector a token, in absorbed form:
//
//   S[r,s]  = sm * (q[r, 0:512] . c[s] + q[r, 512:576] . rope[s])
//   out[r]  = sum_s softmax_s(S[r,:]) c[s],   lse[r] = log sum_s exp(S[r,s])
//
// for the rows r = (query, head) of one query, over the keys of the query's
// list or over its visible keys. All heads of a query read the same keys, and
// a key row is its own value row.
#include <algorithm>

#include "latent_device.h"

namespace misa {

// Joins the splits of a row: each split's sums and total weigh 2^(its reference
// - the largest). COLS / 4 threads hold COLS of a row's WIDTH values; SG such groups
// take the splits in turn and are added through LDS in a fixed order, and the rest of
// the workgroup takes further rows. Bound by memory where there is much (4096 rows of
// 512 values in 4 splits: 34 MB in 7 us), by latency where there is little (4 us).
template <int WIDTH, int COLS, int SG>
__global__ __launch_bounds__(256) void k_join(const float* part, const float* part_ml, int splits, int64_t rows,
                                              uint16_t* out, float* lse) {
  constexpr int TPR = COLS / 4, ROWS = 256 / TPR / SG, PARTS = WIDTH / COLS;
  __shared__ __attribute__((aligned(16))) float sums[ROWS][SG][COLS];
  __shared__ float tots[ROWS][SG];
  const int c = threadIdx.x % TPR, sg = threadIdx.x / TPR % SG, rr = threadIdx.x / TPR / SG;
  const int64_t row = (int64_t)(blockIdx.x / PARTS) * ROWS + rr, r = min(row, rows - 1);
  const int col = (int)(blockIdx.x % PARTS) * COLS + c * 4;
  float top = -INFINITY;
  for (int s = threadIdx.x & 31; s < splits; s += 32) {
    const f32x2 ml = *reinterpret_cast<const f32x2*>(part_ml + ((int64_t)s * rows + r) * 2);
    top = fmaxf(top, no_keys(ml.y) ? -INFINITY : ml.x);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));  // (32 lanes share a row)
  const bool keys = top > -INFINITY;
  top = fmaxf(top, kNoMax);
  float tot = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = sg; s < splits; s += SG) {
    const float* ml = part_ml + ((int64_t)s * rows + r) * 2;
    const float f = exp2_fast(ml[0] - top);
    tot += f * ml[1];
    acc += *reinterpret_cast<const f32x4*>(part + ((int64_t)s * rows + r) * WIDTH + col) * f;
  }
  if constexpr (SG > 1) {
    *reinterpret_cast<f32x4*>(&sums[rr][sg][c * 4]) = acc;
    if (c == 0) tots[rr][sg] = tot;
    __syncthreads();
    if (sg != 0) return;
#pragma unroll
    for (int i = 1; i < SG; ++i) {
      acc += *reinterpret_cast<const f32x4*>(&sums[rr][i][c * 4]);
      tot += tots[rr][i];
    }
  }
  if (row >= rows) return;
  tot = row_total(keys, tot);
  const float inv = row_inverse(tot);
  *reinterpret_cast<bf16x4*>(out + r * WIDTH + col) = __builtin_convertvector(acc * inv, bf16x4);
  if (lse && col == 0) lse[r] = row_log_sum(top, tot);
}

template <int WIDTH, int COLS, int SG>
static hipError_t join_as(const LaunchCtx& cx, const float* part, const float* part_ml, int splits, int64_t rows,
                          uint16_t* out, float* lse) {
  constexpr int ROWS = 256 / (COLS / 4) / SG;
  return cx.launch("k_join", k_join<WIDTH, COLS, SG>, dim3((unsigned)((rows + ROWS - 1) / ROWS * (WIDTH / COLS))), dim3(256),
                   0, part, part_ml, splits, rows, out, lse);
}

// A workgroup for 128 values of a row where a row has many splits or there are few
// rows to fill the card with, otherwise whole rows.
hipError_t launch_join(const LaunchCtx& cx, const float* part, const float* part_ml, int splits, int64_t rows,
                       int width, uint16_t* out, float* lse) {
  if (width == kLatent)
    return splits > 8 || rows < 1024 ? join_as<kLatent, 128, 8>(cx, part, part_ml, splits, rows, out, lse)
                                     : join_as<kLatent, kLatent, 1>(cx, part, part_ml, splits, rows, out, lse);
  return splits > 8 || rows < 1024 ? join_as<kValue, kValue, 8>(cx, part, part_ml, splits, rows, out, lse)
                                   : join_as<kValue, kValue, 1>(cx, part, part_ml, splits, rows, out, lse);
}

static int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Rows per workgroup and splits of the keys: the cheapest of four widths by what
// they cost on this card, in us. A workgroup starts and ends in `fixed`, a tile
// of 64 keys takes `tile` (more rows amortise the gather of a tile, fewer leave
// less to write where the keys are split), 256 run at a time, and partial sums
// (2 KB a row and split) are written and joined at 2.3 TB/s after 3.5 of launch and
// 0.05 a split. The constants are fitted to 500 measured calls (1 to 1024 queries, 3
// to 128 heads, lists and prefixes of 100 to 100003 keys, codes and bf16); what this
// rule chooses is 1% off the fastest cut in the mean and 16% at worst.
// Measured, each width with the cheapest of its splits, lists of 2048 coded keys, 128
// heads (16 / 32 / 64 / 128 rows): 8 queries 30 / 31 / 31 / 39 us, 32 queries
// 69 / 54 / 43 / 49, 256 queries 535 / 329 / 184 / 163, 1024 queries
// 2158 / 1318 / 733 / 641; 4 queries of 32 heads over 100003 bf16 keys
// 153 / 91 / 62 / 61; 512 causal queries of 16 heads over 4096 keys, where a unit of
// 32 rows is half empty, 247 / 157 / 152 / 157.
AttnPlan latent_plan(int T, int H, int keys, bool shared_keys) {
  struct Width {
    int rows, unit;
    double fixed, tile;
  };
  static const Width widths[] = {{16, 16, 9.0, 1.8}, {32, 16, 11.0, 2.2}, {64, 32, 13.0, 2.25}, {128, 32, 12.0, 3.8}};
  const int tiles = std::max(1, cdiv(keys, kAttnTile));
  AttnPlan best{};
  double least = 0.0;
  for (const Width& w : widths) {
    AttnPlan pl{};
    pl.nq = w.rows;
    // units of queries that read the same keys share a tile
    pl.head_tiles = shared_keys ? 0 : cdiv(H, w.rows);
    const int64_t row_tiles = shared_keys ? ((int64_t)cdiv(H, w.unit) * w.unit * T + w.rows - 1) / w.rows
                                          : (int64_t)T * pl.head_tiles;
    pl.row_tiles = (int)row_tiles;
    const int most = (int)std::max<int64_t>(1, std::min<int64_t>(256 / row_tiles, tiles));
    for (int want = 1;; want = std::min(2 * want, most)) {
      const int share = cdiv(tiles, want);  // tiles of a split
      pl.splits = cdiv(tiles, share);
      const double rounds = (double)((row_tiles * pl.splits + 255) / 256);
      double cost = rounds * (w.fixed + share * w.tile);
      if (pl.splits > 1) cost += 3.5 + 0.05 * pl.splits + (double)pl.splits * T * H * (kLatent * 4) / 2.3e6;
      if (best.nq == 0 || cost < least) best = pl, least = cost;
      if (want == most) break;
    }
  }
  return best;
}

size_t latent_ws_bytes(const AttnPlan& pl, int T, int H) {
  if (pl.splits <= 1) return 256;
  const size_t rows = (size_t)T * H;
  return 256 + rows * pl.splits * (kLatent + 2) * 4;
}

// (launches are named by the rows of a workgroup, so that a profile says how a call was cut)
template <int NQ, bool FP8>
static hipError_t launch_latent_nq(const LaunchCtx& cx, const LatentArgs& a, dim3 grid) {
  const char* name = NQ == 16 ? "k_latent_16" : "k_latent_32";
  return a.idx ? cx.launch(name, k_latent<NQ, FP8, ListForm>, grid, dim3(256), 0, a)
               : cx.launch(name, k_latent<NQ, FP8, PrefixForm>, grid, dim3(256), 0, a);
}

template <int G, bool FP8>
static hipError_t launch_latent_wide(const LaunchCtx& cx, const LatentArgs& a, dim3 grid) {
  const char* name = G == 2 ? "k_latent_wide_64" : "k_latent_wide_128";
  return a.idx ? cx.launch(name, k_latent_wide<G, FP8, ListForm>, grid, dim3(256), 0, a)
               : cx.launch(name, k_latent_wide<G, FP8, PrefixForm>, grid, dim3(256), 0, a);
}

template <bool FP8>
static hipError_t launch_latent_t(const LaunchCtx& cx, const LatentArgs& a, int nq, dim3 grid) {
  switch (nq) {
    case 16: return launch_latent_nq<16, FP8>(cx, a, grid);
    case 32: return launch_latent_nq<32, FP8>(cx, a, grid);
    case 64: return launch_latent_wide<2, FP8>(cx, a, grid);
    default: return launch_latent_wide<4, FP8>(cx, a, grid);
  }
}

hipError_t launch_latent(const LaunchCtx& cx, LatentArgs a, const AttnPlan& pl, bool fp8, void* ws) {
  const int64_t rows = (int64_t)a.T * a.H;
  a.splits = pl.splits;
  a.head_tiles = pl.head_tiles;
  a.row_tiles = pl.row_tiles;
  if (pl.splits > 1) {
    a.part = static_cast<float*>(ws);
    a.part_ml = a.part + rows * pl.splits * kLatent;
  }
  const int64_t n = (int64_t)pl.row_tiles * pl.splits;
  const dim3 grid((unsigned)((n + 7) / 8 * 8));
  const hipError_t e = fp8 ? launch_latent_t<true>(cx, a, pl.nq, grid) : launch_latent_t<false>(cx, a, pl.nq, grid);
  if (e != hipSuccess || pl.splits <= 1) return e;
  return launch_join(cx, a.part, a.part_ml, pl.splits, rows, kLatent, a.out, a.lse);
}

}  // namespace misa
