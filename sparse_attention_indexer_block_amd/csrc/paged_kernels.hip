// Rows of latents or indexer keys into the pages of their sequences, normed, rotated
// by their position and coded on the way, and the rotation of queries.
//
//   lat = x[0:d] * weight / sqrt(mean(x[0:d]^2) + eps)   (or x[0:d])
//   (a, b) -> (a cos - b sin, b cos + a sin)             the 64 rotary values, in 32 pairs
//   code = lat / scale                                   scale as misa_cache_write
//
// Values are formed in fp32 and rounded once, as they are stored.
#include "attention.h"
#include "row_device.h"

namespace misa {

// D / 8 lanes a row, eight values a lane. What a row waits for is two loads one after
// the other (its position, then its page and its angles), beside which the row itself
// is read and normed. Several rows a wave with all their loads in flight gained nothing
// (16383 coded latents: 11.7 us with one row a wave, 12.4 with two, 13.9 with four; 33.7 MB,
// 2.9 TB/s: bound by that chain, and the launch). 32 rows 3.6 us, 5015 keys of 128 3.2, of
// which the launch is 1.7.
template <int D, int DR, bool FP8>
__global__ __launch_bounds__(256) void k_paged_append(AppendArgs p) {
  constexpr int LPR = D / 8, RPB = 256 / LPR;
  const int tid = threadIdx.x, sub = tid % LPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + tid / LPR, rr = min(row, (int64_t)p.cache.n - 1);
  const int seq = p.seq[rr], pos = p.pos[rr], turn = p.turn[rr];
  const uint16_t* xr = p.x + rr * p.x_ld;
  const u32x4 v = *reinterpret_cast<const u32x4*>(xr + sub * 8);
  u32x4 vr = {0u, 0u, 0u, 0u};
  if (DR && sub < DR / 8) vr = *reinterpret_cast<const u32x4*>(xr + D + sub * 8);
  float w[8];
  if (p.weight) load_weights(p.weight, p.weight_f32, sub * 8, w);
  const int lg = p.pages.page_log2, page = pos >> lg;
  bool live = row < p.cache.n && seq >= 0 && seq < p.pages.seqs && pos >= 0 && page < p.pages.per;
  const int entry = live ? p.pages.table[(int64_t)seq * p.pages.per + page] : -1;
  const bool turns = p.rot.rot != nullptr, placed = turn >= 0 && turn < p.rot.positions;
  const float* cs = p.rot.rot + (int64_t)(placed ? turn : 0) * kRotary;
  live = live && (placed || !turns);

  float x[8], rot[8];
  unpack8(v, x);
  unpack8(vr, rot);
  if (DR && turns) rotate8(rot, sub & 7, cs, p.rot.pairs);
  if (p.weight) scale_row(x, inverse_rms(sum_of<LPR>(squares(x, 0.0)), p.inv_width, p.eps), w);
  if (!DR && turns) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    rotate8(y, sub & 7, cs, p.rot.pairs);
    const bool turned = (unsigned)(sub * 8 - p.rot_at) < (unsigned)kRotary;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = turned ? y[i] : x[i];
  }
  const RowCode code(FP8 ? max_of<LPR>(magnitude_bits(x)) : 0u);
  const int64_t slot = ((int64_t)entry << lg) + (pos & ((1 << lg) - 1));
  if (!live || entry < 0 || slot >= p.cache.rows) return;
  if constexpr (FP8) {
    *reinterpret_cast<u32x2*>(static_cast<unsigned char*>(p.cache.c) + slot * D + sub * 8) = code.eight(x);
    if (DR && sub < DR / 8) *reinterpret_cast<u32x4*>(p.cache.rope + slot * DR + sub * 8) = pack8(rot);
    if (sub == 0) p.cache.scale[slot] = code.scale;
  } else {
    uint16_t* to = static_cast<uint16_t*>(p.cache.c) + slot * (D + DR);
    *reinterpret_cast<u32x4*>(to + sub * 8) = pack8(x);
    if (DR && sub < DR / 8) *reinterpret_cast<u32x4*>(to + D + sub * 8) = pack8(rot);
  }
}

// Eight lanes a row of 64 values: a workgroup's 32 rows are 4 KB in a piece where heads are
// dense, and a position's 256 bytes of cosines and sines come from the caches for all heads
// but its first. Bound by memory: 8192 x 64 rows, 136 MB in 30.5 us, 4.5 TB/s; 64 x 128 rows 2.8.
__global__ __launch_bounds__(256) void k_rotate(RotateArgs p) {
  const int64_t rows = (int64_t)p.T * p.H;
  const int64_t row = (int64_t)blockIdx.x * 32 + threadIdx.x / 8, rr = min(row, rows - 1);
  const int sub = threadIdx.x & 7, t = (int)(rr / p.H), h = (int)(rr % p.H);
  const int pos = p.pos[t];
  const bool live = row < rows && pos >= 0 && pos < p.rot.positions;
  float x[8];
  unpack8(*reinterpret_cast<const u32x4*>(p.x + t * p.x_t + h * p.x_h + sub * 8), x);
  rotate8(x, sub, p.rot.rot + (int64_t)(live ? pos : 0) * kRotary, p.rot.pairs);
  if (live) *reinterpret_cast<u32x4*>(p.out + t * p.out_t + h * p.out_h + sub * 8) = pack8(x);
}

template <int D, int DR>
static hipError_t append_shape(const LaunchCtx& cx, const AppendArgs& a, bool fp8) {
  constexpr int RPB = 2048 / D;
  const dim3 grid((unsigned)(((int64_t)a.cache.n + RPB - 1) / RPB));
  return fp8 ? cx.launch("k_paged_append", k_paged_append<D, DR, true>, grid, dim3(256), 0, a)
             : cx.launch("k_paged_append", k_paged_append<D, DR, false>, grid, dim3(256), 0, a);
}

hipError_t launch_paged_append(const LaunchCtx& cx, AppendArgs a, bool fp8) {
  a.inv_width = 1.0 / a.cache.d;
  if (a.cache.d == kLatent)
    return a.cache.dr ? append_shape<kLatent, kRotary>(cx, a, fp8) : append_shape<kLatent, 0>(cx, a, fp8);
  return a.cache.dr ? append_shape<kHeadDim, kRotary>(cx, a, fp8) : append_shape<kHeadDim, 0>(cx, a, fp8);
}

hipError_t launch_rotate(const LaunchCtx& cx, const RotateArgs& a) {
  const int64_t rows = (int64_t)a.T * a.H;
  return cx.launch("k_rotate", k_rotate, dim3((unsigned)((rows + 31) / 32)), dim3(256), 0, a);
}

}  // namespace misa
