// Root-mean-square norm of rows, with the addition of a residual before it and, if
// asked for, a result coded to E4M3FN with a scale for each row or each 128 columns:
//
//   h = x + residual,  sum = h in bf16,  y = (h / sqrt(mean(h^2) + eps)) * weight
//
// h, y and the scales are formed in fp32 and each result is rounded once.
#include "attention.h"
#include "row_device.h"

namespace misa {

// W waves a row, CH chunks of eight values a lane (chunk = thread + 64 W i); a
// workgroup of four waves takes 4 / W rows, or one of more waves. A row is read once
// and stays in registers; the squares are summed in fp64, so that the root, and the scales of
// codes with it, depend on the order only next to a rounding border (see squares). Bound by memory: 16,384 rows of 4096 with residual, to
// codes with a scale for 128 columns, 472 MB in 84 us, 5.6 TB/s (a plain copy, which writes
// as much as it reads, 4.9); eight rows 3.7 us, of which 1.7 are the launch and the rest the
// loads and two barriers one after the other.
template <int W, int CH, NormOut OUT>
__global__ __launch_bounds__(W > 4 ? 64 * W : 256) void k_rms_norm(NormArgs p) {
  constexpr int ROWS = W > 4 ? 1 : 4 / W, TPR = 64 * W;
  __shared__ double sums[ROWS * W];
  __shared__ uint32_t tops[ROWS * W];
  const int tid = threadIdx.x, lane = tid & 63, in_row = tid % TPR, rr = tid / TPR, wave = tid / 64;
  const int64_t row = (int64_t)blockIdx.x * ROWS + rr;
  const bool live = row < p.n;
  const int64_t r = live ? row : p.n - 1;
  const int chunks = p.width / 8;
  u32x4 vx[CH], vr[CH];
  float w[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = min(in_row + TPR * i, chunks - 1);
    vx[i] = *reinterpret_cast<const u32x4*>(p.x + r * p.x_ld + c * 8);
    if (p.residual) vr[i] = *reinterpret_cast<const u32x4*>(p.residual + r * p.width + c * 8);
    load_weights(p.weight, p.weight_f32, c * 8, w[i]);
  }
  float h[CH][8];
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = in_row + TPR * i;
    unpack8(vx[i], h[i]);
    if (p.residual) {
      float b[8];
      unpack8(vr[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += b[j];
    }
    if (c < chunks) {
      sum = squares(h[i], sum);
      if (p.sum && live) *reinterpret_cast<u32x4*>(p.sum + row * p.width + c * 8) = pack8(h[i]);
    }
  }
  sum = sum_of<64>(sum);
  if constexpr (W > 1) {
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) sum += sums[rr * W + i];
  }
  const float inv = inverse_rms(sum, p.inv_width, p.eps);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = in_row + TPR * i;
    scale_row(h[i], inv, w[i]);
    if constexpr (OUT == NormOut::kBf16) {
      if (c < chunks && live) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.y) + row * p.width + c * 8) = pack8(h[i]);
    } else if constexpr (OUT == NormOut::kGroupCodes) {
      const RowCode code(max_of_16(c < chunks ? magnitude_bits(h[i]) : 0u));
      if (c < chunks && live) {
        *reinterpret_cast<u32x2*>(static_cast<unsigned char*>(p.y) + row * p.width + c * 8) = code.eight(h[i]);
        if ((lane & 15) == 0) p.scale[row * ((chunks + 15) / 16) + c / 16] = code.scale;
      }
    } else {
      if (c < chunks) top = max(top, magnitude_bits(h[i]));
    }
  }
  if constexpr (OUT == NormOut::kRowCodes) {
    top = wave_max_u32(top);
    if constexpr (W > 1) {
      if (lane == 0) tops[wave] = top;
      __syncthreads();
      top = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) top = max(top, tops[rr * W + i]);
    }
    const RowCode code(top);
    if (!live) return;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = in_row + TPR * i;
      if (c < chunks) *reinterpret_cast<u32x2*>(static_cast<unsigned char*>(p.y) + row * p.width + c * 8) = code.eight(h[i]);
    }
    if (in_row == 0) p.scale[row] = code.scale;
  }
}

template <int W, int CH>
static hipError_t norm_as(const LaunchCtx& cx, const NormArgs& a, NormOut out) {
  constexpr int ROWS = W > 4 ? 1 : 4 / W;
  const dim3 grid((unsigned)(((int64_t)a.n + ROWS - 1) / ROWS)), block(W > 4 ? 64 * W : 256);
  switch (out) {
    case NormOut::kBf16: return cx.launch("k_rms_norm", k_rms_norm<W, CH, NormOut::kBf16>, grid, block, 0, a);
    case NormOut::kRowCodes: return cx.launch("k_rms_norm", k_rms_norm<W, CH, NormOut::kRowCodes>, grid, block, 0, a);
    default: return cx.launch("k_rms_norm", k_rms_norm<W, CH, NormOut::kGroupCodes>, grid, block, 0, a);
  }
}

// One chunk a lane up to eight waves a row: more and shorter rows in flight hide more of
// the loads, and a row of one wave meets no barrier. Measured with the residual and bf16 out,
// 64 M values (us): 512 columns, one wave 93, four 157; 1024, two 91.5, four 99, one of four
// chunks 92; 2048, four 91, one of four chunks 95; 4096, eight 89, four of two chunks 93.5;
// 8192, eight 92.5, four of four chunks 96; 16384, sixteen 94, eight of four chunks 97. Codes
// of 4096 columns write less a row: four waves 84, eight 86.
hipError_t launch_rms_norm(const LaunchCtx& cx, NormArgs a, NormOut out) {
  a.inv_width = 1.0 / a.width;
  if (a.width <= 512) return norm_as<1, 1>(cx, a, out);
  if (a.width <= 1024) return norm_as<2, 1>(cx, a, out);
  if (a.width <= 2048) return norm_as<4, 1>(cx, a, out);
  if (a.width <= 4096) return out == NormOut::kBf16 ? norm_as<8, 1>(cx, a, out) : norm_as<4, 2>(cx, a, out);
  if (a.width <= 8192) return norm_as<8, 2>(cx, a, out);
  return norm_as<16, 2>(cx, a, out);
}

}  // namespace misa
