// Device helpers of the kernels that make rows: the norm, the rotation and the
// coding of fp32 values (gfx950). Products and sums are rounded one by one here (no
// contraction): a row's scale is a power of two, which a last bit may move.
#pragma once

#include "attention_device.h"

namespace misa {

// Scale of a coded row from the bits of its largest magnitude (NaN above infinity):
// 2^e, the smallest e >= -126 with max|x| <= 448 * 2^e, and what values are divided by.
struct RowCode {
  float scale, inv;
  bool bad;  // an infinity or NaN: the row reads back as NaN
  __device__ __forceinline__ explicit RowCode(uint32_t top) {
    // 448 = 1.75 * 2^8: the exponent of top less 8, one more if its fraction is over 0.75
    const int e = max(-126, (int)(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
    bad = top >= 0x7f800000u;
    scale = bad ? __uint_as_float(0x7fc00000u) : top == 0 ? 1.f : __uint_as_float((uint32_t)(e + 127) << 23);
    inv = top == 0 ? 1.f : __uint_as_float((uint32_t)(127 - e) << 23);
  }
  __device__ __forceinline__ uint32_t four(const float* y) const {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * inv, y[1] * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * inv, y[3] * inv, w, true);
    return bad ? 0x7f7f7f7fu : (uint32_t)w;
  }
  __device__ __forceinline__ u32x2 eight(const float (&y)[8]) const { return u32x2{four(y), four(y + 4)}; }
};
__device__ __forceinline__ uint32_t magnitude_bits(const float (&y)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
  return top;
}

// Maximum over groups of 16 lanes, and over the wave.
__device__ __forceinline__ uint32_t max_of_16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x128, 0xf, 0xf, false));  // row_ror:8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x124, 0xf, 0xf, false));  // row_ror:4
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x122, 0xf, 0xf, false));  // row_ror:2
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x121, 0xf, 0xf, false));  // row_ror:1
}

__device__ __forceinline__ void unpack8(u32x4 v, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_bits_to_f32(v[i] & 0xffffu);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (__bf16)x[i];
  return __builtin_bit_cast(u32x4, r);
}

// Eight weights of a norm, bf16 or fp32.
__device__ __forceinline__ void load_weights(const void* weight, bool f32, int at, float (&w)[8]) {
  if (f32) {
    const float* p = static_cast<const float*>(weight) + at;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = a[i], w[4 + i] = b[i];
  } else {
    unpack8(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(weight) + at), w);
  }
}

// The sum of squares of a row is held in 64 bits: a square of an fp32 value is exact
// there and no magnitude overflows. Each addition rounds (2^-53), up to 38 of them one
// after the other (a lane's values, then lanes, then waves), so the sum is off by less
// than 2^-47 of itself in whatever order, and another order gives another fp32 root only
// where the root lies within 2^-47 of itself from a border of fp32's rounding.
__device__ __forceinline__ double squares(const float (&x)[8], double sum) {
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fma((double)x[i], (double)x[i], sum);
  return sum;
}
// 1 / sqrt(sum * inv_width + eps): the hardware's estimate and two steps of Newton's method,
// which leave it within a few 2^-53, then one rounding. (Library division and root take
// some hundred instructions, which a row's whole workgroup would wait for.)
__device__ __forceinline__ float inverse_rms(double sum, double inv_width, double eps) {
  const double a = fma(sum, inv_width, eps);
  double y = __builtin_amdgcn_rsq(a);
  const double first = y;
#pragma unroll
  for (int i = 0; i < 2; ++i) y = fma(y, fma(-0.5 * a * y, y, 0.5), y);
  return (float)(a > 0.0 && a < (double)INFINITY ? y : first);  // (0 and infinity are exact)
}
// Sum over groups of LANES (16 or 64) lanes, in every lane.
template <int LANES>
__device__ __forceinline__ double sum_of(double v) {
  auto step = [&](auto move) {
    const u32x2 b = __builtin_bit_cast(u32x2, v);
    v += __builtin_bit_cast(double, u32x2{move(b.x), move(b.y)});
  };
  step([](uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xf, 0xf, false); });  // row_ror:8
  step([](uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x124, 0xf, 0xf, false); });  // row_ror:4
  step([](uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x122, 0xf, 0xf, false); });  // row_ror:2
  step([](uint32_t x) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x121, 0xf, 0xf, false); });  // row_ror:1
  if constexpr (LANES == 64) {
    auto lane = [&](int i) {
      const u32x2 b = __builtin_bit_cast(u32x2, v);
      return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)b.x, i), (uint32_t)__builtin_amdgcn_readlane((int)b.y, i)});
    };
    v = (lane(0) + lane(16)) + (lane(32) + lane(48));
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  if constexpr (LANES == 64) return wave_max_u32(v);
  return max_of_16(v);
}
__device__ __forceinline__ void scale_row(float (&x)[8], float r, const float (&w)[8]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (x[i] * r) * w[i];
}

// Turns the eight values that lane `sub` (0..7) of a row's 64 rotary ones holds, by
// the angles whose cosines and sines lie at cs. All lanes of the wave come here; the
// partner of value i is i + 32, four lanes on, or (pairs) its neighbour.
__device__ __forceinline__ void rotate8(float (&x)[8], int sub, const float* cs, bool pairs) {
#pragma clang fp contract(off)
  float other[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) other[i] = __shfl_xor(x[i], 4, kWave);
  if (pairs) {
    const f32x4 c = *reinterpret_cast<const f32x4*>(cs + 4 * sub), s = *reinterpret_cast<const f32x4*>(cs + 32 + 4 * sub);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * s[i];
      x[2 * i + 1] = b * c[i] + a * s[i];
    }
  } else {
    const int at = 8 * (sub & 3);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f32x4 c = *reinterpret_cast<const f32x4*>(cs + at + 4 * j), s = *reinterpret_cast<const f32x4*>(cs + 32 + at + 4 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float own = x[4 * j + i] * c[i], cross = other[4 * j + i] * s[i];
        x[4 * j + i] = sub < 4 ? own - cross : own + cross;
      }
    }
  }
}

}  // namespace misa
