// Caches of indexer keys and latent rows: rows go in at given slots, in bf16 or
// coded to E4M3FN with one scale a row, and come back as bf16.
//
// Coded rows: scale = 2^e, the smallest power of two (e >= -126) with
// max|x| <= 448 * 2^e, and code = RNE(x / scale). A power of two makes x /
// scale exact, so a value is rounded once, and code * scale is exact in bf16
// (4 significant bits): what a reader gets is the coded value itself. Against
// max|x| / 448 it costs at most one binade at the bottom of E4M3's range.
#include <algorithm>

#include "attention.h"
#include "attention_device.h"

namespace misa {

// D / 8 lanes a row, eight values a lane.
template <int D, int DR>
__global__ __launch_bounds__(256) void k_cache_write(CacheArgs p, const uint16_t* x) {
  constexpr int LPR = D / 8;           // lanes of a row
  constexpr int RPB = 256 / LPR;       // rows of a workgroup
  const int tid = threadIdx.x, sub = tid % LPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + tid / LPR;
  const bool in = row < p.n;
  const int slot = in ? p.slots[row] : -1;
  const bool live = slot >= 0 && slot < p.rows;
  const uint16_t* xr = x + (in ? row : 0) * (D + DR);
  const u32x4 v = *reinterpret_cast<const u32x4*>(xr + sub * 8);
  u32x4 r = {0u, 0u, 0u, 0u};
  if (DR && sub < DR / 8) r = *reinterpret_cast<const u32x4*>(xr + D + sub * 8);
  uint32_t top = 0;  // magnitude bits order like the magnitudes, NaN above infinity
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(v[i] & 0x7fffu, (v[i] >> 16) & 0x7fffu));
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, kWave));
  if (!live) return;
  // 448 = 1.75 * 2^8: the exponent of top less 8, one more if its fraction is over 0.75
  const int e = max(-126, (int)(top >> 7) - 135 + ((top & 0x7fu) > 96u ? 1 : 0));
  const bool bad = top >= 0x7f80u;  // an infinity or NaN: the row reads back as NaN
  const float scale = bad ? __uint_as_float(0x7fc00000u) : top == 0 ? 1.f : __uint_as_float((uint32_t)(e + 127) << 23);
  const float inv = top == 0 ? 1.f : __uint_as_float((uint32_t)(127 - e) << 23);
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_bits_to_f32(v[2 * i] & 0xffffu) * inv,
                                            __uint_as_float(v[2 * i] & 0xffff0000u) * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_bits_to_f32(v[2 * i + 1] & 0xffffu) * inv,
                                        __uint_as_float(v[2 * i + 1] & 0xffff0000u) * inv, w, true);
    c[i] = bad ? 0x7f7f7f7fu : (uint32_t)w;
  }
  *reinterpret_cast<u32x2*>(static_cast<unsigned char*>(p.c) + (int64_t)slot * D + sub * 8) = c;
  if (DR && sub < DR / 8) *reinterpret_cast<u32x4*>(p.rope + (int64_t)slot * DR + sub * 8) = r;
  if (sub == 0) p.scale[slot] = scale;
}

// bf16 caches: 16 bytes a thread.
template <int W>
__global__ __launch_bounds__(256) void k_cache_copy_in(CacheArgs p, const uint16_t* x) {
  constexpr int CPR = W / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.n * CPR) return;
  const int64_t row = i / CPR;
  const int ch = (int)(i - row * CPR);
  const int slot = p.slots[row];
  if (slot < 0 || slot >= p.rows) return;
  *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.c) + (int64_t)slot * W + ch * 8) =
      *reinterpret_cast<const u32x4*>(x + i * 8);
}

// Eight values of a row a thread.
template <int D, int DR, bool FP8>
__global__ __launch_bounds__(256) void k_cache_read(CacheArgs p, uint16_t* out) {
  constexpr int CPR = (D + DR) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.n * CPR) return;
  const int64_t row = i / CPR;
  const int ch = (int)(i - row * CPR);
  const int slot = p.slots[row];
  u32x4 v = {0u, 0u, 0u, 0u};
  if (slot >= 0 && slot < p.rows) {
    if (!FP8) {
      v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.c) + (int64_t)slot * (D + DR) + ch * 8);
    } else if (ch >= D / 8) {
      v = *reinterpret_cast<const u32x4*>(p.rope + (int64_t)slot * DR + (ch - D / 8) * 8);
    } else {
      const u32x2 c = *reinterpret_cast<const u32x2*>(static_cast<const unsigned char*>(p.c) + (int64_t)slot * D + ch * 8);
      const float s = p.scale[slot];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float a, b;
        bf16x2 r;
        fp8x2_to_f32<false>(c[k], a, b);
        r.x = (__bf16)(a * s), r.y = (__bf16)(b * s);
        v[2 * k] = __builtin_bit_cast(uint32_t, r);
        fp8x2_to_f32<true>(c[k], a, b);
        r.x = (__bf16)(a * s), r.y = (__bf16)(b * s);
        v[2 * k + 1] = __builtin_bit_cast(uint32_t, r);
      }
    }
  }
  *reinterpret_cast<u32x4*>(out + i * 8) = v;
}

static unsigned blocks(int64_t items, int per) { return (unsigned)((items + per - 1) / per); }

template <int D, int DR>
static hipError_t write_shape(const LaunchCtx& cx, const CacheArgs& a, bool fp8, const uint16_t* x) {
  if (fp8) return cx.launch("k_cache_write", k_cache_write<D, DR>, dim3(blocks(a.n, 2048 / D)), dim3(256), 0, a, x);
  return cx.launch("k_cache_copy_in", k_cache_copy_in<D + DR>, dim3(blocks((int64_t)a.n * (D + DR) / 8, 256)),
                   dim3(256), 0, a, x);
}
template <int D, int DR>
static hipError_t read_shape(const LaunchCtx& cx, const CacheArgs& a, bool fp8, uint16_t* out) {
  const dim3 grid(blocks((int64_t)a.n * (D + DR) / 8, 256));
  return fp8 ? cx.launch("k_cache_read", k_cache_read<D, DR, true>, grid, dim3(256), 0, a, out)
             : cx.launch("k_cache_read", k_cache_read<D, DR, false>, grid, dim3(256), 0, a, out);
}

hipError_t launch_cache_write(const LaunchCtx& cx, const CacheArgs& a, bool fp8, const uint16_t* x) {
  if (a.d == kLatent) return a.dr ? write_shape<kLatent, kRotary>(cx, a, fp8, x) : write_shape<kLatent, 0>(cx, a, fp8, x);
  return a.dr ? write_shape<kHeadDim, kRotary>(cx, a, fp8, x) : write_shape<kHeadDim, 0>(cx, a, fp8, x);
}

hipError_t launch_cache_read(const LaunchCtx& cx, const CacheArgs& a, bool fp8, uint16_t* out) {
  if (a.d == kLatent) return a.dr ? read_shape<kLatent, kRotary>(cx, a, fp8, out) : read_shape<kLatent, 0>(cx, a, fp8, out);
  return a.dr ? read_shape<kHeadDim, kRotary>(cx, a, fp8, out) : read_shape<kHeadDim, 0>(cx, a, fp8, out);
}

}  // namespace misa
