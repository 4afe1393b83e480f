// Caches of indexer keys and latent rows: rows go in at given slots, in bf16 or
// coded to E4M3FN with one scale a row, and come back as bf16.
//
// Coded rows: scale = 2^e, the smallest power of two (e >= -126) with
// max|x| <= 448 * 2^e, and code = RNE(x / scale). A power of two makes x /
// scale exact, so a value is rounded once, and code * scale is exact in bf16
// (4 significant bits): what a reader gets is the coded value itself. Against
// max|x| / 448 it costs at most one binade at the bottom of E4M3's range.
#include <algorithm>
#include <type_traits>

#include "attention.h"
#include "attention_device.h"

namespace misa {

// D / 8 lanes a row, eight values a lane: one read, the row's maximum over its
// lanes, one write. Bound by memory from about 16384 latent rows on (29.5 MB in 9.1
// us, 3.2 TB/s, in 6.7 where the rows lie in the caches; 131072 rows 49.5, 4.8 TB/s; keys
// of 128 values 13.1), by the launch below (8 rows 2.0 us, 5001 keys 2.7).
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

// bf16 caches: 16 bytes a thread. A copy, bound as one: 131072 latent rows 59 us (5.1
// TB/s; a plain copy of 1 or 2 GiB reaches 4.9 to 5.1), 16384 10.4, 131072 keys of 128
// values 15.7, 5001 2.6.
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

// A wave reads R = NI * 512 / D rows, eight values a lane at a time, and asks for
// all of them before it uses the first: rows lie anywhere, and the more of them
// are on their way, the less HBM waits.
template <int D, int DR, bool FP8, int NI>
__global__ __launch_bounds__(256) void k_cache_read(CacheArgs p, uint16_t* out) {
  constexpr int LPR = D / 8, RPI = kWave / LPR, R = NI * RPI, W = D + DR;
  constexpr int CPR = DR ? DR / 8 : 1, NR = DR ? (R * CPR + kWave - 1) / kWave : 0;  // rotary chunks of a row and of a lane
  const int lane = threadIdx.x & 63;
  const int64_t row0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * R;
  if (row0 >= p.n) return;
  // the slot of row row0 + lane % R, and whether it names a row
  const int64_t mine = row0 + lane % R;
  const int slot = p.slots[min(mine, (int64_t)p.n - 1)];
  const int held = slot >= 0 && slot < p.rows ? slot : -1;
  const unsigned char* c = static_cast<const unsigned char*>(p.c);
  using Chunk = std::conditional_t<FP8, u32x2, u32x4>;
  Chunk v[NI];
  float sc[NI];
  int at[NI];
  u32x4 rot[NR > 0 ? NR : 1];
  int rat[NR > 0 ? NR : 1];
#pragma unroll
  for (int j = 0; j < NI; ++j) {  // (a row that is not there reads row 0 and is dropped)
    at[j] = __shfl(held, j * RPI + lane / LPR, kWave);
    const int64_t r = max(at[j], 0);
    v[j] = *reinterpret_cast<const Chunk*>(c + r * (FP8 ? D : 2 * W) + (lane % LPR) * sizeof(Chunk));
    if constexpr (FP8) sc[j] = p.scale[r];
  }
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int i = min(j * kWave + lane, R * CPR - 1);
    rat[j] = __shfl(held, i / CPR, kWave);
    const int64_t r = max(rat[j], 0);
    rot[j] = FP8 ? *reinterpret_cast<const u32x4*>(p.rope + r * DR + i % CPR * 8)
                 : *reinterpret_cast<const u32x4*>(c + r * (2 * W) + 2 * D + i % CPR * 16);
  }
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int64_t row = row0 + j * RPI + lane / LPR;
    u32x4 o;
    if constexpr (FP8) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x, y;
        bf16x2 r;
        fp8x2_to_f32<false>(v[j][k], x, y);
        r.x = (__bf16)(x * sc[j]), r.y = (__bf16)(y * sc[j]);
        o[2 * k] = __builtin_bit_cast(uint32_t, r);
        fp8x2_to_f32<true>(v[j][k], x, y);
        r.x = (__bf16)(x * sc[j]), r.y = (__bf16)(y * sc[j]);
        o[2 * k + 1] = __builtin_bit_cast(uint32_t, r);
      }
    } else {
      o = v[j];
    }
    if (at[j] < 0) o = u32x4{0u, 0u, 0u, 0u};
    if (row < p.n) *reinterpret_cast<u32x4*>(out + row * W + (lane % LPR) * 8) = o;
  }
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int i = j * kWave + lane;
    const int64_t row = row0 + i / CPR;
    if (rat[j] < 0) rot[j] = u32x4{0u, 0u, 0u, 0u};
    if (i < R * CPR && row < p.n) *reinterpret_cast<u32x4*>(out + row * W + D + i % CPR * 8) = rot[j];
  }
}

static unsigned blocks(int64_t items, int per) { return (unsigned)((items + per - 1) / per); }

template <int D, int DR>
static hipError_t write_shape(const LaunchCtx& cx, const CacheArgs& a, bool fp8, const uint16_t* x) {
  if (fp8) return cx.launch("k_cache_write", k_cache_write<D, DR>, dim3(blocks(a.n, 2048 / D)), dim3(256), 0, a, x);
  return cx.launch("k_cache_copy_in", k_cache_copy_in<D + DR>, dim3(blocks((int64_t)a.n * (D + DR) / 8, 256)),
                   dim3(256), 0, a, x);
}
template <int D, int DR, bool FP8, int NI>
static hipError_t read_as(const LaunchCtx& cx, const CacheArgs& a, uint16_t* out) {
  return cx.launch("k_cache_read", k_cache_read<D, DR, FP8, NI>, dim3(blocks(a.n, 4 * NI * 512 / D)), dim3(256), 0, a, out);
}
// Four times the rows a wave once there are more than 2^22 values, enough for
// every wave slot. Coded latent rows, cold, one / four: 2048 rows 2.3 / 2.5 us,
// 8192 4.3 / 4.4, 16384 6.7 / 6.2, 131072 54.6 / 47.4 (47 to 50 us, 4.7 to 5.0 TB/s, from
// run to run, what a plain copy reaches; a thread for each eight values took 67.0); keys
// of 128 values: 32768 rows 4.1 / 4.4, 131072 14.7 / 12.7. bf16 rows: 131072 latents
// 63.6 us (4.75 TB/s), 131072 keys 15.3, 2048 latents 3.0.
template <int D, int DR>
static hipError_t read_shape(const LaunchCtx& cx, const CacheArgs& a, bool fp8, uint16_t* out) {
  if ((int64_t)a.n * D > ((int64_t)1 << 22))
    return fp8 ? read_as<D, DR, true, 4>(cx, a, out) : read_as<D, DR, false, 4>(cx, a, out);
  return fp8 ? read_as<D, DR, true, 1>(cx, a, out) : read_as<D, DR, false, 1>(cx, a, out);
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
