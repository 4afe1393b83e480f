// Attention over latent vectors in expanded form: every head has its own keys
// [nope 128 | rotary 64, shared by the heads] and values [128],
//
//   S[t,s]  = sm * (q[t,h, 0:128] . kv[s,h, 0:128] + q[t,h, 128:192] . rope[s])
//   out[t,h] = sum_s softmax_s(S[t,:]) kv[s,h, 128:256],  lse[t,h] = log sum_s exp(S[t,s])
//
// over the keys base[t] .. base[t] + pos[t] of query t.
#include <algorithm>

#include "attention.h"
#include "attention_device.h"

namespace misa {

constexpr int kExpRows = 128;            // queries of a workgroup (32 a wave)
constexpr int kKvRow = 2 * (kNope + kValue);  // bytes of a head's key and value row

// Order of the 16-byte chunks of a key/value row (32 chunks) and of a rotary
// row (8 chunks) in LDS: 32 rows of one chunk column fall on 32 distinct
// chunks modulo 512 bytes, and four neighbouring rows of a transposing read
// four chunks apart.
__device__ __forceinline__ int swz_kv(int row) { return ((row & 3) << 2) | ((row >> 2) & 3) | (row & 16); }
__device__ __forceinline__ int swz_rot(int row) { return (row >> 2) & 7; }

// 128 queries of one head and a share of the keys per workgroup; each wave owns
// 32 queries and walks every key tile (64 keys, shared through LDS). The
// scores are formed transposed (S^T = K Q^T), so a lane holds weights of one
// query only, its reference and total are lane values, and the weights are the
// B operand of O^T = V^T P^T as they stand: the order of the keys inside an
// MFMA's contraction is free, and the transposing LDS reads of V take the same
// order as the result rows of S^T.
__global__ __launch_bounds__(256, 2) void k_expanded(ExpandedArgs p) {
  constexpr int kTileBytes = kAttnTile * (kKvRow + 2 * kRotary);
  constexpr int kRope = kAttnTile * kKvRow;
  __shared__ __attribute__((aligned(1024))) unsigned char tile[2][kTileBytes];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h2 = lane >> 5, lo = lane & 15;

  // each XCD takes a run of (head, split, row tile): the row tiles of a head
  // share its keys; the last row tiles, with the most keys under a causal mask, first
  const int per = (int)(gridDim.x / 8);
  const int lid = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  const int head = lid / (p.row_tiles * p.splits);
  if (head >= p.H) return;
  const int rem = lid % (p.row_tiles * p.splits);
  const int split = rem % p.splits;
  const int rt = p.row_tiles - 1 - rem / p.splits;

  // ---- key ranges: of the lane's query, of the wave and of the workgroup
  auto range = [&](int t, int& a, int& b) {
    a = 0, b = 0;
    if (t >= p.T) return;
    const int64_t s0 = p.base ? p.base[t] : 0;
    const int64_t s1 = min((int64_t)p.L, s0 + (int64_t)p.pos[t] + 1);
    if (s0 < 0 || s1 <= s0) return;
    a = (int)s0, b = (int)s1;
  };
  const int t = rt * kExpRows + 32 * w + c;
  int s_lo, s_hi;
  range(t, s_lo, s_hi);
  const uint32_t kBig = 0x7fffffffu;
  const bool some = s_hi > s_lo;
  const int w_lo = (int)wave_min_u32(some ? (uint32_t)s_lo : kBig);    // the wave's first key
  const int w_hi = (int)wave_max_u32((uint32_t)s_hi);                  // and end
  // keys that every query of the wave sees (none if one sees none)
  const int f_lo = (int)wave_max_u32(some ? (uint32_t)s_lo : kBig), f_hi = (int)wave_min_u32((uint32_t)s_hi);
  int g_lo = (int)kBig, g_hi = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int a, b;
    range(rt * kExpRows + 64 * i + lane, a, b);
    if (b > a) g_lo = min(g_lo, a), g_hi = max(g_hi, b);
  }
  g_lo = (int)wave_min_u32((uint32_t)g_lo);
  g_hi = (int)wave_max_u32((uint32_t)g_hi);
  int tile0 = g_lo / kAttnTile, tile1 = (g_hi + kAttnTile - 1) / kAttnTile;
  tile0 = max(tile0, split * p.tiles_per_split);
  tile1 = min(tile1, (split + 1) * p.tiles_per_split);

  const unsigned char* kv = reinterpret_cast<const unsigned char*>(p.kv) + (int64_t)head * kKvRow;
  const unsigned char* rope = reinterpret_cast<const unsigned char*>(p.rope);
  const int64_t kv_ld = (int64_t)p.H * kKvRow, rope_ld = p.rope_ld * 2;
  const uint32_t tile_lds = lds_addr(&tile[0][0]);
  // copies keys 16 w .. 16 w + 15 of tile ti into buffer b; keys past the last
  // repeat it (they are masked)
  auto stage = [&](int b, int ti) {
    const uint32_t dst = tile_lds + b * kTileBytes;
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // two rows a copy
      const int row = 16 * w + 2 * i + h2;
      const int64_t s = min(ti * kAttnTile + row, p.L - 1);
      copy16_to_lds(kv + s * kv_ld + ((c ^ swz_kv(row)) * 16), dst + (16 * w + 2 * i) * kKvRow);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // eight rotary rows a copy
      const int row = 16 * w + 8 * i + (lane >> 3);
      const int64_t s = min(ti * kAttnTile + row, p.L - 1);
      copy16_to_lds(rope + s * rope_ld + (((lane & 7) ^ swz_rot(row)) * 16), dst + kRope + (16 * w + 8 * i) * (2 * kRotary));
    }
  };
  if (tile0 < tile1) stage(0, tile0);

  // Q as the B operand: K step ks, lane (query c, half h2): values 16 ks + 8 h2 .. + 7
  const float sm = scale_magnitude(p.sm_log2);
  bf16x8 qf[12];
  {
    const uint32_t sign = p.sm_log2 < 0.f ? 0x80008000u : 0u;
    const uint16_t* qr = p.q + ((int64_t)min(t, p.T - 1) * p.H + head) * (kNope + kRotary) + 8 * h2;
#pragma unroll
    for (int ks = 0; ks < 12; ++ks) qf[ks] = flip_sign(*reinterpret_cast<const bf16x8*>(qr + 16 * ks), sign);
  }
  f32x16 o[4];
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  float m = kNoMax, l = 0.f;
  wait_copies();
  __syncthreads();

  // The lane's addresses in a tile: its key row, its rotary row, and its row of
  // the transposing reads (rows 16 j + 4 h2 + lo / 4 and eight further on). Every
  // other chunk is an exclusive-or of the address, every other row an offset.
  const uint32_t a_key = c * kKvRow + ((h2 ^ swz_kv(c)) * 16);
  const uint32_t a_rot = kRope + c * (2 * kRotary) + ((h2 ^ swz_rot(c)) * 16);
  const int vrow = 4 * h2 + (lo >> 2);
  const uint32_t a_val =
      vrow * kKvRow + (((kNope / 8 + 2 * ((lane >> 4) & 1) + ((lo & 3) >> 1)) ^ swz_kv(vrow)) * 16) + (lo & 1) * 8;

  for (int ti = tile0; ti < tile1; ++ti) {
    const uint32_t tb = tile_lds + ((ti - tile0) & 1) * kTileBytes;
    if (ti + 1 < tile1) stage((ti + 1 - tile0) & 1, ti + 1);
    const int k0 = ti * kAttnTile;
    if (k0 < w_hi && k0 + kAttnTile > w_lo) {
      // ---- scores of keys 32 n + 8 (e / 4) + 4 h2 + e % 4 (result rows) for query c
      f32x16 s[2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[n][e] = 0.f;
      const uint32_t ka = tb + a_key, ra = tb + a_rot, va = tb + a_val;
      // Operand reads run kAhead steps before their products, in one sequence:
      // key rows 32 n + c of K step ks (2 ks + n), then values 32 d .. + 31 of
      // keys 16 i .. + 15 (4 i + d)
      constexpr int kKeyReads = 24, kAhead = 8;
      bf16x8 ring[kAhead];
      auto read = [&](int i) -> bf16x8 {
        if (i < 16) return lds_read<bf16x8>((ka ^ (32 * (i >> 1))) + (i & 1) * 32 * kKvRow);
        if (i < 24) return lds_read<bf16x8>((ra ^ (32 * ((i >> 1) - 8))) + (i & 1) * 32 * 2 * kRotary);
        const int k = (i - 24) >> 2, d = (i - 24) & 3;
        const uint32_t at = va ^ (64 * d) ^ (256 * (k & 1));
        return join_rows(lds_read_tr16(at + 16 * k * kKvRow), lds_read_tr16((at ^ 32) + (16 * k + 8) * kKvRow));
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ring[i] = read(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kKeyReads; ++i) {
        s[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[i % kAhead], qf[i >> 1], s[i & 1], 0, 0, 0);
        ring[i % kAhead] = read(i + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      }
      const bool mixed = k0 < f_lo || k0 + kAttnTile > f_hi;  // not every query sees every key
      bool odd = false;                                       // and a value is not finite
      if (__builtin_expect(mixed, 0)) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int key = k0 + 32 * n + 8 * (e >> 2) + 4 * h2 + (e & 3);
            s[n][e] = key >= s_lo && key < s_hi ? s[n][e] : -INFINITY;
          }
#pragma unroll 1
        for (int i = 0; i < 16; ++i) odd |= any_odd(read(kKeyReads + i));
        odd = __any(odd);
      }
      float top = fmaxf(s[0][0], s[1][0]);
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, fmaxf(s[0][e], s[1][e]));
      top = max_halves(top) * sm;
      if (__builtin_expect(__any(top > m + kSlack), 0)) {
        const float mm = fmaxf(m, top), f = exp2_fast(m - mm);
        m = mm;
        l *= f;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] *= f;
      }
      bf16x8 pb[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x = exp2_fast(fmaf(s[n][e], sm, -m));
          l += x;  // the total keeps 32 bits; the weights are rounded to bf16 for the matrix cores
          pb[2 * n + (e >> 3)][e & 7] = (__bf16)x;
        }
      // ---- sums of values 32 d + (result row) for query c
      if (__builtin_expect(!odd, 1)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i & 3] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[(kKeyReads + i) % kAhead], pb[i >> 2], o[i & 3], 0, 0, 0);
          if (i + kAhead < 16) ring[(kKeyReads + i) % kAhead] = read(kKeyReads + i + kAhead);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {  // each key with such a value adds it to the queries that see the key
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const bf16x8 a = read(kKeyReads + 4 * i + d);
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
              const bf16x8 one = part_of<true>(a, h2 == (k >> 3) ? (k & 7) : -1);
              f32x16 z;
#pragma unroll
              for (int e = 0; e < 16; ++e) z[e] = 0.f;
              z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(one, pb[i], z, 0, 0, 0);
              const int key = k0 + 16 * i + 8 * ((k & 7) >> 2) + 4 * (k >> 3) + (k & 3);
              if (key >= s_lo && key < s_hi) o[d] += z;
            }
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(part_of<false>(a, 0), pb[i], o[d], 0, 0, 0);
          }
      }
    }
    wait_copies();
    lds_barrier();
  }

  // ---- result: lane holds values 32 d + 8 i + 4 h2 + 0..3 of query c
  const float tot = sum_halves(l);
  if (t >= p.T) return;
  const int64_t R = (int64_t)t * p.H + head;
  if (p.splits > 1) {
    const int64_t pr = (int64_t)split * p.T * p.H + R;
    float* po = p.part + pr * kValue + 4 * h2;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(po + 32 * d + 8 * i) =
            f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    if (h2 == 0) p.part_ml[pr * 2] = m, p.part_ml[pr * 2 + 1] = tot;
  } else {
    const float inv = tot > 0.f ? 1.f / tot : (tot == 0.f ? 0.f : tot);  // no key: zeros; NaN stays
    uint16_t* po = p.out + R * kValue + 4 * h2;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 v = {o[d][4 * i] * inv, o[d][4 * i + 1] * inv, o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv};
        *reinterpret_cast<bf16x4*>(po + 32 * d + 8 * i) = __builtin_convertvector(v, bf16x4);
      }
    if (p.lse && h2 == 0) p.lse[R] = tot == 0.f ? -INFINITY : (m + log2_fast(tot)) * 0.6931471805599453f;
  }
}

AttnPlan expanded_plan(int T, int H, int L) {
  AttnPlan pl{};
  pl.nq = kExpRows;
  pl.row_tiles = (T + kExpRows - 1) / kExpRows;
  const int tiles = std::max(1, (L + kAttnTile - 1) / kAttnTile);
  const int64_t wgs = std::max<int64_t>(1, (int64_t)pl.row_tiles * H);
  const int want = (int)std::max<int64_t>(1, 512 / wgs);
  pl.tiles_per_split = (tiles + std::min(want, tiles) - 1) / std::min(want, tiles);
  pl.splits = (tiles + pl.tiles_per_split - 1) / pl.tiles_per_split;
  return pl;
}

size_t expanded_ws_bytes(const AttnPlan& pl, int T, int H) {
  return pl.splits <= 1 ? 256 : 256 + (size_t)T * H * pl.splits * (kValue + 2) * 4;
}

hipError_t launch_expanded(const LaunchCtx& cx, ExpandedArgs a, const AttnPlan& pl, void* ws) {
  const int64_t rows = (int64_t)a.T * a.H;
  a.splits = pl.splits;
  a.tiles_per_split = pl.tiles_per_split;
  a.row_tiles = pl.row_tiles;
  if (pl.splits > 1) {
    a.part = static_cast<float*>(ws);
    a.part_ml = a.part + rows * pl.splits * kValue;
  }
  const int64_t n = (int64_t)pl.row_tiles * pl.splits * a.H;
  const hipError_t e = cx.launch("k_expanded", k_expanded, dim3((unsigned)((n + 7) / 8 * 8)), dim3(256), 0, a);
  if (e != hipSuccess || pl.splits <= 1) return e;
  return launch_join(cx, a.part, a.part_ml, pl.splits, rows, kValue, a.out, a.lse);
}

}  // namespace misa
