// Attention over latent vectors in expanded form: every head has its own keys
// [nope 128 | rotary 64, shared by the heads] and values [128],
//
//   S[t,s]  = sm * (q[t,h, 0:128] . kv[s,h, 0:128] + q[t,h, 128:192] . rope[s])
//   out[t,h] = sum_s softmax_s(S[t,:]) kv[s,h, 128:256],  lse[t,h] = log sum_s exp(S[t,s])
//
// over the keys base[t] .. base[t] + pos[t] of query t.
#include <algorithm>
#include <type_traits>

#include "attention.h"
#include "attention_device.h"

namespace misa {

constexpr int kKvRow = 2 * (kNope + kValue);  // bytes of a head's key and value row

// Order of the 16-byte chunks of a key/value row (32 chunks) and of a rotary
// row (8 chunks) in LDS: 32 rows of one chunk column fall on 32 distinct
// chunks modulo 512 bytes, and four neighbouring rows of a transposing read
// four chunks apart.
__device__ __forceinline__ int swz_kv(int row) { return ((row & 3) << 2) | ((row >> 2) & 3) | (row & 16); }
__device__ __forceinline__ int swz_rot(int row) { return (row >> 2) & 7; }

// 32 NW queries of one head and a share of the keys per workgroup of NW waves; each
// wave owns 32 queries and walks every key tile (64 keys, shared through LDS). The
// scores are formed transposed (S^T = K Q^T), so a lane holds weights of one
// query only, its reference and total are lane values, and the weights are the
// B operand of O^T = V^T P^T as they stand: the order of the keys inside an
// MFMA's contraction is free, and the transposing LDS reads of V take the same
// order as the result rows of S^T.
//
// Bound by matrix and vector issue together: the two waves of a SIMD take turns (a
// product of one does not run beside the exponentials of the other, only beside
// vector work of its own wave), so a tile costs the sum, 40 products of 32 cycles and
// about 500 of softmax a wave. 8192 causal queries of 16 heads: 323-350 us, 0.98-1.06
// PFLOP/s (up to 444 us in the first thirty calls of a process, while the clock
// recovers from the onset of the load), against 1.15 of a library product of 8192^3 (under this load the clock
// falls to 2.0 GHz). Few queries over a long context are bound by memory: 100 over
// 32768 keys of 16 heads read 268 MB in 59 us (4.6 TB/s; a copy reaches 4.9), and
// join in 5. Tried and left out: waves half a tile apart (402 us against 399), halves
// of a tile interleaved in a wave (500, registers), four LDS buffers (73 against 60 on
// the long context).
template <int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_expanded(ExpandedArgs p) {
  constexpr int kRows = 32 * NW;
  constexpr int kTileBytes = kAttnTile * (kKvRow + 2 * kRotary);
  constexpr int kRope = kAttnTile * kKvRow;
  constexpr int kMyRows = kAttnTile / NW;                        // tile rows a wave copies
  constexpr int kKvCopies = kMyRows / 2, kCopies = kKvCopies + kMyRows / 8;
  __shared__ __attribute__((aligned(1024))) unsigned char tile[2][kTileBytes];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h2 = lane >> 5, lo = lane & 15;

  // each XCD takes a run of (split, head, row tile): the row tiles of a head
  // share its keys, the heads of a split the rows that hold them side by side;
  // the last row tiles, with the most keys under a causal mask, first
  const int per = (int)(gridDim.x / 8);
  const int lid = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  const int rt = p.row_tiles - 1 - lid % p.row_tiles;
  const int head = lid / p.row_tiles % p.H, split = lid / p.row_tiles / p.H;
  if (split >= p.splits) return;

  // ---- key ranges of the workgroup's queries, 64 a load, and Q: all asked for at
  // once from rows that are there (a read under a condition would be waited for by itself)
  const int t = rt * kRows + 32 * w + c;
  int n_pos[kRows / 64], n_base[kRows / 64];
#pragma unroll
  for (int i = 0; i < kRows / 64; ++i) n_pos[i] = p.pos[min(rt * kRows + 64 * i + lane, p.T - 1)];
#pragma unroll
  for (int i = 0; i < kRows / 64; ++i) n_base[i] = 0;
  if (p.base) {
#pragma unroll
    for (int i = 0; i < kRows / 64; ++i) n_base[i] = p.base[min(rt * kRows + 64 * i + lane, p.T - 1)];
  }
  // Q as the B operand: K step ks, lane (query c, half h2): values 16 ks + 8 h2 .. + 7
  bf16x8 qf[12];
  {
    const uint16_t* qr = p.q + ((int64_t)min(t, p.T - 1) * p.H + head) * (kNope + kRotary) + 8 * h2;
#pragma unroll
    for (int ks = 0; ks < 12; ++ks) qf[ks] = *reinterpret_cast<const bf16x8*>(qr + 16 * ks);
  }
  const uint32_t kBig = 0x7fffffffu;
  int g_lo = (int)kBig, g_hi = 0, s_lo = 0, s_hi = 0;  // of the workgroup; of the lane's query (0, 0: no key)
#pragma unroll
  for (int i = 0; i < kRows / 64; ++i) {
    const int64_t s0 = n_base[i], s1 = min((int64_t)p.L, s0 + (int64_t)n_pos[i] + 1);
    const bool any = rt * kRows + 64 * i + lane < p.T && s0 >= 0 && s1 > s0;
    const int lo_i = any ? (int)s0 : 0, hi_i = any ? (int)s1 : 0;
    if (any) g_lo = min(g_lo, lo_i), g_hi = max(g_hi, hi_i);
    const int from = 32 * (w & 1) + c;  // (rows 32 w .. of the workgroup)
    const int own_lo = __shfl(lo_i, from, kWave), own_hi = __shfl(hi_i, from, kWave);
    s_lo = w >> 1 == i ? own_lo : s_lo;
    s_hi = w >> 1 == i ? own_hi : s_hi;
  }
  const bool some = s_hi > s_lo;
  const int w_lo = (int)wave_min_u32(some ? (uint32_t)s_lo : kBig);    // the wave's first key
  const int w_hi = (int)wave_max_u32((uint32_t)s_hi);                  // and end
  // keys that every query of the wave sees; a query that sees none is set to its
  // result at the end, whatever it gathers
  const int f_lo = (int)wave_max_u32(some ? (uint32_t)s_lo : 0u);
  const int f_hi = w_hi == 0 ? 0 : (int)wave_min_u32(some ? (uint32_t)s_hi : kBig);
  g_lo = (int)wave_min_u32((uint32_t)g_lo);
  g_hi = (int)wave_max_u32((uint32_t)g_hi);
  int tile0 = min(g_lo, g_hi) / kAttnTile, tile1 = (g_hi + kAttnTile - 1) / kAttnTile;
  // an equal share of the tiles that this row tile has
  const int share = (max(tile1 - tile0, 0) + p.splits - 1) / p.splits;
  tile0 += split * share;
  tile1 = min(tile1, tile0 + share);

  const uint64_t kv = (uint64_t)(uintptr_t)p.kv + (uint64_t)head * kKvRow, rope = (uint64_t)(uintptr_t)p.rope;
  const uint32_t kv_ld = (uint32_t)p.H * kKvRow, rope_ld = (uint32_t)p.rope_ld * 2;
  const uint32_t tile_lds = lds_addr(&tile[0][0]);
  // copy j of the wave's rows of the tile that starts at key k0, to LDS at dst;
  // keys past the last repeat it (they are masked)
  auto copy = [&](uint32_t dst, int k0, int j, int ln) {
    if (j < kKvCopies) {  // two rows a copy
      const int r0 = kMyRows * w + 2 * j, row = r0 + (ln >> 5);
      const int sb = min(k0 + r0, p.L - 1);
      const uint32_t step = sb + 1 < p.L ? kv_ld : 0u;
      copy16_to_lds_at(reinterpret_cast<const void*>(kv + (uint64_t)(uint32_t)sb * kv_ld),
                       (ln >= 32 ? step : 0u) + (((ln & 31) ^ swz_kv(row)) * 16), dst + r0 * kKvRow);
    } else {              // eight rotary rows a copy
      const int r0 = kMyRows * w + 8 * (j - kKvCopies), row = r0 + (ln >> 3);
      const int sb = min(k0 + r0, p.L - 1);
      copy16_to_lds_at(reinterpret_cast<const void*>(rope + (uint64_t)(uint32_t)sb * rope_ld),
                       (uint32_t)min(ln >> 3, p.L - 1 - sb) * rope_ld + (((ln & 7) ^ swz_rot(row)) * 16),
                       dst + kRope + r0 * (2 * kRotary));
    }
  };
  if (tile0 < tile1) {
#pragma unroll
    for (int j = 0; j < kCopies; ++j) copy(tile_lds, tile0 * kAttnTile, j, lane);
  }

  const float sm = scale_magnitude(p.sm_log2);
  {
    const uint32_t sign = p.sm_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int ks = 0; ks < 12; ++ks) qf[ks] = flip_sign(qf[ks], sign);
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

  // one tile; MIXED: not every query of the wave sees every key (or none does)
  auto step = [&](int ti, auto mixed) {
    constexpr bool MIXED = decltype(mixed)::value;
    const uint32_t tb = tile_lds + ((ti - tile0) & 1) * kTileBytes, next_lds = tile_lds + ((ti + 1 - tile0) & 1) * kTileBytes;
    const int k0 = ti * kAttnTile;
    const int k_next = ti + 1 < tile1 ? k0 + kAttnTile : p.L;  // (no next tile: the last key's row, unused)
    const int ln = anew(lane);
    if (!MIXED || (k0 < w_hi && k0 + kAttnTile > w_lo)) {
      // ---- scores of keys 32 n + 8 (e / 4) + 4 h2 + e % 4 (result rows) for query c.
      // Operand reads run kAhead steps before their products, in one sequence:
      // key rows 32 n + c of K step ks (2 ks + n), then values 32 d .. + 31 of
      // keys 16 i .. + 15 (4 i + d)
      constexpr int kKeyReads = 24, kAhead = 4;
      const uint32_t ka = tb + a_key, ra = tb + a_rot, va = tb + a_val;
      bf16x8 ring[kAhead];
      auto read = [&](int i) -> bf16x8 {
        if (i < 16) return lds_read<bf16x8>((ka ^ (32 * (i >> 1))) + (i & 1) * 32 * kKvRow);
        if (i < 24) return lds_read<bf16x8>((ra ^ (32 * ((i >> 1) - 8))) + (i & 1) * 32 * 2 * kRotary);
        const int k = (i - 24) >> 2, d = (i - 24) & 3;
        const uint32_t at = va ^ (64 * d) ^ (256 * (k & 1));
        return join_rows(lds_read_tr16(at + 16 * k * kKvRow), lds_read_tr16((at ^ 32) + (16 * k + 8) * kKvRow));
      };
      f32x16 s[2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[n][e] = 0.f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ring[i] = read(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kKeyReads; ++i) {
        s[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[i % kAhead], qf[i >> 1], s[i & 1], 0, 0, 0);
        if (i + kAhead < kKeyReads) ring[i % kAhead] = read(i + kAhead);
        // the next tile's copies, spread over these products
        if ((i + 1) * kCopies / kKeyReads != i * kCopies / kKeyReads) copy(next_lds, k_next, i * kCopies / kKeyReads, ln);
        __builtin_amdgcn_sched_barrier(0);
      }
      bool odd = false;  // a value is not finite
      if constexpr (MIXED) {
        const uint32_t first = (uint32_t)(k0 + 4 * h2 - s_lo), seen = (uint32_t)(s_hi - s_lo);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[n][e] = first + (32 * n + 8 * (e >> 2) + (e & 3)) < seen ? s[n][e] : -INFINITY;
        // the largest magnitude among the tile's values, in whatever order they lie
        u16x2 most = {0, 0};
#pragma unroll
        for (int i = 0; i < kAttnTile / 4; ++i) {
          const u32x4 v = lds_read<u32x4>(tb + (ln >> 4) * kKvRow + (ln & 15) * 16 + 4 * i * kKvRow + ((16 ^ (4 * i & 16)) * 16));
#pragma unroll
          for (int x = 0; x < 4; ++x) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, v[x] & 0x7fff7fffu));
        }
        odd = __any(max(most.x, most.y) >= 0x7f80);
      }
      float top = max_or_nan(s[0][0], s[1][0]);
#pragma unroll
      for (int e = 1; e < 16; ++e) top = max_or_nan(max_or_nan(top, s[0][e]), s[1][e]);
      top = max_halves(top) * sm;
      if (__builtin_expect(__any(top > m + kSlack), 0)) {
        const float mm = top > m + kSlack ? top : m, f = exp2_fast(m - mm);
        m = mm;
        l *= f;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] *= f;
      }
      bf16x8 pb[4];
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x = exp2_fast(fmaf(s[n][e], sm, -m));
          sum[e & 3] += x;  // the total keeps 32 bits; the weights are rounded to bf16 for the matrix cores
          pb[2 * n + (e >> 3)][e & 7] = (__bf16)x;
        }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      // ---- sums of values 32 d + (result row) for query c
      if (!MIXED || __builtin_expect(!odd, 1)) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ring[i] = read(kKeyReads + i);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i & 3] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[i % kAhead], pb[i >> 2], o[i & 3], 0, 0, 0);
          if (i + kAhead < 16) ring[i % kAhead] = read(kKeyReads + i + kAhead);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {  // each key with such a value adds it to the queries that see the key
        f32x16 sums[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) sums[d] = o[d];
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          const bf16x8 a = read(kKeyReads + i);
          const bf16x8 pi = i < 8 ? (i < 4 ? pb[0] : pb[1]) : (i < 12 ? pb[2] : pb[3]);
          f32x16 acc = sums[i & 3];
#pragma unroll 1
          for (int k = 0; k < 16; ++k) {
            f32x16 z;
#pragma unroll
            for (int e = 0; e < 16; ++e) z[e] = 0.f;
            z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(part_of<true>(a, h2 == (k >> 3) ? (k & 7) : -1), pi, z, 0, 0, 0);
            const int key = k0 + 16 * (i >> 2) + 8 * ((k & 7) >> 2) + 4 * (k >> 3) + (k & 3);
            if (key >= s_lo && key < s_hi) acc += z;
          }
          sums[i & 3] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(part_of<false>(a, 0), pi, acc, 0, 0, 0);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = sums[d];
      }
    } else {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) copy(next_lds, k_next, j, ln);
    }
    wait_copies();
    lds_barrier();
  };
  for (int ti = tile0; ti < tile1; ++ti) {
    for (; ti < tile1 && ti * kAttnTile >= f_lo && (ti + 1) * kAttnTile <= f_hi; ++ti) step(ti, std::false_type{});
    if (ti < tile1) step(ti, std::true_type{});
  }

  // ---- result, through LDS (the wave's own 8 KB) so that rows leave in whole lines:
  // 256 bytes of each of 32 rows at a time, chunks in an order that depends on the row
  if (!some) {
    m = kNoMax;
    l = 0.f;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  }
  const float tot = row_total(some, sum_halves(l));
  const uint32_t mine = tile_lds + w * 32 * 256;
  const int rows_here = min(32, p.T - (rt * kRows + 32 * w));
  const int64_t R0 = (int64_t)(rt * kRows + 32 * w) * p.H + head;
  auto put = [&](unsigned char* dst, int64_t stride) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int rr = 4 * i + (lane >> 4);
      const u32x4 v = lds_read<u32x4>(mine + rr * 256 + ((lo ^ (rr & 15)) * 16));
      if (rr < rows_here) *reinterpret_cast<u32x4*>(dst + rr * stride + lo * 16) = v;
    }
  };
  if (p.splits > 1) {
    const int64_t pr = (int64_t)split * p.T * p.H + R0;
#pragma unroll
    for (int d0 = 0; d0 < 4; d0 += 2) {
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(mine + c * 256 + (((8 * d + 2 * i + h2) ^ (c & 15)) * 16)) =
              f32x4{o[d0 + d][4 * i], o[d0 + d][4 * i + 1], o[d0 + d][4 * i + 2], o[d0 + d][4 * i + 3]};
      put(reinterpret_cast<unsigned char*>(p.part + pr * kValue + 32 * d0), (int64_t)p.H * kValue * 4);
    }
    if (c < rows_here && h2 == 0) {
      p.part_ml[(pr + (int64_t)c * p.H) * 2] = m;
      p.part_ml[(pr + (int64_t)c * p.H) * 2 + 1] = tot;
    }
  } else {
    const float inv = row_inverse(tot);
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 v = {o[d][4 * i] * inv, o[d][4 * i + 1] * inv, o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv};
        *(__attribute__((address_space(3))) bf16x4*)(uintptr_t)(mine + c * 256 + (((4 * d + i) ^ (c & 15)) * 16) + h2 * 8) =
            __builtin_convertvector(v, bf16x4);
      }
    put(reinterpret_cast<unsigned char*>(p.out + R0 * kValue), (int64_t)p.H * kValue * 2);
    if (p.lse && c < rows_here && h2 == 0)
      p.lse[R0 + (int64_t)c * p.H] = row_log_sum(m, tot);
  }
}

// Queries per workgroup and splits of the keys, by what they cost on this card, in
// us: a tile takes 1.55 of a compute unit with 128 queries (two such workgroups share
// it) and 1.4 with 256, and 1.3 and 1.45 in a workgroup whose keys are the longest;
// partial sums (512 bytes a row and split) are written and joined at 2.6 TB/s after 3
// of launch. The constants are fitted to 111 measured calls (1 to 8192 queries, 1 to
// 128 heads, 100 to 32768 keys, packed ones among them); what this rule chooses is 3%
// off the fastest cut in the mean and 23% at worst. The queries are taken to be the last
// of the keys, which is the most work. Measured, us a call (four / eight waves, splits):
// 300 queries of 16 heads in one piece 13 / 16, in four 16 / 18; 2048 of 16 heads in one
// 51 / 64, in two 55 / 50; 8192 of 16 heads 389 / 348; 100 over 32768 keys 70 in 32 /
// 70 in 16; three packed prompts of 1000, 5 heads, 30 / 30 in four.
AttnPlan expanded_plan(int T, int H, int L) {
  const double tiles = std::max(1, (L + kAttnTile - 1) / kAttnTile);
  const double mean = std::max(tiles - T / (2.0 * kAttnTile), 0.5 * tiles);
  AttnPlan best{};
  double least = 0.0;
  for (int nq = 128; nq <= 256; nq += 128) {
    AttnPlan pl{};
    pl.nq = nq;
    pl.row_tiles = (T + nq - 1) / nq;
    const double wgs = (double)pl.row_tiles * H;
    const int most = (int)std::max(1.0, std::min((nq == 256 ? 256 : 512) / wgs, tiles));
    for (int s = 1;; s = std::min(2 * s, most)) {
      pl.splits = s;
      const double all = wgs * mean * (nq == 256 ? 1.4 : 1.55) / 256, longest = tiles / s * (nq == 256 ? 1.45 : 1.3);
      const double cost = std::max(all, longest) + (s > 1 ? 3.0 + (double)s * T * H * (kValue * 4) / 2.6e6 : 0.0);
      if (best.nq == 0 || cost < least) best = pl, least = cost;
      if (s == most) break;
    }
  }
  return best;
}

size_t expanded_ws_bytes(const AttnPlan& pl, int T, int H) {
  return pl.splits <= 1 ? 256 : 256 + (size_t)T * H * pl.splits * (kValue + 2) * 4;
}

hipError_t launch_expanded(const LaunchCtx& cx, ExpandedArgs a, const AttnPlan& pl, void* ws) {
  const int64_t rows = (int64_t)a.T * a.H;
  a.splits = pl.splits;
  a.row_tiles = pl.row_tiles;
  if (pl.splits > 1) {
    a.part = static_cast<float*>(ws);
    a.part_ml = a.part + rows * pl.splits * kValue;
  }
  const int64_t n = (int64_t)pl.row_tiles * pl.splits * a.H;
  const dim3 grid((unsigned)((n + 7) / 8 * 8));
  const hipError_t e = pl.nq == 256 ? cx.launch("k_expanded_256", k_expanded<8>, grid, dim3(512), 0, a)
                                    : cx.launch("k_expanded_128", k_expanded<4>, grid, dim3(256), 0, a);
  if (e != hipSuccess || pl.splits <= 1) return e;
  return launch_join(cx, a.part, a.part_ml, pl.splits, rows, kValue, a.out, a.lse);
}

}  // namespace misa
