// Attention over one shared latent vector a token, in absorbed form:
//
//   S[r,s]  = sm * (q[r, 0:512] . c[s] + q[r, 512:576] . rope[s])
//   out[r]  = sum_s softmax_s(S[r,:]) c[s],   lse[r] = log sum_s exp(S[r,s])
//
// for the rows r = (query, head) of one query, over the keys of the query's
// list or over its visible keys. All heads of a query read the same keys, and
// a key row is its own value row.
#include <algorithm>

#include "attention.h"
#include "attention_device.h"

namespace misa {

// What a key that does not exist is read from.
__device__ const uint4 g_zero_row[(kLatent + kRotary) * 2 / 16] = {};

// Tile in LDS: 64 key rows of 512 values (1024 bytes in bf16, 512 in codes) and
// apart from them their 64 rotary values (128 bytes). Rows are a multiple of
// 128 bytes apart, so 16-byte chunks are stored in an order that depends on
// the row (chunk ^ swizzle): the rows of an operand read, and the rows of a
// transposing read (four in bf16, eight in codes), then fall on distinct banks.
// WIDE: for operands of 32 rows, otherwise of 16.
template <bool FP8, bool WIDE>
struct LatentTile {
  static constexpr int kRow = FP8 ? kLatent : 2 * kLatent;
  static constexpr int kBytes = kAttnTile * (kRow + 2 * kRotary);
  static constexpr int kRope = kAttnTile * kRow;  // offset of the rotary rows
  static constexpr int kRopeRow = 2 * kRotary;
  static __device__ __forceinline__ int swz(int row) {
    if constexpr (WIDE && FP8)
      return ((row & 3) << 1) | (row & 8) | ((row >> 2) & 1) | (row & 16);
    else if constexpr (WIDE)
      return ((row & 3) << 2) | ((row >> 2) & 3) | (row & 16);
    else if constexpr (FP8)
      return ((row & 7) << 1) | ((row & 8) << 1) | ((row >> 3) & 1);
    else
      return ((row & 3) << 1) | (row & 8) | ((row & 4) << 2);
  }
  static __device__ __forceinline__ int swz_rope(int row) { return WIDE ? (row >> 2) & 7 : ((row >> 2) & 3) << 1; }
};

// Where a workgroup's rows and keys are, and the walk over its key tiles.
template <int NQ, bool LIST>
struct LatentWork {
  const LatentArgs& p;
  int lane;
  int64_t r0;      // first row (query * H + head)
  int nv, t;       // rows; their query (when head_tiles)
  int base;
  int j1;          // entries of the list, or visible keys of the rows that see most
  int same;        // keys that every row sees (prefix form)
  int split, cur, tile_end;
  bool valid;

  __device__ __forceinline__ LatentWork(const LatentArgs& a, int lane_) : p(a), lane(lane_) {
    // neighbouring workgroups run on different XCDs; give each XCD a run of
    // neighbouring queries, with the row tiles and splits of one query together
    const int per = (int)(gridDim.x / 8);
    const int lid = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    const int ht = p.head_tiles ? p.head_tiles : 1;
    const int rt = (lid / (ht * p.splits)) * ht + lid % ht;
    split = (lid / ht) % p.splits;
    valid = rt < p.row_tiles;
    if (!valid) return;
    const int64_t nrows = (int64_t)p.T * p.H;
    t = 0;
    if (p.head_tiles) {
      t = rt / p.head_tiles;
      const int h0 = (rt % p.head_tiles) * NQ;
      r0 = (int64_t)t * p.H + h0;
      nv = min(NQ, p.H - h0);
    } else {
      r0 = (int64_t)rt * NQ;
      nv = (int)min((int64_t)NQ, nrows - r0);
    }
    base = (p.base && p.head_tiles) ? p.base[t] : 0;
    same = 0x7fffffff;
    if constexpr (LIST) {
      j1 = p.k;
    } else if (p.head_tiles) {
      j1 = visible_keys(p.pos[t], left());
    } else {
      j1 = 0;
#pragma unroll
      for (int i = 0; i < (NQ + 63) / 64; ++i) {
        const int r = 64 * i + lane;
        const int n = r < nv ? visible_keys(p.pos[(r0 + r) / p.H], left()) : -1;
        j1 = max(j1, n);
        same = n >= 0 ? min(same, n) : same;
      }
      j1 = __builtin_amdgcn_readfirstlane((int)wave_max_u32((uint32_t)j1));
      same = __builtin_amdgcn_readfirstlane((int)wave_min_u32((uint32_t)same));
    }
    j1 = __builtin_amdgcn_readfirstlane(j1);
    tile_end = min((j1 + kAttnTile - 1) / kAttnTile, (split + 1) * p.tiles_per_split);
    cur = split * p.tiles_per_split;
  }
  __device__ __forceinline__ int left() const { return base < 0 ? 0 : max(0, p.rows - base); }
  // visible keys of row r (prefix form)
  __device__ __forceinline__ int limit(int r) const {
    return p.head_tiles ? j1 : r < nv ? visible_keys(p.pos[(r0 + r) / p.H], left()) : 0;
  }
  // entry 64 * ti + lane of the list
  __device__ __forceinline__ int list_entry(int ti) const {
    if constexpr (LIST) {
      const int j = ti * kAttnTile + lane;
      if (j < p.k) return p.idx[(int64_t)t * p.k + j];
    }
    return -1;
  }
  // the cache row of key 64 * ti + lane, or -1; v: its list entry
  __device__ __forceinline__ int row_of(int ti, int v) const {
    if constexpr (LIST) {
      const int64_t row = (int64_t)v + base;
      return (v >= 0 && base >= 0 && row < p.rows) ? (int)row : -1;
    } else {
      const int j = ti * kAttnTile + lane;
      return j < j1 ? base + j : -1;
    }
  }
  // first tile at or after ti that holds a key; v: ti's list entries, rows: the found tile's rows
  __device__ __forceinline__ int find_tile(int ti, int v, int& rows) const {
    rows = -1;
    while (ti < tile_end) {
      rows = row_of(ti, v);
      if (wave_ballot(rows >= 0) != 0) break;
      v = list_entry(++ti);
    }
    return ti;
  }
};

// Copies key rows 16 w .. 16 w + 15 of a tile to LDS at dst; lane i of `rows`
// holds the cache row of the tile's key i, or -1 (zeros then).
template <class Tile, bool FP8>
__device__ __forceinline__ void stage_tile(const LatentArgs& p, uint32_t dst, int w, int lane, int rows) {
  const unsigned char* C = static_cast<const unsigned char*>(p.c);
  const unsigned char* zero = reinterpret_cast<const unsigned char*>(g_zero_row);
  if constexpr (FP8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // two rows a copy
      const int row = 16 * w + 2 * i + (lane >> 5);
      const int s = __shfl(rows, row, kWave);
      const int ch = (lane & 31) ^ Tile::swz(row);
      const unsigned char* src = s >= 0 ? C + (int64_t)s * kLatent : zero;
      copy16_to_lds(src + ch * 16, dst + (16 * w + 2 * i) * Tile::kRow);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = 16 * w + i;
      const int s = __builtin_amdgcn_readlane(rows, row);
      const unsigned char* src = s >= 0 ? C + (int64_t)s * (2 * (kLatent + kRotary)) : zero;
      copy16_to_lds_at(src, (lane ^ Tile::swz(row)) * 16, dst + row * Tile::kRow);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // eight rotary rows a copy
    const int row = 16 * w + 8 * i + (lane >> 3);
    const int s = __shfl(rows, row, kWave);
    const int ch = (lane & 7) ^ Tile::swz_rope(row);
    const unsigned char* src;
    if constexpr (FP8)
      src = s >= 0 ? reinterpret_cast<const unsigned char*>(p.rope) + (int64_t)s * (2 * kRotary) : zero;
    else
      src = s >= 0 ? C + (int64_t)s * (2 * (kLatent + kRotary)) + 2 * kLatent : zero;
    copy16_to_lds(src + ch * 16, dst + Tile::kRope + (16 * w + 8 * i) * Tile::kRopeRow);
  }
}

// NQ = 16 or 32 rows and a share of the keys per workgroup of four waves. Per
// tile of 64 keys: wave w scores keys 16 w .. 16 w + 15 against all NQ rows (S^T
// = C Q^T with Q in registers), the weights cross LDS once, and wave w sums
// values 128 w .. 128 w + 127 over all 64 keys (O^T = C^T P^T, C^T by transposing
// LDS reads). So the tile is read from LDS twice whatever NQ is, the
// accumulators are spread over the waves, and a row's reference and weights stay
// in the lanes that hold its column. The copy of the next tile runs meanwhile.
template <int NQ, bool FP8, bool LIST>
__global__ __launch_bounds__(256, 1) void k_latent(LatentArgs p) {
  using Tile = LatentTile<FP8, false>;
  constexpr int QT = NQ / 16;
  __shared__ __attribute__((aligned(1024))) unsigned char tile[2][Tile::kBytes];
  __shared__ __attribute__((aligned(1024))) uint16_t pt[NQ * kAttnTile];  // weights, 128 bytes a row
  __shared__ float red[4][NQ];
  __shared__ int raise[2];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lo = lane & 15, g = lane >> 4;

  LatentWork<NQ, LIST> wk(p, lane);
  if (!wk.valid) return;
  const int64_t r0 = wk.r0, nrows = (int64_t)p.T * p.H;
  const int nv = wk.nv, tile_end = wk.tile_end;
  int lim[QT];  // visible keys of each of the lane's rows
#pragma unroll
  for (int i = 0; i < QT; ++i) lim[i] = LIST ? 0 : wk.limit(i * 16 + lo);

  const uint32_t tile_lds = lds_addr(&tile[0][0]);
  auto stage = [&](int b, int rows) { stage_tile<Tile, FP8>(p, tile_lds + b * Tile::kBytes, w, lane, rows); };
  auto key_scale = [&](int rows) -> float {
    if constexpr (FP8) return rows >= 0 ? p.scale[rows] : 0.f;
    return 0.f;
  };

  int rows_cur, rows_nxt;
  int cur = wk.find_tile(wk.cur, wk.list_entry(wk.cur), rows_cur);
  int nxt = wk.find_tile(cur + 1, wk.list_entry(cur + 1), rows_nxt);
  float sc_cur = key_scale(rows_cur);
  if (cur < tile_end) stage(0, rows_cur);

  // Q as the B operand: lane (row lo, group g) of K step ks holds values
  // 32 ks + 8 g .. + 7; with codes, whose 16-byte chunk covers two K steps,
  // values 64 (ks / 2) + 16 g + 8 (ks % 2) .. + 7 of the latent part
  const float sm = scale_magnitude(p.sm_log2);
  bf16x8 qf[QT][18];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int r = i * 16 + lo;
    const uint32_t sign = p.sm_log2 < 0.f ? 0x80008000u : 0u;
    const uint16_t* qr = p.q + (r0 + min(r, nv - 1)) * (kLatent + kRotary);
#pragma unroll
    for (int ks = 0; ks < 18; ++ks) {
      const int at = (FP8 && ks < 16) ? 64 * (ks >> 1) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g;
      qf[i][ks] = flip_sign(*reinterpret_cast<const bf16x8*>(qr + at), sign);
    }
  }

  f32x4 o[8][QT];
  float m[QT], l[QT];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    m[i] = kNoMax;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d) o[d][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  if (tid < 2) raise[tid] = 0;
  wait_copies();
  __syncthreads();

  // The lane's addresses in a tile: its key row and rotary row (the A operand of
  // the scores), its row of the transposing reads, its rows of the weights. Other
  // chunks are an exclusive-or of these, other rows an offset.
  const int krow = 16 * w + lo;
  const uint32_t a_key = krow * Tile::kRow + ((g ^ Tile::swz(krow)) * 16);
  const uint32_t a_rot = Tile::kRope + krow * Tile::kRopeRow + ((g ^ Tile::swz_rope(krow)) * 16);
  const int vrow = 8 * g + (FP8 ? lo >> 1 : lo >> 2);
  const uint32_t a_val =
      vrow * Tile::kRow + (lo & 1) * 8 +
      (FP8 ? ((8 * w) ^ Tile::swz(vrow)) * 16 : ((16 * w + ((lo & 3) >> 1)) ^ Tile::swz(vrow)) * 16);
  const uint32_t pt_lds = lds_addr(&pt[0]);
  const uint32_t a_prd = pt_lds + lo * 128 + ((g ^ (lo & 7)) * 16);
  const uint32_t a_pwr = pt_lds + lo * 128 + (((2 * w + (g >> 1)) ^ (lo & 7)) * 16) + (g & 1) * 8;

  int it = 0;
  while (cur < tile_end) {
    const uint32_t tb = tile_lds + (it & 1) * Tile::kBytes;
    const bool mixed = !LIST && (cur + 1) * kAttnTile > wk.same;  // not every row sees every key
    // the list entries after the next tile and the next tile's scales are asked
    // for ahead of its copy and used after the copy has landed
    const int v_nn = wk.list_entry(nxt + 1);
    const float sc_nxt = key_scale(rows_nxt);
    if (nxt < tile_end) stage((it + 1) & 1, rows_nxt);

    // ---- scores of keys 16 w + 4 g + 0..3 (result rows) for rows 16 i + lo (columns)
    f32x4 s[QT];
#pragma unroll
    for (int i = 0; i < QT; ++i) s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t ka = tb + a_key, ra = tb + a_rot, va = tb + a_val;
    if constexpr (FP8) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const u32x4 v = lds_read<u32x4>(ka ^ (64 * c));
        const bf16x8 a0 = codes_to_bf16(u32x2{v.x, v.y}), a1 = codes_to_bf16(u32x2{v.z, v.w});
#pragma unroll
        for (int i = 0; i < QT; ++i) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, qf[i][2 * c], s[i], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < QT; ++i) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, qf[i][2 * c + 1], s[i], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < 16; ++ks) {
        const bf16x8 a = lds_read<bf16x8>((ka ^ (64 * (ks & 7))) + 512 * (ks >> 3));
#pragma unroll
        for (int i = 0; i < QT; ++i) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, qf[i][ks], s[i], 0, 0, 0);
      }
    }
    f32x4 ksc;
    if constexpr (FP8) {  // a key's scale multiplies its latent part only
#pragma unroll
      for (int e = 0; e < 4; ++e) ksc[e] = __shfl(sc_cur, 16 * w + 4 * g + e, kWave);
#pragma unroll
      for (int i = 0; i < QT; ++i) s[i] *= ksc;
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const bf16x8 a = lds_read<bf16x8>(ra ^ (64 * ks));
#pragma unroll
      for (int i = 0; i < QT; ++i) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, qf[i][16 + ks], s[i], 0, 0, 0);
    }

    // ---- weights against the present reference
    const uint64_t live = wave_ballot(rows_cur >= 0);
    const uint32_t mine = (uint32_t)(live >> (16 * w + 4 * g)) & 15u;
    bool high = false;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool ok = LIST ? (mine >> e) & 1u : cur * kAttnTile + 16 * w + 4 * g + e < lim[i];
        s[i][e] = ok ? s[i][e] : -INFINITY;
      }
      const float top = max_over_groups(fmaxf(fmaxf(s[i].x, s[i].y), fmaxf(s[i].z, s[i].w))) * sm;
      high |= top > m[i] + kSlack;
      if (g == 0) red[w][i * 16 + lo] = top;
    }
    float sum[QT];
    auto weigh = [&]() {
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        f32x4 e;
#pragma unroll
        for (int x = 0; x < 4; ++x) e[x] = exp2_fast(fmaf(s[i][x], sm, -m[i]));
        sum[i] = (e.x + e.y) + (e.z + e.w);
        // rounded to bf16 for the matrix cores; the row's total keeps 32 bits
        if constexpr (FP8) {
#pragma unroll
          for (int x = 0; x < 4; ++x) e[x] = mixed && e[x] == 0.f ? 0.f : e[x] * ksc[x];
        }
        *(__attribute__((address_space(3))) bf16x4*)(uintptr_t)(a_pwr + i * 2048) = __builtin_convertvector(e, bf16x4);
      }
    };
    weigh();
    if (__any(high) && lane == 0) raise[it & 1] = 1;
    lds_barrier();
    if (__builtin_expect(raise[it & 1], 0)) {  // the same for all waves: move the references up, weigh again
      float f[QT];
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const int r = i * 16 + lo;
        const float mm = fmaxf(fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r])), m[i]);
        f[i] = exp2_fast(m[i] - mm);
        m[i] = mm;
        l[i] *= f[i];
      }
      weigh();
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int d = 0; d < 8; ++d) o[d][i] *= f[i];
      lds_barrier();
    }
    if (tid == 0) raise[(it + 1) & 1] = 0;
#pragma unroll
    for (int i = 0; i < QT; ++i) l[i] += sum[i];

    // ---- sums of values 128 w + 16 d + 4 g + 0..3 (result rows) for rows 16 i + lo (columns)
    auto values = [&](int j, int d) -> bf16x8 {  // values 16 d .. + 15 of the wave, keys 32 j .. + 31
      if constexpr (FP8)
        return codes_to_bf16(lds_read_tr8((va ^ (16 * d)) + 32 * j * Tile::kRow));
      else
        return join_rows(lds_read_tr16((va ^ (32 * d)) + 32 * j * Tile::kRow),
                         lds_read_tr16((va ^ (32 * d) ^ 256) + (32 * j + 4) * Tile::kRow));
    };
    bool odd = false;
    if (__builtin_expect(mixed, 0)) {
#pragma unroll 1
      for (int i = 0; i < 16; ++i) odd |= any_odd(values(i >> 3, i & 7));
      odd = __any(odd);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      bf16x8 pb[QT];
#pragma unroll
      for (int i = 0; i < QT; ++i) pb[i] = lds_read<bf16x8>((a_prd ^ (64 * j)) + i * 2048);
      if (__builtin_expect(!odd, 1)) {
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const bf16x8 a = values(j, d);
#pragma unroll
          for (int i = 0; i < QT; ++i) o[d][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, pb[i], o[d][i], 0, 0, 0);
        }
      } else {  // each key with a value that is not finite adds it to the rows that see the key
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const bf16x8 a = values(j, d);
#pragma unroll 1
          for (int k = 0; k < 32; ++k) {
            const bf16x8 one = part_of<true>(a, g == (k >> 3) ? (k & 7) : -1);
#pragma unroll
            for (int i = 0; i < QT; ++i) {
              const f32x4 z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one, pb[i], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
              if (cur * kAttnTile + 32 * j + k < lim[i]) o[d][i] += z;
            }
          }
#pragma unroll
          for (int i = 0; i < QT; ++i)
            o[d][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(part_of<false>(a, 0), pb[i], o[d][i], 0, 0, 0);
        }
      }
    }
    wait_copies();
    lds_barrier();
    cur = nxt;
    rows_cur = rows_nxt;
    sc_cur = sc_nxt;
    nxt = wk.find_tile(nxt + 1, v_nn, rows_nxt);
    ++it;
  }

  // ---- totals over the waves, then the result
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const float x = sum_over_groups(l[i]);
    if (g == 0) red[w][i * 16 + lo] = x;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int r = i * 16 + lo;
    const float tot = (red[0][r] + red[1][r]) + (red[2][r] + red[3][r]);
    if (r >= nv) continue;
    const int64_t R = r0 + r;
    if (p.splits > 1) {
      float* po = p.part + ((int64_t)wk.split * nrows + R) * kLatent + 128 * w + 4 * g;
#pragma unroll
      for (int d = 0; d < 8; ++d) *reinterpret_cast<f32x4*>(po + 16 * d) = o[d][i];
      if (w == 0 && g == 0) {
        p.part_ml[((int64_t)wk.split * nrows + R) * 2] = m[i];
        p.part_ml[((int64_t)wk.split * nrows + R) * 2 + 1] = tot;
      }
    } else {
      const float inv = tot > 0.f ? 1.f / tot : (tot == 0.f ? 0.f : tot);  // no key: zeros; NaN stays
      uint16_t* po = p.out + R * kLatent + 128 * w + 4 * g;
#pragma unroll
      for (int d = 0; d < 8; ++d)
        *reinterpret_cast<bf16x4*>(po + 16 * d) = __builtin_convertvector(o[d][i] * inv, bf16x4);
      if (p.lse && w == 0 && g == 0)
        p.lse[R] = tot == 0.f ? -INFINITY : (m[i] + log2_fast(tot)) * 0.6931471805599453f;
    }
  }
}

// The same for 32 G rows (G = 2 or 4) per workgroup of four waves: each wave owns
// 32 rows and 64 G / 4 keys of a tile, with its own reference and total, so the
// weights never leave the lanes that formed them (result rows of S^T = C Q^T are
// keys; the contraction of O^T = C^T P^T takes the keys in that order). With G =
// 4 a tile serves 128 rows. With G = 2 the two waves of a row group take
// alternate halves of each tile and are joined at the end.
template <int G, bool FP8, bool LIST>
__global__ __launch_bounds__(256, 1) void k_latent_wide(LatentArgs p) {
  using Tile = LatentTile<FP8, true>;
  constexpr int NQ = 32 * G, NS = G / 2;  // rows; 32-key steps of a wave per tile
  __shared__ __attribute__((aligned(1024))) unsigned char tile[2][Tile::kBytes];
  __shared__ __attribute__((aligned(16))) float ksc[2][kAttnTile];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h2 = lane >> 5, lo = lane & 15;
  const int grp = w % G, half = w / G;  // row group, key half of a tile (G = 2)

  LatentWork<NQ, LIST> wk(p, lane);
  if (!wk.valid) return;
  const int64_t r0 = wk.r0, nrows = (int64_t)p.T * p.H;
  const int nv = wk.nv, tile_end = wk.tile_end;
  const int r = 32 * grp + c;  // the lane's row
  const int lim = LIST ? 0 : wk.limit(r);

  const uint32_t tile_lds = lds_addr(&tile[0][0]);
  auto stage = [&](int b, int rows) { stage_tile<Tile, FP8>(p, tile_lds + b * Tile::kBytes, w, lane, rows); };
  auto key_scale = [&](int rows) -> float {
    if constexpr (FP8) return w == 0 && rows >= 0 ? p.scale[rows] : 0.f;
    return 0.f;
  };

  int rows_cur, rows_nxt;
  int cur = wk.find_tile(wk.cur, wk.list_entry(wk.cur), rows_cur);
  int nxt = wk.find_tile(cur + 1, wk.list_entry(cur + 1), rows_nxt);
  if (FP8 && w == 0) ksc[0][lane] = key_scale(rows_cur);
  if (cur < tile_end) stage(0, rows_cur);

  // Q as the B operand: K step ks, lane (row c, half h2): values 16 ks + 8 h2 .. + 7; with
  // codes, whose 16-byte chunk covers two K steps, 32 (ks / 2) + 16 h2 + 8 (ks % 2) .. + 7
  const float sm = scale_magnitude(p.sm_log2);
  bf16x8 qf[36];
  {
    const uint32_t sign = p.sm_log2 < 0.f ? 0x80008000u : 0u;
    const uint16_t* qr = p.q + (r0 + min(r, nv - 1)) * (kLatent + kRotary);
#pragma unroll
    for (int ks = 0; ks < 36; ++ks) {
      const int at = (FP8 && ks < 32) ? 32 * (ks >> 1) + 16 * h2 + 8 * (ks & 1) : 16 * ks + 8 * h2;
      qf[ks] = flip_sign(*reinterpret_cast<const bf16x8*>(qr + at), sign);
    }
  }
  f32x16 o[16];
#pragma unroll
  for (int d = 0; d < 16; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
#pragma unroll
  for (int d = 0; d < 16; ++d) in_agprs(o[d]);
  float m = kNoMax, l = 0.f;
  wait_copies();
  __syncthreads();

  // the lane's addresses in a tile (see k_latent)
  const uint32_t a_key = c * Tile::kRow + ((h2 ^ Tile::swz(c)) * 16);
  const uint32_t a_rot = Tile::kRope + c * Tile::kRopeRow + ((h2 ^ Tile::swz_rope(c)) * 16);
  const int vrow = FP8 ? 4 * h2 + ((lo >> 1) & 3) + 8 * (lo >> 3) : 4 * h2 + (lo >> 2);
  const uint32_t a_val = vrow * Tile::kRow + (lo & 1) * 8 +
                         (FP8 ? ((lane >> 4) & 1) ^ Tile::swz(vrow)
                              : (2 * ((lane >> 4) & 1) + ((lo & 3) >> 1)) ^ Tile::swz(vrow)) * 16;

  int it = 0;
  while (cur < tile_end) {
    const uint32_t tb = tile_lds + (it & 1) * Tile::kBytes;
    const bool mixed = !LIST && (cur + 1) * kAttnTile > wk.same;
    const int v_nn = wk.list_entry(nxt + 1);
    const float sc_nxt = key_scale(rows_nxt);
    if (nxt < tile_end) stage((it + 1) & 1, rows_nxt);
    const uint64_t live = wave_ballot(rows_cur >= 0);

#pragma unroll 1
    for (int n0 = 0; n0 < NS; ++n0) {
      const int n = G == 2 ? half : n0;  // keys 32 n .. + 31 of the tile
      const uint32_t nb = tb + n * 32 * Tile::kRow;
      const uint32_t ka = nb + a_key, ra = tb + a_rot + n * 32 * Tile::kRopeRow, va = nb + a_val;
      f32x16 s;
      f32x4 sc4[4];
      if constexpr (FP8) {
#pragma unroll
        for (int cc = 0; cc < 16; ++cc) {
          const u32x4 v = lds_read<u32x4>(ka ^ (32 * cc));
          const bf16x8 a0 = codes_to_bf16(u32x2{v.x, v.y}), a1 = codes_to_bf16(u32x2{v.z, v.w});
          if (cc == 0)
            mfma_vgpr_first(s, a0, qf[0]);
          else
            mfma_vgpr(s, a0, qf[2 * cc]);
          mfma_vgpr(s, a1, qf[2 * cc + 1]);
        }
        // a key's scale multiplies its latent part only
        mfma_done(s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc4[i] = *reinterpret_cast<const f32x4*>(&ksc[it & 1][32 * n + 8 * i + 4 * h2]);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[4 * i + e] *= sc4[i][e];
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < 32; ++ks) {
          const bf16x8 a = lds_read<bf16x8>((ka ^ (32 * (ks & 15))) + 512 * (ks >> 4));
          if (ks == 0)
            mfma_vgpr_first(s, a, qf[0]);
          else
            mfma_vgpr(s, a, qf[ks]);
        }
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) mfma_vgpr(s, lds_read<bf16x8>(ra ^ (32 * ks)), qf[32 + ks]);
      mfma_done(s);

      // ---- weights of keys 32 n + 8 (e / 4) + 4 h2 + e % 4
      auto values = [&](int j, int d) -> bf16x8 {  // values 32 d .. + 31, keys 32 n + 16 j .. + 15
        if constexpr (FP8)
          return codes_to_bf16(lds_read_tr8((va ^ (32 * d) ^ (256 * j)) + 16 * j * Tile::kRow));
        else
          return join_rows(
              lds_read_tr16((va ^ (64 * (d & 7)) ^ (256 * j)) + 512 * (d >> 3) + 16 * j * Tile::kRow),
              lds_read_tr16((va ^ (64 * (d & 7)) ^ (256 * j) ^ 32) + 512 * (d >> 3) + (16 * j + 8) * Tile::kRow));
      };
      const uint32_t mine = (uint32_t)(live >> (32 * n));
      bool odd = false;
      if (mixed || mine != 0xffffffffu) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int key = 8 * (e >> 2) + 4 * h2 + (e & 3);
          const bool ok = LIST ? (mine >> key) & 1u : cur * kAttnTile + 32 * n + key < lim;
          s[e] = ok ? s[e] : -INFINITY;
        }
        if (__builtin_expect(mixed, 0)) {
#pragma unroll 1
          for (int i = 0; i < 32; ++i) odd |= any_odd(values(i >> 4, i & 15));
          odd = __any(odd);
        }
      }
      float top = s[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
      top = max_halves(top) * sm;
      if (__builtin_expect(__any(top > m + kSlack), 0)) {
        const float mm = fmaxf(m, top), f = exp2_fast(m - mm);
        m = mm;
        l *= f;
#pragma unroll
        for (int d = 0; d < 16; ++d) {
          in_agprs(o[d]);
          o[d] *= f;
          in_agprs(o[d]);
        }
      }
      bf16x8 pb[2];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float x = exp2_fast(fmaf(s[e], sm, -m));
        l += x;  // the total keeps 32 bits; the weights are rounded to bf16 for the matrix cores
        if constexpr (FP8) x = mixed && x == 0.f ? 0.f : x * sc4[e >> 2][e & 3];
        pb[e >> 3][e & 7] = (__bf16)x;
      }
      // ---- sums of values 32 d + (result row) for row c
      if (__builtin_expect(!odd, 1)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int d = 0; d < 16; ++d)
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(values(j, d), pb[j], o[d], 0, 0, 0);
      } else {  // each key with a value that is not finite adds it to the rows that see the key
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int d = 0; d < 16; ++d) {
            in_agprs(o[d]);
            const bf16x8 a = values(j, d);
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
              const bf16x8 one = part_of<true>(a, h2 == (k >> 3) ? (k & 7) : -1);
              f32x16 z;
#pragma unroll
              for (int e = 0; e < 16; ++e) z[e] = 0.f;
              z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(one, pb[j], z, 0, 0, 0);
              const int key = cur * kAttnTile + 32 * n + 16 * j + 8 * ((k & 7) >> 2) + 4 * (k >> 3) + (k & 3);
              if (key < lim) o[d] += z;
            }
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(part_of<false>(a, 0), pb[j], o[d], 0, 0, 0);
            in_agprs(o[d]);
          }
      }
    }
    wait_copies();
    if (FP8 && w == 0) ksc[(it + 1) & 1][lane] = sc_nxt;
    lds_barrier();
    cur = nxt;
    rows_cur = rows_nxt;
    nxt = wk.find_tile(nxt + 1, v_nn, rows_nxt);
    ++it;
  }

  // ---- result: lane holds values 32 d + 8 i + 4 h2 + 0..3 of its row
  float tot = sum_halves(l);
  if constexpr (G == 2) {  // the two waves of a row group, through LDS
    constexpr int kPass = FP8 ? 4 : 8;  // accumulator tiles (4 KB a wave) at a time
    static_assert(2 * kPass * 4096 <= 2 * Tile::kBytes, "exchange space");
    f32x4* ex = reinterpret_cast<f32x4*>(&tile[0][0]) + grp * kPass * 256;
    float* ml = &ksc[0][0];
    if (half == 1 && h2 == 0) ml[32 * grp + c] = m, ml[64 + 32 * grp + c] = tot;
    __syncthreads();
    const float m1 = ml[32 * grp + c], t1 = ml[64 + 32 * grp + c];
    const float mm = fmaxf(m, m1), f0 = exp2_fast(m - mm), f1 = exp2_fast(m1 - mm);
#pragma unroll
    for (int d0 = 0; d0 < 16; d0 += kPass) {
      if (half == 1) {
#pragma unroll
        for (int d = 0; d < kPass; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ex[(d * 4 + i) * 64 + lane] =
                f32x4{o[d0 + d][4 * i], o[d0 + d][4 * i + 1], o[d0 + d][4 * i + 2], o[d0 + d][4 * i + 3]};
      }
      __syncthreads();
      if (half == 0) {
#pragma unroll
        for (int d = 0; d < kPass; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 x = ex[(d * 4 + i) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d0 + d][4 * i + e] = o[d0 + d][4 * i + e] * f0 + x[e] * f1;
          }
      }
      __syncthreads();
    }
    if (half == 1) return;
    m = mm;
    tot = tot * f0 + t1 * f1;
  }
  if (r >= nv) return;
  const int64_t R = r0 + r;
  if (p.splits > 1) {
    float* po = p.part + ((int64_t)wk.split * nrows + R) * kLatent + 4 * h2;
#pragma unroll
    for (int d = 0; d < 16; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(po + 32 * d + 8 * i) =
            f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    if (h2 == 0) {
      p.part_ml[((int64_t)wk.split * nrows + R) * 2] = m;
      p.part_ml[((int64_t)wk.split * nrows + R) * 2 + 1] = tot;
    }
  } else {
    const float inv = tot > 0.f ? 1.f / tot : (tot == 0.f ? 0.f : tot);  // no key: zeros; NaN stays
    uint16_t* po = p.out + R * kLatent + 4 * h2;
#pragma unroll
    for (int d = 0; d < 16; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 v = {o[d][4 * i] * inv, o[d][4 * i + 1] * inv, o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv};
        *reinterpret_cast<bf16x4*>(po + 32 * d + 8 * i) = __builtin_convertvector(v, bf16x4);
      }
    if (p.lse && h2 == 0) p.lse[R] = tot == 0.f ? -INFINITY : (m + log2_fast(tot)) * 0.6931471805599453f;
  }
}

// Joins the splits of a row: each split's sums and total weigh 2^(its reference
// - the largest). One workgroup a row, `width` / 4 threads wide; the threads
// beyond take further splits and are added through LDS in a fixed order.
template <int WIDTH>
__global__ __launch_bounds__(256) void k_join(const float* part, const float* part_ml, int splits, int64_t rows,
                                              uint16_t* out, float* lse) {
  constexpr int TPR = WIDTH / 4, SG = 256 / TPR;
  __shared__ __attribute__((aligned(16))) float sums[SG][WIDTH];
  __shared__ float tots[SG];
  const int64_t r = blockIdx.x;
  const int c = threadIdx.x % TPR, sg = threadIdx.x / TPR;
  float top = kNoMax;
  for (int s = threadIdx.x & 63; s < splits; s += 64) top = fmaxf(top, part_ml[((int64_t)s * rows + r) * 2]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
  float tot = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = sg; s < splits; s += SG) {
    const float* ml = part_ml + ((int64_t)s * rows + r) * 2;
    const float f = exp2_fast(ml[0] - top);
    tot += f * ml[1];
    acc += *reinterpret_cast<const f32x4*>(part + ((int64_t)s * rows + r) * WIDTH + c * 4) * f;
  }
  *reinterpret_cast<f32x4*>(&sums[sg][c * 4]) = acc;
  if (c == 0) tots[sg] = tot;
  __syncthreads();
  if (sg != 0) return;
#pragma unroll
  for (int i = 1; i < SG; ++i) {
    acc += *reinterpret_cast<const f32x4*>(&sums[i][c * 4]);
    tot += tots[i];
  }
  const float inv = tot > 0.f ? 1.f / tot : (tot == 0.f ? 0.f : tot);
  *reinterpret_cast<bf16x4*>(out + r * WIDTH + c * 4) = __builtin_convertvector(acc * inv, bf16x4);
  if (lse && c == 0) lse[r] = tot == 0.f ? -INFINITY : (top + log2_fast(tot)) * 0.6931471805599453f;
}

hipError_t launch_join(const LaunchCtx& cx, const float* part, const float* part_ml, int splits, int64_t rows,
                       int width, uint16_t* out, float* lse) {
  const dim3 grid((unsigned)rows);
  return width == kLatent
             ? cx.launch("k_join", k_join<kLatent>, grid, dim3(256), 0, part, part_ml, splits, rows, out, lse)
             : cx.launch("k_join", k_join<kValue>, grid, dim3(256), 0, part, part_ml, splits, rows, out, lse);
}

static int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

AttnPlan latent_plan(int T, int H, int keys, bool lists, bool fp8, bool shared_keys) {
  AttnPlan pl{};
  // rows of different queries share a tile where they read the same keys
  const int64_t rows = shared_keys ? (int64_t)T * H : H;
  pl.nq = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  pl.head_tiles = shared_keys ? 0 : cdiv(H, pl.nq);
  pl.row_tiles = shared_keys ? cdiv(rows, pl.nq) : T * pl.head_tiles;
  const int tiles = std::max(1, cdiv(keys, kAttnTile));
  const int want = std::max(1, 256 / std::max(1, pl.row_tiles));
  pl.tiles_per_split = std::max(1, cdiv(tiles, std::min(want, tiles)));
  pl.splits = cdiv(tiles, pl.tiles_per_split);
  return pl;
}

size_t latent_ws_bytes(const AttnPlan& pl, int T, int H) {
  if (pl.splits <= 1) return 256;
  const size_t rows = (size_t)T * H;
  return 256 + rows * pl.splits * (kLatent + 2) * 4;
}

template <int NQ, bool FP8>
static hipError_t launch_latent_nq(const LaunchCtx& cx, const LatentArgs& a, dim3 grid) {
  return a.idx ? cx.launch("k_latent", k_latent<NQ, FP8, true>, grid, dim3(256), 0, a)
               : cx.launch("k_latent", k_latent<NQ, FP8, false>, grid, dim3(256), 0, a);
}

template <int G, bool FP8>
static hipError_t launch_latent_wide(const LaunchCtx& cx, const LatentArgs& a, dim3 grid) {
  return a.idx ? cx.launch("k_latent_wide", k_latent_wide<G, FP8, true>, grid, dim3(256), 0, a)
               : cx.launch("k_latent_wide", k_latent_wide<G, FP8, false>, grid, dim3(256), 0, a);
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
  a.tiles_per_split = pl.tiles_per_split;
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
