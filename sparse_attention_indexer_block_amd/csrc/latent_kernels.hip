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
// the row (chunk ^ swizzle): the 16 rows of an operand read, and the rows of a
// transposing read, then fall on distinct banks.
template <bool FP8>
struct LatentTile {
  static constexpr int kRow = FP8 ? kLatent : 2 * kLatent;
  static constexpr int kBytes = kAttnTile * (kRow + 2 * kRotary);
  static constexpr int kRope = kAttnTile * kRow;  // offset of the rotary rows
  static __device__ __forceinline__ int swz(int row) {
    if constexpr (FP8)
      return ((row & 7) << 1) | ((row & 8) << 1) | ((row >> 3) & 1);
    else
      return ((row & 3) << 1) | (row & 8) | ((row & 4) << 2);
  }
  static __device__ __forceinline__ int swz_rope(int row) { return ((row >> 2) & 3) << 1; }
};

// NQ rows and a share of the keys per workgroup of four waves. Per tile of 64
// keys: wave w scores keys 16 w .. 16 w + 15 against all NQ rows (S^T = C Q^T
// with Q in registers), the weights cross LDS once, and wave w sums values
// 128 w .. 128 w + 127 over all 64 keys (O^T = C^T P^T, C^T by transposing LDS
// reads). So the tile is read from LDS twice whatever NQ is, the accumulators
// are spread over the waves, and a row's reference and weights stay in the
// lanes that hold its column. The copy of the next tile runs meanwhile.
template <int NQ, bool FP8, bool LIST>
__global__ __launch_bounds__(256, 1) void k_latent(LatentArgs p) {
  using Tile = LatentTile<FP8>;
  constexpr int QT = NQ / 16;
  __shared__ __attribute__((aligned(1024))) unsigned char tile[2][Tile::kBytes];
  __shared__ __attribute__((aligned(16))) uint16_t pt[NQ * kAttnTile];  // weights, 128 bytes a row
  __shared__ float red[4][NQ];
  __shared__ int raise[2];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lo = lane & 15, g = lane >> 4;

  // neighbouring workgroups run on different XCDs; give each XCD a run of
  // neighbouring queries, with the row tiles and splits of one query together
  const int per = (int)(gridDim.x / 8);
  const int lid = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  const int ht = p.head_tiles ? p.head_tiles : 1;
  const int rt = (lid / (ht * p.splits)) * ht + lid % ht;
  const int split = (lid / ht) % p.splits;
  if (rt >= p.row_tiles) return;

  const int64_t nrows = (int64_t)p.T * p.H;
  int64_t r0;
  int nv, t = 0;
  if (p.head_tiles) {
    t = rt / p.head_tiles;
    const int h0 = (rt % p.head_tiles) * NQ;
    r0 = (int64_t)t * p.H + h0;
    nv = min(NQ, p.H - h0);
  } else {
    r0 = (int64_t)rt * NQ;
    nv = (int)min((int64_t)NQ, nrows - r0);
  }
  const int base = (p.base && p.head_tiles) ? p.base[t] : 0;

  // keys of this workgroup: entries j0 .. j1 - 1 of the list or of the prefix
  int lim[QT];  // visible keys of each of the lane's rows
  int j1;
  if constexpr (LIST) {
    j1 = p.k;
  } else {
    j1 = 0;
    const int left = base < 0 ? 0 : max(0, p.rows - base);
    if (p.head_tiles) {
      j1 = visible_keys(p.pos[t], left);
#pragma unroll
      for (int i = 0; i < QT; ++i) lim[i] = j1;
    } else {
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const int r = i * 16 + lo;
        lim[i] = r < nv ? visible_keys(p.pos[(r0 + r) / p.H], left) : 0;
        j1 = max(j1, lim[i]);
      }
      j1 = (int)wave_max_u32((uint32_t)j1);
    }
    j1 = __builtin_amdgcn_readfirstlane(j1);
  }
  // tiles from here on hold keys that not every row sees
  int same = 0x7fffffff;
  if constexpr (!LIST) {
    if (!p.head_tiles) {
#pragma unroll
      for (int i = 0; i < QT; ++i) same = min(same, i * 16 + lo < nv ? lim[i] : 0x7fffffff);
      same = __builtin_amdgcn_readfirstlane((int)wave_min_u32((uint32_t)same));
    }
  }
  const int tile_end = min((j1 + kAttnTile - 1) / kAttnTile, (split + 1) * p.tiles_per_split);
  int cur = split * p.tiles_per_split;

  // entry 64 * ti + lane of the list, and the cache row it names or -1
  auto list_entry = [&](int ti) -> int {
    if constexpr (LIST) {
      const int j = ti * kAttnTile + lane;
      if (j < p.k) return p.idx[(int64_t)t * p.k + j];
    }
    return -1;
  };
  auto row_of = [&](int ti, int v) -> int {
    if constexpr (LIST) {
      const int64_t row = (int64_t)v + base;
      return (v >= 0 && base >= 0 && row < p.rows) ? (int)row : -1;
    } else {
      const int j = ti * kAttnTile + lane;
      return j < j1 ? base + j : -1;
    }
  };
  // first tile at or after ti that holds a key; v: ti's list entries, rows: the found tile's rows
  auto find_tile = [&](int ti, int v, int& rows) -> int {
    rows = -1;
    while (ti < tile_end) {
      rows = row_of(ti, v);
      if (wave_ballot(rows >= 0) != 0) break;
      v = list_entry(++ti);
    }
    return ti;
  };

  const unsigned char* C = static_cast<const unsigned char*>(p.c);
  const unsigned char* zero = reinterpret_cast<const unsigned char*>(g_zero_row);
  const uint32_t tile_lds = lds_addr(&tile[0][0]);

  // copies key rows 16 w .. 16 w + 15 of a tile (rows: see entry) into buffer b
  auto stage = [&](int b, int rows) {
    const uint32_t dst = tile_lds + b * Tile::kBytes;
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
        copy16_to_lds(src + ((lane ^ Tile::swz(row)) * 16), dst + row * Tile::kRow);
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
      copy16_to_lds(src + ch * 16, dst + Tile::kRope + (16 * w + 8 * i) * (2 * kRotary));
    }
  };
  auto key_scale = [&](int rows) -> float {
    if constexpr (FP8) return rows >= 0 ? p.scale[rows] : 0.f;
    return 0.f;
  };

  int rows_cur, rows_nxt;
  cur = find_tile(cur, list_entry(cur), rows_cur);
  int nxt = find_tile(cur + 1, list_entry(cur + 1), rows_nxt);
  float sc_cur = key_scale(rows_cur);
  if (cur < tile_end) stage(0, rows_cur);

  // Q as the B operand: lane (row lo, group g) of K step ks holds values
  // 32 ks + 8 g .. + 7; with codes, whose 16-byte chunk covers two K steps,
  // values 64 (ks / 2) + 16 g + 8 (ks % 2) .. + 7 of the latent part
  bf16x8 qf[QT][18];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int r = i * 16 + lo;
    const uint16_t* qr = p.q + (r0 + min(r, nv - 1)) * (kLatent + kRotary);
#pragma unroll
    for (int ks = 0; ks < 18; ++ks) {
      const int at = (FP8 && ks < 16) ? 64 * (ks >> 1) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g;
      qf[i][ks] = *reinterpret_cast<const bf16x8*>(qr + at);
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

  int it = 0;
  const int krow = 16 * w + lo;  // the lane's key row as the A operand of the scores
  while (cur < tile_end) {
    const unsigned char* tb = tile[it & 1];
    const bool mixed = !LIST && (cur + 1) * kAttnTile > same;
    // the list entries after the next tile and the next tile's scales are asked
    // for ahead of its copy and used after the copy has landed
    const int v_nn = list_entry(nxt + 1);
    const float sc_nxt = key_scale(rows_nxt);
    if (nxt < tile_end) stage((it + 1) & 1, rows_nxt);

    // ---- scores of keys 16 w + 4 g + 0..3 (result rows) for rows 16 i + lo (columns)
    f32x4 s[QT];
#pragma unroll
    for (int i = 0; i < QT; ++i) s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (FP8) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(tb + krow * Tile::kRow + (((4 * c + g) ^ Tile::swz(krow)) * 16));
        const bf16x8 a0 = codes_to_bf16(u32x2{v.x, v.y}), a1 = codes_to_bf16(u32x2{v.z, v.w});
#pragma unroll
        for (int i = 0; i < QT; ++i) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, qf[i][2 * c], s[i], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < QT; ++i) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, qf[i][2 * c + 1], s[i], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < 16; ++ks) {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(tb + krow * Tile::kRow + (((4 * ks + g) ^ Tile::swz(krow)) * 16));
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
    for (int ks = 16; ks < 18; ++ks) {
      const bf16x8 a = *reinterpret_cast<const bf16x8*>(
          tb + Tile::kRope + krow * (2 * kRotary) + (((4 * (ks - 16) + g) ^ Tile::swz_rope(krow)) * 16));
#pragma unroll
      for (int i = 0; i < QT; ++i) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, qf[i][ks], s[i], 0, 0, 0);
    }

    // ---- weights against the present reference
    const uint64_t live = wave_ballot(rows_cur >= 0);
    const uint32_t mine = (uint32_t)(live >> (16 * w + 4 * g)) & 15u;
    float top[QT];
    bool high = false;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      s[i] *= p.sm_log2;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        bool ok = (mine >> e) & 1u;
        if constexpr (!LIST) ok = cur * kAttnTile + 16 * w + 4 * g + e < lim[i];
        s[i][e] = ok ? s[i][e] : -INFINITY;
      }
      top[i] = max_over_groups(fmaxf(fmaxf(s[i].x, s[i].y), fmaxf(s[i].z, s[i].w)));
      high |= top[i] > m[i] + kSlack;
      if (g == 0) red[w][i * 16 + lo] = top[i];
    }
    float sum[QT];
    auto weigh = [&]() {
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        f32x4 e;
#pragma unroll
        for (int x = 0; x < 4; ++x) e[x] = exp2_fast(s[i][x] - m[i]);
        sum[i] = (e.x + e.y) + (e.z + e.w);
        // rounded to bf16 for the matrix cores; the row's total keeps 32 bits
        if constexpr (FP8) {
#pragma unroll
          for (int x = 0; x < 4; ++x) e[x] = mixed && e[x] == 0.f ? 0.f : e[x] * ksc[x];
        }
        const bf16x4 b = __builtin_convertvector(e, bf16x4);
        const int r = i * 16 + lo;
        const int ch = (2 * w + (g >> 1)) ^ (r & 7);
        *reinterpret_cast<bf16x4*>(reinterpret_cast<unsigned char*>(pt) + r * 128 + ch * 16 + (g & 1) * 8) = b;
      }
    };
    weigh();
    if (__any(high) && lane == 0) raise[it & 1] = 1;
    lds_barrier();
    if (raise[it & 1]) {  // the same for all waves: move the references up, weigh again
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
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      bf16x8 pb[QT];
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const int r = i * 16 + lo;
        pb[i] = *reinterpret_cast<const bf16x8*>(reinterpret_cast<const unsigned char*>(pt) + r * 128 +
                                                 (((4 * j + g) ^ (r & 7)) * 16));
      }
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        bf16x8 a;
        if constexpr (FP8) {
          const int row = 32 * j + 8 * g + (lo >> 1);
          const int ch = (8 * w + d) ^ Tile::swz(row);
          const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds_i32x2*)(tb + row * Tile::kRow + ch * 16 + (lo & 1) * 8));
          a = codes_to_bf16(__builtin_bit_cast(u32x2, v));
        } else {
          const int row = 32 * j + 8 * g + (lo >> 2);
          const int c0 = 16 * w + 2 * d + ((lo & 3) >> 1);
          const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4*)(tb + row * Tile::kRow + (c0 ^ Tile::swz(row)) * 16 + (lo & 1) * 8));
          const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4*)(tb + (row + 4) * Tile::kRow + (c0 ^ Tile::swz(row + 4)) * 16 + (lo & 1) * 8));
          a = __builtin_bit_cast(bf16x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        if (mixed && __any(any_odd(a))) {
          // each key with such a value adds it to the rows that see the key
          for (int k = 0; k < 32; ++k) {
            const bf16x8 one = part_of<true>(a, g == (k >> 3) ? (k & 7) : -1);
#pragma unroll
            for (int i = 0; i < QT; ++i) {
              const f32x4 z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one, pb[i], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
              const bool sees = cur * kAttnTile + 32 * j + k < (LIST ? 0 : lim[i]);
              if (sees) o[d][i] += z;
            }
          }
          a = part_of<false>(a, 0);
        }
#pragma unroll
        for (int i = 0; i < QT; ++i) o[d][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, pb[i], o[d][i], 0, 0, 0);
      }
    }
    wait_copies();
    lds_barrier();
    cur = nxt;
    rows_cur = rows_nxt;
    sc_cur = sc_nxt;
    nxt = find_tile(nxt + 1, v_nn, rows_nxt);
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
      float* po = p.part + ((int64_t)split * nrows + R) * kLatent + 128 * w + 4 * g;
#pragma unroll
      for (int d = 0; d < 8; ++d) *reinterpret_cast<f32x4*>(po + 16 * d) = o[d][i];
      if (w == 0 && g == 0) {
        p.part_ml[((int64_t)split * nrows + R) * 2] = m[i];
        p.part_ml[((int64_t)split * nrows + R) * 2 + 1] = tot;
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

// One workgroup of width / 4 threads joins the splits of a row: each split's
// sums and total weigh 2^(its reference - the largest).
__global__ __launch_bounds__(128) void k_join(const float* part, const float* part_ml, int splits, int64_t rows,
                                              int width, uint16_t* out, float* lse) {
  const int64_t r = blockIdx.x;
  const int c = threadIdx.x * 4;
  float top = kNoMax;
  for (int s = 0; s < splits; ++s) {
    const float* ml = part_ml + ((int64_t)s * rows + r) * 2;
    if (ml[1] != 0.f) top = fmaxf(top, ml[0]);
  }
  float tot = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const float* ml = part_ml + ((int64_t)s * rows + r) * 2;
    const f32x4 v = *reinterpret_cast<const f32x4*>(part + ((int64_t)s * rows + r) * width + c);
    if (ml[1] == 0.f) continue;
    const float f = exp2_fast(ml[0] - top);
    tot += f * ml[1];
    acc += v * f;
  }
  const float inv = tot > 0.f ? 1.f / tot : (tot == 0.f ? 0.f : tot);
  *reinterpret_cast<bf16x4*>(out + r * width + c) = __builtin_convertvector(acc * inv, bf16x4);
  if (lse && c == 0) lse[r] = tot == 0.f ? -INFINITY : (top + log2_fast(tot)) * 0.6931471805599453f;
}

hipError_t launch_join(const LaunchCtx& cx, const float* part, const float* part_ml, int splits, int64_t rows,
                       int width, uint16_t* out, float* lse) {
  return cx.launch("k_join", k_join, dim3((unsigned)rows), dim3(width / 4), 0, part, part_ml, splits, rows, width, out,
                   lse);
}

static int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

AttnPlan latent_plan(int T, int H, int keys, bool lists, bool fp8, bool shared_keys) {
  AttnPlan pl{};
  // rows of different queries share a tile where they read the same keys
  const int64_t rows = shared_keys ? (int64_t)T * H : H;
  pl.nq = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
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

template <bool FP8>
static hipError_t launch_latent_t(const LaunchCtx& cx, const LatentArgs& a, int nq, dim3 grid) {
  switch (nq) {
    case 16: return launch_latent_nq<16, FP8>(cx, a, grid);
    case 32: return launch_latent_nq<32, FP8>(cx, a, grid);
    default: return launch_latent_nq<64, FP8>(cx, a, grid);
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
