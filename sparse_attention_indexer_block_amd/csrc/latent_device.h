// The kernels of attention over one shared latent vector a token, in absorbed form:
//
//   S[r,s]  = sm * (q[r, 0:512] . c[s] + q[r, 512:576] . rope[s])
//   out[r]  = sum_s softmax_s(S[r,:]) c[s],   lse[r] = log sum_s exp(S[r,s])
//
// for the rows r = (query, head) of one query, over the query's keys. All heads of
// a query read the same keys, and a key row is its own value row. What the keys are
// is a Form (ListForm, PrefixForm here; drafted trees over pages in tree_kernels.hip),
// whose Work walks the tiles of a workgroup.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attention.h"
#include "attention_device.h"

namespace misa {

// What a key that does not exist is read from.
static __device__ const uint4 g_zero_row[(kLatent + kRotary) * 2 / 16] = {};

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

// Where a workgroup's rows and keys are, and the walk over its key tiles. Rows
// come in units of U heads of one query, so that the rows of a unit see the
// same keys; the units of a workgroup belong to one query, or (units of queries
// that share their keys) to consecutive ones.
template <int NQ, int U, bool LIST>
struct LatentWork {
  const LatentArgs& p;
  int lane;
  int rt, t;       // row tile; its query (when head_tiles)
  int base;
  int j1;          // entries of the list, or visible keys of the unit that sees most
  int same;        // keys that every unit sees (prefix form)
  i32x4 ulim;      // visible keys of each unit (units of several queries)
  static_assert(NQ / U <= 4, "at most four units");
  int split, cur, tile_end;
  bool valid;

  struct Unit {
    int64_t row;   // first row (query * H + head)
    int rows, lim; // rows (0: none), visible keys (prefix form)
  };
  __device__ __forceinline__ Unit unit(int i) const {
    const int hc = (p.H + U - 1) / U;
    int tu = t, c;
    if (p.head_tiles) {
      c = (rt % p.head_tiles) * (NQ / U) + i;
    } else {
      const int64_t g = (int64_t)rt * (NQ / U) + i;
      tu = (int)(g / hc);
      c = (int)(g % hc);
    }
    Unit u{0, 0, 0};
    if (tu >= p.T || c >= hc) return u;
    u.row = (int64_t)tu * p.H + c * U;
    u.rows = min(U, p.H - c * U);
    if constexpr (!LIST) u.lim = p.head_tiles ? j1 : visible_keys(p.pos[tu], left());
    return u;
  }

  __device__ __forceinline__ LatentWork(const LatentArgs& a, int lane_) : p(a), lane(lane_) {
    // neighbouring workgroups run on different XCDs; give each XCD a run of
    // neighbouring queries, with the row tiles and splits of one query together
    const int per = (int)(gridDim.x / 8);
    const int lid = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    const int ht = p.head_tiles ? p.head_tiles : 1;
    rt = (lid / (ht * p.splits)) * ht + lid % ht;
    split = (lid / ht) % p.splits;
    valid = rt < p.row_tiles;
    if (!valid) return;
    t = p.head_tiles ? rt / p.head_tiles : 0;
    base = (p.base && p.head_tiles) ? p.base[t] : 0;
    same = 0x7fffffff;
    if constexpr (LIST) {
      j1 = p.k;
    } else if (p.head_tiles) {
      j1 = visible_keys(p.pos[t], left());
    } else {
      j1 = 0;
#pragma unroll
      for (int i = 0; i < NQ / U; ++i) {
        const Unit u = unit(i);
        ulim[i] = __builtin_amdgcn_readfirstlane(u.lim);
        j1 = max(j1, u.lim);
        same = u.rows ? min(same, u.lim) : same;
      }
    }
    j1 = __builtin_amdgcn_readfirstlane(j1);
    same = __builtin_amdgcn_readfirstlane(same);
    // an equal share of the tiles that there are here
    const int tiles = (j1 + kAttnTile - 1) / kAttnTile, share = (tiles + p.splits - 1) / p.splits;
    cur = split * share;
    tile_end = min(tiles, cur + share);
  }
  __device__ __forceinline__ int left() const { return base < 0 ? 0 : max(0, p.rows - base); }
  // keys of tile ti (bits) that a unit with limit lim sees, of those that the tile holds
  __device__ __forceinline__ uint64_t sees(int ti, int lim, uint64_t held) const {
    const int n = lim - ti * kAttnTile;
    return n >= kAttnTile ? held : n <= 0 ? 0 : held & ((1ull << n) - 1);
  }
  // entry 64 * ti + lane of the list (the last one past its end; row_of knows).
  // A load without a branch: it is asked for a tile ahead, and a branch around
  // it would wait for what is in flight.
  __device__ __forceinline__ int list_entry(int ti) const {
    if constexpr (LIST) return p.idx[(int64_t)t * p.k + min(ti * kAttnTile + lane, p.k - 1)];
    return -1;
  }
  // the list entries of the tile after `next`, which was found after tile ti; v: those of
  // tile ti + 2. To be called when v's load has landed, and says so to the compiler:
  // it would wait for copies in flight where v is used otherwise.
  __device__ __forceinline__ int list_after(int ti, int next, int v) const {
    if constexpr (!LIST) return -1;
    asm volatile("" : "+v"(v));
    if (next != ti + 1) {
      v = list_entry(next + 1);
      asm volatile("" : "+v"(v));
    }
    return v;
  }
  // the cache row of key 64 * ti + lane, or -1; v: its list entry
  __device__ __forceinline__ int row_of(int ti, int v) const {
    if constexpr (LIST) {
      const int64_t row = (int64_t)v + base;
      return (v >= 0 && base >= 0 && row < p.rows && ti * kAttnTile + lane < p.k) ? (int)row : -1;
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
  // whether every unit sees what tile ti holds, and the keys of it (bits) that unit u sees of those it holds
  __device__ __forceinline__ bool common(int ti) const { return LIST || (ti + 1) * kAttnTile <= same; }
  __device__ __forceinline__ uint64_t sees(int ti, const Unit& u, uint64_t held) const { return sees(ti, u.lim, held); }
  // where unit u's partial sums go (its first row), and whether there are any
  __device__ __forceinline__ int64_t part_row(const Unit& u, int64_t nrows) const { return (int64_t)split * nrows + u.row; }
  __device__ __forceinline__ bool in_parts() const { return p.splits > 1; }
};
// What a query's keys are: a list, or the prefix that ends at its position.
struct ListForm {
  using Args = LatentArgs;
  static constexpr bool kList = true, kTree = false;
  template <int NQ, int U>
  using Work = LatentWork<NQ, U, true>;
};
struct PrefixForm {
  using Args = LatentArgs;
  static constexpr bool kList = false, kTree = false;
  template <int NQ, int U>
  using Work = LatentWork<NQ, U, false>;
};

// Masks for an operand of eight bf16 values: element e stays if bit key(e) of
// `keep` is set.
template <typename Key>
__device__ __forceinline__ u32x4 keep_mask(uint64_t keep, Key key) {
  u32x4 m;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m[i] = ((keep >> key(2 * i)) & 1 ? 0xffffu : 0u) | ((keep >> key(2 * i + 1)) & 1 ? 0xffff0000u : 0u);
  return m;
}
__device__ __forceinline__ bf16x8 masked(bf16x8 a, u32x4 m) {
  return __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, a) & m);
}

// Copies a tile to LDS, one instruction (1 KB) at a time: a wave that issues them
// back to back stalls, so they are spread over the products of the tile before.
// Wave w copies key rows 16 w .. 16 w + 15, eight at a time, in two halves. aim()
// takes the tile's cache rows (lane i: key i, or -1, which reads zeros) and
// leaves little to do per copy: the addresses of a half's rows lie in the first
// lanes of every 16, from where a copy takes its one (a lane read) or two (spread
// over 32 lanes each by row_newbcast), and flip() brings up the other half's.
template <class Tile, bool FP8>
struct TileCopy {
  static constexpr int kPerEight = FP8 ? 5 : 9;  // copies of eight rows: the rows, then their rotary values
  static constexpr int kCopies = 2 * kPerEight;
  static constexpr int kRowsACopy = FP8 ? 2 : 1;
  const LatentArgs& p;
  int w, lane;
  int half;            // the half that is up
  uint32_t off;        // the lane's chunk of a copy, in the order of the half's first row
  uint64_t held;       // address of key row own_row()
  int rot[2];          // the lane's rotary rows, counted from rot_base
  uint64_t rot_base;

  __device__ __forceinline__ TileCopy(const LatentArgs& a, int w_, int lane_) : p(a), w(w_), lane(lane_), half(0) {
    off = FP8 ? ((lane & 31) ^ Tile::swz(16 * w + (lane >> 5))) * 16 : (lane ^ Tile::swz(16 * w)) * 16;
  }
  // the row of the tile whose address lane i holds
  __device__ __forceinline__ int own_row() const {
    const int i = lane & 7;
    return 16 * w + (lane & 8) + (FP8 ? 2 * (i & 3) + (lane >> 5) : i);
  }
  __device__ __forceinline__ uint64_t address(const void* from, int row, int stride, int offset) const {
    return row >= 0 ? (uint64_t)(uintptr_t)from + (uint64_t)(uint32_t)row * (uint32_t)stride + offset
                    : (uint64_t)(uintptr_t)g_zero_row;
  }
  // copies from q instead, with the layout of bf16 key rows: row i is row i % 32 of unit u0 or u1
  template <typename Unit>
  __device__ __forceinline__ void aim_q(const Unit& u0, const Unit& u1) {
    static_assert(!FP8, "queries are bf16 rows");
    constexpr int kStride = 2 * (kLatent + kRotary);
    const Unit& u = w < 2 ? u0 : u1;
    rot_base = (uint64_t)(uintptr_t)p.q + (uint64_t)u.row * kStride;
    const int own = own_row() & 31;
    held = own < u.rows ? rot_base + (uint64_t)(uint32_t)own * kStride : (uint64_t)(uintptr_t)g_zero_row;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 16 * (w & 1) + 8 * i + (lane >> 3);
      rot[i] = r < u.rows ? r : -1;
    }
  }
  __device__ __forceinline__ void aim(int rows) {
    rot_base = (uint64_t)(uintptr_t)(FP8 ? (const void*)p.rope : p.c);
    held = address(p.c, __shfl(rows, own_row(), kWave), FP8 ? kLatent : 2 * (kLatent + kRotary), 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) rot[i] = __shfl(rows, 16 * w + 8 * i + (lane >> 3), kWave);
  }
  // the other half's rows (twice a tile)
  __device__ __forceinline__ void flip() {
    held = (uint64_t)(uint32_t)__builtin_amdgcn_mov_dpp((int)(held >> 32), 0x128, 0xf, 0xf, true) << 32 |  // row_ror:8
           (uint32_t)__builtin_amdgcn_mov_dpp((int)held, 0x128, 0xf, 0xf, true);
    off ^= Tile::swz(8) * 16;
    half ^= 1;
  }
  template <int I>
  __device__ __forceinline__ uint64_t spread_address() const {  // what lane I of every 16 holds
    return (uint64_t)__builtin_amdgcn_mov_dpp((long)held, 0x150 + I, 0xf, 0xf, true);  // row_newbcast:I
  }
  __device__ __forceinline__ uint64_t spread_address(int i) const {
    switch (i) {  // (i is known when this is compiled)
      case 0: return spread_address<0>();
      case 1: return spread_address<1>();
      case 2: return spread_address<2>();
      default: return spread_address<3>();
    }
  }
  // copy j of the half that is up
  __device__ __forceinline__ void copy(uint32_t dst, int j) const {
    const int r0 = 16 * w + 8 * half;
    if (j < kPerEight - 1) {
      // (swz() permutes bits, so a row's order is an exclusive-or of its parts')
      const uint32_t at = off ^ (uint32_t)(Tile::swz(kRowsACopy * j) * 16);
      const uint32_t to = dst + r0 * Tile::kRow + kRowsACopy * j * Tile::kRow;
      if constexpr (FP8) {
        copy16_to_lds(reinterpret_cast<const void*>(spread_address(j) + at), to);
      } else {
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)held, j), hi = __builtin_amdgcn_readlane((uint32_t)(held >> 32), j);
        copy16_to_lds_at(reinterpret_cast<const void*>((uint64_t)hi << 32 | lo), at, to);
      }
    } else {
      const int row = r0 + (lane >> 3), s = half ? rot[1] : rot[0];
      const void* from = reinterpret_cast<const void*>(rot_base);
      const uint64_t src = FP8 ? address(from, s, 2 * kRotary, 0) : address(from, s, 2 * (kLatent + kRotary), 2 * kLatent);
      copy16_to_lds(reinterpret_cast<const void*>(src + (((lane & 7) ^ Tile::swz_rope(row)) * 16)),
                    dst + Tile::kRope + r0 * Tile::kRopeRow);
    }
  }
  // copy i of both halves, in order
  __device__ __forceinline__ void next(uint32_t dst, int i) {
    copy(dst, i % kPerEight);
    if (i % kPerEight == kPerEight - 1) flip();
  }
  __device__ __forceinline__ void all(uint32_t dst) {
#pragma unroll
    for (int i = 0; i < kCopies; ++i) next(dst, i);
  }
};

// NQ = 16 or 32 rows and a share of the keys per workgroup of four waves. Per
// tile of 64 keys: wave w scores keys 16 w .. 16 w + 15 against all NQ rows (S^T
// = C Q^T with Q in registers), the weights cross LDS once, and wave w sums
// values 128 w .. 128 w + 127 over all 64 keys (O^T = C^T P^T, C^T by transposing
// LDS reads). So the tile is read from LDS twice whatever NQ is, the
// accumulators are spread over the waves, and a row's reference and weights stay
// in the lanes that hold its column. The copy of the next tile runs meanwhile.
//
// It serves calls with few rows, which the chain of dependent steps bounds (list,
// rows, products, weights, products, partial sums), not a rate: one query of 16
// heads over 2048 coded keys takes 9 us as 32 workgroups of a tile each, and 4 to
// join them. A tile more costs 1.8 us with 16 rows and 2.2 with 32, of which the
// products are 0.3 and 0.5: the rest is the copy's latency and the barriers.
template <int NQ, bool FP8, class Form>
__global__ __launch_bounds__(256, 1) void k_latent(typename Form::Args p) {
  constexpr bool LIST = Form::kList, TREE = Form::kTree;
  using Work = typename Form::template Work<NQ, 16>;
  using Tile = LatentTile<FP8, false>;
  constexpr int QT = NQ / 16;
  __shared__ __attribute__((aligned(1024))) unsigned char tile[2][Tile::kBytes];
  __shared__ __attribute__((aligned(1024))) uint16_t pt[NQ * kAttnTile];  // weights, 128 bytes a row
  __shared__ float red[4][NQ];
  __shared__ int raise[2];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lo = lane & 15, g = lane >> 4;

  Work wk(p, lane);
  if (!wk.valid) return;
  const int64_t nrows = (int64_t)p.T * p.H;
  const int tile_end = wk.tile_end;
  typename Work::Unit un[QT];
#pragma unroll
  for (int i = 0; i < QT; ++i) un[i] = wk.unit(i);

  const uint32_t tile_lds = lds_addr(&tile[0][0]);
  TileCopy<Tile, FP8> copies{p, w, lane};
  auto key_scale = [&](int rows) -> float {
    if constexpr (FP8) return p.scale[max(rows, 0)];  // (what a row that is no key is scaled by is dropped)
    return 0.f;
  };

  int rows_cur, rows_nxt;
  const int v0 = wk.list_entry(wk.cur), v1 = wk.list_entry(wk.cur + 1);
  int cur = wk.find_tile(wk.cur, v0, rows_cur);
  int nxt = wk.find_tile(cur + 1, cur == wk.cur ? v1 : wk.list_entry(cur + 1), rows_nxt);
  float sc_cur = rows_cur >= 0 ? key_scale(rows_cur) : 0.f;
  copies.aim(rows_cur);
  if (cur < tile_end) copies.all(tile_lds);
  copies.aim(rows_nxt);

  // Q as the B operand: lane (row lo, group g) of K step ks holds values
  // 32 ks + 8 g .. + 7; with codes, whose 16-byte chunk covers two K steps,
  // values 64 (ks / 2) + 16 g + 8 (ks % 2) .. + 7 of the latent part
  const float sm = scale_magnitude(p.sm_log2);
  bf16x8 qf[QT][18];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const uint32_t sign = p.sm_log2 < 0.f ? 0x80008000u : 0u;
    const uint16_t* qr = p.q + (un[i].row + min(lo, max(un[i].rows - 1, 0))) * (kLatent + kRotary);
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
  bool has[QT] = {};  // whether a unit has seen a key (trees)
  // one tile; PART: not every unit sees every key that the tile holds
  auto step = [&](auto part) {
    constexpr bool PART = decltype(part)::value;
    const uint32_t tb = tile_lds + (it & 1) * Tile::kBytes;
    // the list entries after the next tile and the next tile's scales are asked
    // for ahead of its copy and used after the copy has landed
    const int v_nn = wk.list_entry(nxt + 1);
    const float sc_nxt = key_scale(rows_nxt);
    copies.lane = anew(lane);
    uint32_t next_lds = tile_lds + ((it + 1) & 1) * Tile::kBytes;  // (no next tile: zeros, unused)
    if constexpr (TREE) next_lds = __builtin_amdgcn_readfirstlane(next_lds);  // (the same for all lanes, which the compiler does not see here)
    // the next tile's copies, spread over the 16 products of the scores and the 16 of the sums
    auto spread = [&](int i) {
      using Copy = TileCopy<Tile, FP8>;
#pragma unroll
      for (int j = i * Copy::kCopies / 32; j < (i + 1) * Copy::kCopies / 32; ++j)
        copies.next(next_lds, j);
    };

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
        spread(2 * c);
        spread(2 * c + 1);
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < 16; ++ks) {
        const bf16x8 a = lds_read<bf16x8>((ka ^ (64 * (ks & 7))) + 512 * (ks >> 3));
#pragma unroll
        for (int i = 0; i < QT; ++i) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, qf[i][ks], s[i], 0, 0, 0);
        spread(ks);
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
    const uint64_t held = wave_ballot(rows_cur >= 0);
    uint64_t seen[QT];
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      seen[i] = PART ? wk.sees(cur, un[i], held) : held;
      if constexpr (TREE) has[i] |= seen[i] != 0;
    }
    bool high = false;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool ok = (seen[i] >> (16 * w + 4 * g + e)) & 1u;
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
          for (int x = 0; x < 4; ++x)  // (a key that the unit does not see is scaled by 0, whatever its scale is)
            e[x] *= !PART || (seen[i] >> (16 * w + 4 * g + x)) & 1u ? ksc[x] : 0.f;
        }
        *(__attribute__((address_space(3))) bf16x4*)(uintptr_t)(a_pwr + i * 2048) = __builtin_convertvector(e, bf16x4);
      }
    };
    weigh();
    if (__any(high) && lane == 0) raise[it & 1] = 1;
    lds_barrier();
    // the same for all waves: move up the references of the rows that passed theirs (of
    // no other: a row's bits are its own) and weigh again
    if (__builtin_expect(raise[it & 1], 0)) {
      float f[QT];
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const int r = i * 16 + lo;
        const float most = fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r]));
        const float mm = most > m[i] + kSlack ? most : m[i];
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
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      bf16x8 pb[QT];
      u32x4 keep[QT];  // a key that a unit does not see is no value for it, whatever it holds
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        pb[i] = lds_read<bf16x8>((a_prd ^ (64 * j)) + i * 2048);
        if constexpr (PART) keep[i] = keep_mask(seen[i], [&](int e) { return 32 * j + 8 * g + e; });
      }
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const bf16x8 a = values(j, d);
#pragma unroll
        for (int i = 0; i < QT; ++i)
          o[d][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(PART ? masked(a, keep[i]) : a, pb[i], o[d][i], 0, 0, 0);
        spread(16 + 8 * j + d);
      }
    }
    wait_copies();
    lds_barrier();
    cur = nxt;
    sc_cur = rows_nxt >= 0 ? sc_nxt : 0.f;
    rows_cur = rows_nxt;
    nxt = wk.find_tile(nxt + 1, v_nn, rows_nxt);
    copies.aim(rows_nxt);
    ++it;
  };
  while (cur < tile_end && wk.common(cur)) step(std::false_type{});
  if constexpr (!LIST) {
    while (cur < tile_end) step(std::true_type{});
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
    // (a list's tiles are taken only if they hold a key)
    bool keys;
    if constexpr (TREE) {
      keys = has[i] && un[i].live;
      if (!un[i].live) {  // padding, whatever its queries hold
        m[i] = kNoMax;
#pragma unroll
        for (int d = 0; d < 8; ++d) o[d][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    } else {
      keys = LIST ? it > 0 : un[i].lim > 0;
    }
    const float tot = row_total(keys, (red[0][r] + red[1][r]) + (red[2][r] + red[3][r]));
    const int64_t R = un[i].row + lo;
    // (the conditions stand side by side: of nested ones the compiler has left
    // out the end of the inner, and put a copy of a register under its mask)
    const bool live = lo < un[i].rows, first = live && w == 0 && g == 0;
    if (wk.in_parts()) {
      const int64_t P = wk.part_row(un[i], nrows) + lo;
      float* po = p.part + P * kLatent + 128 * w + 4 * g;
      if (live) {
#pragma unroll
        for (int d = 0; d < 8; ++d) *reinterpret_cast<f32x4*>(po + 16 * d) = o[d][i];
      }
      if (first) {
        p.part_ml[P * 2] = m[i];
        p.part_ml[P * 2 + 1] = tot;
      }
    } else {
      const float inv = row_inverse(tot);
      uint16_t* po = p.out + R * kLatent + 128 * w + 4 * g;
      if (live) {
#pragma unroll
        for (int d = 0; d < 8; ++d)
          *reinterpret_cast<bf16x4*>(po + 16 * d) = __builtin_convertvector(o[d][i] * inv, bf16x4);
      }
      if (p.lse && first) p.lse[R] = row_log_sum(m[i], tot);
    }
  }
}

// The same for 32 G rows (G = 2 or 4) per workgroup of four waves: each wave owns
// 32 rows and 64 G / 4 keys of a tile, with its own reference and total, so the
// weights never leave the lanes that formed them (result rows of S^T = C Q^T are
// keys; the contraction of O^T = C^T P^T takes the keys in that order). With G =
// 4 a tile serves 128 rows. With G = 2 the two waves of a row group take
// a half of each tile each and are joined at the end. Where the units of a
// workgroup see different numbers of keys (queries side by side in the prefix
// form), the few tiles that not all of them see in full are taken once for each
// number, with the keys beyond it left out, by the waves that it belongs to.
//
// Bound by the products and what feeds them. A tile and wave of G = 4 has 136
// products of 32 cycles (4352) and takes about 8700: 470 for the weights' exponentials of
// each half, which nothing overlaps (a wave fills its SIMD, and its 512 registers
// leave no room for a second half in flight), 500 at its end, where the copies are
// waited for and the tile after them is found, one after the other: the search's loop
// holds a load of list entries, and the compiler waits for all that is in flight at
// its head (with the search after the barrier, from list entries a tile younger, 1190
// us against 1145), and the products
// themselves run at 0.6 of their rate beside the LDS reads (1 KB a product for each
// of four waves, all that the LDS gives) and copies.
// 2048 queries of 128 heads, 2048 bf16 keys each: 1085-1145 us, 1.02-1.08 PFLOP/s (up
// to 1435 in the first ten calls of a process, while the clock recovers from the onset
// of the load), against 1.15 that a library product of 8192^3 reaches here; coded keys
// 1200-1225 us. A
// workgroup starts and ends in 20 us when all do at once (its queries and results,
// 278 KB, move at the rate of HBM), which is what a short list costs. With G = 2, 32
// queries of 128 heads over 2048 coded keys each take 38 us and 7 to join four splits:
// half of it is the start, the exchange between the waves and 2 KB of sums a row and split.
// Registers: all 512 are taken, and 1 to 7 more with 64 rows and 16 to 19 with 128 are
// spilled, before and after the tile loop; inside it only the bits that mask a tile which
// is not full are reloaded (64 rows, prefixes).
// Tried and left out: queries straight to registers (short lists 5% faster, decode
// batches 4% slower), more LDS reads in flight and weights of half a tile beside the
// products of the other (both spill inside the loop).
template <int G, bool FP8, class Form>
__global__ __launch_bounds__(256, 1) void k_latent_wide(typename Form::Args p) {
  constexpr bool LIST = Form::kList, TREE = Form::kTree;
  using Tile = LatentTile<FP8, true>;
  constexpr int NQ = 32 * G, NS = G / 2;  // rows; 32-key steps of a wave per tile
  constexpr int kAhead = FP8 ? 4 : G == 2 && !LIST ? 5 : 6;  // LDS reads in flight
  __shared__ __attribute__((aligned(1024))) unsigned char tile[2][Tile::kBytes];
  __shared__ __attribute__((aligned(16))) float ksc[2][kAttnTile];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h2 = lane >> 5, lo = lane & 15;
  const int grp = w % G, half = w / G;  // row group, key half of a tile (G = 2)

  typename Form::template Work<NQ, 32> wk(p, lane);
  if (!wk.valid) return;
  const int64_t nrows = (int64_t)p.T * p.H;
  const int tile_end = wk.tile_end;
  const auto un = wk.unit(grp);  // the wave's rows; lane's row un.row + c

  const uint32_t tile_lds = lds_addr(&tile[0][0]);
  TileCopy<Tile, FP8> copies{p, w, lane};
  auto key_scale = [&](int rows) -> float {
    if constexpr (FP8) return p.scale[max(rows, 0)];
    return 0.f;
  };

  // the pass after (tile, number): the next tile that holds a key, or the next
  // number of a tile that is taken by number (who: the unit it is of, -1: all)
  auto next_pass = [&](int ti, int who, int v, int& who_next, int& rows) -> int {
    if constexpr (TREE) {
      return wk.next_pass(ti, who, v, who_next, rows);
    } else if constexpr (!LIST) {
      if (!p.head_tiles) {
        ++who;
        for (; ti < tile_end; ++ti, who = 0) {
          if ((ti + 1) * kAttnTile <= wk.same) {
            who_next = -1;
            rows = wk.row_of(ti, 0);
            return ti;
          }
#pragma unroll
          for (int u = 0; u < G; ++u) {
            bool first = u >= who && wk.ulim[u] > ti * kAttnTile;
#pragma unroll
            for (int x = 0; x < u; ++x) first = first && wk.ulim[x] != wk.ulim[u];
            if (first) {
              who_next = u;
              const int j = ti * kAttnTile + lane;
              rows = j < wk.ulim[u] ? j : -1;
              return ti;
            }
          }
        }
        who_next = -1;
        rows = -1;
        return ti;
      }
    }
    who_next = -1;
    return wk.find_tile(ti, v, rows);
  };
  auto ulim_of = [&](int who) {
    if constexpr (TREE) return 0;
    else {
      int x = wk.ulim[0];
#pragma unroll
      for (int u = 1; u < G; ++u) x = who == u ? wk.ulim[u] : x;
      return x;
    }
  };
  // whether the wave's rows see the keys of this pass
  auto in_pass = [&](int ti, int who) {
    if constexpr (TREE) return wk.in_pass(ti, who, un);
    else return LIST || who < 0 || un.lim == ulim_of(who);
  };
  // (a tile taken by number may have another pass)
  auto after = [&](int ti, int who) { return who < 0 ? ti + 1 : ti; };
  int rows_cur, rows_nxt;
  int who_cur, who_nxt;
  const int v0 = wk.list_entry(wk.cur), v1 = wk.list_entry(wk.cur + 1);
  int cur = next_pass(wk.cur, -1, v0, who_cur, rows_cur);
  int nxt = next_pass(after(cur, who_cur), who_cur, cur == wk.cur ? v1 : wk.list_entry(cur + 1), who_nxt, rows_nxt);
  int v_nn = wk.list_entry(nxt + 1);
  if (FP8 && w == 0) ksc[0][lane] = rows_cur >= 0 ? key_scale(rows_cur) : 0.f;

  // Q as the B operand: K step ks, lane (row c, half h2): values 16 ks + 8 h2 .. + 7; with
  // codes, whose 16-byte chunk covers two K steps, 32 (ks / 2) + 16 h2 + 8 (ks % 2) .. + 7.
  // The rows come through LDS in the layout of bf16 key rows, 64 at a time: loads of
  // 16 bytes a row would touch 32 lines each.
  const float sm = scale_magnitude(p.sm_log2);
  bf16x8 qf[36];
  {
    using QTile = LatentTile<false, true>;
    constexpr int kFit = FP8 ? 1 : 2;  // tiles of 64 rows that fit at once
    static_assert(kFit * QTile::kBytes <= 2 * Tile::kBytes, "query rows fit the key tiles");
    TileCopy<QTile, false> qc{p, w, lane};
    const uint32_t sign = p.sm_log2 < 0.f ? 0x80008000u : 0u;
    const int qrow = 32 * (grp & 1) + c;
#pragma unroll
    for (int q0 = 0; q0 < NQ / 64; q0 += kFit) {
#pragma unroll
      for (int i = q0; i < q0 + kFit && i < NQ / 64; ++i) {
        qc.aim_q(wk.unit(2 * i), wk.unit(2 * i + 1));
        qc.all(tile_lds + (i - q0) * QTile::kBytes);
      }
      wait_copies();
      __syncthreads();
      if (grp / 2 >= q0 && grp / 2 < q0 + kFit) {
        const uint32_t qb = tile_lds + (grp / 2 - q0) * QTile::kBytes + qrow * QTile::kRow;
        const uint32_t qr = tile_lds + (grp / 2 - q0) * QTile::kBytes + QTile::kRope + qrow * QTile::kRopeRow;
#pragma unroll
        for (int ks = 0; ks < 36; ++ks) {
          const int ch = FP8 ? 4 * (ks >> 1) + (ks & 1) : 2 * ks;
          const uint32_t at = ks < 32 ? ((qb + (((FP8 ? 2 * h2 : h2) ^ QTile::swz(qrow)) * 16)) ^ (16 * (ch & 31))) + 512 * (ch >> 5)
                                      : (qr + ((h2 ^ QTile::swz_rope(qrow)) * 16)) ^ (32 * (ks - 32));
          qf[ks] = flip_sign(lds_read<bf16x8>(at), sign);
        }
      }
      lds_barrier();
    }
  }
  copies.aim(rows_cur);
  if (cur < tile_end) copies.all(tile_lds);
  copies.aim(rows_nxt);

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
  bool has = false;  // whether the wave's rows have seen a key (trees)
  while (cur < tile_end) {
    const uint32_t tb = tile_lds + (it & 1) * Tile::kBytes;
    int v_two = wk.list_entry(nxt + 2);
    const float sc_nxt = key_scale(rows_nxt);
    copies.lane = anew(lane);
    const uint32_t next_lds = tile_lds + ((it + 1) & 1) * Tile::kBytes;  // (no next tile: zeros, unused)
    const uint64_t held = wave_ballot(rows_cur >= 0);
    const bool mine_to_do = in_pass(cur, who_cur);
    if constexpr (TREE) has |= mine_to_do;
    if (!LIST && !mine_to_do) copies.all(next_lds);

#pragma unroll 1
    for (int n0 = 0; n0 < (mine_to_do ? NS : 0); ++n0) {
      const int n = G == 2 ? half : n0;  // keys 32 n .. + 31 of the tile
      const uint32_t nb = tb + n * 32 * Tile::kRow;
      const uint32_t ka = nb + a_key, ra = tb + a_rot + n * 32 * Tile::kRopeRow, va = nb + a_val;
      // Operand reads run kAhead steps before their products, in one sequence
      // over the scores and the sums: first the key rows (two K steps a read with
      // codes), then the rotary rows, then the transposed values.
      constexpr int kKeyReads = (FP8 ? 16 : 32) + 4, kReads = kKeyReads + 32;
      u32x4 ring[kAhead];
      auto read = [&](int i) -> u32x4 {
        if (i < kKeyReads - 4)
          return FP8 ? lds_read<u32x4>(ka ^ (32 * i)) : lds_read<u32x4>((ka ^ (32 * (i & 15))) + 512 * (i >> 4));
        if (i < kKeyReads) return lds_read<u32x4>(ra ^ (32 * (i - (kKeyReads - 4))));
        const int j = (i - kKeyReads) >> 4, d = (i - kKeyReads) & 15;
        if constexpr (FP8) {
          const u32x2 v = lds_read_tr8((va ^ (32 * d) ^ (256 * j)) + 16 * j * Tile::kRow);
          return u32x4{v.x, v.y, 0u, 0u};
        }
        const uint32_t at = va ^ (64 * (d & 7)) ^ (256 * j);
        const int off = 512 * (d >> 3) + 16 * j * Tile::kRow;
        return __builtin_bit_cast(u32x4, join_rows(lds_read_tr16(at + off), lds_read_tr16((at ^ 32) + off + 8 * Tile::kRow)));
      };
      // this step's share of the next tile's copies, evenly over the kReads products
      constexpr int kMine = TileCopy<Tile, FP8>::kCopies / NS;
      auto spread = [&](int i) {
        if ((i + 1) * kMine / kReads != i * kMine / kReads) {
          copies.next(next_lds, i * kMine / kReads);
        }
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ring[i] = read(i);
      __builtin_amdgcn_sched_barrier(0);
      f32x16 s;
      f32x4 sc4[4];
#pragma unroll
      for (int i = 0; i < kKeyReads; ++i) {
        const u32x4 v = ring[i % kAhead];
        if (FP8 && i < 16) {
          const bf16x8 a0 = codes_to_bf16(u32x2{v.x, v.y}), a1 = codes_to_bf16(u32x2{v.z, v.w});
          if (i == 0)
            mfma_vgpr_first(s, a0, qf[0]);
          else
            mfma_vgpr(s, a0, qf[2 * i]);
          mfma_vgpr(s, a1, qf[2 * i + 1]);
        } else if (i == 0) {
          mfma_vgpr_first(s, __builtin_bit_cast(bf16x8, v), qf[0]);
        } else {
          mfma_vgpr(s, __builtin_bit_cast(bf16x8, v), qf[36 - kKeyReads + i]);
        }
        ring[i % kAhead] = read(i + kAhead);
        spread(i);
        if (FP8 && i == 15) {  // a key's scale multiplies its latent part only
          mfma_done(s);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sc4[k] = *reinterpret_cast<const f32x4*>(&ksc[it & 1][32 * n + 8 * k + 4 * h2]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[4 * k + e] *= sc4[k][e];
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      mfma_done(s);

      // ---- weights of keys 32 n + 8 (e / 4) + 4 h2 + e % 4
      auto operand = [&](u32x4 v) -> bf16x8 {
        if constexpr (FP8) return codes_to_bf16(u32x2{v.x, v.y});
        return __builtin_bit_cast(bf16x8, v);
      };
      const uint32_t mine = (uint32_t)(held >> (32 * n));
      if (mine != 0xffffffffu) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = (mine >> (8 * (e >> 2) + 4 * h2 + (e & 3))) & 1u ? s[e] : -INFINITY;
      }
      float top = s[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = max_or_nan(top, s[e]);
      top = max_halves(top) * sm;
      if (__builtin_expect(__any(top > m + kSlack), 0)) {
        const float mm = top > m + kSlack ? top : m, f = exp2_fast(m - mm);
        const bool begun = __any(l != 0.f);  // (before a key weighs anything the sums are zero)
        m = mm;
        l *= f;
        if (begun) {
#pragma unroll
          for (int d = 0; d < 16; ++d) {
            in_agprs(o[d]);
            o[d] *= f;
            in_agprs(o[d]);
          }
        }
      }
      bf16x8 pb[2];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float x = exp2_fast(fmaf(s[e], sm, -m));
        l += x;  // the total keeps 32 bits; the weights are rounded to bf16 for the matrix cores
        if constexpr (FP8) x *= sc4[e >> 2][e & 3];
        pb[e >> 3][e & 7] = (__bf16)x;
      }
      // ---- sums of values 32 d + (result row) for row c
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const bf16x8 v = operand(ring[(kKeyReads + i) % kAhead]);
        o[i & 15] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, pb[i >> 4], o[i & 15], 0, 0, 0);
        if (i + kAhead < 32) ring[(kKeyReads + i) % kAhead] = read(kKeyReads + i + kAhead);
        spread(kKeyReads + i);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    int rows_nn, who_nn;
    const int nn = next_pass(after(nxt, who_nxt), who_nxt, v_nn, who_nn, rows_nn);
    copies.aim(rows_nn);
    wait_copies();
    v_nn = wk.list_after(nxt, nn, v_two);
    if (FP8 && w == 0) ksc[(it + 1) & 1][lane] = rows_nxt >= 0 ? sc_nxt : 0.f;  // (no key: zeros, scaled by none)
    lds_barrier();
    cur = nxt;
    rows_cur = rows_nxt;
    who_cur = who_nxt;
    nxt = nn;
    rows_nxt = rows_nn;
    who_nxt = who_nn;
    ++it;
  }

  // ---- result: lane holds values 32 d + 8 i + 4 h2 + 0..3 of its row
  float tot = sum_halves(l);
  if constexpr (G == 2) {
    // the two waves of a row group, through LDS: each takes the other's sums of its
    // own half of the values, so that both add and both write
    constexpr int kPass = FP8 ? 4 : 8;  // accumulator tiles (4 KB a wave) at a time
    constexpr int kSums = 4 * kPass * 4096;
    static_assert(kSums + 1024 <= 2 * Tile::kBytes, "exchange space");
    f32x4* ex = reinterpret_cast<f32x4*>(&tile[0][0]) + w * kPass * 256 + lane;
    const f32x4* from = reinterpret_cast<const f32x4*>(&tile[0][0]) + (w ^ 2) * kPass * 256 + lane;
    float* ml = reinterpret_cast<float*>(&tile[0][0] + kSums);
    if (h2 == 0) ml[64 * half + 32 * grp + c] = m, ml[128 + 64 * half + 32 * grp + c] = tot;
    float f_own, f_other;
#pragma unroll
    for (int d0 = 0; d0 < 8; d0 += kPass) {
#pragma unroll
      for (int d = 0; d < kPass; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 x;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = half ? o[d0 + d][4 * i + e] : o[8 + d0 + d][4 * i + e];
          ex[(d * 4 + i) * 64] = x;
        }
      __syncthreads();
      if (d0 == 0) {
        const float m0 = ml[32 * grp + c], m1 = ml[64 + 32 * grp + c], mm = fmaxf(m0, m1);
        const float f0 = exp2_fast(m0 - mm), f1 = exp2_fast(m1 - mm);
        m = mm;
        tot = ml[128 + 32 * grp + c] * f0 + ml[192 + 32 * grp + c] * f1;
        f_own = half ? f1 : f0, f_other = half ? f0 : f1;
      }
#pragma unroll
      for (int d = 0; d < kPass; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 x = from[(d * 4 + i) * 64];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float own = half ? o[8 + d0 + d][4 * i + e] : o[d0 + d][4 * i + e];
            o[d0 + d][4 * i + e] = own * f_own + x[e] * f_other;  // (o[0..7]: the wave's half from here on)
          }
        }
      __syncthreads();
    }
  }
  if constexpr (TREE) tot = row_total(has, tot);
  else tot = row_total(LIST ? it > 0 : un.lim > 0, tot);
  // through LDS (the wave's own part of the tiles), so that rows leave in whole
  // lines: 16-byte chunks in an order that depends on the row, `seg` bytes of each row at a time
  constexpr int kRoom = FP8 ? 512 : 1024;  // bytes a row
  static_assert(4 * 32 * kRoom <= 2 * Tile::kBytes, "room for every wave's rows");
  const uint32_t mine = tile_lds + w * 32 * kRoom;
  const int rows_here = un.rows;
  const int64_t R = un.row;
  auto put = [&](unsigned char* dst, int64_t stride, auto seg) {  // what is in LDS to rows `stride` apart
    constexpr int kSeg = decltype(seg)::value, kChunks = kSeg / 16, kRows = 64 / kChunks;  // rows a store
#pragma unroll 8
    for (int i = 0; i < rows_here; i += kRows) {
      const int rr = i + lane / kChunks;
      const u32x4 v = lds_read<u32x4>(mine + rr * kSeg + (((lane % kChunks) ^ (rr & 31)) * 16));
      if (rr < rows_here) *reinterpret_cast<u32x4*>(dst + rr * stride + (lane % kChunks) * 16) = v;
    }
  };
  constexpr int kN = G == 2 ? 8 : 16;  // accumulator tiles of the wave: values 32 (8 half) .. of its rows
  const int col = G == 2 ? 8 * half : 0;
  {
    if (wk.in_parts()) {
      constexpr int kSeg = std::min(kRoom, kN * 128), kD = kSeg / 128;  // accumulator tiles a pass (32 values, 128 bytes a row)
      unsigned char* dst = reinterpret_cast<unsigned char*>(p.part + wk.part_row(un, nrows) * kLatent);
#pragma unroll
      for (int d0 = 0; d0 < kN; d0 += kD) {
#pragma unroll
        for (int d = 0; d < kD; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(mine + c * kSeg + (((8 * d + 2 * i + h2) ^ c) * 16)) =
                f32x4{o[d0 + d][4 * i], o[d0 + d][4 * i + 1], o[d0 + d][4 * i + 2], o[d0 + d][4 * i + 3]};
        put(dst + (col + d0) * 128, kLatent * 4, std::integral_constant<int, kSeg>{});
      }
    } else {
      constexpr int kSeg = std::min(kRoom, kN * 64), kD = kSeg / 64;
      const float inv = row_inverse(tot);
      unsigned char* dst = reinterpret_cast<unsigned char*>(p.out + R * kLatent);
#pragma unroll
      for (int d0 = 0; d0 < kN; d0 += kD) {
#pragma unroll
        for (int d = 0; d < kD; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x16& x = o[d0 + d];
            const f32x4 v = {x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv};
            *(__attribute__((address_space(3))) bf16x4*)(uintptr_t)(mine + c * kSeg + (((4 * d + i) ^ c) * 16) + h2 * 8) =
                __builtin_convertvector(v, bf16x4);
          }
        put(dst + (col + d0) * 64, kLatent * 2, std::integral_constant<int, kSeg>{});
      }
    }
  }
  const bool first = half == 0 && h2 == 0 && c < rows_here;
  if (wk.in_parts() && first) {
    p.part_ml[(wk.part_row(un, nrows) + c) * 2] = m;
    p.part_ml[(wk.part_row(un, nrows) + c) * 2 + 1] = tot;
  }
  if (!wk.in_parts() && p.lse && first) p.lse[R + c] = row_log_sum(m, tot);
}

}  // namespace misa
