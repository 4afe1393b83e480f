// Latent attention of drafted tokens over a paged cache: the queries of a sequence
// are the N nodes of a tree, and node i sees the committed keys of its sequence
// (all of them, or a list) and the nodes that its mask names:
//
//   S[i,h,j] = sm * (q[i,h, 0:512] . c[j] + q[i,h, 512:576] . rope[j]),  j in keys(i)
//   out[i,h] = sum_j softmax_j(S[i,h,:]) c[j]
//
// The matrix work is that of the latent kernels (latent_device.h); here is where
// the keys of a workgroup's rows lie, and how sequences of different lengths are
// shared out.
#include <algorithm>

#include "latent_pair.h"

namespace misa {

// The largest batch whose keys are split: one lane of a wave holds kPlanSeqs / 64 sequences.
// Past it a sequence's row tiles are whole: one token of 16 heads over 8000 coded keys each
// takes 323 us with 256 sequences and 607 with 257 (of 200 to 2000 keys beside one of 8000:
// 103 and 275), 128 sequences 183.
constexpr int kPlanSeqs = 256;

// The walk of a workgroup: a row tile of one sequence (units of U heads of one node)
// and a share of its key tiles. Tiles below np hold 64 committed positions each,
// which all nodes see; tile np + w holds the positions of word w of the masks.
//
// Which share: all workgroups work the same cut out from the sequences' lengths,
// which lie on the device. With c tiles a split, a sequence of n tiles takes
// max(1, ceil(n / c)) of them, and c is the smallest (to within a 32nd of its range)
// whose splits fit the budget. Two budgets are held against each other, one of which
// fills the card once more: it pays where lengths differ, since the longest sequence
// is cut and not the others, and costs twice the partial sums to join (24 sequences of up
// to 8000 keys, 4 tokens x 128 heads, codes: splits of 37 tiles 198 us, of 16 206).
template <int NQ, int U>
struct TreeWork {
  const TreeArgs& p;
  int lane;
  int s, r;                // sequence, row tile of it
  int prefix, np;          // committed keys, their tiles
  bool padded;             // no sequence: no query of it has a key
  int slot, splits;        // the split's place among all sequences' splits; splits of this sequence
  int cur, tile_end;
  bool valid;
  uint32_t alive;          // bit i: unit i is not padding
  static constexpr int kUnits = NQ / U;

  struct Unit {
    int64_t row;           // first row (query * H + head)
    int rows, node, i;     // rows (0: none), node, unit of the row tile
    bool live;             // not padding
  };
  __device__ __forceinline__ Unit unit(int i) const { return unit_of(i, r); }
  __device__ __forceinline__ Unit unit_of(int i, int tile) const {
    const int hc = (p.H + U - 1) / U;
    const int g = tile * kUnits + i, node = g / hc, c = g % hc;
    Unit u{0, 0, 0, i, false};
    if (node >= p.N) return u;
    u.row = ((int64_t)s * p.N + node) * p.H + c * U;
    u.rows = min(U, p.H - c * U);
    u.node = node;
    u.live = alive >> i & 1;
    return u;
  }
  // Word w of the node's mask, the same for all lanes. It has landed where this ends: where
  // paths with and without a load meet, the compiler would wait for copies in flight.
  __device__ __forceinline__ uint64_t mask_word(int node, int w) const {
    uint64_t x = p.mask[((int64_t)s * p.N + node) * p.words + w];
    asm volatile("" : "+v"(x));
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(x >> 32)) << 32 |
           (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)x);
  }
  // which positions of tile ti (at or past np) the node sees
  __device__ __forceinline__ uint64_t bits(int node, int ti) const {
    const int w = ti - np;
    if (p.mask) return mask_word(node, w);
    const int n = node + 1 - 64 * w;
    return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
  }

  static __device__ __forceinline__ int committed(const TreeArgs& p, int s) {
    return min(p.prefix[s], p.pages.per << p.pages.page_log2);
  }
  static __device__ __forceinline__ int tiles(const TreeArgs& p, int prefix) {
    return prefix < 0 ? 0 : (prefix + kAttnTile - 1) / kAttnTile + p.words;
  }
  // ceil(n / c), n < 2^25
  static __device__ __forceinline__ int shares(int n, int c, float inv) {
    int q = (int)((float)n * inv);
    q -= q * c > n;
    q += (q + 1) * c <= n;
    return q + (q * c < n);
  }
  struct Cut {
    int c, slots;
  };
  // (lane l holds the tiles of sequences l, l + 64, ...; -1: no sequence)
  static __device__ __forceinline__ int slots_of(const int (&n)[kPlanSeqs / 64], int seqs, int c) {
    const float inv = 1.f / (float)c;
    int m = 0;
#pragma unroll
    for (int i = 0; i < kPlanSeqs / 64; ++i)
      if (64 * i < seqs) m += n[i] < 0 ? 0 : max(1, shares(n[i], c, inv));
    return (int)wave_total_u32((uint32_t)m);
  }
  static __device__ __forceinline__ Cut cut(const int (&n)[kPlanSeqs / 64], int total, int most, int seqs, int budget, int least) {
    int lo = max(least, (total + budget - 1) / budget);
    int hi = budget > seqs ? min(most, (total + budget - seqs - 1) / (budget - seqs)) : most;
    int at = slots_of(n, seqs, lo);
    if (at <= budget) return {lo, at};
    // lo's splits do not fit, hi's do: sum of ceil(n / c) < total / c + seqs
    at = slots_of(n, seqs, hi);
#pragma unroll 1
    for (int i = 0; i < 5 && hi - lo > 1; ++i) {
      const int mid = (lo + hi) / 2, k = slots_of(n, seqs, mid);
      if (k <= budget) hi = mid, at = k;
      else lo = mid;
    }
    return {hi, at};
  }

  __device__ __forceinline__ TreeWork(const TreeArgs& a, int lane_) : p(a), lane(lane_) {
    // neighbouring workgroups run on different XCDs; give each XCD a run of
    // neighbouring slots, with the row tiles that read the same keys together
    const int R = p.tiles_a_seq, seqs = p.pages.seqs;
    const bool whole = p.budget[1] <= seqs;  // no sequence is split
    int n[kPlanSeqs / 64], lens[kPlanSeqs / 64];
    int total = 0, slots = seqs, c = 0;
    if (!whole) {
      int most = 1;
#pragma unroll
      for (int i = 0; i < kPlanSeqs / 64; ++i) {
        const int j = lane + 64 * i;
        n[i] = -1;
        if (64 * i >= seqs) continue;
        lens[i] = committed(p, min(j, seqs - 1));
        if (j < seqs) n[i] = tiles(p, lens[i]);
        total += max(n[i], 0);
        most = max(most, n[i]);
      }
      total = (int)wave_total_u32((uint32_t)total);
      most = (int)wave_max_u32((uint32_t)most);
      Cut best = cut(n, total, most, seqs, p.budget[0], p.least);
      if (p.budget[1] > p.budget[0]) {
        const Cut more = cut(n, total, most, seqs, p.budget[1], p.least);
        auto cost = [&](const Cut& x) {
          return (float)((x.slots * R + 255) / 256) * (p.fixed + (float)x.c * p.tile) + (float)x.slots * p.join;
        };
        if (cost(more) < cost(best)) best = more;
      }
      c = __builtin_amdgcn_readfirstlane(best.c);
      slots = __builtin_amdgcn_readfirstlane(best.slots);
    }
    const int64_t used = (int64_t)slots * R;
    const int each = (int)((used + 7) / 8);
    const int64_t lid = (int64_t)(blockIdx.x & 7) * each + (blockIdx.x >> 3);
    valid = (int)(blockIdx.x >> 3) < each && lid < used;
    if (!valid) return;
    slot = (int)(lid / R);
    r = (int)(lid % R);
    int split = 0;
    s = slot;
    splits = 1;
    int len = 0;
    if (!whole) {
      const float inv = 1.f / (float)c;
      int before = 0;
#pragma unroll
      for (int i = 0; i < kPlanSeqs / 64; ++i) {
        if (64 * i >= seqs) break;
        const int m = n[i] < 0 ? 0 : max(1, shares(n[i], c, inv));
        const int end = before + wave_inclusive_scan(m);
        const uint64_t here = wave_ballot(slot >= end - m && slot < end);
        if (here) {
          const int l = __builtin_ctzll(here);
          s = 64 * i + l;
          splits = __builtin_amdgcn_readlane(m, l);
          len = __builtin_amdgcn_readlane(lens[i], l);
          split = slot - (__builtin_amdgcn_readlane(end, l) - splits);
        }
        before = __builtin_amdgcn_readlane(end, 63);
      }
      if (split == 0 && r == 0 && threadIdx.x == 0) {
        p.rec[2 * s] = slot;
        p.rec[2 * s + 1] = splits;
      }
    }
    // (the same for all lanes, which the compiler does not see through a scan)
    s = __builtin_amdgcn_readfirstlane(s);
    splits = __builtin_amdgcn_readfirstlane(splits);
    split = __builtin_amdgcn_readfirstlane(split);
    len = __builtin_amdgcn_readfirstlane(whole ? committed(p, s) : len);
    padded = len < 0;
    prefix = max(len, 0);
    np = (prefix + kAttnTile - 1) / kAttnTile;
    const int t = tiles(p, len), share = (t + splits - 1) / splits;
    cur = split * share;
    tile_end = min(t, cur + share);
    // (a lane a unit, so that the masks are waited for once)
    const int hc = (p.H + U - 1) / U, node = (r * kUnits + lane) / hc;
    bool live = lane < kUnits && node < p.N && !padded;
    if (p.mask && live) {
      uint64_t any = 0;
      for (int w = 0; w < p.words; ++w) any |= p.mask[((int64_t)s * p.N + node) * p.words + w];
      live = any != 0;
    }
    alive = (uint32_t)wave_ballot(live);
    if (!alive) tile_end = cur;
  }

  // position of key 64 * ti + lane
  __device__ __forceinline__ int position(int ti) const {
    return (ti < np ? ti * kAttnTile : prefix + (ti - np) * kAttnTile) + lane;
  }
  // its page, or one past the table's end for it (row_at knows). A load without a
  // branch: it is asked for a tile ahead, and a branch around it would wait for
  // what is in flight.
  __device__ __forceinline__ const int32_t* entry_at(int ti) const {
    return p.pages.table + (int64_t)s * p.pages.per + min(position(ti) >> p.pages.page_log2, p.pages.per - 1);
  }
  __device__ __forceinline__ int list_entry(int ti) const { return *entry_at(ti); }
  __device__ __forceinline__ int list_after(int ti, int next, int v) const {
    asm volatile("" : "+v"(v));
    if (next != ti + 1) {
      v = list_entry(next + 1);
      asm volatile("" : "+v"(v));
    }
    return v;
  }
  // the cache row of key 64 * ti + lane in page v, or -1; a committed one, or a position of a mask's word
  __device__ __forceinline__ int row_at(int ti, int v) const {
    return (position(ti) >> p.pages.page_log2) < p.pages.per ? row_in(ti, v, position(ti)) : -1;
  }
  // the same for a tile below np, whose positions the table has
  __device__ __forceinline__ int plain_row(int ti, int v) const { return row_in(ti, v, ti * kAttnTile + lane); }
  __device__ __forceinline__ int row_in(int ti, int v, int j) const {
    const int lg = p.pages.page_log2, pages = (p.rows + (1 << lg) - 1) >> lg;
    const int row = (int)((uint32_t)v << lg) + (j & ((1 << lg) - 1));  // (below 2^31 if v is a page)
    return (ti >= np || j < prefix) && (uint32_t)v < (uint32_t)pages && row < p.rows ? row : -1;
  }
  // the same, if any unit sees it
  __device__ __forceinline__ int row_of(int ti, int v) const {
    const int row = row_at(ti, v);
    if (ti < np) return row;
    uint64_t any = 0;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const Unit u = unit(i);
      any |= u.live ? bits(u.node, ti) : 0ull;
    }
    return (any >> lane) & 1 ? row : -1;
  }
  __device__ __forceinline__ int find_tile(int ti, int v, int& rows) const {
    rows = -1;
    while (ti < tile_end) {
      rows = row_of(ti, v);
      if (wave_ballot(rows >= 0) != 0) break;
      v = list_entry(++ti);
    }
    return ti;
  }
  __device__ __forceinline__ bool common(int ti) const { return ti < np; }
  __device__ __forceinline__ uint64_t sees(int ti, const Unit& u, uint64_t held) const {
    return ti < np ? held : u.live ? held & bits(u.node, ti) : 0ull;
  }

  // The wide kernel's walk: a tile of a word is taken once for all units if they
  // see the same of it, otherwise once for each kind (who: the unit it is of).
  __device__ __forceinline__ int next_pass(int ti, int who, int v, int& who_next, int& rows) const {
    // (what follows of the units is rare; it is formed here, not kept from before the loop)
    const int tile = __builtin_amdgcn_readfirstlane(anew(r));
    bool asked = who < 0;  // v is tile ti's
    ++who;
    for (; ti < tile_end; ++ti, who = 0) {
      if (!asked) {
        v = list_entry(ti);
        asm volatile("" : "+v"(v));  // (waited for here, not where the paths meet)
      }
      asked = false;
      const int row = row_at(ti, v);
      if (ti < np) {
        rows = row;
        who_next = -1;
        if (wave_ballot(rows >= 0) != 0) return ti;
        continue;
      }
      uint64_t b[kUnits];
      bool live[kUnits], alike = true;
      int first = -1;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const Unit u = unit_of(i, tile);
        live[i] = u.live;
        b[i] = u.live ? bits(u.node, ti) : 0ull;
        if (u.live && first < 0) first = i;
#pragma unroll
        for (int x = 0; x < i; ++x) alike = alike && (!live[i] || !live[x] || b[x] == b[i]);
      }
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        bool take = i >= who && (alike ? i == first : live[i]);
        if (!alike) {
#pragma unroll
          for (int x = 0; x < i; ++x) take = take && !(live[x] && b[x] == b[i]);
        }
        if (take) {
          rows = (b[i] >> lane) & 1 ? row : -1;
          if (wave_ballot(rows >= 0) != 0) {
            who_next = alike ? -1 : i;
            return ti;
          }
        }
      }
    }
    who_next = -1;
    rows = -1;
    return ti;
  }
  __device__ __forceinline__ bool in_pass(int ti, int who, const Unit& u) const {
    return u.live && (who < 0 || bits(u.node, ti) == bits(unit(who).node, ti));
  }

  // partial sums: the rows of a row tile side by side, a slot's row tiles one after the other
  __device__ __forceinline__ int64_t part_row(const Unit& u, int64_t) const {
    return ((int64_t)slot * p.tiles_a_seq + r) * NQ + u.i * U;
  }
  __device__ __forceinline__ bool in_parts() const { return splits > 1; }
};

struct TreeForm {
  using Args = TreeArgs;
  static constexpr bool kList = false, kTree = true;
  template <int NQ, int U>
  using Work = TreeWork<NQ, U>;
};

// Joins the splits of the sequences that were split (rec says which, and where). As
// k_join: a workgroup's threads hold COLS of a row's values, SG groups take the
// splits in turn and are added in a fixed order. Bound by memory where there is much (67 MB
// in 20.5 us), by latency where there is little (16 rows of 64 splits: 5). Asking for the
// first sums before their weights are known gained 0.9 of the 20 and cost as much of the 5.
template <int COLS, int SG>
__global__ __launch_bounds__(256) void k_tree_join(TreeArgs p, int nq, int unit_rows) {
  constexpr int TPR = COLS / 4, ROWS = 256 / TPR / SG, PARTS = kLatent / COLS;
  __shared__ __attribute__((aligned(16))) float sums[ROWS][SG][COLS];
  __shared__ float tots[ROWS][SG];
  const int c = threadIdx.x % TPR, sg = threadIdx.x / TPR % SG, rr = threadIdx.x / TPR / SG;
  const int64_t rows = (int64_t)p.T * p.H;
  const int64_t row = (int64_t)(blockIdx.x / PARTS) * ROWS + rr, rw = min(row, rows - 1);
  const int col = (int)(blockIdx.x % PARTS) * COLS + c * 4;
  const int q = (int)(rw / p.H), h = (int)(rw % p.H), s = q / p.N;
  const int hc = (p.H + unit_rows - 1) / unit_rows, units = nq / unit_rows;
  const int g = (q % p.N) * hc + h / unit_rows;
  const int first = p.rec[2 * s], splits = p.rec[2 * s + 1];
  const int64_t step = (int64_t)p.tiles_a_seq * nq;  // from one split's row to the next one's
  const int64_t at = ((int64_t)first * p.tiles_a_seq + g / units) * nq + (g % units) * unit_rows + h % unit_rows;
  const int mine = splits > 1 ? splits : 0;  // (whole sequences are done)
  float top = -INFINITY;
  for (int i = threadIdx.x & 31; i < mine; i += 32) {
    const f32x2 ml = *reinterpret_cast<const f32x2*>(p.part_ml + (at + i * step) * 2);
    top = fmaxf(top, no_keys(ml.y) ? -INFINITY : ml.x);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));  // (32 lanes share a row)
  const bool keys = top > -INFINITY;
  top = fmaxf(top, kNoMax);
  float tot = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int i = sg; i < mine; i += SG) {
    const int64_t x = at + i * step;
    const float f = exp2_fast(p.part_ml[x * 2] - top);
    tot += f * p.part_ml[x * 2 + 1];
    acc += *reinterpret_cast<const f32x4*>(p.part + x * kLatent + col) * f;
  }
  if constexpr (SG > 1) {
    *reinterpret_cast<f32x4*>(&sums[rr][sg][c * 4]) = acc;
    if (c == 0) tots[rr][sg] = tot;
    __syncthreads();
    if (sg != 0) return;
#pragma unroll
    for (int i = 1; i < SG; ++i) {
      acc += *reinterpret_cast<const f32x4*>(&sums[rr][i][c * 4]);
      tot += tots[rr][i];
    }
  }
  if (row >= rows || !mine) return;
  tot = row_total(keys, tot);
  const float inv = row_inverse(tot);
  *reinterpret_cast<bf16x4*>(p.out + rw * kLatent + col) = __builtin_convertvector(acc * inv, bf16x4);
  if (p.lse && col == 0) p.lse[rw] = row_log_sum(top, tot);
}

// The rows of the keys of each query: its list's positions (those that are
// committed), then the nodes of its mask one after the other, then -1. A workgroup
// takes 1024 entries of one query's list; the one of its end takes the nodes. A chain of
// dependent loads (position, page) that 1024 entries a workgroup cover: 56 queries of 2048, 4.4
// us, 1.7 of them the launch. (A list of rows lets k_latent_wide walk it as any other: its
// 40 us would not be shorter for resolving pages itself.)
constexpr int kListPart = 1024;
__global__ __launch_bounds__(256) void k_tree_lists(TreeArgs p, int32_t* lists) {
  const int parts = (p.k + kListPart - 1) / kListPart + 1;
  const int t = blockIdx.x / parts, part = blockIdx.x % parts;
  const int s = t / p.N, node = t % p.N, lane = threadIdx.x & 63;
  const int lg = p.pages.page_log2, len = p.k + 64 * p.words;
  const int prefix = min(p.prefix[s], p.pages.per << lg);
  const uint64_t* mask = p.mask ? p.mask + (int64_t)t * p.words : nullptr;
  auto bits = [&](int w) -> uint64_t {
    if (prefix < 0) return 0ull;
    if (mask) return mask[w];
    const int n = node + 1 - 64 * w;
    return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
  };
  auto row_of = [&](int j) -> int {
    if (j < 0 || (j >> lg) >= p.pages.per) return -1;
    const int v = p.pages.table[(int64_t)s * p.pages.per + (j >> lg)];
    const int64_t row = ((int64_t)v << lg) + (j & ((1 << lg) - 1));
    return v >= 0 && row < p.rows ? (int)row : -1;
  };
  int32_t* out = lists + (int64_t)t * len;
  if (part < parts - 1) {
    bool live = false;
    for (int w = 0; w < p.words; ++w) live |= bits(w) != 0;
#pragma unroll
    for (int i = 0; i < kListPart / 256; ++i) {
      const int e = part * kListPart + i * 256 + (int)threadIdx.x;
      if (e >= p.k) break;
      const int j = p.idx[(int64_t)t * p.k + e];
      out[e] = live && j < prefix ? row_of(j) : -1;
    }
    return;
  }
  if (threadIdx.x >= 64) return;
  int at = p.k;
  for (int w = 0; w < p.words; ++w) {
    const uint64_t b = bits(w);
    if ((b >> lane) & 1) out[at + lanes_below(b)] = row_of(prefix + 64 * w + lane);
    at += __popcll(b);
  }
  for (int e = at + lane; e < len; e += 64) out[e] = -1;
}

hipError_t launch_tree_lists(const LaunchCtx& cx, const TreeArgs& a, int32_t* lists) {
  const int64_t parts = (a.k + kListPart - 1) / kListPart + 1;
  return cx.launch("k_tree_lists", k_tree_lists, dim3((unsigned)(a.T * parts)), dim3(256), 0, a, lists);
}

static int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Rows per workgroup and the budget of splits: the cheapest of four widths, by the
// costs of the latent kernels (see latent_plan; 128 rows: of k_latent_pair), for sequences
// that are all as long as the longest. 128 rows of few heads are of several nodes, and the pair
// kernel takes a word's keys anew for each kind of mask, which it finds by loads one after the
// other: 7 us each (29 sequences x 41 nodes x 16 heads, 24 keys: 102 us, 51 with 32 rows;
// 20 x 16 x 3 heads, 700 keys: 59, 41 with 64). That is charged to every workgroup, though with
// split keys only the last splits of a sequence meet words: such calls may be given a narrower
// width than the fastest. How many splits a sequence gets of the budget
// is found on the device, from the lengths.
TreePlan tree_plan(int seqs, int N, int H, int words, int longest) {
  struct Width {
    int rows, unit;
    double fixed, tile, kind;
  };
  static const Width widths[] = {{16, 16, 9.0, 1.8, 0.0}, {32, 16, 11.0, 2.2, 0.0}, {64, 32, 13.0, 2.25, 0.0}, {128, 32, 12.0, 3.5, 7.0}};
  const int tiles = cdiv(longest, kAttnTile) + words;
  TreePlan best{};
  double least = 0.0;
  for (const Width& w : widths) {
    TreePlan pl{};
    pl.nq = w.rows;
    pl.tiles_a_seq = cdiv((int64_t)N * cdiv(H, w.unit), w.rows / w.unit);
    const int nodes = std::min(N, std::max(1, w.rows / w.unit / cdiv(H, w.unit)));  // of a row tile
    const double fixed = w.fixed + (double)(nodes - 1) * words * w.kind;
    pl.fixed = (float)fixed;
    pl.tile = (float)w.tile;
    const int64_t row_tiles = (int64_t)seqs * pl.tiles_a_seq;
    const int most = seqs > kPlanSeqs ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(256 / row_tiles, tiles));
    for (int want = 1;; want = std::min(2 * want, most)) {
      const int share = cdiv(tiles, want), splits = cdiv(tiles, share);
      const double rounds = (double)((row_tiles * splits + 255) / 256);
      double cost = rounds * (fixed + share * w.tile);
      if (splits > 1) cost += 3.5 + 0.05 * splits + (double)splits * seqs * N * H * (kLatent * 4) / 2.3e6;
      if (best.nq == 0 || cost < least) {
        least = cost;
        best = pl;
        best.least = std::max(1, std::min(share, w.rows / 16));
        best.budget[0] = splits == most && splits > 1 ? std::max(seqs * splits, 256 / pl.tiles_a_seq) : seqs * splits;
      }
      if (want == most) break;
    }
  }
  best.budget[1] = best.budget[0];
  const int64_t row_tiles = (int64_t)seqs * best.tiles_a_seq;
  if (seqs > 1 && seqs <= kPlanSeqs && row_tiles > 64 && row_tiles <= 512 && tiles >= 16)
    best.budget[1] = std::max<int64_t>(best.budget[0], 512 * ((row_tiles + 255) / 256) / best.tiles_a_seq);
  return best;
}

size_t tree_ws_bytes(const TreePlan& pl, int seqs) {
  if (pl.budget[1] <= seqs) return 256;
  const size_t rows = (size_t)pl.budget[1] * pl.tiles_a_seq * pl.nq;
  return 256 + ((size_t)seqs * 8 + 255) / 256 * 256 + rows * (kLatent + 2) * 4;
}

template <bool FP8>
static hipError_t launch_tree_t(const LaunchCtx& cx, const TreeArgs& a, int nq, dim3 grid) {
  switch (nq) {
    case 16: return cx.launch("k_tree_16", k_latent<16, FP8, TreeForm>, grid, dim3(256), 0, a);
    case 32: return cx.launch("k_tree_32", k_latent<32, FP8, TreeForm>, grid, dim3(256), 0, a);
    case 64: return cx.launch("k_tree_64", k_latent_wide<2, FP8, TreeForm>, grid, dim3(256), 0, a);
    default: return cx.launch("k_tree_128", k_latent_pair<FP8, TreeForm>, grid, dim3(256), 0, a);
  }
}

hipError_t launch_tree(const LaunchCtx& cx, TreeArgs a, const TreePlan& pl, bool fp8, void* ws) {
  const int seqs = a.pages.seqs;
  a.tiles_a_seq = pl.tiles_a_seq;
  a.budget[0] = pl.budget[0];
  a.budget[1] = pl.budget[1];
  a.least = pl.least;
  a.fixed = pl.fixed;
  a.tile = pl.tile;
  a.join = (float)(pl.tiles_a_seq * pl.nq * (kLatent * 4 / 4.8e6));  // (read once more, at the rate of a copy)
  const bool split = pl.budget[1] > seqs;
  if (split) {
    a.rec = static_cast<int32_t*>(ws);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + ((size_t)seqs * 8 + 255) / 256 * 256);
    a.part_ml = a.part + (int64_t)pl.budget[1] * pl.tiles_a_seq * pl.nq * kLatent;
  }
  const int64_t n = (int64_t)std::max(pl.budget[1], seqs) * pl.tiles_a_seq;
  const dim3 grid((unsigned)((n + 7) / 8 * 8));
  const hipError_t e = fp8 ? launch_tree_t<true>(cx, a, pl.nq, grid) : launch_tree_t<false>(cx, a, pl.nq, grid);
  if (e != hipSuccess || !split) return e;
  const int64_t rows = (int64_t)a.T * a.H;
  const int unit = pl.nq <= 32 ? 16 : 32;
  if (pl.budget[1] > 8 * seqs || rows < 1024)
    return cx.launch("k_tree_join", k_tree_join<128, 8>, dim3((unsigned)(rows * 4)), dim3(256), 0, a, pl.nq, unit);
  return cx.launch("k_tree_join", k_tree_join<kLatent, 1>, dim3((unsigned)((rows + 1) / 2)), dim3(256), 0, a, pl.nq, unit);
}

}  // namespace misa
