// Latent attention of 128 rows a workgroup where many rows share their keys: the
// kernel that long contexts of drafted tokens run on.
#pragma once

#include "latent_device.h"

namespace misa {

// Starts a copy of 4 bytes a lane from global memory to LDS at lds + 4 * lane (see copy16_to_lds).
__device__ __forceinline__ void copy4_to_lds(const void* src, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, off"
      :
      : "s"(lds), "v"(src)
      : "memory");
}
// copy16_to_lds of what lies OFFSET further than src, to LDS at at + LDS (the instruction
// adds its offset on both sides).
template <int OFFSET, int LDS>
__device__ __forceinline__ void copy_piece_to_lds(uint64_t src, uint32_t at) {
  asm volatile(
      "s_add_u32 m0, %0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off offset:%3"
      :
      : "s"(at), "v"(src), "n"(LDS - OFFSET), "n"(OFFSET)
      : "memory", "scc");
}
// f(0), f(1), .. f(N - 1), each with its number as a constant: what a long body would not
// be unrolled for.
template <class F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

// A product whose operands are no vector instruction's results of the two before it: what
// is read from LDS, and queries (a test reads the generated code for it).
__device__ __forceinline__ void mfma_loaded(f32x16& d, bf16x8 a, bf16x8 b) {
  asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(d) : "v"(a), "v"(b));
}

// LDS of the pair kernel: keys in steps of 32, and what waves hand each other. A copy brings
// 256 bytes of four rows, side by side. An operand read takes 16 bytes of 16 rows at a time, a
// transposing one 64 (codes: 32) bytes of four (eight) rows, and each should cover the 64
// banks: so the pieces of 64 (32) bytes are stored in an order that depends on the row
// (piece p of row r in place p ^ (r & 3)), and every four rows lie 16 bytes further than
// the ones before (codes: and every eight 128). Only two bits of a piece's number change, so
// that reads are offsets from four addresses. Rotary rows of 128 bytes, eight a copy: chunk c in
// place c ^ (r / 2 & 7).
template <bool FP8>
struct PairLds {
  static constexpr int kKeys = 32, kStages = 4;
  static constexpr int kParts = FP8 ? 2 : 4;              // of 256 bytes, of a row
  static constexpr int kPiece = FP8 ? 5 : 6;              // log2 of a piece's bytes
  static __device__ __forceinline__ constexpr int four_at(int g) {  // where rows 4 g .. + 3 begin
    return g * kParts * 1024 + (FP8 ? (g >> 1) * 128 + (g & 1) * 16 : g * 16);
  }
  static __device__ __forceinline__ int row_at(int r) { return four_at(r >> 2) + (r & 3) * 256; }
  static constexpr int kLat = kKeys / 4 * kParts * 1024 + (FP8 ? 512 : 128);
  static constexpr int kRotRow = 2 * kRotary, kRot = kKeys * kRotRow;
  static constexpr int kRotAt = kStages * kLat, kRotStages = 3;
  // what one step's waves hand each other lies beside what the next one's do
  static constexpr int kWeights = kRotAt + kRotStages * kRot;  // 2 KB a wave, two steps
  static constexpr int kFactors = kWeights + 2 * 8192;         // 32 numbers a wave, two steps
  static constexpr int kPages = kFactors + 2 * 512;            // 64 entries a wave
  static constexpr int kScales = kPages + 1024;                // 256 bytes a wave and stage, its eight numbers first
  static constexpr int kQueries = kScales + (FP8 ? kStages * 1024 : 0);  // codes: rotary queries, 4 KB a wave
  static constexpr int kBytes = kQueries + (FP8 ? 4 * 4096 : 0);
};

// o = sum_k 2^(sm s_k - m) v_k and l = sum_k 2^(sm s_k - m) for 128 rows, with the running
// maximum m lifted only when a score passes it by kSlack: the sums stay in 32 bits, and only
// the weights are rounded to bf16, as the matrix cores take them.
//
// Bound by the matrix cores' issue: 68 products of 32 cycles a wave and step of 32 keys (36 of
// scores, 32 of values), 2176 cycles, beside which one wave a SIMD has to issue all else.
// k_latent_wide, with 16 of the values' columns a wave and all waves' weights through LDS,
// stops at two barriers a step with nothing to issue. Here
//   - a wave scores its own 32 rows alone (queries in registers, keys as the other operand), so
//     that maximum, sum and weights are its own lanes' and need no one else;
//   - values cost a transposing read each, so waves go in pairs: each sums half of the values,
//     256 columns, of both waves' rows, which halves those reads, and the partner's weights and
//     rescaling come through LDS, 4 KB and one barrier a step;
//   - the next step's scores run beside this one's softmax, the copies three steps ahead
//     beside the values' products, the reads of LDS ahead of both.
// A second wave a SIMD to issue beside does not fit: 256 sums and 144 of queries a lane.
// 2 sequences x 64 tokens x 128 heads over 32,000 keys, bf16: 936 us in the median of the first
// thirty calls of a process, 1.22 PFLOP/s, and 893 under a longer load (a
// library's product of 8192^3 reaches 1.32, and the clock falls as the kernel gains: the
// last step took 9 % of its cycles and 2.4 % of its time); k_latent_wide 1060 under that load. A step of 32
// keys: 70 cycles until the scores, 1670 with them, 1670 of values. With codes 85, 2550 and
// 1860: the issue of 192 conversions bounds the scores. A workgroup's rest, some 45,000
// cycles: 10,000 to find its share, 9,000 for the queries, 9,000 until the first scores are
// there, 18,000 for its partial sums.
// Tried and left: two barriers a step (960 us), copies spread over scores and values (928
// beside 921), four stages of rotary rows (no room), values' operands shared by four waves
// (bound by LDS).
template <bool FP8, class Form>
__global__ __launch_bounds__(256, 1) void k_latent_pair(typename Form::Args p) {
  using Lds = PairLds<FP8>;
  constexpr int kStride = FP8 ? kLatent : 2 * (kLatent + kRotary);     // bytes of a cache row
  constexpr int kCopies = FP8 ? 6 : 9;                                 // of a wave and step
  constexpr int kKeyReads = FP8 ? 20 : 36, kAhead = FP8 ? 4 : 6, kAheadV = FP8 ? 4 : 3;
  // The waves meet where the weights are done, well before the values, so that the partner's
  // are there when the values begin. With codes no registers are left to hold them through
  // the scores (8 would spill in the loop; 186 us became 192): there the waves meet behind the
  // scores, and the partner's products run two behind the own ones, while its weights come.
  constexpr bool kEarly = !FP8;
  constexpr int kLag = kEarly ? 0 : 2;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[Lds::kBytes];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h2 = lane >> 5, lo = lane & 15, z = w & 1;

  typename Form::template Work<128, 32> wk(p, lane);
  if (!wk.valid) return;
  const int64_t nrows = (int64_t)p.T * p.H;
  const int tile_end = wk.tile_end;
  const auto un = wk.unit(w), mate = wk.unit(w ^ 1);  // the wave's rows, and its partner's
  const uint32_t base = lds_addr(&lds[0]);

  // ---- queries, as in k_latent_wide
  const float sm = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(scale_magnitude(p.sm_log2))));
  constexpr int kHeld = FP8 ? 32 : 36;  // of the 36 operands; with codes the rotary ones stay in LDS
  bf16x8 qf[kHeld], qrot[36 - kHeld + 1];
  {
    using QTile = LatentTile<false, true>;
    constexpr int kFit = FP8 ? 1 : 2;
    static_assert(kFit * QTile::kBytes <= Lds::kBytes, "query rows fit");
    TileCopy<QTile, false> qc{p, w, lane};
    const uint32_t sign = p.sm_log2 < 0.f ? 0x80008000u : 0u;
    const int qrow = 32 * (w & 1) + c;
#pragma unroll
    for (int q0 = 0; q0 < 2; q0 += kFit) {
#pragma unroll
      for (int i = q0; i < q0 + kFit; ++i) {
        qc.aim_q(wk.unit(2 * i), wk.unit(2 * i + 1));
        qc.all(base + (i - q0) * QTile::kBytes);
      }
      wait_copies();
      __syncthreads();
      if (w / 2 >= q0 && w / 2 < q0 + kFit) {
        const uint32_t qb = base + (w / 2 - q0) * QTile::kBytes + qrow * QTile::kRow;
        const uint32_t qr = base + (w / 2 - q0) * QTile::kBytes + QTile::kRope + qrow * QTile::kRopeRow;
#pragma unroll
        for (int ks = 0; ks < 36; ++ks) {
          const int ch = FP8 ? 4 * (ks >> 1) + (ks & 1) : 2 * ks;
          const uint32_t at = ks < 32 ? ((qb + (((FP8 ? 2 * h2 : h2) ^ QTile::swz(qrow)) * 16)) ^ (16 * (ch & 31))) + 512 * (ch >> 5)
                                      : (qr + ((h2 ^ QTile::swz_rope(qrow)) * 16)) ^ (32 * (ks - 32));
          (ks < kHeld ? qf[ks < kHeld ? ks : 0] : qrot[ks < kHeld ? 0 : ks - kHeld]) = flip_sign(lds_read<bf16x8>(at), sign);
        }
      }
      lds_barrier();
    }
  }

  const uint32_t queries = base + Lds::kQueries + w * 4096;
  if constexpr (FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(__attribute__((address_space(3))) bf16x8*)(uintptr_t)(queries + i * 1024 + lane * 16) = qrot[i];
  }

  // ---- the walk: passes of up to 64 keys, two steps each
  struct Pass {
    int ti, who;
    uint64_t held;        // its keys
    uint32_t own, other;  // ~0 if the wave's rows (its partner's) see them, or 0
  };
  auto after = [](const Pass& x) { return x.who < 0 ? x.ti + 1 : x.ti; };
  auto find = [&](int ti, int who, int v, int& rows) __attribute__((always_inline)) {
    Pass x;
    wk.lane = anew(lane);
    x.ti = __builtin_amdgcn_readfirstlane(wk.next_pass(ti, who, v, x.who, rows));
    x.who = __builtin_amdgcn_readfirstlane(x.who);
    x.held = wave_ballot(rows >= 0);
    auto sees = [&](const auto& u) {
      return (uint32_t)__builtin_amdgcn_readfirstlane(x.ti < tile_end && wk.in_pass(x.ti, x.who, u) ? -1 : 0);
    };
    x.own = sees(un);
    x.other = sees(mate);
    return x;
  };
  int rows = -1;  // of the pass that is being copied: lane i has key i

  // ---- copies of a step: the wave's eight keys
  const uint64_t zeros = (uint64_t)(uintptr_t)g_zero_row;
  auto address = [&](const void* from, int row, int stride) -> uint64_t {
    return row >= 0 ? (uint64_t)(uintptr_t)from + (uint64_t)(uint32_t)row * (uint32_t)stride : zeros;
  };
  // the rows of half n of the pass whose pieces the lane copies: of the first and the second
  // four keys, of the rotary rows, and the key whose scale it brings
  int row_a = -1, row_b = -1, row_rot = -1, row_scale = -1;
  auto begin_copies = [&](int n) {
    const int ln = anew(lane), first = 32 * n + 8 * w;
    row_a = __shfl(rows, first + (ln >> 4), kWave);
    row_b = __shfl(rows, first + 4 + (ln >> 4), kWave);
    row_rot = __shfl(rows, first + (ln >> 3), kWave);
    if constexpr (FP8) row_scale = __shfl(rows, first + (ln & 7), kWave);
  };
  uint64_t from = 0;
  // copy J of that half, to stage `at` (its rotary rows to stage `rot_to`)
  auto copy = [&](uint32_t at, uint32_t rot_to, auto number) __attribute__((always_inline)) {
    constexpr int J = decltype(number)::value, G = J / Lds::kParts, K = J % Lds::kParts;
    if constexpr (FP8 && J == 5) {
      copy4_to_lds(reinterpret_cast<const void*>(address(p.scale, row_scale, 4)), base + Lds::kScales + at * 1024 + w * 256);
    } else if constexpr (G == 2) {
      const uint64_t rot = FP8 ? address(p.rope, row_rot, 2 * kRotary) : address(p.c, row_rot, kStride) + 2 * kLatent;
      const int ln = anew(lane);
      copy16_to_lds(reinterpret_cast<const void*>(rot + (uint32_t)(((ln & 7) ^ ((4 * w + (ln >> 4)) & 7)) * 16)),
                    base + Lds::kRotAt + rot_to * Lds::kRot + 8 * w * Lds::kRotRow);
    } else {
      if constexpr (K == 0) {
        const int ln = anew(lane);
        from = address(p.c, G ? row_b : row_a, kStride) + (uint32_t)(((ln & 15) ^ (ln >> 4) << (FP8 ? 1 : 2)) * 16);
      }
      copy_piece_to_lds<256 * K, Lds::four_at(G) + 1024 * K>(from, base + at * Lds::kLat + Lds::four_at(2 * w));
    }
  };
  // the page entries of the tile behind a pass's, for the pass after it
  const uint32_t pages_lds = base + Lds::kPages + w * 256;
  auto ask_entries = [&](const Pass& x) { copy4_to_lds(wk.entry_at(x.ti + 1), pages_lds); };

  f32x16 own[8], oth[8];
#pragma unroll
  for (int d = 0; d < 8; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) own[d][e] = 0.f, oth[d][e] = 0.f;
#pragma unroll
  for (int d = 0; d < 8; ++d) in_agprs(own[d]), in_agprs(oth[d]);
  float m = kNoMax, l = 0.f;
  uint32_t has = 0;

  // the lane's places in a step: its key row, its rotary row, its row of the transposing
  // reads (of values 256 z .. + 255, which the wave sums); and where pieces 0 .. 3 of them
  // lie in the stage that is read
  const uint32_t a_key = Lds::row_at(c) + h2 * 16, x_key = (c & 3) << Lds::kPiece;
  const uint32_t a_rot = c * Lds::kRotRow + ((h2 ^ (c >> 1 & 7)) * 16);
  const int vrow = FP8 ? 4 * h2 + ((lo >> 1) & 3) + 8 * (lo >> 3) : 4 * h2 + (lo >> 2);
  const uint32_t a_val = Lds::row_at(vrow) + (lo & 1) * 8 +
                         (FP8 ? (lane >> 4) & 1 : 2 * ((lane >> 4) & 1) + ((lo & 3) >> 1)) * 16 + (FP8 ? 1024 : 2048) * z;
  const uint32_t x_val = (vrow & 3) << Lds::kPiece;
  uint32_t key_at[4], val_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    key_at[i] = base + a_key + (x_key ^ (uint32_t)(i << Lds::kPiece));
    val_at[i] = base + a_val + (x_val ^ (uint32_t)(i << Lds::kPiece));
  }
  auto weights = [&](int n, int of) { return base + Lds::kWeights + n * 8192 + of * 2048 + (uint32_t)anew(lane) * 16; };
  auto factors = [&](int n, int of) { return base + Lds::kFactors + n * 512 + of * 128 + (uint32_t)(anew(lane) & 31) * 4; };

  // (stage: 0 or 1, of the pair that key_at and val_at point to)
  auto read_key = [&](uint32_t ra, int stage, int i) -> u32x4 {
    if (i >= kKeyReads - 4) return lds_read<u32x4>(ra ^ (32 * (i - (kKeyReads - 4))));
    return FP8 ? lds_read<u32x4>(key_at[i & 3] + (stage * Lds::kLat + 128 * (i >> 2 & 1) + 1024 * (i >> 3)))
               : lds_read<u32x4>(key_at[i >> 1 & 3] + (stage * Lds::kLat + 32 * (i & 1) + 1024 * (i >> 3)));
  };
  // values 32 d .. + 31 of the wave's half, keys 16 j .. + 15 of the step
  auto read_value = [&](int stage, int i) -> u32x4 {
    const int j = i >> 3, d = i & 7;
    const uint32_t at = val_at[d & 3] + (stage * Lds::kLat + (d >> 2) * (FP8 ? 128 : 1024) + j * Lds::four_at(4));
    if constexpr (FP8) {
      const u32x2 x = lds_read_tr8(at);
      return u32x4{x.x, x.y, 0u, 0u};
    }
    return __builtin_bit_cast(u32x4, join_rows(lds_read_tr16(at), lds_read_tr16(at + Lds::four_at(2))));
  };
  auto operand = [&](u32x4 v) -> bf16x8 {
    if constexpr (FP8) return codes_to_bf16(u32x2{v.x, v.y});
    return __builtin_bit_cast(bf16x8, v);
  };

  // Reads of keys run kAhead ahead of their products, in two groups; the last one asked for of
  // a group is used first, so that a group is waited for once.
  u32x4 ring[kAhead];
  constexpr int kGroup = kAhead / 2;
  auto used = [](int t) constexpr { return t / kGroup * kGroup + ((t / kGroup >> 1 & 1) ? t % kGroup : kGroup - 1 - t % kGroup); };
  auto rot_at = [&](uint32_t at) { return base + Lds::kRotAt + at * Lds::kRot + a_rot; };
  // The scores of a step (result rows 8 (e / 4) + 4 h2 + e % 4 of its keys), from stage `at`,
  // which is STAGE of the pair that key_at points to; with work(t) between the products, t = 0 .. 35.
  auto score = [&](f32x16& s, uint32_t at, uint32_t rot, auto of, auto work) __attribute__((always_inline)) {
    constexpr int STAGE = decltype(of)::value;
    const uint32_t ra = rot_at(rot);
    if constexpr (FP8) {
      // a read serves two products, whose operands are converted beside the ones before
      bf16x8 a0, a1;
      {
        const u32x4 v = ring[used(0) % kAhead];
        a0 = codes_to_bf16(u32x2{v.x, v.y}), a1 = codes_to_bf16(u32x2{v.z, v.w});
      }
      each<16>([&](auto number) __attribute__((always_inline)) {
        constexpr int t = decltype(number)::value, i = used(t);
        if constexpr (t == 0)
          mfma_vgpr_first(s, a0, qf[2 * i]);
        else
          mfma_loaded(s, a0, qf[2 * i]);
        if constexpr (i + kAhead < kKeyReads) ring[i % kAhead] = read_key(ra, STAGE, i + kAhead);
        work(std::integral_constant<int, 2 * t>{});
        __builtin_amdgcn_sched_barrier(0);
        bf16x8 b0, b1;
        if constexpr (t < 15) {
          const u32x4 v = ring[used(t + 1) % kAhead];
          b0 = anew(codes_to_bf16(u32x2{v.x, v.y}));
          __builtin_amdgcn_sched_barrier(0);
          b1 = anew(codes_to_bf16(u32x2{v.z, v.w}));
          __builtin_amdgcn_sched_barrier(0);  // (each at least two instructions before its product, and not moved to it)
        }
        mfma_loaded(s, a1, qf[2 * i + 1]);
        __builtin_amdgcn_sched_barrier(0);
        work(std::integral_constant<int, 2 * t + 1>{});
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (t < 15) a0 = b0, a1 = b1;
      });
      bf16x8 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = lds_read<bf16x8>(queries + i * 1024 + (uint32_t)anew(lane) * 16);
      mfma_done(s);
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // a key's scale multiplies its latent part only
        const f32x4 sc = lds_read<f32x4>(base + Lds::kScales + at * 1024 + 256 * k + 16 * h2);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * k + e] *= sc[e];
      }
      each<4>([&](auto number) __attribute__((always_inline)) {
        constexpr int i = decltype(number)::value;
        mfma_vgpr(s, __builtin_bit_cast(bf16x8, ring[(16 + i) % kAhead]), q[i]);
        work(std::integral_constant<int, 32 + i>{});
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      each<36>([&](auto number) __attribute__((always_inline)) {
        constexpr int t = decltype(number)::value, i = used(t);
        const bf16x8 v = __builtin_bit_cast(bf16x8, ring[i % kAhead]);
        if constexpr (t == 0)
          mfma_vgpr_first(s, v, qf[i]);
        else
          mfma_loaded(s, v, qf[i]);
        if constexpr (i + kAhead < 36) ring[i % kAhead] = read_key(ra, STAGE, i + kAhead);
        work(number);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
  };

  // (tiles below this are taken by all rows that are not padding)
  const int plain_end = __builtin_amdgcn_readfirstlane(min(wk.np, tile_end));
  const uint32_t live = __builtin_amdgcn_readfirstlane(un.live ? -1 : 0), live_mate = __builtin_amdgcn_readfirstlane(mate.live ? -1 : 0);
  // the first two passes (the second's other half is copied once more in the first step)
  Pass cur, nxt;
  nxt.ti = wk.cur - 1;
  nxt.who = -1;
#pragma unroll 1
  for (uint32_t at = 0; at < 4; at += 2) {
    cur = nxt;
    const int ti = after(nxt);
    nxt = find(ti, nxt.who, wk.list_entry(ti), rows);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      begin_copies(n);
      // (step 3's rotary rows would take the place of step 0's; it is copied in the first step anyway)
      each<kCopies>([&](auto j) __attribute__((always_inline)) {
        if (at + n < 3 || j != (FP8 ? 4 : 8)) copy(at + n, at + n, j);
      });
    }
  }
  ask_entries(nxt);
  wait_copies();
  lds_barrier();
  f32x16 s0, s1;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ring[i] = read_key(0u, 0, i);
  score(s0, 0u, 0u, std::integral_constant<int, 0>{}, [](auto) {});
  mfma_done(s0);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ring[i] = read_key(0u, 1, i);
  begin_copies(1);
  uint32_t pair = 0;  // the pass's stages are pair, pair + 1
  Pass found = nxt;   // the pass after the next
  uint32_t third = 0;  // the step's number modulo 3

  // Where not all see a pass, the others' products take zeros on both sides: a weight of
  // zero times an infinite value would be NaN, and so is one times a scale that is.
  auto seen_by = [](bf16x8 a, uint32_t who) {
    u32x4 v = __builtin_bit_cast(u32x4, a);
    v &= who;
    return __builtin_bit_cast(bf16x8, v);
  };
  // One step: the weights of its keys from s, beside the scores of the next step (into
  // s_next) and the copies of the one three on; then its values. N: half of the pass.
  // PART: not all rows may see the pass.
  auto take = [&](auto half, auto part, f32x16& s, f32x16& s_next) __attribute__((always_inline)) {
    constexpr int N = decltype(half)::value;
    constexpr bool PART = decltype(part)::value;
    // stages: of the step, the next one, and the one that is copied
    const uint32_t here = pair + N, next = N == 0 ? pair + 1 : pair ^ 2, last = N == 0 ? (pair ^ 2) + 1 : pair;
    const uint32_t third_next = third == 2 ? 0 : third + 1;
    const uint32_t seen = (uint32_t)(cur.held >> (32 * N)) & cur.own;
    has |= cur.own;
    if (__builtin_expect(seen != 0xffffffffu, 0)) {
      // (not sixteen masks kept in registers; with codes not the lane's half either: it was spilled,
      // and its reload waited for the copies in flight)
      const uint32_t bits = seen >> (FP8 ? (__builtin_amdgcn_mbcnt_lo(~0u, anew(0u)) >> 5) * 4 : (uint32_t)anew(4 * h2));
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = (bits >> (8 * (e >> 2) + (e & 3))) & 1u ? s[e] : -INFINITY;
    }
    float top, f = 1.f;
    bf16x8 pb[2], po[2];
    float fo;
    f32x4 sc;
    u32x4 vring[kAheadV];
    // What was copied in the last step has landed, and this one's weights are there. One
    // barrier a step: behind it all waves are done with the last step's values, whose place
    // this step's copies take, and with what they handed each other the step before that.
    auto meet = [&]() __attribute__((always_inline)) {
      wait_copies();
      lds_barrier();
#pragma unroll
      for (int j = 0; j < 2; ++j) po[j] = lds_read<bf16x8>(weights(N, w ^ 1) + j * 1024);
      fo = lds_read<float>(factors(N, w ^ 1));
    };
    auto work = [&](auto number) __attribute__((always_inline)) {
      constexpr int t = decltype(number)::value;
      if constexpr (t < 4) {
        const float x = max_or_nan(max_or_nan(s[4 * t], s[4 * t + 1]), max_or_nan(s[4 * t + 2], s[4 * t + 3]));
        top = t == 0 ? x : max_or_nan(top, x);
      } else if constexpr (t == 4) {
        top = max_halves(top) * sm;
      } else if constexpr (t == 5) {
        if (__builtin_expect(__any(top > m + kSlack), 0)) {
          const float mm = top > m + kSlack ? top : m;
          f = exp2_fast(m - mm);
          m = mm;
          l *= f;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            in_agprs(own[d]);
            own[d] *= f;
            in_agprs(own[d]);
            __builtin_amdgcn_sched_barrier(0);  // (one tile at a time in vector registers)
          }
        }
      } else if constexpr (t < 22) {
        constexpr int e = t - 6;
        if constexpr (FP8 && (e & 3) == 0) sc = lds_read<f32x4>(base + Lds::kScales + here * 1024 + 256 * (e >> 2) + 16 * h2);
        float x = exp2_fast(fmaf(s[e], sm, -m));
        l += x;  // the total keeps 32 bits; the weights are rounded to bf16 for the matrix cores
        if constexpr (FP8) x *= sc[e & 3];
        pb[e >> 3][e & 7] = (__bf16)x;
      } else if constexpr (t == 22 || t == 23) {
        if constexpr (FP8 && PART) pb[t - 22] = seen_by(pb[t - 22], cur.own);
        *(__attribute__((address_space(3))) bf16x8*)(uintptr_t)(weights(N, w) + (t - 22) * 1024) = pb[t - 22];
      } else if constexpr (t == 24) {
        *(__attribute__((address_space(3))) float*)(uintptr_t)factors(N, w) = f;
      } else if constexpr (kEarly && t == 26) {
        meet();
      } else if constexpr (t >= 36 - kAheadV) {
        vring[t - (36 - kAheadV)] = read_value(N, t - (36 - kAheadV));
      }
    };
    score(s_next, next, third_next, std::integral_constant<int, 1 - N>{}, work);
    if constexpr (!kEarly) meet();
    int entry = 0;
    each<16 + kLag>([&](auto number) __attribute__((always_inline)) {
      constexpr int i = decltype(number)::value;
      if constexpr (i < 16) {
        const bf16x8 a = operand(vring[i % kAheadV]);
        own[i & 7] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(PART ? seen_by(a, cur.own) : a, pb[i >> 3], own[i & 7], 0, 0, 0);
      }
      if constexpr (i == kLag / 2) {
        if (__builtin_expect(__any(fo != 1.f), 0)) {
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            in_agprs(oth[d]);
            oth[d] *= fo;
            in_agprs(oth[d]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      if constexpr (i < kCopies) copy(last, third, number);
      if constexpr (N == 0) {
        // the pass after the next, which the copies of the next two steps are of
        if constexpr (i == 8) entry = lds_read<int>(pages_lds + (uint32_t)anew(lane) * 4);
        if constexpr (i == 10) rows = wk.plain_row(nxt.ti + 1, entry);
        if constexpr (i == 11) {
          found = Pass{nxt.ti + 1, -1, wave_ballot(rows >= 0), live, live_mate};
          if (__builtin_expect((nxt.who >= 0) | (found.ti >= plain_end) | (found.held == 0), 0)) found = find(after(nxt), nxt.who, entry, rows);
        }
        if constexpr (i == 12) ask_entries(found);
        if constexpr (i == 13) {  // the keys that are scored from here on are the next pass's
          const uint32_t by = pair ? -2 * Lds::kLat : 2 * Lds::kLat;
#pragma unroll
          for (int q = 0; q < 4; ++q) key_at[q] += by;
        }
      }
      if constexpr (i == 14) begin_copies(N == 0 ? 0 : 1);  // of the next step
      if constexpr (i >= kLag) {
        constexpr int k = i - kLag;
        const bf16x8 a = operand(vring[k % kAheadV]);
        oth[k & 7] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(PART ? seen_by(a, cur.other) : a, po[k >> 3], oth[k & 7], 0, 0, 0);
        if constexpr (k + kAheadV < 16) vring[k % kAheadV] = read_value(N, k + kAheadV);
        // the next step's first reads come last
        constexpr int kLast = 2 + kLag;
        if constexpr (i >= 14) {  // (behind the step to the next pair)
#pragma unroll
          for (int x = (i - 14) * kAhead / kLast; x < (i - 13) * kAhead / kLast; ++x) ring[x] = read_key(0u, N, x);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    third = third_next;
    s_next = anew(s_next);  // (its last products ended while the values' ran; a test reads the distance)
    if constexpr (N == 1) {
      cur = nxt;
      nxt = found;
      const uint32_t by = pair ? -2 * Lds::kLat : 2 * Lds::kLat;
#pragma unroll
      for (int q = 0; q < 4; ++q) val_at[q] += by;
      pair ^= 2;
    }
  };
  using First = std::integral_constant<int, 0>;
  using Second = std::integral_constant<int, 1>;
  while (cur.ti < tile_end && cur.who < 0) {
    take(First{}, std::false_type{}, s0, s1);
    take(Second{}, std::false_type{}, s1, s0);
  }
  while (cur.ti < tile_end) {
    take(First{}, std::true_type{}, s0, s1);
    take(Second{}, std::true_type{}, s1, s0);
  }

  // ---- result: lane holds values 256 z + 32 d + 8 i + 4 h2 + 0..3 of its two rows
  wait_copies();  // (of steps past the last)
  __syncthreads();
  const float tot = row_total(has != 0, sum_halves(l));
  float* ml = reinterpret_cast<float*>(&lds[Lds::kWeights]);
  if (h2 == 0) ml[64 * w + c] = m, ml[64 * w + 32 + c] = tot;
  __syncthreads();
  const float tot_mate = ml[64 * (w ^ 1) + 32 + c];
  // through LDS (the wave's own part), so that rows leave in whole lines: 512 bytes of
  // each row at a time, 16-byte chunks in an order that depends on the row
  constexpr int kSeg = 512;
  static_assert(4 * 32 * kSeg <= Lds::kWeights, "room for every wave's rows");
  const uint32_t mine = base + w * 32 * kSeg;
  auto put = [&](unsigned char* dst, int64_t stride, int n) {  // what is in LDS to n rows `stride` apart
#pragma unroll 8
    for (int i = 0; i < n; i += 2) {
      const int rr = i + h2;
      const u32x4 v = lds_read<u32x4>(mine + rr * kSeg + ((c ^ (rr & 31)) * 16));
      if (rr < n) *reinterpret_cast<u32x4*>(dst + rr * stride + c * 16) = v;
    }
  };
  // (padding's sums hold what weights of zero left of its keys: NaN, it may be)
  auto leave = [&](f32x16 (&o)[8], const typename Form::template Work<128, 32>::Unit& u, float total, uint32_t keep) {
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = __uint_as_float(__float_as_uint(o[d][e]) & keep);
    if (wk.in_parts()) {
      unsigned char* dst = reinterpret_cast<unsigned char*>(p.part + wk.part_row(u, nrows) * kLatent) + z * 1024;
#pragma unroll
      for (int d0 = 0; d0 < 8; d0 += 4) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *(__attribute__((address_space(3))) f32x4*)(uintptr_t)(mine + c * kSeg + (((8 * d + 2 * i + h2) ^ c) * 16)) =
                f32x4{o[d0 + d][4 * i], o[d0 + d][4 * i + 1], o[d0 + d][4 * i + 2], o[d0 + d][4 * i + 3]};
        put(dst + d0 * 128, kLatent * 4, u.rows);
      }
    } else {
      const float inv = row_inverse(total);
#pragma unroll
      for (int d = 0; d < 8; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 v = {o[d][4 * i] * inv, o[d][4 * i + 1] * inv, o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv};
          *(__attribute__((address_space(3))) bf16x4*)(uintptr_t)(mine + c * kSeg + (((4 * d + i) ^ c) * 16) + h2 * 8) =
              __builtin_convertvector(v, bf16x4);
        }
      put(reinterpret_cast<unsigned char*>(p.out + u.row * kLatent) + z * 512, kLatent * 2, u.rows);
    }
  };
  leave(own, un, tot, live);
  leave(oth, mate, tot_mate, live_mate);
  const bool first = h2 == 0 && c < un.rows;
  if (wk.in_parts() && first) {
    p.part_ml[(wk.part_row(un, nrows) + c) * 2] = m;
    p.part_ml[(wk.part_row(un, nrows) + c) * 2 + 1] = tot;
  }
  if (!wk.in_parts() && p.lse && first) p.lse[un.row + c] = row_log_sum(m, tot);
}

}  // namespace misa
