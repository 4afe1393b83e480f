// What the cache and latent-attention kernels share: fixed widths, argument
// structs and launchers (cache_kernels.hip, latent_kernels.hip,
// expanded_kernels.hip, tree_kernels.hip, norm_kernels.hip, paged_kernels.hip;
// argument checks in api_attention.hip and api_paged.hip).
#pragma once

#include "launch.h"

namespace misa {

constexpr int kLatent = 512;           // values of a latent row
constexpr int kRotary = 64;            // rotary values beside them
constexpr int kNope = 128, kValue = 128;  // expanded key (without rotary part) and value of one head
constexpr int kAttnTile = 64;          // keys per tile, and the grain of a split

// ---- caches (cache_kernels.hip)
struct CacheArgs {
  int32_t n;             // rows to write or read
  int32_t rows;          // rows of the cache
  int32_t d, dr;         // coded and rotary columns
  const int32_t* slots;  // [n]
  void* c;               // [rows, d] codes, or [rows, d + dr] bf16
  float* scale;          // [rows] (codes)
  uint16_t* rope;        // [rows, dr] bf16 (codes with rotary columns)
};
hipError_t launch_cache_write(const LaunchCtx& cx, const CacheArgs& a, bool fp8, const uint16_t* x);
hipError_t launch_cache_read(const LaunchCtx& cx, const CacheArgs& a, bool fp8, uint16_t* out);

// ---- latent attention, absorbed form (latent_kernels.hip)
struct LatentArgs {
  const uint16_t* q;     // [T, H, 576] bf16
  int32_t T, H;
  const void* c;         // [rows, 512] codes, or [rows, 576] bf16
  const float* scale;    // [rows] (codes)
  const uint16_t* rope;  // [rows, 64] bf16 (codes)
  int32_t rows;
  const int32_t* pos;    // [T] (no lists)
  const int32_t* idx;    // [T, k] (lists)
  int32_t k;
  const int32_t* base;   // [T] or null
  float sm_log2;         // softmax scale times log2(e)
  uint16_t* out;         // [T, H, 512]
  float* lse;            // [T, H] or null
  // set by the launcher
  float* part;           // [splits, T * H, 512] partial sums
  float* part_ml;        // [splits, T * H, 2] their reference and weight
  int32_t splits;
  int32_t head_tiles;    // row tiles per query (rows of one query), 0: tiles run over all T * H rows
  int32_t row_tiles;
};
// How a call is cut: rows per workgroup and splits of the key axis.
struct AttnPlan {
  int nq, head_tiles, row_tiles, splits;
};
AttnPlan latent_plan(int T, int H, int keys, bool shared_keys);
size_t latent_ws_bytes(const AttnPlan& pl, int T, int H);
hipError_t launch_latent(const LaunchCtx& cx, LatentArgs a, const AttnPlan& pl, bool fp8, void* ws);

// ---- latent attention, expanded form (expanded_kernels.hip)
struct ExpandedArgs {
  const uint16_t* q;     // [T, H, 192] bf16
  const uint16_t* kv;    // [L, H, 256] bf16
  const uint16_t* rope;  // [L, 64] bf16, rows rope_ld apart
  int64_t rope_ld;
  int32_t T, H, L;
  const int32_t* pos;    // [T]
  const int32_t* base;   // [T] or null
  float sm_log2;
  uint16_t* out;         // [T, H, 128]
  float* lse;            // [T, H] or null
  float* part;           // [splits, T * H, 128]
  float* part_ml;        // [splits, T * H, 2]
  int32_t splits;
  int32_t row_tiles;
};
AttnPlan expanded_plan(int T, int H, int L);
size_t expanded_ws_bytes(const AttnPlan& pl, int T, int H);
hipError_t launch_expanded(const LaunchCtx& cx, ExpandedArgs a, const AttnPlan& pl, void* ws);

// ---- paged caches (paged_kernels.hip): position j of sequence s lies in row
// (table[s, j >> page_log2] << page_log2) + (j & (2^page_log2 - 1))
struct Pages {
  const int32_t* table;  // [seqs, per]
  int32_t seqs, per, page_log2;
};
struct Rotation {
  const float* rot;  // [positions, 64]: cosines, then sines
  int32_t positions;
  bool pairs;        // values 2i, 2i + 1 turn together, instead of i, i + 32
};
struct AppendArgs {
  CacheArgs cache;       // (slots unused)
  Pages pages;
  const uint16_t* x;     // rows of d + dr bf16, x_ld apart
  int64_t x_ld;
  const int32_t* seq;    // [n]
  const int32_t* pos;    // [n] where a row goes
  const int32_t* turn;   // [n] the position that it is rotated by
  const void* weight;    // [d] or null: no norm
  bool weight_f32;
  double eps;
  Rotation rot;          // rot null: no rotation
  int32_t rot_at;        // first rotated column
  double inv_width;      // (set by the launcher) 1 / d
};
hipError_t launch_paged_append(const LaunchCtx& cx, AppendArgs a, bool fp8);
struct RotateArgs {
  int32_t T, H;
  const uint16_t* x;     // [T, H, 64], rows x_h and queries x_t elements apart
  int64_t x_t, x_h;
  uint16_t* out;
  int64_t out_t, out_h;
  const int32_t* pos;    // [T]
  Rotation rot;
};
hipError_t launch_rotate(const LaunchCtx& cx, const RotateArgs& a);

// ---- norm (norm_kernels.hip)
struct NormArgs {
  int32_t n, width;
  const uint16_t* x;         // rows of width bf16, x_ld apart
  int64_t x_ld;
  const uint16_t* residual;  // [n, width] or null
  const void* weight;        // [width]
  bool weight_f32;
  double eps;
  double inv_width;          // (set by the launcher) 1 / width
  void* y;                   // [n, width] bf16 or codes
  float* scale;              // [n] or [n, ceil(width / 128)] (codes)
  uint16_t* sum;             // [n, width] or null
};
enum class NormOut { kBf16, kRowCodes, kGroupCodes };
hipError_t launch_rms_norm(const LaunchCtx& cx, NormArgs a, NormOut out);

// ---- attention of drafted tokens (tree_kernels.hip)
struct TreeArgs : LatentArgs {
  Pages pages;
  int32_t N;              // drafted nodes (queries) of a sequence
  int32_t words;          // 64-bit words of a mask
  const int32_t* prefix;  // [seqs]
  const uint64_t* mask;   // [seqs, N, words] or null (chains)
  // set by the launcher
  int32_t tiles_a_seq;    // row tiles of a sequence
  int32_t budget[2];      // splits over all sequences, in either of two cuts
  int32_t least;          // tiles a split takes at least
  float fixed, tile, join;  // what a workgroup, a tile and the join of a split cost (us)
  int32_t* rec;           // [seqs, 2]: first slot and splits of a sequence
};
struct TreePlan {
  int nq, tiles_a_seq, budget[2], least;
  float fixed, tile;
};
TreePlan tree_plan(int seqs, int N, int H, int words, int longest);
size_t tree_ws_bytes(const TreePlan& pl, int seqs);
hipError_t launch_tree(const LaunchCtx& cx, TreeArgs a, const TreePlan& pl, bool fp8, void* ws);
// The rows of the keys of queries with lists of positions: [T, k + 64 words], -1 where there is none.
hipError_t launch_tree_lists(const LaunchCtx& cx, const TreeArgs& a, int32_t* lists);

// Joins the partial results of the splits of rows of `width` values.
hipError_t launch_join(const LaunchCtx& cx, const float* part, const float* part_ml, int splits, int64_t rows,
                       int width, uint16_t* out, float* lse);

}  // namespace misa
