// What the cache and latent-attention kernels share: fixed widths, argument
// structs and launchers (cache_kernels.hip, latent_kernels.hip,
// expanded_kernels.hip; argument checks in api_attention.hip).
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

// Joins the partial results of the splits of rows of `width` values.
hipError_t launch_join(const LaunchCtx& cx, const float* part, const float* part_ml, int splits, int64_t rows,
                       int width, uint16_t* out, float* lse);

}  // namespace misa
