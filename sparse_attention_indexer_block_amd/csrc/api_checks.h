// Argument checks shared by the entry points of the caches and the attention.
#pragma once

#include <cmath>

#include "attention.h"
#include "status.h"

namespace misa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxRows = (int64_t)1 << 30;  // (query, head) rows of a call

inline misa_status check_ptr(const void* ptr, const char* name, size_t a) {
  if (!ptr) return fail(MISA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(ptr, a)) return fail(MISA_ERR_INVALID_ARG, "%s must be %zu-byte aligned", name, a);
  return MISA_OK;
}

inline misa_status check_cache(const misa_cache* c) {
  if (!c) return fail(MISA_ERR_INVALID_ARG, "cache is NULL");
  if (c->dtype != MISA_K_BF16 && c->dtype != MISA_K_FP8_E4M3FN)
    return fail(MISA_ERR_INVALID_ARG, "cache dtype = %d is not a misa_kdtype", c->dtype);
  if (c->rows < 1) return fail(MISA_ERR_INVALID_ARG, "cache rows = %d must be >= 1", c->rows);
  if (c->rows > (1 << 30)) return fail(MISA_ERR_UNSUPPORTED, "cache rows = %d exceeds 2^30", c->rows);
  if (c->d < 1 || c->dr < 0) return fail(MISA_ERR_INVALID_ARG, "cache d = %d, dr = %d", c->d, c->dr);
  if ((c->d != kHeadDimHost && c->d != kLatent) || (c->dr != 0 && c->dr != kRotary))
    return fail(MISA_ERR_UNSUPPORTED, "cache d = %d, dr = %d (d = 128 or 512, dr = 0 or 64)", c->d, c->dr);
  MISA_TRY(check_ptr(c->c, "cache c", 16));
  const bool fp8 = c->dtype == MISA_K_FP8_E4M3FN;
  if (fp8) MISA_TRY(check_ptr(c->scale, "cache scale", 4));
  if (fp8 && c->dr) MISA_TRY(check_ptr(c->rope, "cache rope", 16));
  if (!fp8 && c->scale) return fail(MISA_ERR_INVALID_ARG, "cache scale must be NULL for bf16 rows");
  if ((!fp8 || !c->dr) && c->rope)
    return fail(MISA_ERR_INVALID_ARG, "cache rope must be NULL (bf16 rows hold their rotary values; dr = 0 has none)");
  return MISA_OK;
}

inline CacheArgs cache_args(const misa_cache* c, int32_t n, const int32_t* slots) {
  CacheArgs a{};
  a.n = n;
  a.rows = c->rows;
  a.d = c->d;
  a.dr = c->dr;
  a.slots = slots;
  a.c = c->c;
  a.scale = c->scale;
  a.rope = static_cast<uint16_t*>(c->rope);
  return a;
}

inline misa_status check_sizes(int32_t T, int32_t H, float sm_scale) {
  if (T < 0) return fail(MISA_ERR_INVALID_ARG, "T = %d is negative", T);
  if (H < 1) return fail(MISA_ERR_INVALID_ARG, "H = %d must be >= 1", H);
  if (T > (1 << 22)) return fail(MISA_ERR_UNSUPPORTED, "T = %d exceeds 2^22 queries", T);
  if ((int64_t)T * H > kMaxRows) return fail(MISA_ERR_UNSUPPORTED, "T * H = %lld exceeds 2^30", (long long)T * H);
  if (!std::isfinite(sm_scale)) return fail(MISA_ERR_INVALID_ARG, "sm_scale is not finite");
  if (!std::isfinite(sm_scale * kLog2e))  // (the kernels' exponentials are powers of two)
    return fail(MISA_ERR_INVALID_ARG, "sm_scale = %g is past 2.35e38 in magnitude", (double)sm_scale);
  return MISA_OK;
}

inline misa_status check_scratch(size_t need, void* ws, size_t ws_bytes) {
  if (ws_bytes < need)
    return fail(MISA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", ws_bytes, need);
  if (!ws) return fail(MISA_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(MISA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return MISA_OK;
}

}  // namespace misa
