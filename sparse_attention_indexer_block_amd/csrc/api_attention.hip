// C ABI of the caches and of latent attention: argument checks, the cut of a
// call into workgroups, and the launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "attention.h"
#include "status.h"

namespace misa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxRows = (int64_t)1 << 30;  // (query, head) rows of a call

static misa_status check_ptr(const void* ptr, const char* name, size_t a) {
  if (!ptr) return fail(MISA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(ptr, a)) return fail(MISA_ERR_INVALID_ARG, "%s must be %zu-byte aligned", name, a);
  return MISA_OK;
}

static misa_status check_cache(const misa_cache* c) {
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

static CacheArgs cache_args(const misa_cache* c, int32_t n, const int32_t* slots) {
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

static misa_status check_sizes(int32_t T, int32_t H, float sm_scale) {
  if (T < 0) return fail(MISA_ERR_INVALID_ARG, "T = %d is negative", T);
  if (H < 1) return fail(MISA_ERR_INVALID_ARG, "H = %d must be >= 1", H);
  if (T > (1 << 22)) return fail(MISA_ERR_UNSUPPORTED, "T = %d exceeds 2^22 queries", T);
  if ((int64_t)T * H > kMaxRows) return fail(MISA_ERR_UNSUPPORTED, "T * H = %lld exceeds 2^30", (long long)T * H);
  if (!std::isfinite(sm_scale)) return fail(MISA_ERR_INVALID_ARG, "sm_scale is not finite");
  if (!std::isfinite(sm_scale * kLog2e))  // (the kernels' exponentials are powers of two)
    return fail(MISA_ERR_INVALID_ARG, "sm_scale = %g is past 2.35e38 in magnitude", (double)sm_scale);
  return MISA_OK;
}

static misa_status check_latent(const misa_latent_problem* p) {
  if (!p) return fail(MISA_ERR_INVALID_ARG, "problem is NULL");
  MISA_TRY(check_sizes(p->T, p->H, p->sm_scale));
  MISA_TRY(check_cache(&p->cache));
  if (p->cache.d != kLatent || p->cache.dr != kRotary)
    return fail(MISA_ERR_UNSUPPORTED, "latent attention reads rows of d = 512, dr = 64 (got %d, %d)", p->cache.d, p->cache.dr);
  if (p->k > (1 << 30)) return fail(MISA_ERR_UNSUPPORTED, "k = %d exceeds 2^30", p->k);
  if (p->T > 0 && (p->idx ? p->k < 1 : p->k != 0))
    return fail(MISA_ERR_INVALID_ARG, "k = %d must be >= 1 with idx and 0 without", p->k);
  return MISA_OK;
}

static AttnPlan plan_of(const misa_latent_problem* p) {
  const bool lists = p->idx != nullptr;
  return latent_plan(p->T, p->H, lists ? p->k : p->cache.rows, !lists && !p->base);
}

static misa_status check_expanded(const misa_expanded_problem* p) {
  if (!p) return fail(MISA_ERR_INVALID_ARG, "problem is NULL");
  MISA_TRY(check_sizes(p->T, p->H, p->sm_scale));
  if (p->L < 1) return fail(MISA_ERR_INVALID_ARG, "L = %d must be >= 1", p->L);
  if (p->H > (1 << 20)) return fail(MISA_ERR_UNSUPPORTED, "H = %d exceeds 2^20 heads", p->H);
  if (p->rope_ld > (1 << 24)) return fail(MISA_ERR_UNSUPPORTED, "rope_ld = %lld exceeds 2^24", (long long)p->rope_ld);
  if (p->L > (1 << 30)) return fail(MISA_ERR_UNSUPPORTED, "L = %d exceeds 2^30 keys", p->L);
  if (p->rope_ld < kRotary || p->rope_ld % 8 != 0)
    return fail(MISA_ERR_INVALID_ARG, "rope_ld = %lld must be a multiple of 8 and >= 64", (long long)p->rope_ld);
  return MISA_OK;
}

static misa_status check_scratch(size_t need, void* ws, size_t ws_bytes) {
  if (ws_bytes < need)
    return fail(MISA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", ws_bytes, need);
  if (!ws) return fail(MISA_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(MISA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return MISA_OK;
}

}  // namespace misa

using namespace misa;

extern "C" {

misa_status misa_cache_write(const misa_cache* cache, const void* x, int32_t n, const int32_t* slots, void* stream) {
  MISA_TRY(check_cache(cache));
  if (n < 0) return fail(MISA_ERR_INVALID_ARG, "n = %d is negative", n);
  if (n > (1 << 25)) return fail(MISA_ERR_UNSUPPORTED, "n = %d exceeds 2^25 rows", n);
  if (n == 0) return MISA_OK;
  MISA_TRY(check_ptr(x, "x", 16));
  MISA_TRY(check_ptr(slots, "slots", 4));
  const LaunchCtx cx{static_cast<hipStream_t>(stream)};
  HIP_TRY(launch_cache_write(cx, cache_args(cache, n, slots), cache->dtype == MISA_K_FP8_E4M3FN,
                             static_cast<const uint16_t*>(x)),
          "cache write");
  return MISA_OK;
}

misa_status misa_cache_read(const misa_cache* cache, const int32_t* slots, int32_t n, void* out, void* stream) {
  MISA_TRY(check_cache(cache));
  if (n < 0) return fail(MISA_ERR_INVALID_ARG, "n = %d is negative", n);
  if (n > (1 << 25)) return fail(MISA_ERR_UNSUPPORTED, "n = %d exceeds 2^25 rows", n);
  if (n == 0) return MISA_OK;
  MISA_TRY(check_ptr(out, "out", 16));
  MISA_TRY(check_ptr(slots, "slots", 4));
  const LaunchCtx cx{static_cast<hipStream_t>(stream)};
  HIP_TRY(launch_cache_read(cx, cache_args(cache, n, slots), cache->dtype == MISA_K_FP8_E4M3FN,
                            static_cast<uint16_t*>(out)),
          "cache read");
  return MISA_OK;
}

size_t misa_latent_workspace_bytes(const misa_latent_problem* p) {
  if (check_latent(p) != MISA_OK) return 0;
  return p->T == 0 ? 256 : latent_ws_bytes(plan_of(p), p->T, p->H);
}

misa_status misa_latent_attention(const misa_latent_problem* p, void* out, float* lse, void* ws, size_t ws_bytes,
                                  void* stream) {
  MISA_TRY(check_latent(p));
  if (p->T == 0) return MISA_OK;
  MISA_TRY(check_ptr(p->q, "q", 16));
  if (p->idx) {
    MISA_TRY(check_ptr(p->idx, "idx", 4));
    if (p->pos) return fail(MISA_ERR_INVALID_ARG, "pos must be NULL with idx (the list names the keys)");
  } else {
    MISA_TRY(check_ptr(p->pos, "pos", 4));
  }
  if (p->base) MISA_TRY(check_ptr(p->base, "base", 4));
  MISA_TRY(check_ptr(out, "out", 16));
  if (lse) MISA_TRY(check_ptr(lse, "lse", 4));
  const AttnPlan pl = plan_of(p);
  MISA_TRY(check_scratch(latent_ws_bytes(pl, p->T, p->H), ws, ws_bytes));
  LatentArgs a{};
  a.q = static_cast<const uint16_t*>(p->q);
  a.T = p->T;
  a.H = p->H;
  a.c = p->cache.c;
  a.scale = p->cache.scale;
  a.rope = static_cast<const uint16_t*>(p->cache.rope);
  a.rows = p->cache.rows;
  a.pos = p->pos;
  a.idx = p->idx;
  a.k = p->k;
  a.base = p->base;
  a.sm_log2 = p->sm_scale * kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  const LaunchCtx cx{static_cast<hipStream_t>(stream)};
  HIP_TRY(launch_latent(cx, a, pl, p->cache.dtype == MISA_K_FP8_E4M3FN, ws), "latent attention");
  return MISA_OK;
}

size_t misa_expanded_workspace_bytes(const misa_expanded_problem* p) {
  if (check_expanded(p) != MISA_OK) return 0;
  return p->T == 0 ? 256 : expanded_ws_bytes(expanded_plan(p->T, p->H, p->L), p->T, p->H);
}

misa_status misa_expanded_attention(const misa_expanded_problem* p, void* out, float* lse, void* ws, size_t ws_bytes,
                                    void* stream) {
  MISA_TRY(check_expanded(p));
  if (p->T == 0) return MISA_OK;
  MISA_TRY(check_ptr(p->q, "q", 16));
  MISA_TRY(check_ptr(p->kv, "kv", 16));
  MISA_TRY(check_ptr(p->rope, "rope", 16));
  MISA_TRY(check_ptr(p->pos, "pos", 4));
  if (p->base) MISA_TRY(check_ptr(p->base, "base", 4));
  MISA_TRY(check_ptr(out, "out", 16));
  if (lse) MISA_TRY(check_ptr(lse, "lse", 4));
  const AttnPlan pl = expanded_plan(p->T, p->H, p->L);
  MISA_TRY(check_scratch(expanded_ws_bytes(pl, p->T, p->H), ws, ws_bytes));
  ExpandedArgs a{};
  a.q = static_cast<const uint16_t*>(p->q);
  a.kv = static_cast<const uint16_t*>(p->kv);
  a.rope = static_cast<const uint16_t*>(p->rope);
  a.rope_ld = p->rope_ld;
  a.T = p->T;
  a.H = p->H;
  a.L = p->L;
  a.pos = p->pos;
  a.base = p->base;
  a.sm_log2 = p->sm_scale * kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  const LaunchCtx cx{static_cast<hipStream_t>(stream)};
  HIP_TRY(launch_expanded(cx, a, pl, ws), "expanded attention");
  return MISA_OK;
}

}  // extern "C"
