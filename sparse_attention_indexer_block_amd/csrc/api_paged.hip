// C ABI of the norm, of paged caches and of the attention of drafted tokens:
// argument checks, workspaces and launches.
#include <hip/hip_runtime.h>

#include "api_checks.h"

namespace misa {

constexpr int64_t kMaxPositions = (int64_t)1 << 28;  // of one sequence
// A launch holds fewer than 2^32 threads: eight a rotated row; 64 a normed row of up to 512
// values (2^25 rows at most), at most one for four values of a wider one.
constexpr int64_t kMaxTurned = (int64_t)1 << 28;
constexpr int64_t kMaxValues = (int64_t)1 << 33;

static misa_status check_ld(int64_t ld, int64_t least, const char* name) {
  if (ld < least || ld % 8 != 0)
    return fail(MISA_ERR_INVALID_ARG, "%s = %lld must be a multiple of 8 and >= %lld", name, (long long)ld, (long long)least);
  if (ld > ((int64_t)1 << 40)) return fail(MISA_ERR_UNSUPPORTED, "%s = %lld exceeds 2^40", name, (long long)ld);
  return MISA_OK;
}

static misa_status check_weight(const void* weight, int32_t w_dtype, double eps) {
  MISA_TRY(check_ptr(weight, "weight", 16));
  if (w_dtype != MISA_W_BF16 && w_dtype != MISA_W_F32)
    return fail(MISA_ERR_INVALID_ARG, "w_dtype = %d is not a misa_wdtype", w_dtype);
  if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(MISA_ERR_INVALID_ARG, "eps = %g must be finite and >= 0", eps);
  return MISA_OK;
}

static misa_status check_rotation(const misa_rotation* r) {
  MISA_TRY(check_ptr(r->rot, "rot", 16));
  if (r->positions < 1) return fail(MISA_ERR_INVALID_ARG, "positions = %d must be >= 1", r->positions);
  if (r->pairs != 0 && r->pairs != 1) return fail(MISA_ERR_INVALID_ARG, "pairs = %d is neither 0 nor 1", r->pairs);
  return MISA_OK;
}

static Rotation rotation_args(const misa_rotation& r) { return Rotation{r.rot, r.positions, r.pairs != 0}; }

static misa_status check_pages(const misa_pages* p) {
  if (p->seqs < 0) return fail(MISA_ERR_INVALID_ARG, "seqs = %d is negative", p->seqs);
  if (p->per < 1) return fail(MISA_ERR_INVALID_ARG, "per = %d must be >= 1", p->per);
  if (p->page < 1 || (p->page & (p->page - 1)) != 0)
    return fail(MISA_ERR_INVALID_ARG, "page = %d must be a power of two", p->page);
  if (p->seqs > (1 << 22)) return fail(MISA_ERR_UNSUPPORTED, "seqs = %d exceeds 2^22", p->seqs);
  if ((int64_t)p->per * p->page > kMaxPositions)
    return fail(MISA_ERR_UNSUPPORTED, "per * page = %lld exceeds 2^28 positions", (long long)p->per * p->page);
  return MISA_OK;
}

static Pages pages_args(const misa_pages& p) { return Pages{p.table, p.seqs, p.per, __builtin_ctz((unsigned)p.page)}; }

static misa_status check_append(const misa_append_problem* p) {
  if (!p) return fail(MISA_ERR_INVALID_ARG, "problem is NULL");
  MISA_TRY(check_cache(&p->cache));
  MISA_TRY(check_pages(&p->pages));
  if (p->n < 0) return fail(MISA_ERR_INVALID_ARG, "n = %d is negative", p->n);
  if (p->n > (1 << 25)) return fail(MISA_ERR_UNSUPPORTED, "n = %d exceeds 2^25 rows", p->n);
  MISA_TRY(check_ld(p->x_ld, p->cache.d + p->cache.dr, "x_ld"));
  if (p->weight) MISA_TRY(check_weight(p->weight, p->w_dtype, p->eps));
  if (p->rotation.rot) {
    MISA_TRY(check_rotation(&p->rotation));
    const int at = p->rot_at, d = p->cache.d;
    if (p->cache.dr ? at != d : at < 0 || at % kRotary != 0 || at + kRotary > d)
      return fail(MISA_ERR_INVALID_ARG, "rot_at = %d must be %s", at,
                  p->cache.dr ? "d, where the rotary columns begin" : "a multiple of 64 inside the row");
  } else if (p->turn) {
    return fail(MISA_ERR_INVALID_ARG, "turn must be NULL without rot");
  }
  return MISA_OK;
}

static misa_status check_tree(const misa_tree_problem* p) {
  if (!p) return fail(MISA_ERR_INVALID_ARG, "problem is NULL");
  MISA_TRY(check_pages(&p->pages));
  if (p->N < 1) return fail(MISA_ERR_INVALID_ARG, "N = %d must be >= 1", p->N);
  if (p->N > (1 << 16)) return fail(MISA_ERR_UNSUPPORTED, "N = %d exceeds 2^16 nodes", p->N);
  if ((int64_t)p->pages.seqs * p->N > (1 << 22))
    return fail(MISA_ERR_UNSUPPORTED, "seqs * N = %lld exceeds 2^22 queries", (long long)p->pages.seqs * p->N);
  MISA_TRY(check_sizes(p->pages.seqs * p->N, p->H, p->sm_scale));
  MISA_TRY(check_cache(&p->cache));
  if (p->cache.d != kLatent || p->cache.dr != kRotary)
    return fail(MISA_ERR_UNSUPPORTED, "latent attention reads rows of d = 512, dr = 64 (got %d, %d)", p->cache.d, p->cache.dr);
  const bool some = p->pages.seqs > 0;  // (empty batches have empty arrays)
  if (some && (p->mask ? p->words < 1 : p->words != 0))
    return fail(MISA_ERR_INVALID_ARG, "words = %d must be >= 1 with mask and 0 without", p->words);
  if (p->words > 1024) return fail(MISA_ERR_UNSUPPORTED, "words = %d exceeds 1024", p->words);
  if (some && p->mask && p->words < (p->N + 63) / 64)  // (a node past the last word could not name itself)
    return fail(MISA_ERR_INVALID_ARG, "words = %d must be >= %d for %d nodes", p->words, (p->N + 63) / 64, p->N);
  if (some && (p->idx ? p->k < 1 : p->k != 0))
    return fail(MISA_ERR_INVALID_ARG, "k = %d must be >= 1 with idx and 0 without", p->k);
  if (p->k > (1 << 24)) return fail(MISA_ERR_UNSUPPORTED, "k = %d exceeds 2^24", p->k);
  if (p->longest < 0) return fail(MISA_ERR_INVALID_ARG, "longest = %d is negative", p->longest);
  return MISA_OK;
}

static int words_of(const misa_tree_problem* p) { return p->mask ? p->words : (p->N + 63) / 64; }
static int list_len(const misa_tree_problem* p) { return p->k + 64 * words_of(p); }
static size_t list_bytes(const misa_tree_problem* p) {
  return ((size_t)p->pages.seqs * p->N * list_len(p) * 4 + 255) / 256 * 256;
}
static misa_status check_lists(const misa_tree_problem* p) {
  if (p->idx && (int64_t)p->pages.seqs * p->N * list_len(p) > ((int64_t)1 << 31))
    return fail(MISA_ERR_UNSUPPORTED, "seqs * N * (k + 64 words) exceeds 2^31 entries");
  return MISA_OK;
}
static AttnPlan list_plan(const misa_tree_problem* p) {
  return latent_plan(p->pages.seqs * p->N, p->H, list_len(p), false);
}
static TreePlan plan_of(const misa_tree_problem* p) {
  const int all = p->pages.per * p->pages.page;
  return tree_plan(p->pages.seqs, p->N, p->H, words_of(p), p->longest > 0 && p->longest < all ? p->longest : all);
}
static size_t need_of(const misa_tree_problem* p) {
  if (p->pages.seqs == 0) return 256;
  if (p->idx) return list_bytes(p) + latent_ws_bytes(list_plan(p), p->pages.seqs * p->N, p->H);
  return tree_ws_bytes(plan_of(p), p->pages.seqs);
}

}  // namespace misa

using namespace misa;

extern "C" {

misa_status misa_rms_norm(const misa_norm_problem* p, void* y, float* scale, void* sum, void* stream) {
  if (!p) return fail(MISA_ERR_INVALID_ARG, "problem is NULL");
  if (p->n < 0) return fail(MISA_ERR_INVALID_ARG, "n = %d is negative", p->n);
  if (p->n > (1 << 25)) return fail(MISA_ERR_UNSUPPORTED, "n = %d exceeds 2^25 rows", p->n);
  if (p->width < 8 || p->width % 8 != 0) return fail(MISA_ERR_INVALID_ARG, "width = %d must be a multiple of 8", p->width);
  if (p->width > 16384) return fail(MISA_ERR_UNSUPPORTED, "width = %d exceeds 16384", p->width);
  if ((int64_t)p->n * p->width > kMaxValues)
    return fail(MISA_ERR_UNSUPPORTED, "n * width = %lld exceeds 2^33 values", (long long)p->n * p->width);
  if (p->dtype != MISA_K_BF16 && p->dtype != MISA_K_FP8_E4M3FN)
    return fail(MISA_ERR_INVALID_ARG, "dtype = %d is not a misa_kdtype", p->dtype);
  const bool fp8 = p->dtype == MISA_K_FP8_E4M3FN;
  if (p->group != 0 && (p->group != 128 || !fp8))
    return fail(MISA_ERR_INVALID_ARG, "group = %d must be 0 (a scale a row) or, for codes, 128", p->group);
  MISA_TRY(check_ld(p->x_ld, p->width, "x_ld"));
  MISA_TRY(check_weight(p->weight, p->w_dtype, p->eps));
  if (!fp8 && scale) return fail(MISA_ERR_INVALID_ARG, "scale must be NULL for a bf16 result");
  if (!p->residual && sum) return fail(MISA_ERR_INVALID_ARG, "sum must be NULL without residual");
  if (p->n == 0) return MISA_OK;
  MISA_TRY(check_ptr(p->x, "x", 16));
  if (p->residual) MISA_TRY(check_ptr(p->residual, "residual", 16));
  MISA_TRY(check_ptr(y, "y", 16));
  if (fp8) MISA_TRY(check_ptr(scale, "scale", 4));
  if (sum) MISA_TRY(check_ptr(sum, "sum", 16));
  NormArgs a{};
  a.n = p->n;
  a.width = p->width;
  a.x = static_cast<const uint16_t*>(p->x);
  a.x_ld = p->x_ld;
  a.residual = static_cast<const uint16_t*>(p->residual);
  a.weight = p->weight;
  a.weight_f32 = p->w_dtype == MISA_W_F32;
  a.eps = p->eps;
  a.y = y;
  a.scale = scale;
  a.sum = static_cast<uint16_t*>(sum);
  const LaunchCtx cx{static_cast<hipStream_t>(stream)};
  HIP_TRY(launch_rms_norm(cx, a, !fp8 ? NormOut::kBf16 : p->group ? NormOut::kGroupCodes : NormOut::kRowCodes), "norm");
  return MISA_OK;
}

misa_status misa_rotate(const misa_rotate_problem* p, void* out, int64_t out_t, int64_t out_h, void* stream) {
  if (!p) return fail(MISA_ERR_INVALID_ARG, "problem is NULL");
  MISA_TRY(check_sizes(p->T, p->H, 0.f));
  if ((int64_t)p->T * p->H > kMaxTurned)
    return fail(MISA_ERR_UNSUPPORTED, "T * H = %lld exceeds 2^28", (long long)p->T * p->H);
  MISA_TRY(check_rotation(&p->rotation));
  MISA_TRY(check_ld(p->x_h, kRotary, "x_h"));
  MISA_TRY(check_ld(p->x_t, kRotary, "x_t"));
  MISA_TRY(check_ld(out_h, kRotary, "out_h"));
  MISA_TRY(check_ld(out_t, kRotary, "out_t"));
  if (p->T == 0) return MISA_OK;
  MISA_TRY(check_ptr(p->x, "x", 16));
  MISA_TRY(check_ptr(p->pos, "pos", 4));
  MISA_TRY(check_ptr(out, "out", 16));
  RotateArgs a{};
  a.T = p->T;
  a.H = p->H;
  a.x = static_cast<const uint16_t*>(p->x);
  a.x_t = p->x_t;
  a.x_h = p->x_h;
  a.out = static_cast<uint16_t*>(out);
  a.out_t = out_t;
  a.out_h = out_h;
  a.pos = p->pos;
  a.rot = rotation_args(p->rotation);
  const LaunchCtx cx{static_cast<hipStream_t>(stream)};
  HIP_TRY(launch_rotate(cx, a), "rotation");
  return MISA_OK;
}

misa_status misa_paged_append(const misa_append_problem* p, void* stream) {
  MISA_TRY(check_append(p));
  if (p->n == 0 || p->pages.seqs == 0) return MISA_OK;
  MISA_TRY(check_ptr(p->x, "x", 16));
  MISA_TRY(check_ptr(p->seq, "seq", 4));
  MISA_TRY(check_ptr(p->pos, "pos", 4));
  if (p->turn) MISA_TRY(check_ptr(p->turn, "turn", 4));
  MISA_TRY(check_ptr(p->pages.table, "table", 4));
  AppendArgs a{};
  a.cache = cache_args(&p->cache, p->n, nullptr);
  a.pages = pages_args(p->pages);
  a.x = static_cast<const uint16_t*>(p->x);
  a.x_ld = p->x_ld;
  a.seq = p->seq;
  a.pos = p->pos;
  a.turn = p->turn ? p->turn : p->pos;
  a.weight = p->weight;
  a.weight_f32 = p->w_dtype == MISA_W_F32;
  a.eps = p->eps;
  if (p->rotation.rot) a.rot = rotation_args(p->rotation);
  a.rot_at = p->rot_at;
  const LaunchCtx cx{static_cast<hipStream_t>(stream)};
  HIP_TRY(launch_paged_append(cx, a, p->cache.dtype == MISA_K_FP8_E4M3FN), "paged append");
  return MISA_OK;
}

size_t misa_tree_workspace_bytes(const misa_tree_problem* p) {
  if (check_tree(p) != MISA_OK || check_lists(p) != MISA_OK) return 0;
  return need_of(p);
}

misa_status misa_tree_attention(const misa_tree_problem* p, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  MISA_TRY(check_tree(p));
  MISA_TRY(check_lists(p));
  if (p->pages.seqs == 0) return MISA_OK;
  MISA_TRY(check_ptr(p->q, "q", 16));
  MISA_TRY(check_ptr(p->prefix, "prefix", 4));
  MISA_TRY(check_ptr(p->pages.table, "table", 4));
  if (p->mask) MISA_TRY(check_ptr(p->mask, "mask", 8));
  if (p->idx) MISA_TRY(check_ptr(p->idx, "idx", 4));
  MISA_TRY(check_ptr(out, "out", 16));
  if (lse) MISA_TRY(check_ptr(lse, "lse", 4));
  MISA_TRY(check_scratch(need_of(p), ws, ws_bytes));
  TreeArgs a{};
  a.q = static_cast<const uint16_t*>(p->q);
  a.T = p->pages.seqs * p->N;
  a.H = p->H;
  a.c = p->cache.c;
  a.scale = p->cache.scale;
  a.rope = static_cast<const uint16_t*>(p->cache.rope);
  a.rows = p->cache.rows;
  a.idx = p->idx;
  a.k = p->k;
  a.sm_log2 = p->sm_scale * kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.pages = pages_args(p->pages);
  a.N = p->N;
  a.words = words_of(p);
  a.prefix = p->prefix;
  a.mask = reinterpret_cast<const uint64_t*>(p->mask);
  const LaunchCtx cx{static_cast<hipStream_t>(stream)};
  const bool fp8 = p->cache.dtype == MISA_K_FP8_E4M3FN;
  if (!p->idx) {
    HIP_TRY(launch_tree(cx, a, plan_of(p), fp8, ws), "tree attention");
    return MISA_OK;
  }
  // the keys of each query as rows of the cache, then the attention over lists
  int32_t* lists = static_cast<int32_t*>(ws);
  HIP_TRY(launch_tree_lists(cx, a, lists), "tree attention's lists");
  LatentArgs l = a;
  l.idx = lists;
  l.k = list_len(p);
  HIP_TRY(launch_latent(cx, l, list_plan(p), fp8, static_cast<char*>(ws) + list_bytes(p)), "tree attention");
  return MISA_OK;
}

}  // extern "C"
