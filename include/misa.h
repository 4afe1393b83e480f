/*
 * misa.h - C ABI of the MI355X (gfx950) lightning-indexer library.
 *
 * The library computes, on one GPU, the token selection that a DeepSeek
 * sparse-attention indexer hands to sparse attention, in the three forms the
 * MISA and HISA write-ups describe:
 *
 *   misa_route      block-mean router: pick A of the H indexer heads per query
 *                   (MISA technical summary, "Metodologia: MISA", first stage).
 *   misa_score_topk routed heads score every visible key, then top-k
 *                   (same section, second stage "sparse token scoring").
 *   misa_hier_topk  routed pass keeps k' candidates, all H heads rescore them,
 *                   then top-k (MISA technical summary, "Variante Jerarquica").
 *   hisa_topk       top-m key blocks by their mean-pooled representative, then
 *                   the full indexer on the tokens of those blocks, then top-k
 *                   (HISA write-up, section 3, Stage 1 and Stage 2).
 *   hisa_maxpool_topk  HISA with max-pooled block representatives (HISA
 *                   write-up, limitations).
 *   misa_hisa_topk  HISA with the routed heads in both stages: the head axis
 *                   of MISA and the token axis of HISA combined.
 *   misa_block_means  the query-independent block means the router pools.
 *
 * Around the selection it keeps the caches that it and its consumer read, and
 * computes the attention that consumes it:
 *
 *   misa_cache_write, misa_cache_read  rows of indexer keys or of latents,
 *                   coded as they are written, and read back.
 *   misa_latent_attention    attention over one shared latent vector a token
 *                   (absorbed form), on the selected or on all visible keys.
 *   misa_expanded_attention  the same attention over per-head keys and values
 *                   expanded from the latents.
 *   misa_paged_append  rows of latents or indexer keys into the pages of their
 *                   sequences, normed, rotated by position and coded on the way.
 *   misa_rotate     the same rotation of queries.
 *   misa_tree_attention  latent attention of drafted tokens (a tree of them, a
 *                   chain, or one) over a paged cache.
 *   misa_rms_norm   the norm before a layer, with the residual's addition and a
 *                   result in bf16 or coded.
 *
 * Definitions (the pages give the structure; the exact formulas are fixed here):
 *   z(t,h,s)  = q[t,h,:] . k[s,:]
 *   I_S(t,s)  = sum_{h in S} w[t,h] * max(0, z(t,h,s))        (no renormalisation)
 *   visible   : key s is visible to query t iff s <= pos[t]; n_t = pos[t]+1
 *   blocks    : M_t = ceil(n_t/B); block b = [b*B, min((b+1)*B, n_t)); its
 *               representative Kbar_{t,b} is the mean of those keys (so the
 *               last block of a query may be partial)
 *   router    : r(t,h) = w[t,h] * max_b max(0, q[t,h] . Kbar_{t,b}); keep the
 *               first A heads under (-r, h)
 *   HISA block score: beta(t,b) = sum_h w[t,h] * max(0, q[t,h] . Kbar_{t,b})
 *   selection : the first min(k, count) items under (-score, index); -0.0 == +0.0
 *
 * Conventions shared by every entry point:
 *   - Every array argument is caller-owned, contiguous, row-major DEVICE memory;
 *     the struct misa_problem itself lives in host memory. The library never
 *     allocates or frees device memory: scratch comes from the caller's
 *     workspace `ws` of `ws_bytes` bytes (size it with misa_workspace_bytes,
 *     the attention's with misa_latent_workspace_bytes,
 *     misa_expanded_workspace_bytes and misa_tree_workspace_bytes; 256-byte
 *     alignment is required). Outputs and workspace must not overlap each other
 *     or an input.
 *   - `stream` is a hipStream_t (NULL = the legacy default stream). Calls only
 *     enqueue work and return; they never synchronise the host.
 *   - Argument errors are reported synchronously, before anything is enqueued,
 *     and leave every output untouched. MISA_ERR_HIP reports a failed launch.
 *   - Outputs: idx[T,k] int32 and scores[T,k] float32. Row t holds its
 *     k_t = min(k, count) selected keys in ascending key order, followed by
 *     k - k_t padding entries (idx = -1, score = -inf).
 *   - pos values outside [0, L) are clamped: pos < 0 gives a row with no
 *     visible key (all padding), pos >= L behaves as pos = L-1.
 *   - Supported on the GPU: d = 128; 1 <= H <= 64; 1 <= A <= H; B >= 1;
 *     q bf16, or OCP E4M3FN codes with a per-(query, head) fp32 scale;
 *     K bf16 or OCP E4M3FN with a per-token fp32 scale (any finite scale
 *     value; the sign of a negative scale is honoured).
 *   - fp8 queries (q_dtype MISA_Q_FP8_E4M3FN) need fp8 keys (the contraction
 *     runs on fp8 x fp8 matrix cores) and decode-shaped batches wherever heads
 *     are routed or keys are scored over the whole prefix (misa_route,
 *     misa_score_topk, misa_hier_topk, misa_hisa_topk: T * A' <= 256 with A'
 *     = A rounded up to a power of two >= 4, and the few-query router);
 *     hisa_topk and hisa_maxpool_topk take any T. Otherwise
 *     MISA_ERR_UNSUPPORTED.
 *   - Calls that share a workspace must be ordered on one stream; otherwise the
 *     library is stateless and reentrant.
 */
#ifndef MISA_H
#define MISA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum misa_status {
  MISA_OK = 0,
  MISA_ERR_INVALID_ARG = -1, /* null pointer, negative size, A > H, k' < k ... */
  MISA_ERR_UNSUPPORTED = -2, /* valid request outside what the kernels support (d != 128, H > 64) */
  MISA_ERR_WORKSPACE = -3,   /* ws too small or misaligned */
  MISA_ERR_HIP = -4          /* a HIP launch or runtime call failed */
} misa_status;

typedef enum misa_kdtype {
  MISA_K_BF16 = 0,        /* K[L,d] as bf16 bit patterns (uint16) */
  MISA_K_FP8_E4M3FN = 1   /* K[L,d] as OCP E4M3FN bytes; value = code * k_scale[s] */
} misa_kdtype;

typedef enum misa_qdtype {
  MISA_Q_BF16 = 0,        /* q[T,H,d] as bf16 bit patterns (uint16) */
  MISA_Q_FP8_E4M3FN = 1   /* q[T,H,d] as OCP E4M3FN bytes; value = code * q_scale[t,h] */
} misa_qdtype;

typedef enum misa_op {
  MISA_OP_ROUTE = 0,
  MISA_OP_SCORE_TOPK = 1,
  MISA_OP_HIER_TOPK = 2,
  MISA_OP_HISA_TOPK = 3,
  MISA_OP_BLOCK_MEANS = 4,
  MISA_OP_MISA_HISA_TOPK = 5,
  MISA_OP_BLOCK_SCORES = 6
} misa_op;

/* One indexer problem. All pointers are device pointers. */
typedef struct misa_problem {
  int32_t T;               /* queries (>= 0; T == 0 is a no-op) */
  int32_t H;               /* indexer heads per query */
  int32_t d;               /* head dim (128) */
  int32_t L;               /* keys (>= 1) */
  int32_t B;               /* block size of the router / HISA blocks (>= 1) */
  int32_t k_dtype;         /* misa_kdtype */
  const void* q;           /* [T,H,d] bf16 bits, or E4M3FN bytes (q_dtype) */
  const float* w;          /* [T,H]   per-query head weights */
  const void* K;           /* [L,d]   shared indexer keys (bf16 bits or e4m3fn bytes) */
  const float* k_scale;    /* [L]     per-token scale, required iff k_dtype is fp8, else NULL */
  const int32_t* pos;      /* [T]     causal position of each query */
  const float* kbar;       /* [ceil(L/B),d] cached block means, or NULL (see below) */
  int32_t q_dtype;         /* misa_qdtype (MISA_Q_BF16 for bf16 queries) */
  const float* q_scale;    /* [T,H]   per-(query, head) scale, required iff q_dtype is fp8, else NULL */
} misa_problem;

/* Cached block means (kbar). When p->kbar is NULL every call pools the keys
 * itself. When it is set, row b of kbar stands for the mean of block b
 * wherever block b is a complete block before a query's own last block
 * (b < M_t - 1); each query's last block is always pooled from K, since it
 * depends on pos[t]. The library trusts the values: results are those of the
 * definitions evaluated with these means, which is what misa_block_means
 * writes. Pointer must be 16-byte aligned. Used by misa_route,
 * misa_score_topk, misa_hier_topk, hisa_topk and misa_hisa_topk; misa_block_means
 * ignores it. */

/* Bytes of workspace entry point `op` needs for this problem and these
 * parameters (unused parameters are ignored). Returns 0 for an invalid request;
 * a valid request always needs at least 256 bytes. */
size_t misa_workspace_bytes(const misa_problem* p, int32_t op, int32_t A, int32_t kprime,
                            int32_t k, int32_t m);

/* Full-block means of the whole key array (MISA summary, "Metodologia: MISA":
 * the router pools keys block by block; HISA Stage 1 pools each block by its mean).
 * kbar[ceil(L/B), d] float32: row b is the mean of keys [b*B, min((b+1)*B, L)),
 * accumulated in float64 and rounded once. q, w and pos are not read. */
misa_status misa_block_means(const misa_problem* p, float* kbar, void* ws, size_t ws_bytes,
                             void* stream);

/* Incremental form of misa_block_means for a growing key array (the cached
 * block statistics the MISA summary's "Metodologia: MISA" presumes when it
 * calls the router's cost negligible): with p->L the new length, rows
 * first_block .. ceil(L/B) - 1 of kbar are recomputed exactly as
 * misa_block_means computes them, and only those blocks' keys are read; the
 * rows before first_block are left as they are. After keys [L_old, L) were
 * appended, first_block = L_old / B brings kbar up to date. first_block must
 * lie in [0, ceil(L/B)] (MISA_ERR_INVALID_ARG otherwise; ceil(L/B) is a no-op);
 * the workspace is that of misa_block_means. */
misa_status misa_block_means_update(const misa_problem* p, int32_t first_block, float* kbar, void* ws,
                                    size_t ws_bytes, void* stream);

/* Router (MISA summary, "Metodologia: MISA", block-pooled router): heads[T,A]
 * int32 receives the routed heads of each query in ascending order; r[T,H]
 * float32 (may be NULL) receives r(t,h). The selection is taken in float64
 * from exact block sums, so it matches an exact evaluation except where two
 * heads' scores agree to float64 rounding. */
misa_status misa_route(const misa_problem* p, int32_t A, int32_t* heads, float* r, void* ws,
                       size_t ws_bytes, void* stream);

/* MISA selection (MISA summary, "Metodologia: MISA", sparse token scoring):
 * the A routed heads of each query score every visible key with I_R; the
 * top-k keys are returned. `heads` [T,A] may supply the routed heads (any
 * distinct values in [0,H)); NULL routes inside the call. A == H with
 * heads == NULL is the dense DSA indexer. scores[] hold I_R. */
misa_status misa_score_topk(const misa_problem* p, int32_t A, const int32_t* heads, int32_t k,
                            int32_t* idx, float* scores, void* ws, size_t ws_bytes, void* stream);

/* MISA-dagger (MISA summary, "Variante Jerarquica"): the routed pass keeps the
 * top-kprime keys by I_R, all H heads rescore those candidates with I_all and
 * the top-k of them are returned (scores hold I_all). Requires kprime >= k. */
misa_status misa_hier_topk(const misa_problem* p, int32_t A, const int32_t* heads, int32_t kprime,
                           int32_t k, int32_t* idx, float* scores, void* ws, size_t ws_bytes,
                           void* stream);

/* Size in bytes of the library's static device scratch (see
 * misa_hier_topk_noalloc). */
#define MISA_STATIC_SCRATCH_BYTES (32u << 20)

/* misa_hier_topk for callers that cannot allocate device memory: code being
 * captured into a HIP graph, tight serving loops, and harnesses that forbid
 * hipMalloc. Same arguments, results, validation and errors as
 * misa_hier_topk, except that there is no workspace argument: the scratch is
 * a static device array of MISA_STATIC_SCRATCH_BYTES bytes inside the library
 * (one copy per GPU, held from the library's first use on that GPU until the
 * process ends). The call allocates and frees nothing.
 *   - A problem whose scratch need (misa_workspace_bytes(p, MISA_OP_HIER_TOPK,
 *     A, kprime, k, 1)) exceeds MISA_STATIC_SCRATCH_BYTES is rejected with
 *     MISA_ERR_WORKSPACE before anything is enqueued (decode batches up to
 *     T = 16 queries over 131,072 keys fit).
 *   - Every call on one GPU shares that GPU's scratch and leaves its own
 *     contents there. Calls ordered on one stream are safe; calls that may
 *     overlap on one GPU (different streams, or threads enqueuing
 *     concurrently) race on the scratch and give undefined results.
 *   - The device is the calling thread's current device. */
misa_status misa_hier_topk_noalloc(const misa_problem* p, int32_t A, const int32_t* heads, int32_t kprime,
                                   int32_t k, int32_t* idx, float* scores, void* stream);

/* HISA (HISA write-up, section 3, Stage 1 and Stage 2): keep the top-m blocks
 * of each query by beta (ties to the lower block), score the visible tokens of
 * those blocks with all H heads (I_all) and return the top-k. */
misa_status hisa_topk(const misa_problem* p, int32_t m, int32_t k, int32_t* idx, float* scores,
                      void* ws, size_t ws_bytes, void* stream);

/* HISA Stage 1 block scores on their own (HISA write-up, section 3, Stage 1:
 * the query is scored against the block representatives only):
 *   beta[t * beta_ld + b] = sum_h w[t,h] * max(0, q[t,h] . Kbar_{t,b})
 * for every visible block b < M_t of query t, formed in float64 and rounded
 * once to float32; entries b >= M_t are not written. These are the values
 * hisa_topk ranks for its top-m blocks (same kernel, same bits). beta is
 * device memory [T, beta_ld] float32 with beta_ld >= ceil(L/B).
 * Workspace: misa_workspace_bytes(p, MISA_OP_BLOCK_SCORES, ...). Cached means
 * (p->kbar) are used as in hisa_topk. */
misa_status hisa_block_scores(const misa_problem* p, float* beta, int64_t beta_ld, void* ws,
                              size_t ws_bytes, void* stream);

/* HISA with max-pooled block representatives (HISA write-up, limitations:
 * max pooling in place of mean pooling, listed as a possible improvement).
 * As hisa_topk, except that the representative of block b of query t is, per
 * dimension, the largest of its visible keys' values (dequantised keys; the
 * tail block over [b*B, n_t) only), so that one key standing out in a block is
 * not averaged away. Workspace: misa_workspace_bytes(p, MISA_OP_HISA_TOPK, ., .,
 * k, m). p->kbar must be NULL (cached means do not apply); otherwise errors,
 * arguments and outputs as hisa_topk. */
misa_status hisa_maxpool_topk(const misa_problem* p, int32_t m, int32_t k, int32_t* idx, float* scores,
                              void* ws, size_t ws_bytes, void* stream);

/* MISA inside HISA. The MISA technical summary presents head routing as an
 * efficiency axis complementary to token-axis hierarchies such as HISA and
 * combinable with them ("Contribuciones Clave", "Significado y Afirmaciones");
 * the plain reading used here puts the A routed heads R_t (as misa_route picks
 * them) in place of all H heads in both HISA stages:
 *   beta_R(t,b) = sum_{h in R_t} w[t,h] * max(0, q[t,h] . Kbar_{t,b}),
 * the top-m blocks by beta_R (ties to the lower block), I_R on the visible
 * tokens of those blocks, and the top-k of those (scores hold I_R).
 * `heads` [T,A] may supply the routed heads (distinct values in [0,H)); NULL
 * routes inside the call. A == H with heads == NULL is hisa_topk. Errors as
 * for misa_score_topk and hisa_topk. */
misa_status misa_hisa_topk(const misa_problem* p, int32_t A, const int32_t* heads, int32_t m, int32_t k,
                           int32_t* idx, float* scores, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ caches
 *
 * A cache holds `rows` rows of d coded columns and dr rotary columns:
 *   indexer keys  d = 128, dr = 0   (misa_problem.K and k_scale read them)
 *   latents       d = 512, dr = 64  (misa_latent_attention reads them)
 * (d = 128 or 512 with dr = 0 or 64 are supported). dtype MISA_K_BF16: c is
 * [rows, d + dr] bf16 bits, scale and rope are NULL. dtype MISA_K_FP8_E4M3FN:
 * c is [rows, d] E4M3FN codes with value = code * scale[row], and rope is
 * [rows, dr] bf16 bits (NULL iff dr == 0). c and rope are 16-byte aligned. */
typedef struct misa_cache {
  int32_t rows;
  int32_t d;
  int32_t dr;
  int32_t dtype;  /* misa_kdtype */
  void* c;
  float* scale;
  void* rope;
} misa_cache;

/* Writes row i of x [n, d + dr] (bf16 bits) to row slots[i] of the cache, for
 * every i with 0 <= slots[i] < rows; other entries write nothing, and rows of
 * the cache that no slot names stay as they are. bf16 rows are copied. Coded
 * rows: with a = max |x[i, 0:d]|, scale = 2^e for the smallest e >= -126 with
 * a <= 448 * 2^e (1 if a == 0), code = x / scale rounded to nearest even; the
 * rotary columns are copied. A power-of-two scale leaves one rounding per
 * value, and code * scale is exact in bf16. A row with an infinity or NaN among
 * its d columns gets scale NaN and NaN codes. Slots >= 0 must be distinct:
 * a row named twice holds either row's values, possibly mixed. n == 0 is a no-op.
 * One scale serves all d columns: caches with a scale for each part of a row
 * (128 columns, say) are another format, which nothing here reads or writes.
 * Limits (MISA_ERR_UNSUPPORTED past them): 2^30 rows of cache, n <= 2^25. */
misa_status misa_cache_write(const misa_cache* cache, const void* x, int32_t n, const int32_t* slots, void* stream);

/* Reads row slots[i] of the cache into row i of out [n, d + dr] (bf16 bits):
 * code * scale formed in fp32 and rounded to bf16 (exact for the scales that
 * misa_cache_write writes); rotary columns and bf16 rows are copied. A slot
 * outside [0, rows) gives a row of zeros; a slot may occur more than once. */
misa_status misa_cache_read(const misa_cache* cache, const int32_t* slots, int32_t n, void* out, void* stream);

/* --------------------------------------------------------- latent attention
 *
 * Absorbed form: the cache row of a token holds its latent vector c (512) and
 * its rotary key (64), shared by all heads; q[t,h] holds the head's query taken
 * into the latent space (512) and its rotary part (64):
 *   S(t,h,s)  = sm_scale * (q[t,h,0:512] . c[s] + q[t,h,512:576] . rope[s])
 *   out[t,h]  = sum_s p(t,h,s) c[s],  p = softmax of S over the query's keys
 *   lse[t,h]  = log sum_s exp S(t,h,s)
 * The query's keys are, with b = base[t] (0 if base is NULL) the cache row where
 * its sequence begins,
 *   idx given:  rows b + idx[t,j], j < k, for idx[t,j] >= 0 (as the selection
 *               entry points write them: -1 is padding; an index that occurs
 *               twice counts twice; order does not matter). pos must be NULL.
 *   idx NULL:   rows b .. b + pos[t]; k must be 0.
 * Rows outside [0, rows) of the cache are no keys, and base[t] < 0 leaves no
 * key; what a row holds that is not a key of a query (infinities and NaN too)
 * has no effect on that query. A query without keys gets out = 0
 * and lse = -inf; one whose keys all score -inf gets out = NaN
 * (0 / 0) and lse = -inf. Scores, weights' totals and sums are held in fp32; a weight is
 * rounded to bf16 for its product with the values. The values are summed before
 * they are divided by the total, with weights below 2^32: where the keys of a query
 * times the largest magnitude of their values (of coded rows: 448 times the scale)
 * passes 2^96, sums may overflow. Results do not depend on
 * what else runs; the same call gives the same bits.
 * Limits (MISA_ERR_UNSUPPORTED past them): T <= 2^22, T * H <= 2^30, k <= 2^30. */
typedef struct misa_latent_problem {
  int32_t T;              /* queries (T == 0 is a no-op) */
  int32_t H;              /* heads per query, >= 1 */
  int32_t k;              /* entries of a query's list (idx), or 0 */
  float sm_scale;         /* softmax scale, at most 2.35e38 in magnitude (0 weighs all keys
                           * alike, but those that score -inf: they weigh 0 as ever) */
  const void* q;          /* [T,H,576] bf16 bits, 16-byte aligned */
  const int32_t* idx;     /* [T,k] or NULL */
  const int32_t* pos;     /* [T], required iff idx is NULL */
  const int32_t* base;    /* [T] or NULL */
  misa_cache cache;       /* d = 512, dr = 64 */
} misa_latent_problem;

/* Bytes of workspace a call needs (0 for an invalid request; at least 256).
 * q, pos and base's contents do not matter, but whether idx and base are NULL does. */
size_t misa_latent_workspace_bytes(const misa_latent_problem* p);

/* out [T,H,512] bf16 bits (16-byte aligned); lse [T,H] float32 or NULL. */
misa_status misa_latent_attention(const misa_latent_problem* p, void* out, float* lse, void* ws, size_t ws_bytes,
                                  void* stream);

/* Expanded form, for prompts: every head has its own key (128 values, then the
 * rotary key shared by the heads) and value (128):
 *   S(t,h,s)  = sm_scale * (q[t,h,0:128] . kv[s,h,0:128] + q[t,h,128:192] . rope[s])
 *   out[t,h]  = sum_s p(t,h,s) kv[s,h,128:256]
 * over the keys b .. b + pos[t] of query t that lie in [0, L), b = base[t] (0 if
 * base is NULL; b < 0 leaves no key): packed sequences have their own base each, pos < 0 marks a
 * padded row. Queries may come in any order; neighbours with overlapping keys
 * run fastest. Otherwise as misa_latent_attention.
 * Limits (MISA_ERR_UNSUPPORTED past them): T <= 2^22, T * H <= 2^30, H <= 2^20,
 * L <= 2^30, rope_ld <= 2^24. */
typedef struct misa_expanded_problem {
  int32_t T;
  int32_t H;
  int32_t L;              /* keys, >= 1 */
  float sm_scale;
  const void* q;          /* [T,H,192] bf16 bits */
  const void* kv;         /* [L,H,256] bf16 bits: key (without rotary part), value */
  const void* rope;       /* [L,64] bf16 bits, rows rope_ld elements apart */
  int64_t rope_ld;        /* >= 64, a multiple of 8 */
  const int32_t* pos;     /* [T] */
  const int32_t* base;    /* [T] or NULL */
} misa_expanded_problem;

size_t misa_expanded_workspace_bytes(const misa_expanded_problem* p);

/* out [T,H,128] bf16 bits (16-byte aligned); lse [T,H] float32 or NULL. */
misa_status misa_expanded_attention(const misa_expanded_problem* p, void* out, float* lse, void* ws, size_t ws_bytes,
                                    void* stream);

/* ------------------------------------------------------------ paged caches
 *
 * A misa_cache whose rows belong to pages of `page` rows each; a sequence's
 * positions lie in the pages that its row of the table names: position j of
 * sequence s is row table[s, j / page] * page + j % page. A page number below 0 or
 * whose row lies outside the cache is no page: its positions are not written and are
 * no keys. A page may belong to several sequences (a shared prompt).
 * Limits (MISA_ERR_UNSUPPORTED past them): 2^22 sequences, per * page <= 2^28. */
typedef struct misa_pages {
  const int32_t* table;   /* [seqs, per] */
  int32_t seqs;           /* sequences (0 is a no-op) */
  int32_t per;            /* pages of a sequence, >= 1 */
  int32_t page;           /* rows of a page, a power of two */
} misa_pages;

/* The rotation of 64 rotary values by a position: 32 pairs (a, b) become
 * (a cos - b sin, b cos + a sin) with the cosines and sines of the position's row
 * of rot; products and sums are formed in fp32. Values i and i + 32 are a pair, or
 * (pairs = 1) values 2i and 2i + 1; pair i turns by angle i either way. */
typedef struct misa_rotation {
  const float* rot;       /* [positions, 64]: 32 cosines, then 32 sines; 16-byte aligned; NULL: no rotation */
  int32_t positions;      /* >= 1 */
  int32_t pairs;          /* 0 or 1 */
} misa_rotation;

typedef enum misa_wdtype {
  MISA_W_BF16 = 0,
  MISA_W_F32 = 1
} misa_wdtype;

/* Appends row i of x to position pos[i] of sequence seq[i], on the way
 *   1. normed, if weight is given: v = v / sqrt(mean(v^2) + eps) * weight over the
 *      d coded columns (a latent's rotary values stay out of it),
 *   2. rotated, if rotation.rot is given, by position turn[i] (pos[i] if turn is
 *      NULL; a drafted token's place in the cache is not its place in the text):
 *      columns rot_at .. rot_at + 63, which are the rotary ones of caches that have
 *      them (rot_at = d) and any aligned 64 of those that do not (dr = 0; rot_at a
 *      multiple of 64),
 *   3. coded, if the cache holds codes, as misa_cache_write does, with the scale that
 *      the values of steps 1 and 2 call for.
 * Steps 1 and 2 are formed in fp32, and a value is rounded once, as it is stored.
 * The selections read a sequence's keys as a flat K[L,128]: indexer keys are selected from
 * where the pages of their sequence lie one after the other, and misa_cache_read reads them
 * from any pages.
 * A row whose seq lies outside [0, seqs), whose pos outside [0, per * page), whose
 * turn outside the rotation's positions (if it is rotated) or whose page is none
 * writes nothing. Rows must name distinct places: one named twice holds either row's
 * values, possibly mixed. n == 0 is a no-op. Limit: n <= 2^25. */
typedef struct misa_append_problem {
  int32_t n;
  const void* x;          /* rows of d + dr bf16 bits, x_ld elements apart; 16-byte aligned */
  int64_t x_ld;           /* >= d + dr, a multiple of 8 */
  const int32_t* seq;     /* [n] */
  const int32_t* pos;     /* [n] */
  const int32_t* turn;    /* [n] or NULL */
  const void* weight;     /* [d] or NULL; 16-byte aligned */
  int32_t w_dtype;        /* misa_wdtype */
  int32_t rot_at;
  double eps;             /* >= 0 */
  misa_rotation rotation;
  misa_pages pages;
  misa_cache cache;
} misa_append_problem;

misa_status misa_paged_append(const misa_append_problem* p, void* stream);

/* Rotates the 64 rotary values of H heads of T queries, query t by position pos[t]:
 * x and out are [T, H, 64] bf16 bits whose queries and heads are x_t and x_h (out_t
 * and out_h) elements apart (multiples of 8 that are at least 64; 16-byte aligned), so
 * that both may be columns of wider rows; no two rows of out may overlap. out may be x
 * itself, with its distances; otherwise they must not overlap. A query whose position
 * lies outside the rotation's is not written. Limits (MISA_ERR_UNSUPPORTED past them):
 * T <= 2^22, T * H <= 2^28. */
typedef struct misa_rotate_problem {
  int32_t T;
  int32_t H;
  const void* x;
  int64_t x_t, x_h;
  const int32_t* pos;     /* [T] */
  misa_rotation rotation;
} misa_rotate_problem;

misa_status misa_rotate(const misa_rotate_problem* p, void* out, int64_t out_t, int64_t out_h, void* stream);

/* Latent attention (absorbed form, formula and precision as misa_latent_attention) of
 * N drafted tokens in each of pages.seqs sequences over a paged latent cache. Node i of
 * sequence s is query s * N + i. Its keys are, with n = prefix[s] committed tokens
 * (at positions 0 .. n - 1; at most per * page),
 *   idx NULL:   positions 0 .. n - 1,
 *   idx given:  positions idx[s,i,j], j < k, with 0 <= idx[s,i,j] < n (a selection of
 *               the committed tokens; -1 is padding, what occurs twice counts twice),
 * and the drafted tokens that it sees, at positions n + b for the bits b of its mask
 * (bit b % 64 of word b / 64), which is to name the node itself and its ancestors; mask
 * NULL: nodes 0 .. i (a chain; N = 1 is a decode step). The drafted tokens' rows are
 * appended before. A query whose mask is 0 in every word is padding, and all queries of
 * a sequence with prefix < 0: they have no key (out = 0, lse = -inf), whatever q holds.
 * Positions past the table or in no page are no keys. What is not a key of a query has
 * no effect on it. Sequences may differ in length; the call is planned for a longest
 * prefix of `longest` (0: per * page), which may be exceeded: it decides how the call
 * is cut and never what it returns, to within rounding. Results do not depend on what
 * else runs, and the same call gives the same bits. The keys of up to 256 sequences are
 * split over the card by the sequences' lengths; past 256 every sequence is worked
 * whole, and a batch of few more, or of very unequal lengths, takes less time in two calls.
 * Limits (MISA_ERR_UNSUPPORTED past them): N <= 2^16, words <= 1024, seqs * N <= 2^22,
 * seqs * N * H <= 2^30, k <= 2^24, seqs * N * (k + 64 words) <= 2^31 with idx (words =
 * ceil(N / 64) where mask is NULL). */
typedef struct misa_tree_problem {
  int32_t N;              /* nodes a sequence, >= 1 */
  int32_t H;              /* heads, >= 1 */
  int32_t k;              /* entries of a query's list (idx), or 0 */
  int32_t words;          /* 64-bit words of a mask, >= ceil(N / 64), or 0 */
  float sm_scale;         /* as in misa_latent_problem */
  int32_t longest;        /* >= 0 */
  const void* q;          /* [seqs,N,H,576] bf16 bits, 16-byte aligned */
  const int32_t* prefix;  /* [seqs] */
  const int64_t* mask;    /* [seqs,N,words] or NULL; 8-byte aligned */
  const int32_t* idx;     /* [seqs,N,k] or NULL */
  misa_pages pages;
  misa_cache cache;       /* d = 512, dr = 64 */
} misa_tree_problem;

/* Bytes of workspace a call needs (0 for an invalid request; at least 256). Pointers'
 * contents do not matter, but whether idx and mask are NULL does. */
size_t misa_tree_workspace_bytes(const misa_tree_problem* p);

/* out [seqs,N,H,512] bf16 bits (16-byte aligned); lse [seqs,N,H] float32 or NULL. */
misa_status misa_tree_attention(const misa_tree_problem* p, void* out, float* lse, void* ws, size_t ws_bytes,
                                void* stream);

/* -------------------------------------------------------------------- norm
 *
 * Root-mean-square norm of n rows, with a residual added before it:
 *   h = x + residual (x without one),  sum = h,  y = h / sqrt(mean(h^2) + eps) * weight
 * h and y are formed in fp32 (a sum past its range is infinite), the mean square in
 * fp64, its reciprocal root in fp32 (infinite where mean(h^2) + eps is below 2^-256),
 * and each result is rounded once. dtype MISA_K_BF16: y is [n, width] bf16 bits.
 * MISA_K_FP8_E4M3FN: y is [n, width] codes with y = code * scale, scale [n] for the row
 * (group 0) or [n, ceil(width / 128)] for each 128 columns (group 128), a power of two
 * chosen as misa_cache_write chooses a row's; what holds an infinity or NaN gets scale
 * NaN and NaN codes. sum may be residual itself (each value is read before it is
 * written); no other overlap is allowed.
 * Limits (MISA_ERR_UNSUPPORTED past them): width <= 16384, n <= 2^25, n * width <= 2^33. */
typedef struct misa_norm_problem {
  int32_t n;              /* rows (0 is a no-op) */
  int32_t width;          /* a multiple of 8 */
  const void* x;          /* rows of width bf16 bits, x_ld elements apart; 16-byte aligned */
  int64_t x_ld;           /* >= width, a multiple of 8 */
  const void* residual;   /* [n,width] bf16 bits or NULL; 16-byte aligned */
  const void* weight;     /* [width], 16-byte aligned */
  int32_t w_dtype;        /* misa_wdtype */
  int32_t dtype;          /* misa_kdtype of y */
  int32_t group;          /* 0 or 128 */
  double eps;             /* >= 0 */
} misa_norm_problem;

/* y 16-byte aligned; scale NULL iff y is bf16; sum [n,width] bf16 bits (16-byte aligned)
 * or NULL (NULL without residual). */
misa_status misa_rms_norm(const misa_norm_problem* p, void* y, float* scale, void* sum, void* stream);

/* Short static text for a status code. */
const char* misa_status_str(int32_t status);

/* Detail of the most recent error reported on the calling host thread
 * ("" if none). The pointer stays valid until the thread's next call. */
const char* misa_last_error(void);

/* Kernel timing instrumentation. While enabled, every kernel the library
 * enqueues is bracketed by a pair of HIP events on the same stream; this adds
 * a little launch overhead, so time whole calls with it disabled.
 * misa_profile_read synchronises the recorded events and returns, for kernels
 * whose name contains `name_substr`, the summed duration in milliseconds and
 * the launch count; misa_profile_reset drops all records. The names of the
 * attention's kernels end in the rows of a workgroup (k_latent_16, k_latent_32,
 * k_latent_wide_64, k_latent_wide_128, k_expanded_128, k_expanded_256; k_tree_16,
 * k_tree_32, k_tree_64, k_tree_128), and k_join or k_tree_join runs where the keys
 * were split. */
misa_status misa_profile_enable(int32_t on);
misa_status misa_profile_read(const char* name_substr, double* total_ms, int64_t* launches);
misa_status misa_profile_reset(void);

#ifdef __cplusplus
}
#endif

#endif /* MISA_H */
