/*
 * verify_ops.h — C ABI of the operators a decode or speculative-verify round calls beside its MoE
 * feed-forward (moe_round.h), on MI355X (gfx950), from the same library:
 *   verify_round_slots     once per round: block table, slot map, positions and tree masks of the
 *                          round's rows, on the GPU, from the requests' lengths;
 *   verify_qk_norm_rope    per layer: RMS norm of each query and key head and the rotary position in
 *                          one pass, keys and values written into the paged cache;
 *   verify_tree_attention  per layer: attention of each request's tree of drafted rows over its cached
 *                          tokens (plain decode is a tree of one row);
 *   verify_token_logprobs  at the end of the round: log probabilities of given tokens, entropy and the
 *                          top alternatives of each row of logits.
 *
 * The pages these follow: "How AlphaInfer makes local decoding fast", section 2 (a verify round is one
 * forward pass over the committed row and its drafts; per-request data is written into fixed buffers)
 * and section 4 (a row's result must not depend on the other rows); infero README, "Continuous
 * batching" (requests of different lengths over a paged cache in one step).
 *
 * Every call is stateless: it enqueues on `stream` and returns; nothing is allocated, synchronised or
 * kept, so calls may be captured into a graph and may run at once on several streams as long as their
 * outputs and workspaces are distinct.  All pointers are DEVICE memory of the current HIP device, which
 * must be the stream's; lengths, tables and masks are read on the GPU when the call executes, so a
 * captured graph follows their contents.  `stream` is a hipStream_t, NULL the null stream.
 *
 * Outputs may not share memory with inputs or with each other unless a call says so.
 *
 * Contents that cannot be checked without waiting for the GPU are bounded there: no index read from
 * device memory is followed outside its array (see each call for what happens instead).
 *
 * Errors: a moe_status as in moe_round.h; nothing aborts, prints or throws.  A rejected call enqueues
 * nothing.  verify_last_hip_error() has the hipError_t behind this thread's last MOE_ERR_HIP.
 *
 * Each argument struct starts with its own size in bytes (checked: MOE_ERR_INVALID_ARG if it differs).
 * Strides are in elements; a tensor's last dimension is contiguous.
 */
#ifndef VERIFY_OPS_H
#define VERIFY_OPS_H

#include "moe_round.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define VERIFY_F32 0
#define VERIFY_BF16 1
#define VERIFY_F16 2

#define VERIFY_MAX_TREE_ROWS 64      /* rows of one request in a tree (bits of a mask word)   */
#define VERIFY_MAX_REQUESTS 65536    /* B                                                     */
#define VERIFY_MAX_TOTAL_ROWS 16777215 /* rows of one call: a block of 256 each, below 2^32 threads */
#define VERIFY_MAX_ALTERNATIVES 16   /* top alternatives per row                              */

/*
 * Block table, slot map, positions and tree masks of one round.
 *
 * c_b = max(cached[b], 0), r_b = max(rows[b], 0); request b's rows are S_b .. S_b + r_b - 1 of the
 * round, S_b the sum of r over the requests before b.  Its cache then holds c_b + r_b tokens in
 * ceil((c_b + r_b) / P) pages of P tokens, of which ceil(c_b / P) are in the table already; the others
 * are taken from `free_pages` in request order, starting at *free_head, and written into the table (all
 * other table entries stay as they are).  Row i of request b is token c_b + i of the cache:
 *   slots[S_b + i]     = table[b][(c_b + i) / P] * P + (c_b + i) % P
 *   positions[S_b + i] = c_b + depth(i)     (at most 2^31 - 1)
 *   masks[S_b + i]     = bit i, and the bits of all of row i's ancestors
 * With `parents`, parents[S_b + i] in -1 .. i - 1 is the row of the same request that row i hangs
 * below (-1, or any value outside that range: directly below the cached tokens) and depth counts row
 * i's ancestors; without, each request's rows are a chain (depth(i) = i) and `masks` must be NULL.
 *
 * row_start[b] = min(S_b, total_rows), b = 0..B.  counts[0] = S_B and counts[1] = the pages needed:
 * compare them with total_rows and the pages that were free.  What does not fit is left out: a page
 * past the end of free_pages is -1 in the table, columns past the table's width take no page, and
 * rows on either get slot -1; rows past total_rows are dropped.  With `parents`, rows past the 64th of
 * a request get slot -1, position c_b and mask 0.  Rows S_B .. total_rows - 1 (padding) get slot -1,
 * position 0, mask 0.
 *
 * Errors: MOE_ERR_INVALID_ARG (NULL or misaligned pointer, negative or zero size, masks and parents
 * not given together), MOE_ERR_UNSUPPORTED (a size past the limits above), MOE_ERR_HIP (launch).
 * B = 0 is an empty round: all rows are padding.
 */
typedef struct verify_slots_args {
  int64_t struct_bytes;       /* sizeof(verify_slots_args)                                    */
  const int32_t* cached;      /* [B] tokens in each request's cache before the round          */
  const int32_t* rows;        /* [B] new rows of each request                                 */
  int32_t* table;             /* [B][width] block table, rows table_stride apart; updated     */
  int64_t table_stride;
  const int32_t* free_pages;  /* [n_free] (may be NULL if n_free = 0)                         */
  const int32_t* free_head;   /* first free page to take (device), NULL = 0                   */
  const int32_t* parents;     /* [total_rows] or NULL                                         */
  int32_t* row_start;         /* [B + 1]                                                      */
  int32_t* slots;             /* [total_rows]                                                 */
  int32_t* positions;         /* [total_rows]                                                 */
  int64_t* masks;             /* [total_rows], NULL without parents                           */
  int32_t* counts;            /* [2] rows, pages                                              */
  int32_t n_requests;         /* B: 0..VERIFY_MAX_REQUESTS                                    */
  int32_t width;              /* columns of the table, >= 1                                   */
  int32_t n_free;             /* >= 0                                                         */
  int32_t page_size;          /* P: 1..65536                                                  */
  int32_t total_rows;         /* 0..VERIFY_MAX_TOTAL_ROWS                                     */
  int32_t reserved;           /* 0                                                            */
} verify_slots_args;

MOE_ROUND_API moe_status verify_round_slots(const verify_slots_args* a, void* stream);

/*
 * Norm and rotary position of query and key heads, and the cache write, in one pass.  For each row t and
 * each query or key head x of D values (float32 arithmetic):
 *   y = x * rsqrt(mean(x^2) + eps) * weight          (weight NULL: y = x)
 *   the first R = 2 * n_freq values of y are rotated by the angles positions[t] * inv_freq[i], i < R/2
 *   (angle and its reduction in float64): pairs (i, i + R/2), or (2i, 2i + 1) with `interleaved`;
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * rounded once to the cache's type: query heads into q_out, key heads into k_cache at slots[t]; value
 * heads are copied (rounded) into v_cache.  Slot s is token s % P of page s / P.  A row whose slot is
 * outside 0 .. n_pages * P - 1 is skipped: neither q_out's row nor the caches are written.  Slots of one
 * call must differ (two rows of one slot leave that token's values undefined, nothing else).
 *
 * q_out may be q itself (same type and strides); any other overlap of inputs and outputs is the
 * caller's mistake, and one of q_out and q is refused.
 *
 * Supported: D 64, 128 or 256; R a multiple of 16 up to D; in_type = cache_type, or VERIFY_F32 in;
 * cache_type VERIFY_BF16 or VERIFY_F16; pointers 16-byte aligned, strides multiples of 16 bytes.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP.  n_rows = 0: nothing is enqueued.
 */
typedef struct verify_rope_args {
  int64_t struct_bytes;
  const void* q;              /* [n_rows][heads][D]    */
  const void* k;              /* [n_rows][kv_heads][D] */
  const void* v;              /* [n_rows][kv_heads][D] */
  void* q_out;                /* [n_rows][heads][D], the cache's type */
  void* k_cache;              /* [n_pages][kv_heads][P][D] */
  void* v_cache;
  const int32_t* positions;   /* [n_rows] */
  const int32_t* slots;       /* [n_rows] */
  const float* inv_freq;      /* [n_freq] */
  const float* q_weight;      /* [D] or NULL */
  const float* k_weight;      /* [D] or NULL */
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;         /* strides */
  int64_t kc_page, kc_head, kc_token, vc_page, vc_head, vc_token;             /* cache strides */
  int64_t n_pages;
  int32_t n_rows, heads, kv_heads, dim, page_size, n_freq;
  int32_t in_type, cache_type;
  int32_t interleaved;        /* 0 or 1 */
  float eps;                  /* >= 0 */
} verify_rope_args;

MOE_ROUND_API moe_status verify_qk_norm_rope(const verify_rope_args* a, void* stream);

/*
 * Attention of each request's drafted rows over its paged cache.  Request b's rows are row_start[b] ..
 * row_start[b + 1] - 1 of q and out; they are tokens cached[b] .. of its cache, written there before
 * (verify_qk_norm_rope).  For row i of request b and head h (kv head h / (heads / kv_heads)):
 *   s_j = scale * q . k_j       over the tokens j the row sees: every j < cached[b], and cached[b] + i'
 *                               for each set bit i' < rows_b of the row's mask
 *   out = sum_j softmax(s)_j v_j
 * Without masks the rows are a chain: row i sees drafted rows 0..i.  A row that sees no token gets zeros.
 * A token that a row does not see has no effect on it, whatever the cache holds there (infinities and
 * NaN included).  Token j lies at token j % P of page table[b][j / P]; tokens past the table's width, or
 * on pages outside 0 .. n_pages - 1, count as not seen.
 * Rows past row_start[B], and rows past max_rows of a request, are left as they were.
 *
 * Arithmetic: products of 16-bit values summed in float32, softmax statistics and the output sums in
 * float32, each probability rounded to the cache's type for its product with the values (relative to
 * the row's running maximum), the output rounded once.
 * Results do not depend on timing (no atomics); how the context is split depends on the lengths of all
 * requests of the call, and changes results within the rounding of the probabilities (each part has its
 * own running maximum).
 *
 * Supported: D 64, 128 or 256; heads a multiple of kv_heads; P a power of two from 16 to 65536; max_rows
 * 1..VERIFY_MAX_TREE_ROWS; heads / kv_heads up to 64; type VERIFY_BF16 or VERIFY_F16 (q, cache and out
 * alike); pointers 16-byte aligned, strides multiples of 16 bytes; scale > 0; out may be q itself (the
 * same strides; any other overlap of the two is refused). A launch of 2^32 threads or more is refused
 * (MOE_ERR_UNSUPPORTED): n_rows * heads above 2^26 - 4 where the context may be split, or some millions of
 * blocks of 32 to 256 query rows of one kv head.
 * `workspace` is device memory of at least verify_tree_attention_workspace(a) bytes (0 if none is
 * needed), 16-byte aligned, free for other use when the call has executed; its contents do not matter.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP.  n_rows = 0 or n_requests = 0: nothing is
 * enqueued.
 */
typedef struct verify_attention_args {
  int64_t struct_bytes;
  const void* q;              /* [n_rows][heads][D]        */
  const void* k_cache;        /* [n_pages][kv_heads][P][D] */
  const void* v_cache;
  const int32_t* table;       /* [B][width], rows table_stride apart */
  const int32_t* cached;      /* [B] */
  const int32_t* row_start;   /* [B + 1] */
  const int64_t* masks;       /* [n_rows] or NULL (chains) */
  void* out;                  /* [n_rows][heads][D] */
  int64_t q_row, q_head, o_row, o_head;
  int64_t kc_page, kc_head, kc_token, vc_page, vc_head, vc_token;
  int64_t table_stride, n_pages;
  int32_t n_rows, n_requests, heads, kv_heads, dim, page_size, width, max_rows;
  int32_t type;
  float scale;
} verify_attention_args;

/* Bytes of workspace the call needs, or a negative moe_status if it would be refused (host only). */
MOE_ROUND_API int64_t verify_tree_attention_workspace(const verify_attention_args* a);
MOE_ROUND_API moe_status verify_tree_attention(const verify_attention_args* a, void* workspace,
                                               int64_t workspace_bytes, void* stream);

/*
 * Log probabilities of given tokens, entropy, and the top alternatives of each row of logits.  Per row,
 * z = log sum_v exp(x_v) (float32; exact in the order of the sums for a given shape):
 *   logprobs[t][n]     = x[tokens[t][n]] - z   (-inf for a token outside 0 .. vocab - 1)
 *   entropy[t]         = z - sum_v softmax(x)_v x_v     (a logit of -inf adds nothing)
 *   top_ids[t][j], top_logprobs[t][j], j < top: the largest logits in descending order, equal ones by
 *                        ascending id, and their log probabilities
 * A row whose logits are all -inf has log probabilities -inf and entropy 0.  A NaN or +inf logit makes the
 * row's log probabilities (but -inf ones of tokens outside the vocabulary) and entropy NaN; NaN logits
 * are never alternatives (an id of -1, NaN, where too few others are left).
 * logprobs/tokens may be NULL with n_tokens = 0, top_* with top = 0, entropy may be NULL.
 *
 * Supported: any vocab >= 1, any alignment the element type has; top up to min(vocab,
 * VERIFY_MAX_ALTERNATIVES).  `workspace` as for the attention (16-byte aligned).
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP.  n_rows = 0: nothing is enqueued.
 */
typedef struct verify_logprobs_args {
  int64_t struct_bytes;
  const void* logits;         /* [n_rows][vocab], rows row_stride apart */
  const void* tokens;         /* [n_rows][n_tokens] int32, or int64 with tokens_64 */
  float* logprobs;            /* [n_rows][n_tokens] */
  float* entropy;             /* [n_rows] or NULL */
  int32_t* top_ids;           /* [n_rows][top] */
  float* top_logprobs;        /* [n_rows][top] */
  int64_t row_stride;
  int32_t n_rows, vocab, n_tokens, top;
  int32_t type;               /* VERIFY_F32, VERIFY_BF16 or VERIFY_F16 */
  int32_t tokens_64;          /* 0 or 1 */
} verify_logprobs_args;

MOE_ROUND_API int64_t verify_token_logprobs_workspace(const verify_logprobs_args* a);
MOE_ROUND_API moe_status verify_token_logprobs(const verify_logprobs_args* a, void* workspace,
                                               int64_t workspace_bytes, void* stream);

/* The hipError_t (as int) of this thread's last MOE_ERR_HIP from a call above, 0 if none. */
MOE_ROUND_API int32_t verify_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* VERIFY_OPS_H */
