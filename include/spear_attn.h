/*
 * spear_attn.h - the paged key-value cache of libspear and the attention that
 * reads it, for the two phases that spear.h's compensated linears serve:
 * prompt chunks (prefill) and single new tokens (decode).
 *
 * Conventions are spear.h's: device pointers owned by the caller, every call
 * asynchronous on the stream it is given, no device memory allocated and
 * nothing copied between host and device, arguments validated on the host
 * before anything is launched, spear_last_error() for the detail.  What only
 * the device can see (lengths, table entries, slots) is checked by the
 * kernels: a bad value never makes them read or write outside the arrays
 * described here; each call says what it does instead.
 *
 * Element types: queries, keys, values, cache and output share SPEAR_F16 or
 * SPEAR_BF16.  Scores, the running maximum and sum of the softmax and the
 * output sums are fp32.  The softmax's weights are rounded to the element type
 * once, each relative to its own size, before they meet the values (their sum
 * takes them unrounded); a SPEAR_F16 weight below 2^-27 of its row's largest is
 * off by up to 2^-38 of that instead.
 */
#ifndef SPEAR_ATTN_H
#define SPEAR_ATTN_H

#include "spear.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A paged cache: for each layer, num_pages pages of page_size tokens, each
 * token a key and a value of head_dim elements per key-value head.  Element
 * d of token t, head h, page p, layer l of either array is at
 *     l * stride_layer + p * stride_page + h * stride_head + t * stride_token + d
 * (strides in elements), so pages may be head-major ([head][token][dim]) or
 * token-major ([token][head][dim]), in an array of their own or inside a
 * larger one.
 *   head_dim    64 or 128.
 *   page_size   a multiple of 16, at most 65536.
 *   strides     multiples of 8; no two elements may share an address; one
 *               layer's page spans at most 2^29 elements.
 *   k, v        16-byte aligned.
 * A multi-token call may address past 2^31 elements; offsets are 64-bit.
 * The attention and append calls take one layer (n_layers == 1: offset k and
 * v to it); the page calls move a page of all layers at once.
 */
typedef struct spear_kv_cache {
  void *k, *v;
  int32_t dtype; /* a spear_dtype_t */
  int32_t n_layers, num_pages, n_kv_heads, page_size, head_dim;
  int64_t stride_layer, stride_page, stride_head, stride_token;
} spear_kv_cache_t;

/*
 * The sequences of one step, in device memory.
 *   block_table  [n_seqs][table_width]: the pages that hold tokens
 *                0..page_size-1, page_size..2*page_size-1, ... of a sequence.
 *   kv_lens      [n_seqs]: tokens in the cache, the step's own included.
 *                Taken as 0 when negative and as table_width * page_size when
 *                larger than that.
 *   q_starts     [n_seqs + 1], ascending from 0: sequence b's new tokens are
 *                rows q_starts[b] .. q_starts[b+1]-1 of q (of the new keys
 *                and values), its last positions in order.  NULL: one row
 *                per sequence.  Sequences without new tokens are fine.  Taken
 *                as 0 when negative and as n_tokens when larger than that, by
 *                the attention and by append.
 *   n_tokens     rows of q (n_seqs when q_starts is NULL).  Rows that no
 *                sequence covers are left as they are.
 * n_seqs <= SPEAR_ATTN_MAX_SEQS, n_tokens <= 2^24 (times n_q_heads: 2^30),
 * table_width * page_size <= 2^30 (times n_seqs: 2^35).  A table entry outside 0..num_pages-1 hides the tokens of its page.
 */
#define SPEAR_ATTN_MAX_SEQS 4096
typedef struct spear_kv_batch {
  int32_t n_seqs, table_width, n_tokens;
  const int32_t *block_table;
  const int32_t *kv_lens;
  const int32_t *q_starts;
} spear_kv_batch_t;

/*
 * Queries and output of an attention call.  Row t, head h, element d of q is
 * at t * q_stride_token + h * q_stride_head + d (elements); out alike.  q and
 * out are 16-byte aligned with strides that are multiples of 8; out's
 * elements may not share addresses, q's may (a broadcast query).
 *   n_q_heads   a multiple of n_kv_heads; query head h reads key-value head
 *               h / (n_q_heads / n_kv_heads).
 *   scale       factor of the scores before the softmax.
 *   window      0: none.  w > 0: a query at position p sees positions
 *               p-w+1..p,
 *   sinks       and the first `sinks` positions of its sequence (>= 0; with
 *               window == 0 it has no effect).
 *   lse         NULL, or fp32 [n_tokens][n_q_heads]: the natural logarithm of
 *               the sum of exp(score) over what the row sees (for joining
 *               with attention over other keys).
 */
typedef struct spear_attn_args {
  int32_t n_q_heads, window, sinks;
  float scale;
  const void *q;
  int64_t q_stride_token, q_stride_head;
  void *out;
  int64_t out_stride_token, out_stride_head;
  float *lse;
} spear_attn_args_t;

/*
 * Workspace bytes that spear_attn_decode and spear_attn_prefill need for this
 * cache and number of query heads with at most n_seqs sequences and n_tokens
 * rows; 0 when an argument is invalid.  256-byte aligned, its first
 * SPEAR_ATTN_HEADER_BYTES ZEROED ONCE before its first use, left ready by
 * every call; any attention call of at most these sizes may use it.  It is not interchangeable with
 * spear_workspace_bytes' workspace.  Calls that may overlap need different
 * ones.
 */
#define SPEAR_ATTN_HEADER_BYTES 16384
size_t spear_attn_workspace_bytes(const spear_kv_cache_t *cache, int32_t n_q_heads,
                                  int32_t n_seqs, int32_t n_tokens);

/*
 * Attention of one new token per sequence (q_starts == NULL) over its cached
 * keys and values, its own included (append first).  The query is at position
 * kv_len - 1.  A row that sees nothing gives zeros, and -infinity in lse.
 * What a row does not see never reaches its output, whatever it holds.
 */
spear_status_t spear_attn_decode(const spear_kv_cache_t *cache, const spear_kv_batch_t *batch,
                                 const spear_attn_args_t *args, void *workspace,
                                 size_t workspace_bytes, spear_stream_t stream);

/*
 * Causal attention of the batch's new tokens, any number per sequence, over
 * the cached keys and values, their own included (append first): row i of
 * sequence b's n rows is at position kv_len - n + i (a row before position 0
 * sees nothing).  Rows that see nothing, and hidden tokens, as above.
 */
spear_status_t spear_attn_prefill(const spear_kv_cache_t *cache, const spear_kv_batch_t *batch,
                                  const spear_attn_args_t *args, void *workspace,
                                  size_t workspace_bytes, spear_stream_t stream);

/*
 * Store the batch's new keys and values in their pages: k and v are
 * [n_tokens][n_kv_heads][head_dim] by strides as q is (multiples of 8,
 * 16-byte aligned).  Bit-exact copies.  A token whose position lies before 0
 * or whose page is not in 0..num_pages-1 is dropped.
 */
spear_status_t spear_kv_append(const spear_kv_cache_t *cache, const spear_kv_batch_t *batch,
                               const void *k, const void *v, int64_t k_stride_token,
                               int64_t k_stride_head, int64_t v_stride_token,
                               int64_t v_stride_head, spear_stream_t stream);

/*
 * Copy page src[i] to page dst[i], i < n, of all layers, keys and values (src
 * and dst: device arrays).  A pair with an index outside 0..num_pages-1, or
 * with src == dst, is skipped.  The dst pages must be distinct and none may
 * be a src of the same call.
 */
spear_status_t spear_kv_copy_pages(const spear_kv_cache_t *cache, const int32_t *src,
                                   const int32_t *dst, int32_t n, spear_stream_t stream);

/*
 * The pages' bookkeeping, all of it device memory: which sequence slot holds
 * which pages, and how many rows of the table hold each page.
 *   refs    [num_pages]: 0 for a free page.
 *   table   [n_slots][table_width]: a slot's pages in order, -1 past the last.
 *   lens    [n_slots]: tokens of each slot.
 *   scratch spear_kv_scratch_words(...) int32 words, written before they are
 *           read by each call; calls that may overlap need different ones.
 * A fresh pool has refs 0, table -1, lens 0.  The calls below keep refs[p]
 * equal to the number of table entries that name p; slots and pages outside
 * their ranges are skipped.  Allocation takes the free page of the lowest
 * index, so results do not depend on timing.
 */
typedef struct spear_kv_pool {
  int32_t num_pages, page_size, n_slots, table_width;
  int32_t *refs, *table, *lens, *scratch;
} spear_kv_pool_t;

#define SPEAR_KV_MAX_ENTRIES 1024 /* slots in one spear_kv_reserve call */
size_t spear_kv_scratch_words(int32_t num_pages, int32_t n_slots, int32_t table_width);

/*
 * Slot dst[i] becomes a copy of slot src[i], i < n, that shares all its
 * pages; what dst[i] held is released first.  No page is copied (see
 * spear_kv_reserve).  The dst slots must be distinct and none may be a src of
 * the same call; several may share a src.
 */
spear_status_t spear_kv_fork(const spear_kv_pool_t *pool, const int32_t *src, const int32_t *dst,
                             int32_t n, spear_stream_t stream);

/*
 * Make slots[i] ready to hold new_lens[i] tokens, i < n <=
 * SPEAR_KV_MAX_ENTRIES, in order (distinct slots, so n <= n_slots; new_lens[i]
 * no more than the present length changes nothing): where its last page is part full and
 * other rows hold it too, the slot gets a copy of that page, made here in all
 * layers of the cache; the last holder of such a page keeps it.  Then pages
 * are added up to new_lens[i] and lens[slots[i]] = new_lens[i].
 * *missing (device) = 0; or, when the free pages do not suffice, how many
 * more would be needed, or -1 when an entry asks for more than table_width
 * pages or names no slot: then nothing is changed.  cache: the pool's pages
 * (its num_pages and page_size must agree).
 */
spear_status_t spear_kv_reserve(const spear_kv_pool_t *pool, const spear_kv_cache_t *cache,
                                const int32_t *slots, const int32_t *new_lens, int32_t n,
                                int32_t *missing, spear_stream_t stream);

/* Release slots[i], i < n (distinct): its pages lose a holder, its row and length are cleared. */
spear_status_t spear_kv_free(const spear_kv_pool_t *pool, const int32_t *slots, int32_t n,
                             spear_stream_t stream);

/*
 * Move the used pages to the lowest indices: the highest used page takes the
 * lowest free place, and so on until they meet, so that exactly pages
 * 0..*used-1 are in use (*used: device).  Pages are moved in all layers, the
 * table and refs follow; a page that moves leaves its bytes behind.
 */
spear_status_t spear_kv_compact(const spear_kv_pool_t *pool, const spear_kv_cache_t *cache,
                                int32_t *used, spear_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEAR_ATTN_H */
