// C ABI of the paged cache and its attention (spear_attn.h): host-side
// validation before any launch.
#include <math.h>

#include <algorithm>

#include "api_common.h"
#include "attn_internal.h"

using namespace spear;

namespace {

// Whether an array of these extents and strides (elements, the innermost of
// stride 1 first) gives every element an address of its own, with offsets
// that stay below 2^60.
struct Dim {
  int64_t n, stride;
};
bool separate(int64_t inner, Dim *dims, int count) {
  std::sort(dims, dims + count, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
  int64_t extent = inner;  // elements spanned so far
  for (int i = 0; i < count; ++i) {
    if (dims[i].n <= 1) continue;
    if (dims[i].stride < extent || dims[i].stride > (int64_t(1) << 60) / dims[i].n) return false;
    extent += (dims[i].n - 1) * dims[i].stride;
    if (extent > (int64_t(1) << 60)) return false;
  }
  return true;
}

spear_status_t check_cache(const spear_kv_cache_t *c, bool one_layer) {
  if (!c) return fail(SPEAR_ERR_INVALID_ARGUMENT, "cache is NULL");
  if (c->dtype != SPEAR_F16 && c->dtype != SPEAR_BF16)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "cache dtype=%d is not SPEAR_F16 or SPEAR_BF16", c->dtype);
  if (c->n_layers < 1 || c->num_pages < 1 || c->n_kv_heads < 1 || c->page_size < 1)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "cache n_layers=%d num_pages=%d n_kv_heads=%d page_size=%d must be >= 1",
                c->n_layers, c->num_pages, c->n_kv_heads, c->page_size);
  if (one_layer && c->n_layers != 1)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "this call takes one layer of the cache, got n_layers=%d", c->n_layers);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(SPEAR_ERR_UNSUPPORTED, "head_dim=%d: 64 and 128 are supported", c->head_dim);
  if (c->page_size % 16 != 0 || c->page_size > 65536)
    return fail(SPEAR_ERR_UNSUPPORTED, "page_size=%d: multiples of 16 up to 65536 are supported", c->page_size);
  if (c->n_kv_heads > 1024) return fail(SPEAR_ERR_UNSUPPORTED, "n_kv_heads=%d exceeds 1024", c->n_kv_heads);
  if (!c->k || !c->v) return fail(SPEAR_ERR_INVALID_ARGUMENT, "cache k and v must not be NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "cache k and v must be 16-byte aligned");
  if ((c->stride_layer | c->stride_page | c->stride_head | c->stride_token) % 8 != 0)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "cache strides must be multiples of 8 elements");
  Dim dims[4] = {{c->n_layers, c->stride_layer}, {c->num_pages, c->stride_page},
                 {c->n_kv_heads, c->stride_head}, {c->page_size, c->stride_token}};
  if (!separate(c->head_dim, dims, 4))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "cache strides make elements share addresses");
  // offsets inside a page are 32-bit in the kernels
  if ((c->n_kv_heads - 1) * c->stride_head + (c->page_size - 1) * c->stride_token + c->head_dim >
      (int64_t(1) << 29))
    return fail(SPEAR_ERR_UNSUPPORTED, "a page of a layer spans more than 2^29 elements");
  return SPEAR_OK;
}

spear_status_t check_batch(const spear_kv_batch_t *b, int page_size) {
  if (!b) return fail(SPEAR_ERR_INVALID_ARGUMENT, "batch is NULL");
  if (b->n_seqs < 0 || b->table_width < 1 || b->n_tokens < 0)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "batch n_seqs=%d table_width=%d n_tokens=%d", b->n_seqs,
                b->table_width, b->n_tokens);
  if (b->n_seqs > SPEAR_ATTN_MAX_SEQS)
    return fail(SPEAR_ERR_UNSUPPORTED, "n_seqs=%d exceeds %d", b->n_seqs, SPEAR_ATTN_MAX_SEQS);
  if (b->n_tokens > (1 << 24)) return fail(SPEAR_ERR_UNSUPPORTED, "n_tokens=%d too large", b->n_tokens);
  if ((int64_t)b->table_width * page_size > (int64_t(1) << 30))
    return fail(SPEAR_ERR_UNSUPPORTED, "table_width=%d pages of %d tokens exceed 2^30 tokens",
                b->table_width, page_size);
  if ((int64_t)b->n_seqs * b->table_width * page_size > (int64_t(1) << 35))
    return fail(SPEAR_ERR_UNSUPPORTED, "block_table of %d x %d pages of %d tokens exceeds 2^35 tokens",
                b->n_seqs, b->table_width, page_size);
  if (!b->q_starts && b->n_tokens != b->n_seqs)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "without q_starts n_tokens=%d must equal n_seqs=%d",
                b->n_tokens, b->n_seqs);
  if (b->n_seqs > 0 && (!b->block_table || !b->kv_lens))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "block_table and kv_lens must not be NULL");
  if (!aligned(b->block_table, 4) || !aligned(b->kv_lens, 4) || !aligned(b->q_starts, 4))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "block_table, kv_lens and q_starts must be 4-byte aligned");
  return SPEAR_OK;
}

spear_status_t check_rows(const char *name, const void *p, int64_t s_tok, int64_t s_head) {
  if (!p) return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if (!aligned(p, 16)) return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s must be 16-byte aligned", name);
  if (s_tok < 0 || s_head < 0 || (s_tok | s_head) % 8 != 0 || s_tok > (int64_t(1) << 32) ||
      s_head > (int64_t(1) << 40))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s strides %lld, %lld must be multiples of 8 elements", name,
                (long long)s_tok, (long long)s_head);
  return SPEAR_OK;
}

spear_status_t attention(const spear_kv_cache_t *c, const spear_kv_batch_t *b,
                         const spear_attn_args_t *a, void *ws, size_t ws_bytes, void *stream,
                         bool decode) {
  TRY(check_cache(c, true));
  TRY(check_batch(b, c->page_size));
  if (!a) return fail(SPEAR_ERR_INVALID_ARGUMENT, "args is NULL");
  if (decode && b->q_starts)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "decode takes one token per sequence: q_starts must be NULL");
  if (a->n_q_heads < 1 || a->n_q_heads % c->n_kv_heads != 0)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "n_q_heads=%d is not a multiple of n_kv_heads=%d",
                a->n_q_heads, c->n_kv_heads);
  if ((int64_t)b->n_tokens * a->n_q_heads > (int64_t(1) << 30))
    return fail(SPEAR_ERR_UNSUPPORTED, "n_tokens=%d rows of n_q_heads=%d exceed 2^30", b->n_tokens, a->n_q_heads);
  if (a->n_q_heads > 4096) return fail(SPEAR_ERR_UNSUPPORTED, "n_q_heads=%d exceeds 4096", a->n_q_heads);
  if (a->window < 0 || a->sinks < 0)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "window=%d and sinks=%d must be >= 0", a->window, a->sinks);
  if (!isfinite(a->scale)) return fail(SPEAR_ERR_INVALID_ARGUMENT, "scale is not finite");
  if (b->n_tokens == 0 || b->n_seqs == 0) return ok();
  TRY(check_rows("q", a->q, a->q_stride_token, a->q_stride_head));
  TRY(check_rows("out", a->out, a->out_stride_token, a->out_stride_head));
  Dim dims[2] = {{b->n_tokens, a->out_stride_token}, {a->n_q_heads, a->out_stride_head}};
  if (!separate(c->head_dim, dims, 2))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "out strides make elements share addresses");
  if (a->q == a->out) return fail(SPEAR_ERR_INVALID_ARGUMENT, "out must not alias q");
  if (!aligned(a->lse, 4)) return fail(SPEAR_ERR_INVALID_ARGUMENT, "lse must be 4-byte aligned");
  const size_t need = decode ? attn_decode_workspace(c->head_dim, a->n_q_heads, c->n_kv_heads, b->n_seqs)
                             : attn_prefill_workspace(c->head_dim, a->n_q_heads, c->n_kv_heads,
                                                      b->n_seqs, b->n_tokens);
  if (need > 0) {
    if (!ws) return fail(SPEAR_ERR_WORKSPACE, "workspace of %zu bytes required, got NULL", need);
    if (!aligned(ws, 256)) return fail(SPEAR_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (ws_bytes < need)
      return fail(SPEAR_ERR_WORKSPACE, "workspace of %zu bytes required, got %zu", need, ws_bytes);
  }
  AttnDesc d{};
  d.dtype = c->dtype;
  d.D = c->head_dim;
  d.Hq = a->n_q_heads;
  d.Hkv = c->n_kv_heads;
  d.G = d.Hq / d.Hkv;
  d.page_size = c->page_size;
  d.num_pages = c->num_pages;
  // with 2^(s-1) < p <= 2^s, mul = ceil(2^(31+s) / p) exceeds the quotient by
  // less than one, so i mul / 2^(31+s) is less than 1 / p above i / p
  if (const uint32_t p16 = c->page_size / 16; p16 > 1) {
    const int sh = 32 - __builtin_clz(p16 - 1);
    d.p16_mul = (uint32_t)(((uint64_t(1) << (31 + sh)) + p16 - 1) / p16);
    d.p16_shift = sh - 1;
  }
  d.k = (const uint16_t *)c->k;
  d.v = (const uint16_t *)c->v;
  d.s_page = c->stride_page;
  d.s_head = c->stride_head;
  d.s_token = c->stride_token;
  d.n_seqs = b->n_seqs;
  d.width = b->table_width;
  d.n_tokens = b->n_tokens;
  d.table = b->block_table;
  d.kv_lens = b->kv_lens;
  d.q_starts = b->q_starts;
  d.window = a->window;
  d.sinks = a->window > 0 ? a->sinks : 0;
  d.scale = a->scale;
  d.q = (const uint16_t *)a->q;
  d.q_tok = a->q_stride_token;
  d.q_head = a->q_stride_head;
  d.out = (uint16_t *)a->out;
  d.o_tok = a->out_stride_token;
  d.o_head = a->out_stride_head;
  d.lse = a->lse;
  return decode ? hip_status(launch_attn_decode(d, ws, (hipStream_t)stream), "attention decode launch")
                : hip_status(launch_attn_prefill(d, ws, (hipStream_t)stream), "attention prefill launch");
}

// A page of the cache for the copies; extents whose strides continue one
// another are joined, so that a dense page is one run.
PageDesc page_desc(const spear_kv_cache_t &c) {
  PageDesc p{(uint16_t *)c.k, (uint16_t *)c.v, c.n_layers, c.num_pages, c.n_kv_heads, c.page_size,
             c.head_dim, c.stride_layer, c.stride_page, c.stride_head, c.stride_token};
  if (p.S > 1 && p.s_token == p.D) {  // tokens of a head in one run
    p.D *= p.S;
    p.S = 1;
  } else if (p.H > 1 && p.s_head == p.D) {  // heads of a token in one run
    p.D *= p.H;
    p.H = 1;
    if (p.s_token == p.D) {
      p.D *= p.S;
      p.S = 1;
    }
  }
  if (p.S == 1 && p.H > 1 && p.s_head == p.D) {
    p.D *= p.H;
    p.H = 1;
  }
  return p;
}

spear_status_t check_pool(const spear_kv_pool_t *p) {
  if (!p) return fail(SPEAR_ERR_INVALID_ARGUMENT, "pool is NULL");
  if (p->num_pages < 1 || p->page_size < 1 || p->n_slots < 1 || p->table_width < 1)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "pool num_pages=%d page_size=%d n_slots=%d table_width=%d must be >= 1",
                p->num_pages, p->page_size, p->n_slots, p->table_width);
  if (p->num_pages > (1 << 24) || (int64_t)p->n_slots * p->table_width > (int64_t(1) << 30) ||
      (int64_t)p->table_width * p->page_size > (int64_t(1) << 30))
    return fail(SPEAR_ERR_UNSUPPORTED, "pool num_pages=%d n_slots=%d table_width=%d too large",
                p->num_pages, p->n_slots, p->table_width);
  if (!p->refs || !p->table || !p->lens || !p->scratch)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "pool refs, table, lens and scratch must not be NULL");
  if (!aligned(p->refs, 4) || !aligned(p->table, 4) || !aligned(p->lens, 4) || !aligned(p->scratch, 4))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "pool arrays must be 4-byte aligned");
  return SPEAR_OK;
}

spear_status_t check_pool_cache(const spear_kv_pool_t *p, const spear_kv_cache_t *c) {
  TRY(check_pool(p));
  TRY(check_cache(c, false));
  if (c->num_pages != p->num_pages || c->page_size != p->page_size)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "pool has %d pages of %d tokens, the cache %d of %d",
                p->num_pages, p->page_size, c->num_pages, c->page_size);
  return SPEAR_OK;
}

spear_status_t check_list(const char *name, const int32_t *p, int32_t n, int32_t most) {
  if (n < 0 || n > most) return fail(SPEAR_ERR_INVALID_ARGUMENT, "n=%d outside 0..%d", n, most);
  if (n > 0 && !p) return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if (!aligned(p, 4)) return fail(SPEAR_ERR_INVALID_ARGUMENT, "%s must be 4-byte aligned", name);
  return SPEAR_OK;
}

constexpr int32_t kMaxList = 1 << 24;

}  // namespace

extern "C" {

size_t spear_attn_workspace_bytes(const spear_kv_cache_t *cache, int32_t n_q_heads, int32_t n_seqs,
                                  int32_t n_tokens) {
  if (check_cache(cache, false) != SPEAR_OK) return 0;
  if (n_q_heads < 1 || n_q_heads > 4096 || n_q_heads % cache->n_kv_heads != 0 || n_seqs < 0 ||
      n_seqs > SPEAR_ATTN_MAX_SEQS || n_tokens < 0 || n_tokens > (1 << 24)) {
    fail(SPEAR_ERR_INVALID_ARGUMENT, "n_q_heads=%d n_seqs=%d n_tokens=%d", n_q_heads, n_seqs, n_tokens);
    return 0;
  }
  const size_t a = attn_decode_workspace(cache->head_dim, n_q_heads, cache->n_kv_heads, n_seqs);
  const size_t b = attn_prefill_workspace(cache->head_dim, n_q_heads, cache->n_kv_heads, n_seqs, n_tokens);
  return std::max<size_t>(256, std::max(a, b));
}

spear_status_t spear_attn_decode(const spear_kv_cache_t *cache, const spear_kv_batch_t *batch,
                                 const spear_attn_args_t *args, void *workspace,
                                 size_t workspace_bytes, spear_stream_t stream) {
  return attention(cache, batch, args, workspace, workspace_bytes, stream, true);
}

spear_status_t spear_attn_prefill(const spear_kv_cache_t *cache, const spear_kv_batch_t *batch,
                                  const spear_attn_args_t *args, void *workspace,
                                  size_t workspace_bytes, spear_stream_t stream) {
  return attention(cache, batch, args, workspace, workspace_bytes, stream, false);
}

spear_status_t spear_kv_append(const spear_kv_cache_t *c, const spear_kv_batch_t *b, const void *k,
                               const void *v, int64_t k_stride_token, int64_t k_stride_head,
                               int64_t v_stride_token, int64_t v_stride_head,
                               spear_stream_t stream) {
  TRY(check_cache(c, true));
  TRY(check_batch(b, c->page_size));
  if (b->n_tokens == 0 || b->n_seqs == 0) return ok();
  TRY(check_rows("k", k, k_stride_token, k_stride_head));
  TRY(check_rows("v", v, v_stride_token, v_stride_head));
  const AppendDesc d{c->n_kv_heads, c->head_dim, c->page_size, c->num_pages,
                     (uint16_t *)c->k, (uint16_t *)c->v, c->stride_page, c->stride_head,
                     c->stride_token, b->n_seqs, b->table_width, b->n_tokens, b->block_table,
                     b->kv_lens, b->q_starts, (const uint16_t *)k, (const uint16_t *)v,
                     k_stride_token, k_stride_head, v_stride_token, v_stride_head};
  return hip_status(launch_kv_append(d, (hipStream_t)stream), "append launch");
}

spear_status_t spear_kv_copy_pages(const spear_kv_cache_t *cache, const int32_t *src,
                                   const int32_t *dst, int32_t n, spear_stream_t stream) {
  TRY(check_cache(cache, false));
  TRY(check_list("src", src, n, kMaxList));
  TRY(check_list("dst", dst, n, kMaxList));
  if (n == 0) return ok();
  return hip_status(launch_kv_copy_pages(page_desc(*cache), src, dst, n, (hipStream_t)stream),
                    "page copy launch");
}

size_t spear_kv_scratch_words(int32_t num_pages, int32_t n_slots, int32_t table_width) {
  if (num_pages < 1 || n_slots < 1 || table_width < 1 || num_pages > (1 << 24)) return 0;
  // compact: three lists of num_pages and a count per block of pages; reserve:
  // the pages it takes and its copies
  return 3 * (size_t)num_pages + num_pages / 1024 + 2 * SPEAR_KV_MAX_ENTRIES + 64;
}

spear_status_t spear_kv_fork(const spear_kv_pool_t *pool, const int32_t *src, const int32_t *dst,
                             int32_t n, spear_stream_t stream) {
  TRY(check_pool(pool));
  TRY(check_list("src", src, n, kMaxList));
  TRY(check_list("dst", dst, n, kMaxList));
  if (n == 0) return ok();
  return hip_status(launch_kv_fork(*pool, src, dst, n, (hipStream_t)stream), "fork launch");
}

spear_status_t spear_kv_reserve(const spear_kv_pool_t *pool, const spear_kv_cache_t *cache,
                                const int32_t *slots, const int32_t *new_lens, int32_t n,
                                int32_t *missing, spear_stream_t stream) {
  TRY(check_pool_cache(pool, cache));
  TRY(check_list("slots", slots, n, SPEAR_KV_MAX_ENTRIES));
  TRY(check_list("new_lens", new_lens, n, SPEAR_KV_MAX_ENTRIES));
  // (distinct slots ask for at most n_slots * table_width <= 2^30 pages, which the plan's sums hold)
  if (n > pool->n_slots)
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "n=%d entries of a pool of %d slots are not distinct", n, pool->n_slots);
  if (!missing || !aligned(missing, 4))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "missing must be a 4-byte aligned device pointer");
  return hip_status(launch_kv_reserve(*pool, page_desc(*cache), slots, new_lens, n, missing,
                                      (hipStream_t)stream),
                    "reserve launch");
}

spear_status_t spear_kv_free(const spear_kv_pool_t *pool, const int32_t *slots, int32_t n,
                             spear_stream_t stream) {
  TRY(check_pool(pool));
  TRY(check_list("slots", slots, n, kMaxList));
  if (n == 0) return ok();
  return hip_status(launch_kv_free(*pool, slots, n, (hipStream_t)stream), "free launch");
}

spear_status_t spear_kv_compact(const spear_kv_pool_t *pool, const spear_kv_cache_t *cache,
                                int32_t *used, spear_stream_t stream) {
  TRY(check_pool_cache(pool, cache));
  if (!used || !aligned(used, 4))
    return fail(SPEAR_ERR_INVALID_ARGUMENT, "used must be a 4-byte aligned device pointer");
  return hip_status(launch_kv_compact(*pool, page_desc(*cache), used, (hipStream_t)stream),
                    "compact launch");
}

}  // extern "C"
