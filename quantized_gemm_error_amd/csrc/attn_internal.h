// Host-side declarations shared by the attention and cache entry points and
// their kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/spear_attn.h"

namespace spear {

// Records the calling thread's last error and returns the status (api.hip).
spear_status_t set_last_error(spear_status_t st, const char *text);

// Everything an attention launcher needs, already validated.
struct AttnDesc {
  int dtype, D, Hq, Hkv, G;  // G = Hq / Hkv
  int page_size, num_pages;
  uint32_t p16_mul, p16_shift;  // i / (page_size / 16) = mulhi(i, mul) >> shift for i < 2^31; mul 0: i
  const uint16_t *k, *v;
  int64_t s_page, s_head, s_token;
  int n_seqs, width, n_tokens;
  const int32_t *table, *kv_lens, *q_starts;
  int window, sinks;
  float scale;
  const uint16_t *q;
  int64_t q_tok, q_head;
  uint16_t *out;
  int64_t o_tok, o_head;
  float *lse;
};

hipError_t launch_attn_decode(const AttnDesc &d, void *ws, hipStream_t s);
hipError_t launch_attn_prefill(const AttnDesc &d, void *ws, hipStream_t s);
size_t attn_decode_workspace(int D, int Hq, int Hkv, int n_seqs);
size_t attn_prefill_workspace(int D, int Hq, int Hkv, int n_seqs, int n_tokens);

struct AppendDesc {
  int H, D, page_size, num_pages;
  uint16_t *k, *v;
  int64_t s_page, s_head, s_token;
  int n_seqs, width, n_tokens;
  const int32_t *table, *kv_lens, *q_starts;
  const uint16_t *nk, *nv;
  int64_t k_tok, k_head, v_tok, v_head;
};
hipError_t launch_kv_append(const AppendDesc &d, hipStream_t s);

// A page of the cache as the copies see it: `layers` x [H][S] rows of D elements.
struct PageDesc {
  uint16_t *k, *v;
  int layers, num_pages, H, S, D;
  int64_t s_layer, s_page, s_head, s_token;
};
hipError_t launch_kv_copy_pages(const PageDesc &p, const int32_t *src, const int32_t *dst, int n,
                                hipStream_t s);
hipError_t launch_kv_fork(const spear_kv_pool_t &pool, const int32_t *src, const int32_t *dst,
                          int n, hipStream_t s);
hipError_t launch_kv_free(const spear_kv_pool_t &pool, const int32_t *slots, int n, hipStream_t s);
hipError_t launch_kv_reserve(const spear_kv_pool_t &pool, const PageDesc &p, const int32_t *slots,
                             const int32_t *new_lens, int n, int32_t *missing, hipStream_t s);
hipError_t launch_kv_compact(const spear_kv_pool_t &pool, const PageDesc &p, int32_t *used,
                             hipStream_t s);

}  // namespace spear
