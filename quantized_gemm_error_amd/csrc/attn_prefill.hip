// Causal attention of the batch's new tokens over the paged cache.
//
// The simplest form: one wave per row and query head goes through the keys
// that the row sees, one at a time, with the running maximum m, sum l and
// output o of the softmax in fp32:
//   m' = max(m, s), l' = l e^(m - m') + e^(s - m'), o' = o e^(m - m') + e^(s - m') v.
#include "attn_device.h"

namespace spear {

namespace {

template <int DT, int D>
__global__ __launch_bounds__(64) void attn_rows_kernel(AttnDesc d) {
  constexpr int E = D / 64;  // elements per lane
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  int b = t, n = 1, i = 0;
  if (d.q_starts) {
    int lo = 0, hi = d.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (d.q_starts[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    if (t < d.q_starts[b] || t >= d.q_starts[b + 1]) return;
    n = d.q_starts[b + 1] - d.q_starts[b];
    i = t - d.q_starts[b];
  }
  const int p = cached_len(d, b) - n + i;
  const Seen see = seen_by(p, d.window, d.sinks);
  float q[E], o[E], m = -1e30f, l = 0.f;  // (a finite m: a score of -inf weighs 0)
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_f32<DT>(d.q[t * d.q_tok + h * d.q_head + lane * E + e]) * d.scale;
    o[e] = 0.f;
  }
  for (int j = see.sink > 0 ? 0 : see.lo; j <= p; ++j) {
    if (j == see.sink) j = see.lo;
    const int pi = j / d.page_size;
    const int page = d.table[(int64_t)b * d.width + pi];
    if ((uint32_t)page >= (uint32_t)d.num_pages) continue;
    const int64_t at = page * d.s_page + (h / d.G) * d.s_head + (j - pi * d.page_size) * d.s_token + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * to_f32<DT>(d.k[at + e]);
#pragma unroll
    for (int o2 = 32; o2 > 0; o2 >>= 1) s += __shfl_xor(s, o2);
    const float m2 = fmaxf(m, s), c = __expf(m - m2), w = __expf(s - m2);
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * to_f32<DT>(d.v[at + e]);
    m = m2;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    d.out[t * d.o_tok + h * d.o_head + lane * E + e] = from_f32<DT>(l != 0.f ? o[e] / l : 0.f);
  if (d.lse && lane == 0) d.lse[(int64_t)t * d.Hq + h] = l != 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attn_prefill_workspace(int D, int Hq, int Hkv, int n_seqs, int n_tokens) { return 0; }

hipError_t launch_attn_prefill(const AttnDesc &d, void *ws, hipStream_t s) {
  auto *k = d.D == 64 ? (d.dtype == DT_F16 ? attn_rows_kernel<DT_F16, 64> : attn_rows_kernel<DT_BF16, 64>)
                      : (d.dtype == DT_F16 ? attn_rows_kernel<DT_F16, 128> : attn_rows_kernel<DT_BF16, 128>);
  hipLaunchKernelGGL(k, dim3(d.n_tokens, d.Hq), dim3(64), 0, s, d);
  return hipGetLastError();
}

}  // namespace spear
