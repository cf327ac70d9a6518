// The paged cache's bookkeeping and data movement: append, page copies, fork,
// reserve (allocation with copy on write), free, compact.
//
// All of it is index work and 16-byte copies, bound by memory or, at the
// sizes of one decode step, by launches: each call is one launch for the
// bookkeeping and, where pages move, one for the bytes.  Measured (MI355X):
// append of 32 tokens of 32 heads 3.0 us, of 5 chunks with 5672 tokens of 8
// heads 10.2 us (4.6 TB/s); fork and reserve of 32 samples with their part-full
// pages in 32 layers 28 us, of which the copies 17 us (5.8 TB/s); free and
// compact of a 2.5 GB cache of 8 layers 231 us, the copies 217 us (5.7 TB/s).
#include <algorithm>

#include "attn_internal.h"

namespace spear {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

__device__ __forceinline__ bool in_range(int v, int n) { return (uint32_t)v < (uint32_t)n; }

// ------------------------------------------------------------------ append

// One 16-byte piece per thread: piece c of head h of row t, keys and values.  (The
// blocks are numbered over both extents of the grid, one of which holds fewer than
// 2^32 threads.)
__global__ __launch_bounds__(kThreads) void append_kernel(AppendDesc d) {
  const int per_head = d.D / 8, per_row = per_head * d.H;
  const int64_t i = (blockIdx.x + (int64_t)gridDim.x * blockIdx.y) * kThreads + threadIdx.x;
  const int t = (int)(i / per_row);
  if (t >= d.n_tokens) return;
  const int rest = (int)(i - (int64_t)t * per_row), h = rest / per_head, c = rest - h * per_head;
  int b = t, pos;
  if (d.q_starts) {
    // the last sequence that starts at or before t
    int lo = 0, hi = d.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (d.q_starts[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    // (within the call's rows, as the attention has it)
    const int end = min(d.q_starts[b + 1], d.n_tokens);
    if (t < d.q_starts[b] || t >= end) return;
    pos = max(0, min(d.kv_lens[b], d.width * d.page_size)) - (end - t);
  } else {
    pos = max(0, min(d.kv_lens[b], d.width * d.page_size)) - 1;
  }
  if (pos < 0) return;
  const int pi = pos / d.page_size;
  const int page = d.table[(int64_t)b * d.width + pi];
  if (!in_range(page, d.num_pages)) return;
  const int64_t to = page * d.s_page + h * d.s_head + (pos - pi * d.page_size) * d.s_token + 8 * c;
  *(u32x4 *)(d.k + to) = *(const u32x4 *)(d.nk + t * d.k_tok + h * d.k_head + 8 * c);
  *(u32x4 *)(d.v + to) = *(const u32x4 *)(d.nv + t * d.v_tok + h * d.v_head + 8 * c);
}

// -------------------------------------------------------------- page copies

// What compaction changes besides the pages' bytes: the table's entries and
// the counts follow their pages.
struct Rename {
  spear_kv_pool_t pool;
  const int32_t *rank, *used;  // place of a moved page in src and dst; pages in use
};

__device__ void rename(const Rename &n, const int32_t *src, const int32_t *dst, int moves, int64_t i,
                       int64_t step) {
  const spear_kv_pool_t &p = n.pool;
  const int64_t entries = (int64_t)p.n_slots * p.table_width;
  const int used = *n.used;
  for (int64_t e = i; e < entries; e += step) {
    const int page = p.table[e];
    if (!in_range(page, p.num_pages) || page < used) continue;
    // (an entry that names a page nobody counts is left as it is)
    const int r = n.rank[page];
    if (in_range(r, moves) && src[r] == page) p.table[e] = dst[r];
  }
  for (int64_t r = i; r < moves; r += step) {
    const int a = src[r], b = dst[r];
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
}

// Workgroup (x, layer and array, z): pairs x, x + gridDim.x, ... of one array
// of one layer, 16 bytes per thread and step, bound by HBM: 5.4 TB/s of reads
// and writes for 1.25 GB in 8 layers.  The copies go past the caches (252 ->
// 237 us there), and so do compaction's sources, each read once (-> 230); a
// fork's are read once for every child and stay cached (read past the caches
// 29 -> 42 us for 8 children).  RENAME: planes of y past the arrays'
// rename the table.
template <bool RENAME>
__global__ __launch_bounds__(kThreads) void copy_pages_kernel(PageDesc p, const int32_t *src,
                                                              const int32_t *dst, int n,
                                                              const int32_t *count, Rename names) {
  if (count) n = min(n, *count);
  if constexpr (RENAME) {
    if ((int)blockIdx.y >= 2 * p.layers) {
      const int64_t block = blockIdx.x + (int64_t)gridDim.x * blockIdx.z;
      rename(names, src, dst, n, block * kThreads + threadIdx.x, (int64_t)gridDim.x * gridDim.z * kThreads);
      return;
    }
  }
  const int per_row = p.D / 8, pieces = per_row * p.H * p.S;
  uint16_t *base = ((blockIdx.y & 1) ? p.v : p.k) + (int64_t)(blockIdx.y >> 1) * p.s_layer;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int a = src[i], b = dst[i];
    if (a == b || !in_range(a, p.num_pages) || !in_range(b, p.num_pages)) continue;
    const uint16_t *from = base + a * p.s_page;
    uint16_t *to = base + b * p.s_page;
#pragma unroll 4
    for (int j = blockIdx.z * kThreads + threadIdx.x; j < pieces; j += gridDim.z * kThreads) {
      const int row = j / per_row, c = j - row * per_row;
      const int h = row / p.S, s = row - h * p.S;
      const int64_t off = h * p.s_head + s * p.s_token + 8 * c;
      const u32x4 *at = (const u32x4 *)(from + off);
      __builtin_nontemporal_store(RENAME ? __builtin_nontemporal_load(at) : *at, (u32x4 *)(to + off));
    }
  }
}

// n pairs; the renaming, if any, goes with the last launch (launches of 65534
// planes: the grid's second extent is 16 bits).
hipError_t copy_pages(const PageDesc &p, const int32_t *src, const int32_t *dst, int n, const int32_t *count,
                      const Rename *names, hipStream_t s) {
  if (n == 0) return hipSuccess;
  const int64_t pieces = (int64_t)p.D / 8 * p.H * p.S;
  const int x = std::min(n, 1024), z = (int)std::min<int64_t>((pieces + 4 * kThreads - 1) / (4 * kThreads), 64);
  constexpr int kMostLayers = 32766;
  for (int l = 0; l < p.layers; l += kMostLayers) {
    PageDesc q = p;
    q.layers = std::min(p.layers - l, kMostLayers);
    q.k += (int64_t)l * p.s_layer;
    q.v += (int64_t)l * p.s_layer;
    if (names && l + q.layers == p.layers)
      hipLaunchKernelGGL(copy_pages_kernel<true>, dim3(x, 2 * q.layers + 1, z), dim3(kThreads), 0, s, q, src, dst,
                         n, count, *names);
    else
      hipLaunchKernelGGL(copy_pages_kernel<false>, dim3(x, 2 * q.layers, z), dim3(kThreads), 0, s, q, src, dst,
                         n, count, Rename{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ------------------------------------------------------------ fork and free

// One thread per table entry of a dst slot: its old page loses a holder, the
// entry becomes the source's and that page gains one.  No dst is a src, so
// entries do not meet; the counts are integer atomics, which commute.
__global__ __launch_bounds__(kThreads) void fork_kernel(spear_kv_pool_t p, const int32_t *src,
                                                        const int32_t *dst) {
  const int a = src[blockIdx.y], b = dst[blockIdx.y];
  if (a == b || !in_range(a, p.n_slots) || !in_range(b, p.n_slots)) return;
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c == 0) p.lens[b] = p.lens[a];
  if (c >= p.table_width) return;
  int32_t *to = p.table + (int64_t)b * p.table_width + c;
  const int old = *to, now = p.table[(int64_t)a * p.table_width + c];
  if (old == now) return;
  if (in_range(old, p.num_pages)) atomicSub(&p.refs[old], 1);
  if (in_range(now, p.num_pages)) atomicAdd(&p.refs[now], 1);
  *to = now;
}

__global__ __launch_bounds__(kThreads) void free_kernel(spear_kv_pool_t p, const int32_t *slots) {
  const int b = slots[blockIdx.y];
  if (!in_range(b, p.n_slots)) return;
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c == 0) p.lens[b] = 0;
  if (c >= p.table_width) return;
  int32_t *to = p.table + (int64_t)b * p.table_width + c;
  const int old = *to;
  if (in_range(old, p.num_pages)) atomicSub(&p.refs[old], 1);
  *to = -1;
}

// ---------------------------------------------------------------- reserve

constexpr int kPlanThreads = 1024;

// Exclusive prefix sum over the workgroup's 1024 threads; total to all.
__device__ int block_scan(int v, int &total, int *waves /* 17 ints of LDS */) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();  // the LDS words may still be read from a call before
  if (lane == 63) waves[w] = inc;
  __syncthreads();
  if (threadIdx.x == 0) {
    int run = 0;
    for (int i = 0; i < kPlanThreads / 64; ++i) {
      const int x = waves[i];
      waves[i] = run;
      run += x;
    }
    waves[kPlanThreads / 64] = run;
  }
  __syncthreads();
  total = waves[kPlanThreads / 64];
  return waves[w] + inc - v;
}

// One workgroup: thread i plans entry i, then all find the lowest free pages
// and write them.  `taken`: scratch for the pages in order of use;
// move_src/move_dst: the pages to copy (-1: none), one pair per entry.
__global__ __launch_bounds__(kPlanThreads) void reserve_kernel(spear_kv_pool_t p,
                                                               const int32_t *slots,
                                                               const int32_t *new_lens, int n,
                                                               int32_t *missing, int32_t *taken,
                                                               int32_t *move_src,
                                                               int32_t *move_dst) {
  __shared__ int waves[kPlanThreads / 64 + 1];
  __shared__ int s_last[SPEAR_KV_MAX_ENTRIES], s_base[SPEAR_KV_MAX_ENTRIES + 1];
  __shared__ int s_slot[SPEAR_KV_MAX_ENTRIES], s_col[SPEAR_KV_MAX_ENTRIES];
  __shared__ int s_bad;
  const int i = threadIdx.x, S = p.page_size;
  // the first pages' counts, on their way while the entries are planned
  int ahead[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) ahead[u] = 4 * i + u < p.num_pages ? p.refs[4 * i + u] : 1;
  if (i == 0) s_bad = 0;
  __syncthreads();
  int slot = -1, have = 0, want = 0, last = -1, held = 0, need = 0;
  if (i < n) {
    slot = slots[i];
    want = new_lens[i];
    if (!in_range(slot, p.n_slots)) {
      s_bad = 1;
    } else {
      have = max(0, min(p.lens[slot], p.table_width * S));
      if (want > p.table_width * S) s_bad = 1;
      held = (have + S - 1) / S;
      if (want > have) {
        need = (int)(((int64_t)want + S - 1) / S);
        if (have % S != 0) {
          last = p.table[(int64_t)slot * p.table_width + held - 1];
          if (!in_range(last, p.num_pages)) last = -1;
        }
      }
    }
  }
  s_last[i] = last;
  __syncthreads();
  if (s_bad) {
    if (i == 0) *missing = -1;
    if (i < n) move_src[i] = move_dst[i] = -1;
    return;
  }
  // copy on write, as if entry by entry: an earlier copy leaves a holder less
  bool copies = false;
  if (last >= 0) {
    int holders = p.refs[last];
    for (int e = 0; e < i && holders > 1; ++e) holders -= s_last[e] == last;
    copies = holders > 1;
  }
  const int takes = max(0, need - held) + (copies ? 1 : 0);
  int total;
  const int base = block_scan(takes, total, waves);
  s_base[i] = base;
  if (i == 0) s_base[kPlanThreads] = total;
  s_slot[i] = slot;
  s_col[i] = copies ? held - 1 : held;
  // the lowest free pages, in order
  int found = 0;
  for (int p0 = 0; p0 < p.num_pages && found < total; p0 += 4 * kPlanThreads) {
    const int q = p0 + 4 * i;
    bool f[4];
    int c = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f[u] = p0 == 0 ? ahead[u] == 0 : q + u < p.num_pages && p.refs[q + u] == 0;
      c += f[u];
    }
    int some;
    int at = found + block_scan(c, some, waves);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (f[u] && at < total) taken[at++] = q + u;
    found += some;
  }
  __syncthreads();  // taken, s_base
  if (found < total) {
    if (i == 0) *missing = total - found;
    if (i < n) move_src[i] = move_dst[i] = -1;
    return;
  }
  if (i == 0) *missing = 0;
  if (i < n) {
    move_src[i] = copies ? last : -1;
    move_dst[i] = copies ? taken[base] : -1;
    if (copies) atomicSub(&p.refs[last], 1);
    if (want > have) p.lens[slot] = want;
  }
  for (int r = i; r < total; r += kPlanThreads) {
    int lo = 0, hi = kPlanThreads;  // the last entry whose pages start at or before r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_base[mid] <= r) lo = mid; else hi = mid;
    }
    const int page = taken[r];
    p.table[(int64_t)s_slot[lo] * p.table_width + s_col[lo] + r - s_base[lo]] = page;
    p.refs[page] = 1;
  }
}

// ---------------------------------------------------------------- compact

constexpr int kPagesPerBlock = 1024;

// Used pages in each run of 1024.
__global__ __launch_bounds__(kThreads) void count_used_kernel(const int32_t *refs, int P,
                                                              int32_t *counts) {
  __shared__ int sum;
  if (threadIdx.x == 0) sum = 0;
  __syncthreads();
  int c = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int q = blockIdx.x * kPagesPerBlock + u * kThreads + threadIdx.x;
    c += q < P && refs[q] > 0;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) c += __shfl_xor(c, o);
  if ((threadIdx.x & 63) == 0) atomicAdd(&sum, c);
  __syncthreads();
  if (threadIdx.x == 0) counts[blockIdx.x] = sum;
}

// With U pages in use: used page q has rank U - 1 - (used pages before q), its
// place counted from the highest; free page q has rank q - (used before q),
// counted from the lowest.  A used page at q >= U goes to the free page of
// its rank, which lies below U: both lists have as many entries as there are
// free pages below U.
// Without counts every workgroup counts the whole pool itself.
__global__ __launch_bounds__(kPagesPerBlock) void rank_pages_kernel(
    const int32_t *refs, int P, const int32_t *counts, int blocks, int32_t *src, int32_t *dst,
    int32_t *rank, int32_t *n_moves, int32_t *used) {
  __shared__ int waves[kPlanThreads / 64 + 1];
  int mine = 0, all = 0;  // used pages in the blocks before this one, and in all
  if (counts) {
    for (int k = threadIdx.x; k < blocks; k += kPagesPerBlock) {
      const int c = counts[k];
      all += c;
      if (k < (int)blockIdx.x) mine += c;
    }
  } else {
#pragma unroll 4
    for (int k = 0; k < blocks; ++k) {
      const int q = k * kPagesPerBlock + threadIdx.x;
      const int c = q < P && refs[q] > 0;
      all += c;
      if (k < (int)blockIdx.x) mine += c;
    }
  }
  int before, U;
  block_scan(mine, before, waves);
  block_scan(all, U, waves);
  const int q = blockIdx.x * kPagesPerBlock + threadIdx.x;
  const bool u = q < P && refs[q] > 0;
  int in_block;
  before += block_scan(u, in_block, waves);
  if (q < P) {
    if (u && q >= U) {
      const int r = U - 1 - before;
      src[r] = q;
      rank[q] = r;
    } else if (!u && q < U) {
      dst[q - before] = q;
    }
    if (q == U - 1) *n_moves = q + 1 - before - u;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *used = U;
    if (U == 0) *n_moves = 0;
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendDesc &d, hipStream_t s) {
  const int64_t pieces = (int64_t)d.n_tokens * d.H * (d.D / 8);
  const int64_t blocks = (pieces + kThreads - 1) / kThreads, x = std::min<int64_t>(blocks, 1 << 22);
  hipLaunchKernelGGL(append_kernel, dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(kThreads), 0, s, d);
  return hipGetLastError();
}

hipError_t launch_kv_copy_pages(const PageDesc &p, const int32_t *src, const int32_t *dst, int n,
                                hipStream_t s) {
  return copy_pages(p, src, dst, n, nullptr, nullptr, s);
}

hipError_t launch_kv_fork(const spear_kv_pool_t &pool, const int32_t *src, const int32_t *dst,
                          int n, hipStream_t s) {
  for (int i = 0; i < n; i += 65535) {
    hipLaunchKernelGGL(fork_kernel, dim3((pool.table_width + kThreads - 1) / kThreads, std::min(n - i, 65535)),
                       dim3(kThreads), 0, s, pool, src + i, dst + i);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv_free(const spear_kv_pool_t &pool, const int32_t *slots, int n, hipStream_t s) {
  for (int i = 0; i < n; i += 65535) {
    hipLaunchKernelGGL(free_kernel, dim3((pool.table_width + kThreads - 1) / kThreads, std::min(n - i, 65535)),
                       dim3(kThreads), 0, s, pool, slots + i);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv_reserve(const spear_kv_pool_t &pool, const PageDesc &p, const int32_t *slots,
                             const int32_t *new_lens, int n, int32_t *missing, hipStream_t s) {
  int32_t *move_src = pool.scratch, *move_dst = move_src + SPEAR_KV_MAX_ENTRIES;
  int32_t *taken = move_dst + SPEAR_KV_MAX_ENTRIES;
  hipLaunchKernelGGL(reserve_kernel, dim3(1), dim3(kPlanThreads), 0, s, pool, slots, new_lens, n,
                     missing, taken, move_src, move_dst);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : copy_pages(p, move_src, move_dst, n, nullptr, nullptr, s);
}

hipError_t launch_kv_compact(const spear_kv_pool_t &pool, const PageDesc &p, int32_t *used,
                             hipStream_t s) {
  const int P = pool.num_pages, blocks = (P + kPagesPerBlock - 1) / kPagesPerBlock;
  int32_t *src = pool.scratch, *dst = src + P, *rank = dst + P, *counts = rank + P;
  int32_t *n_moves = counts + blocks;
  // Up to 32 blocks of pages, counting the pool in every block (128 KB of
  // counts at most) takes less than a launch of its own.
  const bool counted = blocks > 32;
  if (counted)
    hipLaunchKernelGGL(count_used_kernel, dim3(blocks), dim3(kThreads), 0, s, pool.refs, P, counts);
  hipLaunchKernelGGL(rank_pages_kernel, dim3(blocks), dim3(kPagesPerBlock), 0, s, pool.refs, P,
                     counted ? counts : nullptr, blocks, src, dst, rank, n_moves, used);
  const hipError_t e = hipGetLastError();
  const Rename names{pool, rank, used};
  return e != hipSuccess ? e : copy_pages(p, src, dst, P, n_moves, &names, s);
}

}  // namespace spear
