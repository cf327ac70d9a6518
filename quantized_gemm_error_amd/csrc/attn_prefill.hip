// Causal attention of the batch's new tokens over the paged cache.
//
// With s = q . k scale log2(e), tiles of 64 keys pass by a block of query rows
// that keeps a reference m >= (row maximum) - 8, l = sum 2^(s - m) and
// o = sum 2^(s - m) v in fp32 (m is raised, and l and o scaled, only when a
// maximum passes it by more than 8: the weights stay below 2^8, and their
// relative rounding is the same); out = o / l, lse = ln 2 (m + log2 l).
//
// The work is two matrix products, 4 D flops per visible pair, so MFMA bounds
// it.  A workgroup of four waves owns 128 rows of one key-value head: the
// query heads of a token that share it are neighbouring rows (row = token x
// G + head), so short chunks of grouped heads fill tiles too and share every
// staged key.  Each wave takes 32 rows with 32x32x16 MFMAs, transposed so that
// no value changes lanes:
//   - S^T = K Q^T, keys as rows, queries as columns: lane (c, h) =
//     (lane % 32, lane / 32) holds the scores of query c with keys
//     8 i + 4 h + 0..3, so a softmax row is one lane's registers and its
//     partner's 32 lanes away.
//   - O^T = V^T P^T, dims as rows: a lane's eight scores of each 16 keys,
//     rounded to the type, are the column operand as they are, if V's row
//     operand takes the keys in that order, 4 h + 0..3 and 8 + 4 h + 0..3:
//     two transposing LDS reads (ds_read_b64_tr_b16) of four keys each.
// K and V go from memory to LDS directly (16 bytes per lane), one 64-key tile
// ahead, into two buffers, so one barrier per tile suffices; a wave stages 16
// keys, which lie in one page.  Such a load stores lane i's bytes at base +
// 16 i, so rows cannot be padded; instead each row's 16-byte chunks are
// permuted by the row on the way in (the lane's source address), so that the
// operand reads spread over the banks.
// Keys past the cached length and pages out of range read as zeros (buffer
// range), so that the 0 weights of hidden keys meet numbers.  A hidden key
// that is in the cache (a later token of the chunk, one before the window) may
// hold infinities or NaN: tiles that need a mask are looked over while staged,
// and take a slower path if they hold any.
#include <algorithm>
#include <type_traits>

#include "attn_device.h"

namespace spear {

namespace {

constexpr int kRows = 128;  // query rows of a workgroup
constexpr int kKeys = 64;   // keys of a tile
constexpr int kWaves = 4;
constexpr float kSlack = 8.f;  // by how much a maximum may pass m

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t *tr_ptr;

// The 32-byte segment permutation of V's row t: with it the four rows of a
// transposing read lie in different banks, also together with their
// neighbouring segments.
template <int D>
__device__ __forceinline__ int v_swizzle(int t) {
  t &= 3;
  return D == 128 ? 2 * t + ((t ^ (t >> 1)) & 1) : t;
}

// Where the rows of work item w (of one key-value head) lie: sequence, its
// rows and the first of them.  Items are blocks of kRows rows; the last
// blocks of a batch, which see the most keys, come first.
struct Block {
  int b, start, n, row0;  // first token, tokens, first row in the block
};
__device__ __forceinline__ bool find_block(const AttnDesc &d, int w, Block &k) {
  const int lane = threadIdx.x & 63;
  const auto span = [&](int b, int &start) {
    start = b;
    if (!d.q_starts) return 1;
    start = max(0, min(d.q_starts[b], d.n_tokens));
    return max(0, min(d.q_starts[b + 1], d.n_tokens) - start);
  };
  const auto blocks_of = [&](int b) {
    int start;
    return b < d.n_seqs ? (int)(((int64_t)span(b, start) * d.G + kRows - 1) / kRows) : 0;
  };
  int total = 0;
  for (int b0 = 0; b0 < d.n_seqs; b0 += 64) total += wave_total(blocks_of(b0 + lane));
  w = total - 1 - w;
  if (w < 0) return false;
  int before = 0;
  for (int b0 = 0; b0 < d.n_seqs; b0 += 64) {
    const int n = blocks_of(b0 + lane), upto = before + wave_scan(n);
    const int all = __builtin_amdgcn_readlane(upto, 63);
    if (w < all) {
      const int at = __builtin_popcountll(__ballot(upto <= w));
      k.b = b0 + at;
      if (k.b >= d.n_seqs) return false;
      k.row0 = kRows * (w - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(n, at)));
      k.n = span(k.b, k.start);
      return k.row0 >= 0 && k.row0 < (int64_t)k.n * d.G;
    }
    before = all;
  }
  return false;
}

template <int DT, int D>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_prefill_kernel(AttnDesc d) {
  constexpr int CH = D / 8;          // 16-byte chunks of a row
  constexpr int KS = D / 16;         // contraction steps of S
  constexpr int DB = D / 32;         // 32-dim blocks of O
  constexpr int RPI = 64 / CH;       // rows a wave's load instruction brings
  constexpr int LOADS = 16 / RPI;    // instructions for 16 keys
  constexpr int TILE = kKeys * D * 2;  // bytes of a staged K or V tile
  __shared__ __attribute__((aligned(256))) char s_kv[4][TILE];  // K tiles of even and odd t, then V's
  __shared__ uint32_t s_weights[D == 64 ? kWaves * 16 * 64 : 1];  // (slow path; D = 128: the K tile)
  __shared__ int s_dirty[2][kWaves];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int kvh = blockIdx.x % d.Hkv;
  Block blk;
  if (!find_block(d, blockIdx.x / d.Hkv, blk)) return;
  blk = {uniform(blk.b), uniform(blk.start), uniform(blk.n), uniform(blk.row0)};

  const int len = uniform(cached_len(d, blk.b)), past = len - blk.n;  // position of the first new token
  const int all_rows = blk.n * d.G;
  const int wrow0 = blk.row0 + 32 * wave;
  const int row = wrow0 + col;
  const bool is_row = row < all_rows;
  const int tok = min(row, all_rows - 1) / d.G, head = kvh * d.G + min(row, all_rows - 1) - tok * d.G;
  const int pos = is_row ? past + tok : -1;
  // positions of the first and last rows, of the block and of the wave
  const int p_min = past + blk.row0 / d.G, p_max = past + (min(blk.row0 + kRows, all_rows) - 1) / d.G;
  const bool active = wrow0 < all_rows;
  const int w_end = min(wrow0 + 32, all_rows);
  const int w_min = past + wrow0 / d.G, w_max = past + (w_end - 1) / d.G;

  // the 64-key tiles that some row sees: from position 0 for the sinks, then
  // from lo_tile on
  const int lo = d.window > 0 ? max(0, p_min - d.window + 1) : 0;
  const int lo_tile = lo / kKeys;
  const int sink_tiles = min((min(d.sinks, lo) + kKeys - 1) / kKeys, lo_tile);
  const int tiles = p_max < 0 ? 0 : sink_tiles + p_max / kKeys + 1 - lo_tile;
  const auto key_of = [&](int t) { return kKeys * (t < sink_tiles ? t : t - sink_tiles + lo_tile); };

  // queries, the column operand of S
  u32x4_t q[KS];
  {
    const uint16_t *from = d.q + (int64_t)(blk.start + tok) * d.q_tok + head * d.q_head + 8 * half;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      q[k] = *(const u32x4_t *)(from + 16 * k);
      if (d.scale < 0.f) q[k] ^= 0x80008000u;
    }
  }
  // scores stay unscaled (a negative scale has turned the query's sign): the
  // weight is 2^(s scale - m scale), one fma
  const float scale = fmaxf(fabsf(d.scale) * kLog2e, 1e-30f), slack = kSlack / scale;

  // staging: this wave's 16 keys of a tile
  int k_src[LOADS], v_src[LOADS];  // byte offsets from the first key
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int t = i * RPI + lane / CH, c = lane % CH;
    k_src[i] = 2 * (t * (int)d.s_token + 8 * (c ^ (t & (CH - 1))));
    v_src[i] = 2 * (t * (int)d.s_token + 8 * ((((c >> 1) ^ v_swizzle<D>(t)) << 1) | (c & 1)));
  }
  const int p16 = d.page_size / 16, halves = d.width * p16;
  // page of 16-key group i of the sequence, -1 where there is none
  const auto page_of = [&](int i) {
    const int page = i < halves ? uniform(scalar_load(d.table, (int64_t)blk.b * d.width + i / p16)) : -1;
    return (uint32_t)page < (uint32_t)d.num_pages ? page : -1;
  };
  // Where this wave's 16 keys of the tile at key0 lie; which of the tile's
  // groups are hidden.
  struct Source {
    int64_t off;
    int bytes, hidden;
  };
  const auto source_of = [&](int key0) {
    Source src;
    int mine = -1;
    src.hidden = 0;
#pragma unroll
    for (int u = 0; u < kKeys / 16; ++u) {
      const int page = page_of(key0 / 16 + u);
      src.hidden |= (page < 0) << u;
      if (u == wave) mine = page;
    }
    const int i = key0 / 16 + wave;
    src.off = max(mine, 0) * d.s_page + (int64_t)kvh * d.s_head + (int64_t)(i % p16) * 16 * d.s_token;
    src.bytes = mine < 0 ? 0 : max(0, min(16, len - 16 * i)) * 2 * (int)d.s_token;
    return src;
  };
  const uint32_t lds = lds_offset(s_kv), mine_at = 16 * wave * D * 2;
  const auto load_tile = [&](const uint16_t *base, const Source &src, uint32_t to, const int *from) {
    const u32x4_t r = buffer_words(base + src.off, src.bytes);
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      load_to_lds(r, (uint32_t)uniform((int)(to + mine_at + j * RPI * D * 2)), from[j]);
  };

  // operand addresses in a tile: K row `col`, step 0 (step k: ^ 32 k); V row
  // 4 half + l/4 % 4, dim block 0 (block b: ^ 64 b)
  const int k_at = col * D * 2 + 16 * (half ^ (col & (CH - 1)));
  const int v_at = (4 * half + ((lane & 15) >> 2)) * D * 2 +
                   32 * (((lane >> 4) & 1) ^ v_swizzle<D>((lane & 15) >> 2)) + 8 * (lane & 3);

  f32x16_t acc[DB], s[2];
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[b][v] = 0.f;
  float m = kNoMax, l = 0.f;
  const int window = d.window > 0 ? d.window : 0x7FFFFFFF;
  // whether some row of positions first..last does not see all of a tile
  const auto partly = [&](int key0, int first, int last) {
    return key0 + kKeys - 1 > first || (last - key0 >= window && key0 + kKeys > d.sinks);
  };
  // scores of a tile's keys 32 u .. 32 u + 31
  const auto scores = [&](const char *kt, int u) {
    f32x16_t c;
#pragma unroll
    for (int v = 0; v < 16; ++v) c[v] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k)
      c = mfma_32x32x16<DT>(*(const u32x4_t *)(kt + (k_at ^ (32 * k)) + u * 32 * D * 2), q[k], c);
    return c;
  };

  // The tiles that some row of this wave sees are the first w_tiles (those
  // that a window hides from all of its rows are computed and masked).
  const int w_tiles = !active || w_max < 0 ? 0 : min(tiles, tiles - (p_max / kKeys - w_max / kKeys));
  if (tiles > 0) {
    Source now = source_of(key_of(0)), next = now;
    load_tile(d.k, now, lds, k_src);
    __builtin_amdgcn_s_waitcnt(0x0F70);
    lds_barrier();
    load_tile(d.v, now, lds + 2 * TILE, v_src);
    if (tiles > 1) {
      next = source_of(key_of(1));
      load_tile(d.k, next, lds + TILE, k_src);
    }
    if (w_tiles > 0) {
      s[0] = scores(s_kv[0], 0);
      s[1] = scores(s_kv[0], 1);
    }
    for (int t = 0; t < tiles; ++t) {
      // here: s holds tile t's scores; V of t and K of t + 1 are on their way
      const int buf = t & 1, key0 = key_of(t), hidden = now.hidden;
      const char *kt = s_kv[buf ^ 1], *vt = s_kv[2 + buf];
      const bool masked = partly(key0, p_min, p_max);
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's parts are in LDS
      if (masked) {  // (only V: a score that is no number is replaced, a weight of 0 is not)
        bool any = false;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          u32x4_t *at = (u32x4_t *)(s_kv[2 + buf] + mine_at + j * RPI * D * 2 + 16 * lane);
          u32x4_t x = *at;
          uint32_t bad = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) bad |= not_finite<DT>(x[e]);
          if (__any(bad != 0)) {  // left out of the products, added below
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] &= ~((not_finite<DT>(x[e]) >> 15) * 0xFFFFu);
            *at = x;
            any = true;
          }
        }
        if (lane == 0) s_dirty[buf][wave] = any;
      }
      lds_barrier();
      now = next;
      if (t + 1 < tiles) load_tile(d.v, now, lds + (2 + (buf ^ 1)) * TILE, v_src);
      if (t + 2 < tiles) {
        next = source_of(key_of(t + 2));
        load_tile(d.k, next, lds + buf * TILE, k_src);
      }
      const bool dirty = masked && (s_dirty[buf][0] | s_dirty[buf][1] | s_dirty[buf][2] | s_dirty[buf][3]);
      const bool mine = t < w_tiles;
      if (!mine && !dirty) continue;

      if (hidden || partly(key0, w_min, w_max) || !is_row) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int j = key0 + 32 * u + 8 * (v >> 2) + 4 * half + (v & 3);
            const bool sees = (j <= pos) & ((pos - j < window) | (j < d.sinks)) &
                              (((hidden >> (2 * u + (v >> 3))) & 1) == 0);
            s[u][v] = sees ? s[u][v] : -INFINITY;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 16; ++v) top = fmaxf(top, s[u][v]);
      if (__any(top > m + slack)) {
        top = over_halves(top, [](float a, float b) { return fmaxf(a, b); });
        const float m2 = fmaxf(m, top), f = __builtin_amdgcn_exp2f((m - m2) * scale);
        m = m2;
        l *= f;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[b][v] *= f;
      }
      // the weights of 16 keys each, as the column operand of O; meanwhile the
      // matrix unit forms the next tile's scores
      u32x4_t p[4];
      const float shift = -m * scale;
      f32x16_t ahead[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        ahead[u] = scores(kt, u);
#pragma unroll
        for (int v = 0; v < 16; v += 2) {
          const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][v], scale, shift));
          const float b = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][v + 1], scale, shift));
          l += a + b;
          p[2 * u + (v >> 3)][(v >> 1) & 3] = pack_pair<DT>(a, b);
        }
      }
      s[0] = ahead[0];
      s[1] = ahead[1];
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          const char *from = vt + (v_at ^ (64 * b)) + g * 16 * D * 2;
          const uint2 x = bitcast<uint2>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)from));
          const uint2 y = bitcast<uint2>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)(from + 8 * D * 2)));
          acc[b] = mfma_32x32x16<DT>(u32x4_t{x.x, x.y, y.x, y.y}, p[g], acc[b]);
        }
      if (!dirty) continue;
      // Values that are not finite, key by key, for the rows that see them.
      // The weights go through LDS (D = 128: where the K tile was, once every
      // wave is past it), the values come from memory again.
      lds_barrier();
      uint32_t *w_at = (D == 64 ? s_weights : (uint32_t *)kt) + wave * 16 * 64;
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) w_at[(4 * g + e) * 64 + lane] = p[g][e];
      lds_barrier();
      if (!mine) continue;
      for (int j = 0; j < kKeys; ++j) {
        const int key = key0 + j, page = page_of(key / 16);
        if (page < 0 || key >= len) continue;
        const int in16 = j & 15, e = (in16 & 3) + 4 * (in16 >> 3);
        const uint32_t pair = w_at[(4 * (j >> 4) + (e >> 1)) * 64 + col + 32 * ((in16 >> 2) & 1)];
        const float w = to_f32<DT>((uint16_t)(e & 1 ? pair >> 16 : pair));
        const bool sees = (key <= pos) & ((pos - key < window) | (key < d.sinks));
        const uint16_t *from = d.v + page * d.s_page + (int64_t)kvh * d.s_head +
                               (int64_t)(key % d.page_size) * d.s_token + 4 * half;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4) {  // dims 32 b + 8 v4 + 4 half + 0..3
            const uint2 x = *(const uint2 *)(from + 32 * b + 8 * v4);
#pragma unroll
            for (int e2 = 0; e2 < 4; ++e2) {
              const uint32_t y = e2 < 2 ? x.x : x.y;
              const uint16_t bits = (uint16_t)(e2 & 1 ? y >> 16 : y);
              if (sees & (not_finite<DT>(bits) != 0)) acc[b][4 * v4 + e2] += w * to_f32<DT>(bits);
            }
          }
      }
    }
  }
  l = over_halves(l, [](float a, float b) { return a + b; });
  if (!is_row) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  uint16_t *to = d.out + (int64_t)(blk.start + tok) * d.o_tok + head * d.o_head + 4 * half;
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int v = 0; v < 16; v += 4)
      *(uint2 *)(to + 32 * b + 2 * v) = uint2{pack_pair<DT>(acc[b][v] * inv, acc[b][v + 1] * inv),
                                              pack_pair<DT>(acc[b][v + 2] * inv, acc[b][v + 3] * inv)};
  if (d.lse && half == 0)
    d.lse[(int64_t)(blk.start + tok) * d.Hq + head] =
        l != 0.f ? (m * scale + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t attn_prefill_workspace(int D, int Hq, int Hkv, int n_seqs, int n_tokens) { return 0; }

hipError_t launch_attn_prefill(const AttnDesc &d, void *ws, hipStream_t s) {
  const int64_t blocks = (int64_t)d.n_tokens * d.G / kRows + d.n_seqs;
  auto *k = d.D == 64 ? (d.dtype == DT_F16 ? attn_prefill_kernel<DT_F16, 64> : attn_prefill_kernel<DT_BF16, 64>)
                      : (d.dtype == DT_F16 ? attn_prefill_kernel<DT_F16, 128> : attn_prefill_kernel<DT_BF16, 128>);
  hipLaunchKernelGGL(k, dim3((unsigned)(blocks * d.Hkv)), dim3(64 * kWaves), 0, s, d);
  return hipGetLastError();
}

}  // namespace spear
