// Attention of one new token per sequence over the paged cache.
//
// With s_j = q . k_j log2(e) scale over the visible keys j, every wave keeps
// a running maximum m, l = sum 2^(s_j - m) and o = sum 2^(s_j - m) v_j over
// its share of the keys; parts join as
//     M = max m_i,  L = sum 2^(m_i - M) l_i,  o = sum 2^(m_i - M) o_i / L.
//
// Each key and value is read once, so the floor is the cache's bytes over the
// HBM rate; the rest is arranged around that stream.
//
// A wave takes 32 keys at a time, for the (up to 16) query heads that share a
// key-value head: S^T = K Q^T as 16x16x32 MFMAs with the keys as rows, and
// O^T = V^T P^T with the head dimension as rows.  Both K and V go from memory
// straight into MFMA operand registers, with no LDS and no cross-lane moves:
//   - K as the row operand: lane (r, g) = (lane % 16, lane / 16) loads 16
//     bytes of key r, at dims 32 c + 8 g for step c.
//   - S^T leaves lane (r, g) the scores of head r with keys 4 g + 0..3 of
//     each 16-key half: eight of the 32 keys, which are taken as the eight
//     contraction places of group g in the second product.  The weights are
//     then already where the column operand wants them.
//   - V as the row operand of that product needs, in lane (r, g), those same
//     eight keys at one head dimension per row r.  The lane loads D / 16
//     neighbouring dims (D/16 r ..) of each of its eight keys (four lanes'
//     groups read four whole rows at once), and pairs of keys are interleaved
//     in registers (v_perm): row r of product j is dim D/16 r + j.
// The matrix units do at most 16/G times the needed work and are still idle
// most of the time (per 32 keys and wave 256 cycles of MFMA at D = 128).
#include <algorithm>

#include "attn_device.h"

namespace spear {

namespace {

constexpr int kTile = 32;        // keys a wave takes at a time
constexpr int kSlots = 512;      // workgroups wanted when sequences are split
constexpr int kMinTiles = 16;    // tiles below which a sequence is not split

// What a sequence's query sees as a list of 32-key tiles: `sink_tiles` from
// position 0, then those from lo_tile on.
struct TileList {
  int len, sink, lo, sink_tiles, lo_tile, tiles;
  __device__ __forceinline__ TileList(int len_, int window, int sinks) : len(len_) {
    const Seen s = seen_by(len - 1, window, sinks);
    sink = s.sink;
    lo = s.lo;
    lo_tile = lo / kTile;
    sink_tiles = min((sink + kTile - 1) / kTile, lo_tile);
    tiles = sink_tiles + (len + kTile - 1) / kTile - lo_tile;
  }
};

// A workgroup's share: tiles [first, last) of sequence b, part `split` of
// `splits`; `slot`: the first of the sequence's places among split parts.
struct Share {
  int b, split, splits, slot, tiles_per;
};

// Share w of the batch's work, the same computation in every wave: the tiles
// of all sequences and heads over kSlots workgroups give the tiles per part,
// raised until the parts fit in the slots (unless the sequences alone
// outnumber them), so that they all run at once.
__device__ __forceinline__ bool find_share(const AttnDesc &d, int w, int heads, bool may_split,
                                           Share &sh) {
  const int lane = threadIdx.x & 63;
  const auto tiles_of = [&](int b) {
    return b < d.n_seqs ? TileList(cached_len(d, b), d.window, d.sinks).tiles : 0;
  };
  const int mine = tiles_of(lane);  // of the first 64 sequences
  int total = wave_total(mine);
  for (int b0 = 64; b0 < d.n_seqs; b0 += 64) total += wave_total(tiles_of(b0 + lane));
  const int room = max(kSlots / heads, 1);  // parts of one head
  int per = max(kMinTiles, (total + room - 1) / room);
  if (may_split) {
    for (int i = 0; i < 6; ++i) {
      int parts = wave_total((mine + per - 1) / per);
      for (int b0 = 64; b0 < d.n_seqs; b0 += 64)
        parts += wave_total((tiles_of(b0 + lane) + per - 1) / per);
      if (parts <= room || parts <= d.n_seqs) break;
      per += (per + 7) / 8;
    }
  } else {
    per = 1 << 30;
  }
  int before = 0, split_before = 0;
  for (int b0 = 0; b0 < d.n_seqs; b0 += 64) {
    const int t = b0 == 0 ? mine : tiles_of(b0 + lane);
    const int n = b0 + lane < d.n_seqs ? max(1, (t + per - 1) / per) : 0;
    const int upto = before + wave_scan(n), split_upto = split_before + wave_scan(n > 1 ? n : 0);
    const int all = __builtin_amdgcn_readlane(upto, 63);
    if (w < all) {
      const int at = __builtin_popcountll(__ballot(upto <= w));
      sh.b = b0 + at;
      sh.splits = __builtin_amdgcn_readlane(n, at);
      sh.split = w - (__builtin_amdgcn_readlane(upto, at) - sh.splits);
      sh.slot = __builtin_amdgcn_readlane(split_upto, at) - (sh.splits > 1 ? sh.splits : 0);
      sh.tiles_per = per;
      return true;
    }
    before = all;
    split_before = __builtin_amdgcn_readlane(split_upto, 63);
  }
  return false;
}

template <int DT, int D, int NW>
__global__ __launch_bounds__(64 * NW) void attn_decode_kernel(AttnDesc d, int heads, int head_blocks,
                                                              bool may_split, uint32_t *counters,
                                                              float *parts, int part_bytes) {
  constexpr int E = D / 16;   // dims a lane holds of a value
  constexpr int KC = D / 32;  // contraction steps of the first product
  typedef uint32_t vec_t __attribute__((ext_vector_type(E / 2)));
  __shared__ float s_o[NW][16][D + 4], s_m[NW][16], s_l[NW][16];
  __shared__ int s_last;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int hd = blockIdx.x % heads;
  Share sh;
  if (!find_share(d, blockIdx.x / heads, heads, may_split, sh)) return;
  const int kvh = hd / head_blocks, h0 = kvh * d.G + 16 * (hd % head_blocks);
  const int rows = min(16, d.G - 16 * (hd % head_blocks));  // query heads of this workgroup

  const TileList tl(cached_len(d, sh.b), d.window, d.sinks);
  const int first = sh.split * sh.tiles_per, last = min(first + sh.tiles_per, tl.tiles);

  // queries: the column operand, column r = head h0 + r
  u32x4_t q[KC];
#pragma unroll
  for (int c = 0; c < KC; ++c)
    q[c] = r < rows ? *(const u32x4_t *)(d.q + sh.b * d.q_tok + (h0 + r) * d.q_head + 32 * c + 8 * g)
                    : u32x4_t{0u, 0u, 0u, 0u};

  const int p16 = d.page_size / 16;  // 16-key halves per page
  const int halves = d.width * p16;
  const int64_t row = (int64_t)sh.b * d.width;
  struct Half {
    int page;     // -1: hidden
    int64_t off;  // of its first key, this head
  };
  const auto half_at = [&](int i) {
    Half h;
    const int pi = i / p16;
    int page = i < halves ? scalar_load(d.table, row + pi) : -1;
    if ((uint32_t)page >= (uint32_t)d.num_pages) page = -1;
    h.page = page;
    h.off = max(page, 0) * d.s_page + (int64_t)kvh * d.s_head + (int64_t)(i - pi * p16) * 16 * d.s_token;
    return h;
  };
  const auto real_tile = [&](int t) { return t < tl.sink_tiles ? t : t - tl.sink_tiles + tl.lo_tile; };
  const uint32_t k_off = r * (uint32_t)d.s_token + 8 * g;
  const uint32_t v_off = 4 * g * (uint32_t)d.s_token + E * r, tok = (uint32_t)d.s_token;

  u32x4_t kr[2][KC];
  vec_t vr[8];
  f32x4_t acc[E];
  float m = kNoMax, l = 0.f;
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const auto load_k = [&](const Half *h) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < KC; ++c) kr[u][c] = *(const u32x4_t *)(d.k + h[u].off + (k_off + 32 * c));
  };
  const auto load_v = [&](const Half *h) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) vr[4 * u + i] = *(const vec_t *)(d.v + h[u].off + (v_off + i * tok));
  };

  const float scale = d.scale * kLog2e;
  int t = first + wave;
  Half now[2], next[2];
  if (t < last) {
    now[0] = half_at(2 * real_tile(t));
    now[1] = half_at(2 * real_tile(t) + 1);
    load_k(now);
    load_v(now);
  }
  for (; t < last; t += NW) {
    const int key0 = real_tile(t) * kTile;
    const bool more = t + NW < last;
    if (more) {
      next[0] = half_at(2 * real_tile(t + NW));
      next[1] = half_at(2 * real_tile(t + NW) + 1);
    }
    f32x4_t s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KC; ++c) s[u] = mfma_16x16x32<DT>(kr[u][c], q[c], s[u]);
    }
    if (more) load_k(next);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s[e >> 2][e & 3] * scale;
    // hidden keys: weight 0, and no value of theirs meets that 0
    if (!((key0 >= tl.lo || key0 + kTile <= tl.sink) && key0 + kTile <= tl.len && now[0].page >= 0 &&
          now[1].page >= 0)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = key0 + 16 * (e >> 2) + 4 * g + (e & 3);
        if (!((j < tl.sink || j >= tl.lo) && j < tl.len && now[e >> 2].page >= 0)) {
          x[e] = -INFINITY;
          vr[e] = vec_t(0u);
        }
      }
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
    if (__any(top > m)) {
      const float m2 = fmaxf(m, columns_max(top)), f = __builtin_amdgcn_exp2f(m - m2);
      m = m2;
      l *= f;
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] *= f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = __builtin_amdgcn_exp2f(x[e] - m);
      l += x[e];
    }
    // the weights rounded to the type, as the second product's column operand
    u32x4_t p;
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = pack_pair<DT>(x[2 * e], x[2 * e + 1]);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      u32x4_t a;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        a[e] = __builtin_amdgcn_perm(vr[2 * e + 1][j / 2], vr[2 * e][j / 2],
                                     (j & 1) ? 0x07060302u : 0x05040100u);
      acc[j] = mfma_16x16x32<DT>(a, p, acc[j]);
    }
    if (more) {
      load_v(next);
      now[0] = next[0];
      now[1] = next[1];
    }
  }
  l = columns_sum(l);

  // the waves' parts, joined in wave order
  if (r < rows) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int j = 0; j < E; ++j) s_o[wave][r][E * (4 * g + v) + j] = acc[j][v];
    if (g == 0) {
      s_m[wave][r] = m;
      s_l[wave][r] = l;
    }
  }
  __syncthreads();
  constexpr int Q4 = D / 4;
  const auto part_rs = __builtin_amdgcn_make_buffer_rsrc(parts, (short)0, part_bytes, 0x00020000);
  const auto part_at = [&](int split, int h) {  // byte offset of a part's row
    return (((sh.slot + split) * heads + hd) * 16 + h) * (D + 4) * 4;
  };
  for (int i = threadIdx.x; i < rows * Q4; i += 64 * NW) {
    const int h = i / Q4, c = 4 * (i % Q4);
    float M = s_m[0][h], L = 0.f;
#pragma unroll
    for (int w = 1; w < NW; ++w) M = fmaxf(M, s_m[w][h]);
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = __builtin_amdgcn_exp2f(s_m[w][h] - M);
      L += f * s_l[w][h];
      o += f * *(const f32x4_t *)&s_o[w][h][c];
    }
    if (sh.splits == 1) {
      const float inv = L != 0.f ? 1.f / L : 0.f;
      uint32_t *to = (uint32_t *)(d.out + sh.b * d.o_tok + (h0 + h) * d.o_head + c);
      to[0] = pack_pair<DT>(o[0] * inv, o[1] * inv);
      to[1] = pack_pair<DT>(o[2] * inv, o[3] * inv);
      if (d.lse && c == 0)
        d.lse[(int64_t)sh.b * d.Hq + h0 + h] = L != 0.f ? (M + __builtin_amdgcn_logf(L)) * kLn2 : -INFINITY;
    } else {
      store_partials4(o, part_rs, part_at(sh.split, h) + c * 4);
      if (c == 0) store_partials4(f32x4_t{M, L, 0.f, 0.f}, part_rs, part_at(sh.split, h) + D * 4);
    }
  }
  if (sh.splits == 1) return;

  // the sequence's parts: the workgroup that completes them joins them, in
  // the order of the splits
  publish_wait();
  __syncthreads();
  uint32_t *counter = counters + (sh.b * heads + hd);
  if (threadIdx.x == 0)
    s_last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             (uint32_t)sh.splits - 1;
  __syncthreads();
  if (!s_last) return;
  if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = threadIdx.x; i < rows * Q4; i += 64 * NW) {
    const int h = i / Q4, c = 4 * (i % Q4);
    float M = kNoMax, L = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < sh.splits; s0 += 8) {
      f32x4_t po[8], ml[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = part_at(min(s0 + u, sh.splits - 1), h);
        po[u] = load_partials4(part_rs, at + c * 4);
        ml[u] = load_partials4(part_rs, at + D * 4);
      }
      float M2 = M;
#pragma unroll
      for (int u = 0; u < 8; ++u) M2 = fmaxf(M2, ml[u][0]);
      const float f = __builtin_amdgcn_exp2f(M - M2);
      o *= f;
      L *= f;
      M = M2;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (s0 + u >= sh.splits) continue;
        const float w = __builtin_amdgcn_exp2f(ml[u][0] - M);
        o += w * po[u];
        L += w * ml[u][1];
      }
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    uint32_t *to = (uint32_t *)(d.out + sh.b * d.o_tok + (h0 + h) * d.o_head + c);
    to[0] = pack_pair<DT>(o[0] * inv, o[1] * inv);
    to[1] = pack_pair<DT>(o[2] * inv, o[3] * inv);
    if (d.lse && c == 0)
      d.lse[(int64_t)sh.b * d.Hq + h0 + h] = L != 0.f ? (M + __builtin_amdgcn_logf(L)) * kLn2 : -INFINITY;
  }
}

int head_blocks_of(int Hq, int Hkv) { return (Hq / Hkv + 15) / 16; }

// The parts of split sequences: each head's number at most twice the slots
// over the heads (a sequence of n > 1 parts has more than n - 1 >= n / 2
// times the tiles of one).
size_t part_bytes(int D, int Hq, int Hkv) {
  const size_t heads = (size_t)Hkv * head_blocks_of(Hq, Hkv);
  return 2 * std::max<size_t>(kSlots / heads, 1) * heads * 16 * (D + 4) * sizeof(float);
}

template <int DT, int D>
hipError_t launch(const AttnDesc &d, void *ws, hipStream_t s) {
  const int hb = head_blocks_of(d.Hq, d.Hkv), heads = d.Hkv * hb;
  const bool may_split = (int64_t)heads * d.n_seqs <= kAttnCounters;
  const int shares = d.n_seqs + (may_split ? (kSlots + heads - 1) / heads : 0);
  constexpr int NW = 8;
  hipLaunchKernelGGL((attn_decode_kernel<DT, D, NW>), dim3((unsigned)shares * heads), dim3(64 * NW), 0, s, d,
                     heads, hb, may_split, (uint32_t *)ws, (float *)((char *)ws + kAttnDataOff),
                     (int)part_bytes(D, d.Hq, d.Hkv));
  return hipGetLastError();
}

}  // namespace

size_t attn_decode_workspace(int D, int Hq, int Hkv, int n_seqs) {
  return kAttnDataOff + part_bytes(D, Hq, Hkv);
}

hipError_t launch_attn_decode(const AttnDesc &d, void *ws, hipStream_t s) {
  if (d.D == 64)
    return d.dtype == DT_F16 ? launch<DT_F16, 64>(d, ws, s) : launch<DT_BF16, 64>(d, ws, s);
  return d.dtype == DT_F16 ? launch<DT_F16, 128>(d, ws, s) : launch<DT_BF16, 128>(d, ws, s);
}

}  // namespace spear
