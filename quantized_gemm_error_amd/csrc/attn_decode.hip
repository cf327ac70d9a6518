// Attention of one new token per sequence over the paged cache.
//
// With s_j = q . k_j log2(e) scale over the visible keys j, every wave keeps
// a reference m, its maximum so far less kLift, l = sum 2^(s_j - m) and
// o = sum 2^(s_j - m) v_j over its share of the keys; parts join as
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
// most of the time (per 32 keys and wave 256 cycles of MFMA at D = 128).  The
// weights are rounded to the type once, for the second product; with random
// values that adds less than the output's own rounding (error against 64 bits
// 0.0019 with it, 0.0017 without, bf16).
//
// The work of a head is one list: the 32-key tiles that the sequences' queries
// see, one sequence after the other.  It is cut into R equal runs, whatever the
// lengths, R such that the workgroups (R runs x heads) fill the last of one to
// four rounds of them (see runs_of), and the heads go through it in step, which
// keeps the reads of one moment in the same pages (one list over heads and
// sequences: 212 us where this takes 190).  A workgroup's waves stream through
// their run without a pause: the next tile's loads are issued before the
// present one's products, across the ends of sequences too.  Where a run ends
// inside a sequence, the parts meet in the workspace and the workgroup that
// completes them joins them in list order.
//
// Measured (MI355X, graph-replayed): 32 rows of 32 heads over 512..4144 keys
// 190 us for 1.22 GB (6.4 TB/s; a device copy reaches 5.2), 4 rows of 64 / 8
// heads over up to 32768 keys 79 us (5.7 TB/s), 48 rows in windows of 4096 in
// token-major pages 139 us (5.4 TB/s), one row over 257 keys 6.2 us.
// Tried: four-wave workgroups, three to a CU, 230 us; 128 registers at D = 128
// for twice the waves 344 us (spills); K past the caches too 166 -> 180 us for
// the windowed rows (its 64-byte pieces of a row come by two instructions).
#include <algorithm>

#include "attn_device.h"

namespace spear {

namespace {

constexpr int kTile = 32;      // keys a wave takes at a time
// Short calls: no less than this to a workgroup, two tiles a wave.  Measured: 8
// instead of 16 costs a row over 257 keys 2 us more and one over 8192 keys 3,
// for the joins; 32 takes 3 to 5 us more for one to four rows over 2048 to 8192.
constexpr int kMinTiles = 16;

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

// The list of a head, in units of one tile, or of kMinTiles where that gives
// every sequence workgroups of its own.  Lane i of every wave holds the tiles
// of sequence b0 + i and the inclusive sum of the units.
struct WorkList {
  const AttnDesc &d;
  int unit = 1, b0, mine, upto;
  int length;  // of the list, in units

  __device__ __forceinline__ int tiles_of(int b) const {
    return b < d.n_seqs ? TileList(cached_len(d, b), d.window, d.sinks).tiles : 0;
  }
  __device__ __forceinline__ int units(int tiles) const {
    return unit == 1 ? tiles : (tiles + kMinTiles - 1) / kMinTiles;
  }
  __device__ __forceinline__ void load(int first, int before) {
    b0 = first;
    mine = tiles_of(first + (int)(threadIdx.x & 63));
    upto = before + wave_scan(units(mine));
  }
  __device__ __forceinline__ int sum() const { return __builtin_amdgcn_readlane(upto, 63); }
  __device__ __forceinline__ WorkList(const AttnDesc &desc, int runs) : d(desc) {
    load(0, 0);
    if (d.n_seqs <= 64) {
      const int coarse = wave_total((mine + kMinTiles - 1) / kMinTiles);
      if (coarse <= runs) {
        unit = kMinTiles;
        upto = wave_scan(units(mine));
      }
    }
    length = sum();
    for (int b = 64; b < d.n_seqs; b += 64) {
      load(b, length);
      length = sum();
    }
  }
  // The sequence that holds list position f (< length), its first position
  // and its tiles.
  __device__ __forceinline__ void find(int f, int &b, int &begin, int &tiles) {
    if (b0 > 0 && f < sum() - wave_total(units(mine))) load(0, 0);
    while (f >= sum()) load(b0 + 64, sum());
    const int at = __builtin_popcountll(__ballot(upto <= f));
    b = b0 + at;
    tiles = __builtin_amdgcn_readlane(mine, at);
    begin = __builtin_amdgcn_readlane(upto, at) - units(tiles);
  }
};

// A run's stretch inside one sequence: tiles [first, last) of `tiles`.
struct Stretch {
  int b, first, last, tiles;
  int begin, next;  // list positions of the sequence's start and end
};

// (D = 64 in 128 registers, for two workgroups a CU, spills two pairs of them, each
// read again once a stretch.)
template <int DT, int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 64 ? 4 : 2) void attn_decode_kernel(AttnDesc d, int heads, int head_blocks,
                                                              int runs, uint32_t *counters, float *parts,
                                                              int part_bytes) {
  constexpr int E = D / 16;   // dims a lane holds of a value
  constexpr int KC = D / 32;  // contraction steps of the first product
  constexpr int Q4 = D / 4;
  typedef uint32_t vec_t __attribute__((ext_vector_type(E / 2)));
  __shared__ float s_o[NW][16][D + 4], s_m[NW][16], s_l[NW][16];
  __shared__ int s_last;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;

  const int hd = blockIdx.x % heads, run = blockIdx.x / heads;
  const int kvh = hd / head_blocks, h0 = kvh * d.G + 16 * (hd % head_blocks);
  const int rows = min(16, d.G - 16 * (hd % head_blocks));  // query heads of this workgroup

  WorkList list(d, runs);
  const int per = max(1, (int)(((uint32_t)list.length + runs - 1) / (uint32_t)runs));
  const int begin = (int)min((int64_t)run * per, (int64_t)list.length);
  const int end = min(begin + per, list.length);

  // sequences without tokens see nothing
  for (int b = blockIdx.x; b < d.n_seqs; b += gridDim.x) {
    if (cached_len(d, b) > 0) continue;
    for (int i = threadIdx.x; i < d.Hq * Q4; i += 64 * NW) {
      const int h = i / Q4, c = 4 * (i % Q4);
      *(uint2 *)(d.out + b * d.o_tok + h * d.o_head + c) = uint2{0u, 0u};
      if (d.lse && c == 0) d.lse[(int64_t)b * d.Hq + h] = -INFINITY;
    }
  }
  if (begin >= end) return;

  const auto part_rs = __builtin_amdgcn_make_buffer_rsrc(parts, (short)0, part_bytes, 0x00020000);
  const int part_rows = min(16, d.G);
  const int p16 = d.page_size / 16;  // 16-key halves per page
  const int halves = d.width * p16;
  const uint32_t k_off = r * (uint32_t)d.s_token + 8 * g;
  const uint32_t v_off = 4 * g * (uint32_t)d.s_token + E * r, tok = (uint32_t)d.s_token;
  const float scale = d.scale * kLog2e;

  const auto stretch_at = [&](int f) {  // the stretch that begins at list position f
    Stretch s;
    list.find(f, s.b, s.begin, s.tiles);
    s.next = s.begin + list.units(s.tiles);
    s.first = (f - s.begin) * list.unit;
    s.last = min(s.tiles, (end - s.begin) * list.unit);
    return s;
  };

  struct Half {
    int page;     // -1: hidden
    int64_t off;  // of its first key, this head
  };
  struct TileAt {  // of one wave
    Half half[2];
    int key0;
  };
  const auto tile_at = [&](const Stretch &s, const TileList &tl, int t) {
    TileAt a;
    const int real = t < tl.sink_tiles ? t : t - tl.sink_tiles + tl.lo_tile;
    a.key0 = real * kTile;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = 2 * real + u, pi = column_of(d, i);
      int page = i < halves ? scalar_load(d.table, (int64_t)s.b * d.width + pi) : -1;
      if ((uint32_t)page >= (uint32_t)d.num_pages) page = -1;
      a.half[u].page = page;
      a.half[u].off = max(page, 0) * d.s_page + (int64_t)kvh * d.s_head +
                      (int64_t)(i - pi * p16) * 16 * d.s_token;
    }
    return a;
  };

  u32x4_t kr[2][KC], q[KC];
  vec_t vr[8];
  const auto load_q = [&](int b) {  // the column operand, column r = head h0 + r
    const uint16_t *from = d.q + b * d.q_tok + (h0 + (r < rows ? r : 0)) * d.q_head + 8 * g;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      q[c] = *(const u32x4_t *)(from + 32 * c);
      if (r >= rows) q[c] = u32x4_t{0u, 0u, 0u, 0u};
    }
  };
  const auto load_k = [&](const TileAt &a) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < KC; ++c) kr[u][c] = *(const u32x4_t *)(d.k + a.half[u].off + (k_off + 32 * c));
  };
  // (values come in whole rows and are not read again: past the caches)
  const auto load_v = [&](const TileAt &a) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        vr[4 * u + i] = __builtin_nontemporal_load((const vec_t *)(d.v + a.half[u].off + (v_off + i * tok)));
  };

  Stretch s = stretch_at(begin);
  TileList tl(cached_len(d, s.b), d.window, d.sinks);
  bool have = s.first + wave < s.last;  // whether `now` is a tile of this stretch
  TileAt now;
  load_q(s.b);
  if (have) {
    now = tile_at(s, tl, s.first + wave);
    load_k(now);
    load_v(now);
  }

  for (;;) {  // stretches
    const bool ends = s.next >= end;  // the run's last stretch
    const Stretch s_next = ends ? s : stretch_at(s.next);
    const TileList tl_next = ends ? tl : TileList(cached_len(d, s_next.b), d.window, d.sinks);
    const bool have_next = !ends && s_next.first + wave < s_next.last;

    f32x4_t acc[E];
    float m = kNoMax, l = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    for (int t = s.first + wave; t < s.last; t += NW) {
      const bool here = t + NW < s.last, more = here || have_next;
      TileAt next;
      if (more) next = here ? tile_at(s, tl, t + NW) : tile_at(s_next, tl_next, s_next.first + wave);
      f32x4_t sc[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        sc[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KC; ++c) sc[u] = mfma_16x16x32<DT>(kr[u][c], q[c], sc[u]);
      }
      if (more) load_k(next);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = sc[e >> 2][e & 3] * scale;
      // hidden keys: weight 0, and no value of theirs meets that 0
      if (!((now.key0 >= tl.lo || now.key0 + kTile <= tl.sink) && now.key0 + kTile <= tl.len &&
            now.half[0].page >= 0 && now.half[1].page >= 0)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = now.key0 + 16 * (e >> 2) + 4 * g + (e & 3);
          if (!((j < tl.sink || j >= tl.lo) && j < tl.len && now.half[e >> 2].page >= 0)) {
            x[e] = -INFINITY;
            vr[e] = vec_t(0u);
          }
        }
      }
      float top = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
      if (__any(top - m > kLift<DT>)) {
        const float most = columns_max(top);
        float m2 = most - kLift<DT>;
        if (!(most - m2 <= kLift<DT>)) m2 = most;  // (rounded further down, or an infinity)
        m2 = fmaxf(m, m2);
        const float f = __builtin_amdgcn_exp2f(m - m2);
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
        now = next;
      }
    }
    // a wave without a tile in this stretch starts on the next one's
    if (!have && have_next) {
      now = tile_at(s_next, tl_next, s_next.first + wave);
      load_k(now);
      load_v(now);
    }
    if (!ends) load_q(s_next.b);
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
    lds_barrier();
    const bool whole = s.first == 0 && s.last == s.tiles;
    // A sequence's parts: of the runs from `lead`, where it begins, to the one
    // where it ends.  In its run, a part that begins its sequence (after others)
    // has the second place, any other the first.
    const int lead = whole ? 0 : s.begin / per;
    const auto part_at = [&](int i, int h) {  // byte offset of a row of run i's part
      const int place = 2 * i + (s.begin > i * per ? 1 : 0);
      return ((place * heads + hd) * part_rows + h) * (D + 4) * 4;
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
      if (whole) {
        const float inv = L != 0.f ? 1.f / L : 0.f;
        *(uint2 *)(d.out + s.b * d.o_tok + (h0 + h) * d.o_head + c) =
            uint2{pack_pair<DT>(o[0] * inv, o[1] * inv), pack_pair<DT>(o[2] * inv, o[3] * inv)};
        if (d.lse && c == 0)
          d.lse[(int64_t)s.b * d.Hq + h0 + h] = L != 0.f ? (M + __builtin_amdgcn_logf(L)) * kLn2 : -INFINITY;
      } else {
        store_partials4(o, part_rs, part_at(run, h) + c * 4);
        if (c == 0) store_partials4(f32x4_t{M, L, 0.f, 0.f}, part_rs, part_at(run, h) + D * 4);
      }
    }
    if (!whole) {
      const int parts_n = (s.next - 1) / per - lead + 1;
      uint32_t *counter = counters + lead * heads + hd;
      publish_wait();
      lds_barrier();
      if (threadIdx.x == 0)
        s_last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                 (uint32_t)parts_n - 1;
      lds_barrier();
      if (s_last) {
        if (threadIdx.x == 0)
          __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        for (int i = threadIdx.x; i < rows * Q4; i += 64 * NW) {
          const int h = i / Q4, c = 4 * (i % Q4);
          float M = kNoMax, L = 0.f;
          f32x4_t o = {0.f, 0.f, 0.f, 0.f};
          constexpr int AT_ONCE = D == 128 ? 16 : 8;  // parts in flight (as registers allow)
          for (int k0 = 0; k0 < parts_n; k0 += AT_ONCE) {
            f32x4_t po[AT_ONCE];
            f32x2_t ml[AT_ONCE];
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u) {
              const int at = part_at(lead + min(k0 + u, parts_n - 1), h);
              ml[u] = load_partials2(part_rs, at + D * 4);
              po[u] = load_partials4(part_rs, at + c * 4);
            }
            float M2 = M;
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u) M2 = fmaxf(M2, ml[u][0]);
            const float f = __builtin_amdgcn_exp2f(M - M2);
            o *= f;
            L *= f;
            M = M2;
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u) {
              if (k0 + u >= parts_n) continue;
              const float w = __builtin_amdgcn_exp2f(ml[u][0] - M);
              o += w * po[u];
              L += w * ml[u][1];
            }
          }
          const float inv = L != 0.f ? 1.f / L : 0.f;
          *(uint2 *)(d.out + s.b * d.o_tok + (h0 + h) * d.o_head + c) =
              uint2{pack_pair<DT>(o[0] * inv, o[1] * inv), pack_pair<DT>(o[2] * inv, o[3] * inv)};
          if (d.lse && c == 0)
            d.lse[(int64_t)s.b * d.Hq + h0 + h] = L != 0.f ? (M + __builtin_amdgcn_logf(L)) * kLn2 : -INFINITY;
        }
      }
    }
    if (ends) return;
    lds_barrier();  // s_o is free for the next stretch
    s = s_next;
    tl = tl_next;
    have = have_next;
  }
}

int head_blocks_of(int Hq, int Hkv) { return (Hq / Hkv + 15) / 16; }

// Workgroups that run at once: 256 CUs, of which each holds one workgroup of 8
// waves with the registers of D = 128 and two of D = 64.
int slots_of(int D) { return D == 64 ? 512 : 256; }

// Runs per head: the number, up to four rounds of workgroups, from which on no
// larger one fills the last round by 5% of a round more (256 workgroups at once:
// 1 head takes 247 runs, 8 take 32, 12 take 64 in three full rounds, 33 take 15
// in two).
int runs_of(int D, int heads) {
  const int slots = slots_of(D);
  int best = 1;
  double fill = 0;
  for (int r = 1; r * heads <= std::min(4 * slots, kAttnCounters); ++r) {
    const double f = (double)r * heads / ((r * heads + slots - 1) / slots * slots);
    if (f > fill + 0.05) {
      fill = f;
      best = r;
    }
  }
  return best;
}

size_t part_bytes(int D, int Hq, int Hkv) {
  const int heads = Hkv * head_blocks_of(Hq, Hkv);
  return (size_t)2 * runs_of(D, heads) * heads * std::min(16, Hq / Hkv) * (D + 4) * sizeof(float);
}

template <int DT, int D>
hipError_t launch(const AttnDesc &d, void *ws, hipStream_t s) {
  const int hb = head_blocks_of(d.Hq, d.Hkv), heads = d.Hkv * hb;
  // no more runs than the table's tiles can fill
  const int64_t tiles = ((int64_t)d.width * d.page_size + kTile - 1) / kTile;
  const int runs = (int)std::min<int64_t>((tiles + kMinTiles - 1) / kMinTiles * d.n_seqs, runs_of(D, heads));
  constexpr int NW = 8;
  hipLaunchKernelGGL((attn_decode_kernel<DT, D, NW>), dim3((unsigned)runs * heads), dim3(64 * NW), 0, s, d,
                     heads, hb, runs, (uint32_t *)ws, (float *)((char *)ws + kAttnDataOff),
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
