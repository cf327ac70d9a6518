// Causal attention of the batch's new tokens over the paged cache.
//
// With s = q . k scale log2(e), tiles of 64 keys pass by a block of query rows
// that keeps a reference m >= (row maximum) - kSlack, l = sum 2^(s - m + kLift) and
// o = sum 2^(s - m + kLift) v in fp32 (m is raised, and l and o scaled, only when a
// maximum passes it by more than kSlack: the weights stay in the type's range, and
// their relative rounding is the same); out = o / l, lse = ln 2 (m + log2 l - kLift).
//
// The work is two matrix products, 4 D flops per visible pair, so MFMA bounds
// it.  A group of four waves owns 128 rows of one key-value head (a workgroup is
// one group or two, chosen at the launch): the
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
//
// Measured (MI355X, graph-replayed): 2048 rows of 64 / 8 heads over 16384 keys
// 0.92 ms (1.12 PFLOP/s; a large bf16 matrix product of the library reaches
// 1.21), two chunks in windows of 4096 148 us (913 TFLOP/s), a 2048-token first
// chunk of 32 heads 55 us (621 TFLOP/s: its longest blocks set the time),
// chunks of 129..256 tokens with 32 single rows, D = 64, 29 us.  At the first
// the matrix units are busy for 53% of the cycles at about 1.9 GHz; no LDS
// conflicts.  Tried: 8-wave workgroups of 256 rows with four tiles staged ahead
// (939 us and 70 us at the first and third); the compiler's order of the
// products and weights (980 -> 985 us); fewer fragments ahead (no change).
#include <algorithm>
#include <type_traits>

#include "attn_device.h"

namespace spear {

namespace {

constexpr int kRows = 128;  // query rows of a workgroup
constexpr int kKeys = 64;   // keys of a tile
constexpr int kWaves = 4;   // of 32 rows each
// By how much a maximum may pass m: with kLift and the shift's rounding (2^-9) less
// than 2^16, where fp16 ends.  (fp16 with 1 instead 2% slower, with 4 1% faster: m is
// raised and the sums scaled in more or fewer tiles.)
template <int DT>
constexpr float kSlack = DT == DT_F16 ? 2.9f : 8.f;
constexpr float kFar = 65536.f;  // of m from 0: past this m is subtracted from the scores by itself

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

// The 64-key tiles that a block of rows at positions p_min..p_max sees: from
// position 0 for the sinks, then those from lo_tile on.
struct Tiles {  // (p_min <= p_max)
  int sink_tiles, lo_tile, count;
  __device__ __forceinline__ Tiles(const AttnDesc &d, int p_min, int p_max) {
    // (p_min may be negative and the window as large as the type holds)
    const int lo = d.window > 0 && p_min >= d.window ? p_min - d.window + 1 : 0;
    lo_tile = lo / kKeys;
    sink_tiles = min((min(d.sinks, lo) + kKeys - 1) / kKeys, lo_tile);
    count = p_max < 0 ? 0 : sink_tiles + p_max / kKeys + 1 - lo_tile;
  }
};

// A work item of a key-value head: part `part` of `parts` of the tiles of the
// kRows rows from row0 on of a sequence.
struct Item {
  int b, start, n, row0;  // first token, tokens, first row in the block
  int part, parts;
  int part_row;           // of the sequence's parts in the workspace, per head
  int block;              // number of the block in the batch
};

// Item w of a head, the same computation in every wave.  A sequence's blocks
// are each cut into as many parts as its longest block has stretches of `per`
// tiles.  When a call has too few blocks to fill the chip, or some with many
// tiles, parts of `per` tiles take as long as one part if all run at once, and
// otherwise the tiles and the starts and joins of the parts spread over the
// slots, and half a part more at the end; the cheapest of a few sizes is
// taken, whole blocks among them.
constexpr int kSlots = 512;      // groups of four waves that run at once: two to a CU
constexpr int kMinTiles = 4;     // of a part
constexpr int kPartTiles = 3;    // what a part's start and its partial sums cost, in tiles of a group
constexpr int kJoinRows = 100;   // rows of partial sums that are joined in the time of one
constexpr int kMaxParts = 63;
constexpr int kWhole = 1 << 29;  // tiles per part: no block is cut

template <int GROUPS>
__device__ __forceinline__ bool find_item(const AttnDesc &d, int w, int part_rows, int most_items,
                                          Item &k) {
  const int lane = threadIdx.x & 63;
  struct Seq {
    int start, n, blocks, longest, total;  // tiles of the longest block, of all
  };
  const auto seq_of = [&](int b) {
    Seq s{b, b < d.n_seqs, 0, 0, 0};
    if (b >= d.n_seqs) return s;
    if (d.q_starts) {
      s.start = max(0, min(d.q_starts[b], d.n_tokens));
      s.n = max(0, min(d.q_starts[b + 1], d.n_tokens) - s.start);
    }
    if (s.n == 0) return s;
    s.blocks = (s.n * d.G + kRows - 1) / kRows;
    const int len = cached_len(d, b), first = len - s.n, span = (kRows - 1) / d.G;
    s.longest = Tiles(d, max(first, len - 1 - span), len - 1).count;
    s.total = min((s.longest + Tiles(d, first, min(len - 1, first + span)).count + 1) / 2, 1 << 18) *
              min(s.blocks, 1 << 12);
    return s;
  };
  const auto parts_of = [&](const Seq &s, int per) {
    return per >= kWhole ? 1 : min(kMaxParts, max(1, (int)((uint32_t)(s.longest + per - 1) / (uint32_t)per)));
  };
  const Seq mine = seq_of(lane);  // of the first 64 sequences
  const auto sum = [&](auto value) {
    int all = wave_total(value(mine));
    for (int b0 = 64; b0 < d.n_seqs; b0 += 64) all += wave_total(value(seq_of(b0 + lane)));
    return all;
  };
  // (sums that device data of any kind cannot overflow: each term is bounded
  // by more than a whole cut batch may have)
  const int blocks = sum([](const Seq &s) { return min(s.blocks, 1 << 18); });
  const int slots = max(kSlots / GROUPS / d.Hkv, 1);
  int per = kWhole;
  if (blocks <= kAttnCounters / d.Hkv && blocks < most_items) {
    const int total = sum([](const Seq &s) { return s.total; });
    int most = mine.longest;
    for (int b0 = 64; b0 < d.n_seqs; b0 += 64) most = max(most, seq_of(b0 + lane).longest);
    most = wave_max(most);
    const int even = (total + slots - 1) / slots;
    // whole blocks
    int least = blocks <= slots ? most : even + (most + 1) / 2;
    const int tries = d.n_seqs <= 64 ? 6 : 2;
    for (int i = 0; i < tries && most > 3 * kMinTiles; ++i) {
      // the even share times 1, 1.25, 1.5, 2, 4, 8
      const int p = max(kMinTiles, (even * (i < 3 ? 4 + i : 1 << i) + 3) / 4);
      if (p >= most) break;
      const int items = sum([&](const Seq &s) { return s.blocks * parts_of(s, p); });
      const int rows = sum([&](const Seq &s) {
        const int parts = parts_of(s, p);
        return parts > 1 ? (int)min((int64_t)s.n * d.G * parts, (int64_t)1 << 18) : 0;
      });
      // the join of the block with the most partial sums
      int join = 0;
      for (int b0 = 0; b0 < d.n_seqs; b0 += 64) {
        const Seq s = b0 == 0 ? mine : seq_of(b0 + lane);
        const int parts = s.blocks > 0 ? parts_of(s, p) : 1;
        join = max(join, parts > 1 ? parts * min(s.n * d.G, kRows) : 0);
      }
      join = (wave_max(join) * GROUPS + kJoinRows - 1) / kJoinRows;
      const int cost = GROUPS * kPartTiles + join + (items <= slots ? p : even + (p + 1) / 2);
      if (rows <= part_rows && items <= most_items && cost < least) {
        least = cost;
        per = p;
      }
    }
  }
  const int items = sum([&](const Seq &s) { return s.blocks * parts_of(s, per); });
  // The last items, which see the most keys, come first; of up to two
  // workgroups a CU, the second ones, which a launch places after every CU has
  // one, go the other way, so that CUs get like amounts of work.
  const int first_round = max(kSlots / 2 / d.Hkv, 1);
  if (w >= items) return false;
  w = w < first_round || items > 2 * first_round ? items - 1 - w : w - first_round;
  int before = 0, rows_before = 0, blocks_before = 0;
  for (int b0 = 0; b0 < d.n_seqs; b0 += 64) {
    const Seq s = b0 == 0 ? mine : seq_of(b0 + lane);
    const int parts = parts_of(s, per), n = s.blocks * parts;
    const int upto = before + wave_scan(n);
    const int rows_upto = rows_before + wave_scan(parts > 1 ? s.n * d.G * parts : 0);
    const int blocks_upto = blocks_before + wave_scan(s.blocks);
    const int all = __builtin_amdgcn_readlane(upto, 63);
    if (w < all) {
      const int at = __builtin_popcountll(__ballot(upto <= w));
      k.b = b0 + at;
      if (k.b >= d.n_seqs) return false;
      const auto pick = [&](int v) { return __builtin_amdgcn_readlane(v, at); };
      k.start = pick(s.start);
      k.n = pick(s.n);
      k.parts = pick(parts);
      const int i = w - (pick(upto) - pick(n));
      k.part = i % k.parts;
      k.block = i / k.parts;
      k.row0 = kRows * k.block;
      k.block += pick(blocks_upto) - pick(s.blocks);
      k.part_row = pick(rows_upto) - (k.parts > 1 ? k.n * d.G * k.parts : 0);
      return k.row0 >= 0 && k.row0 < k.n * d.G;
    }
    before = all;
    rows_before = __builtin_amdgcn_readlane(rows_upto, 63);
    blocks_before = __builtin_amdgcn_readlane(blocks_upto, 63);
  }
  return false;
}

// GROUPS: groups of four waves.  With two, both have the same rows, with
// buffers of their own, and take the part's tiles by turns; the second's sums
// then join the first's through LDS.
template <int DT, int D, int GROUPS>
__global__ __launch_bounds__(64 * kWaves * GROUPS, 2) void attn_prefill_kernel(
    AttnDesc d, int part_rows, int most_items, uint32_t *counters, float *parts, int part_bytes) {
  constexpr int CH = D / 8;          // 16-byte chunks of a row
  constexpr int KS = D / 16;         // contraction steps of S
  constexpr int DB = D / 32;         // 32-dim blocks of O
  constexpr int RPI = 64 / CH;       // rows a wave's load instruction brings
  constexpr int LOADS = 16 / RPI;    // instructions for 16 keys
  constexpr int TILE = kKeys * D * 2;  // bytes of a staged K or V tile
  static_assert((kMaxParts + 1) * kRows * 4 <= 4 * TILE, "the join's weights");
  static_assert(GROUPS == 1 || kRows * (D + 4) * 4 <= 8 * TILE, "a group's sums");
  constexpr int THREADS = 64 * kWaves * GROUPS;
  // of a group: K tiles of its even and odd t, then V's
  __shared__ __attribute__((aligned(256))) char s_all[GROUPS][4][TILE];
  // of a group's tile, by 16 keys: 1 hidden, 2 not finite
  __shared__ __attribute__((aligned(16))) int s_flags[2][GROUPS][kWaves];

  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = GROUPS == 1 ? wave_all : wave_all % kWaves;  // in its group
  const int team = GROUPS == 1 ? 0 : wave_all / kWaves;
  char (&s_kv)[4][TILE] = s_all[team];
  const int col = lane & 31, half = lane >> 5;
  const int kvh = blockIdx.x % d.Hkv;
  Item blk;
  if (!find_item<GROUPS>(d, blockIdx.x / d.Hkv, part_rows, most_items, blk)) return;
  blk = {uniform(blk.b), uniform(blk.start), uniform(blk.n), uniform(blk.row0), uniform(blk.part),
         uniform(blk.parts), uniform(blk.part_row), uniform(blk.block)};

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

  // the part's tiles, of which this group has every GROUPS-th
  const Tiles list(d, p_min, p_max);
  const int first = blk.parts == 1 ? 0 : (int)((int64_t)list.count * blk.part / blk.parts);
  const int part_tiles =
      (blk.parts == 1 ? list.count : (int)((int64_t)list.count * (blk.part + 1) / blk.parts)) - first;
  const auto of_group = [&](int n) { return max(n + GROUPS - 1 - team, 0) / GROUPS; };
  const int tiles = of_group(part_tiles), steps = (part_tiles + GROUPS - 1) / GROUPS;
  const auto key_of = [&](int t) {
    t = first + GROUPS * t + team;
    return kKeys * (t < list.sink_tiles ? t : t - list.sink_tiles + list.lo_tile);
  };

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
  // scores stay unscaled (a negative scale has turned the query's sign; one of 0 is
  // taken as 1e-37, so that a hidden key's weight is 0 there too, with a slack that
  // any score passes from kNoMax)
  const float scale = fmaxf(fabsf(d.scale) * kLog2e, 1e-37f), slack = kSlack<DT> / scale;

  // Staging this wave's 16 keys of a tile: load j brings the RPI rows from
  // j RPI on, this lane the chunk that belongs where its bytes land.  The
  // chunks of K's row t are permuted by ^ (t & 7), which depends on j's parity
  // (D = 128) or not on j (D = 64); V's by row alone.
  const int lane_row = lane / CH, lane_ch = lane % CH;
  const int row_bytes = 2 * (int)d.s_token;
  int k_src[D == 128 ? 2 : 1];  // byte offsets from the load's first row
#pragma unroll
  for (int j = 0; j < (D == 128 ? 2 : 1); ++j)
    k_src[j] = lane_row * row_bytes + 16 * (lane_ch ^ ((j * RPI + lane_row) & 7));
  const int v_src = lane_row * row_bytes +
                    16 * ((((lane_ch >> 1) ^ v_swizzle<D>(lane_row)) << 1) | (lane_ch & 1));
  // Where this wave's 16 keys of a tile lie, worked out for 64 tiles at a time,
  // one per lane, so that the loop has no table entry to wait for.
  const int p16 = d.page_size / 16;
  const int32_t *row_table = d.table + (int64_t)blk.b * d.width;
  int64_t src_off = 0;  // elements, of tile (sources' first) + lane
  int src_bytes = 0;    // 0: past the cached length; kHidden: on no page
  constexpr int kHidden = -1;
  const auto sources_from = [&](int t0) {
    const int i = key_of(t0 + lane) / 16 + wave, left = len - 16 * i, c = column_of(d, i);
    const bool want = t0 + lane < tiles && left > 0;
    const int page = want ? row_table[c] : -1;
    const bool is = (uint32_t)page < (uint32_t)d.num_pages;
    src_off = (is ? page : 0) * d.s_page + (int64_t)kvh * d.s_head + (int64_t)((i - c * p16) * 16) * d.s_token;
    src_bytes = is ? min(16, left) * row_bytes : want ? kHidden : 0;
  };
  struct Source {
    int64_t off;
    int bytes;
  };
  const auto source_of = [&](int t) {
    if ((t & 63) == 0) sources_from(t);
    return Source{((int64_t)__builtin_amdgcn_readlane((int)(src_off >> 32), t & 63) << 32) |
                      (uint32_t)__builtin_amdgcn_readlane((int)src_off, t & 63),
                  __builtin_amdgcn_readlane(src_bytes, t & 63)};
  };
  const uint32_t lds = lds_offset(s_kv), mine_at = 16 * wave * D * 2;
  static_assert(RPI * D * 2 == 1024, "a load's rows follow the last load's in LDS");
  const auto load_keys = [&](const Source &src, uint32_t to) {
    load_to_lds<LOADS>(buffer_words(d.k + src.off, max(src.bytes, 0)), (uint32_t)uniform((int)(to + mine_at)),
                       k_src[0], k_src[D == 128 ? 1 : 0], uniform(RPI * row_bytes));
  };
  const auto load_values = [&](const Source &src, uint32_t to) {
    load_to_lds<LOADS>(buffer_words(d.v + src.off, max(src.bytes, 0)), (uint32_t)uniform((int)(to + mine_at)),
                       v_src, v_src, uniform(RPI * row_bytes));
  };

  // operand addresses in a tile: K row `col`, step 0 (step k: ^ 32 k); V row
  // 4 half + l/4 % 4, dim block 0 (block b: ^ 64 b)
  const int k_at = col * D * 2 + 16 * (half ^ (col & 7));
  const int v_at = (4 * half + ((lane & 15) >> 2)) * D * 2 +
                   32 * (((lane >> 4) & 1) ^ v_swizzle<D>((lane & 15) >> 2)) + 8 * (lane & 3);

  f32x16_t acc[DB], s_even[2], s_odd[2];  // output sums; scores of even and odd tiles
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
  // The operand fragments in the order the products take them: K by (step,
  // 32-key half), V by (16-key group, dim block).
  const auto k_frag = [&](const char *kt, int i) {
    return *(const u32x4_t *)(kt + (k_at ^ (32 * (i >> 1))) + (i & 1) * 32 * D * 2);
  };
  const auto v_frag = [&](const char *vt, int i) {
    const char *from = vt + (v_at ^ (64 * (i % DB))) + (i / DB) * 16 * D * 2;
    const uint2 x = bitcast<uint2>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)from));
    const uint2 y = bitcast<uint2>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)(from + 8 * D * 2)));
    return u32x4_t{x.x, x.y, y.x, y.y};
  };
  constexpr int NQ = 2 * KS, NP = 4 * DB, AHEAD = 4;  // steps of the products, fragments read ahead
  const f32x16_t zeros = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};

  // The tiles that some row of this wave sees are the first w_tiles (those
  // that a window hides from all of its rows are computed and masked).
  const int w_tiles =
      !active || w_max < 0
          ? 0
          : of_group(min(part_tiles, max(list.count - (p_max / kKeys - w_max / kKeys) - first, 0)));
  if (steps > 0) {
    Source now{0, 0};
    if (tiles > 0) {
      now = source_of(0);
      load_keys(now, lds);
    }
    Source next = now;
    wait_for_lds_loads();
    lds_barrier();
    if (tiles > 0) load_values(now, lds + 2 * TILE);
    if (tiles > 1) {
      next = source_of(1);
      load_keys(next, lds + TILE);
    }
    if (w_tiles > 0) {
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i)
        s_even[i & 1] = mfma_32x32x16<DT>(k_frag(s_kv[0], i), q[i >> 1], i < 2 ? zeros : s_even[i & 1]);
    }
    // Tile t, whose scores s holds; V of t and K of t + 1 are on their way.
    // Leaves the scores of t + 1 in ahead.  (The loop takes two tiles at a time, so
    // that the two sets of scores and buffers are fixed registers and addresses.)
    const auto tile = [&](const int t, const int buf, f32x16_t (&s)[2], f32x16_t (&ahead)[2]) {
      const int key0 = key_of(t);
      const char *kt = s_kv[buf ^ 1], *vt = s_kv[2 + buf];
      const bool masked = (GROUPS == 1 || t < tiles) && partly(key0, p_min, p_max);
      wait_for_lds_loads();  // this wave's parts of V(t) and K(t + 1)
      int flags = now.bytes == kHidden ? 1 : 0;
      if (masked) {  // (only V: a score that is no number is replaced, a weight of 0 is not)
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          const u32x4_t x = *(const u32x4_t *)(vt + mine_at + j * RPI * D * 2 + 16 * lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) bad |= not_finite<DT>(x[e]);
        }
        flags |= __any(bad != 0) ? 2 : 0;
      }
      if (lane == 0) s_flags[buf][team][wave] = flags;
      lds_barrier();
      // (first the reads whose latency the loads' issue covers)
      const u32x4_t group = *(const u32x4_t *)s_flags[buf][team];
      u32x4_t either = group;
      if constexpr (GROUPS == 2) either |= *(const u32x4_t *)s_flags[buf][team ^ 1];
      u32x4_t kf[AHEAD], vf[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) kf[i] = k_frag(kt, i);
      now = next;
      if (t + 1 < tiles) load_values(now, lds + (2 + (buf ^ 1)) * TILE);
      if (t + 2 < tiles) {
        next = source_of(t + 2);
        load_keys(next, lds + buf * TILE);
      }
      const int any = uniform((int)(either[0] | either[1] | either[2] | either[3]));
      const bool dirty = any & 2;  // (of either group: the path has barriers)
      const bool mine = t < w_tiles;
      if (!mine && !dirty) return;
      // a tile that no row sees is masked as any other; past the group's last
      // there is none
      const bool looks = GROUPS == 1 || mine;

      if (looks && ((any & 1) || partly(key0, w_min, w_max))) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int j = key0 + 32 * u + 8 * (v >> 2) + 4 * half + (v & 3);
            const bool sees = (j <= pos) & ((pos - j < window) | (j < d.sinks)) &
                              ((group[2 * u + (v >> 3)] & 1) == 0);
            s[u][v] = sees ? s[u][v] : -INFINITY;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 16; ++v) top = fmaxf(top, s[u][v]);
      if (looks && __any(top - m > slack)) {
        top = over_halves(top, [](float a, float b) { return fmaxf(a, b); });
        const float m2 = fmaxf(m, top), f = __builtin_amdgcn_exp2f((m - m2) * scale);
        m = m2;
        l *= f;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[b][v] *= f;
      }
      if (dirty) {
        // Values that are not finite: how many of a sign (of both, for no
        // number) a row sees of each dim, as products of ones; then they leave
        // the tile.
        constexpr uint32_t kOnes = DT == DT_F16 ? 0x3C003C00u : 0x3F803F80u;
#pragma unroll 1
        for (int sign = looks ? 0 : 2; sign < 2; ++sign) {
          const uint32_t flip = sign ? 0x80008000u : 0u;
#pragma unroll
          for (int b = 0; b < DB; ++b) {
            f32x16_t c = zeros;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              u32x4_t x = v_frag(vt, g * DB + b), w;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t bad = not_finite<DT>(x[e]) >> 15;  // 1 in each half that is not finite
                // exponent bits only: an infinity, of one sign; else no number
                const uint32_t frac = x[e] & ~(kExp<DT> | 0x80008000u);
                const uint32_t nan = (((frac & 0xFFFFu) != 0) | ((uint32_t)((frac >> 16) != 0) << 16)) & bad;
                const uint32_t take = nan | (bad & ~((x[e] ^ flip) >> 15));
                x[e] = kOnes & ((take & 0x00010001u) * 0xFFFFu);
                const float s0 = s[g >> 1][8 * (g & 1) + 2 * e], s1 = s[g >> 1][8 * (g & 1) + 2 * e + 1];
                w[e] = kOnes & ((s0 != -INFINITY ? 0xFFFFu : 0u) | (s1 != -INFINITY ? 0xFFFF0000u : 0u));
              }
              c = mfma_32x32x16<DT>(x, w, c);
            }
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[b][v] += c[v] > 0.f ? (sign ? -INFINITY : INFINITY) : 0.f;
          }
        }
        lds_barrier();
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          u32x4_t *at = (u32x4_t *)(s_kv[2 + buf] + mine_at + j * RPI * D * 2 + 16 * lane);
          u32x4_t x = *at;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] &= ~((not_finite<DT>(x[e]) >> 15) * 0xFFFFu);
          *at = x;
        }
        lds_barrier();
        if (!mine) return;
      }
      // The weight is 2^(s scale - m scale), one fma: m scale is rounded first, which
      // puts every weight of the row off by one factor (sums and lse with them), of at
      // most 2^(2^-9) up to kFar.  Further out the factor would pass what the types
      // span: there m is subtracted first.
      float shift = kLift<DT> - m * scale;
      if (__any(fabsf(shift) > kFar)) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int v = 0; v < 16; ++v) s[u][v] -= m;
        shift = kLift<DT>;
      }
      // The two products in steps of one MFMA, the next fragments' reads and a
      // share of the weights' arithmetic, which keeps both units busy; the
      // compiler's own order bunches each kind.  The next tile's scores go
      // along with the weights of the first 32 keys, and O's first half of
      // the keys with those of the last 32.
      u32x4_t p[4];  // p: weights of 16 keys each, the column operand of O
      float sum[2] = {0.f, 0.f};
      const auto weights = [&](int e) {  // of scores e and e + 1
        const int u = e >> 4, v = e & 15;
        const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][v], scale, shift));
        const float b = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][v + 1], scale, shift));
        sum[0] += a;
        sum[1] += b;
        p[2 * u + (v >> 3)][(v >> 1) & 3] = pack_pair<DT>(a, b);
      };
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        ahead[i & 1] = mfma_32x32x16<DT>(kf[i % AHEAD], q[i >> 1], i < 2 ? zeros : ahead[i & 1]);
        if (i + AHEAD < NQ)
          kf[i % AHEAD] = k_frag(kt, i + AHEAD);
        else
          vf[i + AHEAD - NQ] = v_frag(vt, i + AHEAD - NQ);
        if (NQ == 8)
          weights(2 * i);
        else if (i & 1)
          weights(i - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      // (the wave goes before the other one of its SIMD while it has mostly
      // products to issue: 980 -> 955 us for 2048 rows of 64 heads over 16384 keys)
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        acc[i % DB] = mfma_32x32x16<DT>(vf[i % AHEAD], p[i / DB], acc[i % DB]);
        if (i + AHEAD < NP) vf[i % AHEAD] = v_frag(vt, i + AHEAD);
        if (i < NP / 2) {
#pragma unroll
          for (int e = 0; e < 32 / NP; e += 2) weights(16 + 32 / NP * i + e);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      l += sum[0] + sum[1];
    };
    for (int t = 0; t < steps; t += 2) {
      tile(t, 0, s_even, s_odd);
      if (t + 1 < steps) tile(t + 1, 1, s_odd, s_even);
    }
  }
  if constexpr (GROUPS == 2) {  // the second group's sums join the first's
    float *at = (float *)s_all + (32 * wave + col) * (D + 4);
    lds_barrier();
    if (team == 1) {
#pragma unroll
      for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int v = 0; v < 16; v += 4)
          *(f32x4_t *)(at + 32 * b + 2 * v + 4 * half) =
              f32x4_t{acc[b][v], acc[b][v + 1], acc[b][v + 2], acc[b][v + 3]};
      at[D + half] = l;  // (a half's l: the other half has the other keys')
      if (half == 0) at[D + 2] = m;
    }
    lds_barrier();
    if (team == 0) {
      const float m1 = at[D + 2], m2 = fmaxf(m, m1);
      const float f0 = __builtin_amdgcn_exp2f((m - m2) * scale), f1 = __builtin_amdgcn_exp2f((m1 - m2) * scale);
      m = m2;
      l = f0 * l + f1 * at[D + half];
#pragma unroll
      for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
          const f32x4_t x = *(const f32x4_t *)(at + 32 * b + 2 * v + 4 * half);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[b][v + i] = f0 * acc[b][v + i] + f1 * x[i];
        }
    }
    if (blk.parts == 1 && team == 1) return;
    lds_barrier();  // (with parts, the sums' LDS is used again)
  }
  l = over_halves(l, [](float a, float b) { return a + b; });
  const auto store = [&](int r, f32x4_t o, int c, float lse) {  // dims c.. of row r
    const int t = r / d.G, h = kvh * d.G + r - t * d.G;
    *(uint2 *)(d.out + (int64_t)(blk.start + t) * d.o_tok + h * d.o_head + c) =
        uint2{pack_pair<DT>(o[0], o[1]), pack_pair<DT>(o[2], o[3])};
    if (d.lse && c == 0) d.lse[(int64_t)(blk.start + t) * d.Hq + h] = lse;
  };
  const auto dims = [&](int b, int v) {
    return f32x4_t{acc[b][v], acc[b][v + 1], acc[b][v + 2], acc[b][v + 3]};
  };
  if (blk.parts == 1) {
    if (!is_row) return;
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const float lse = l != 0.f ? (m * scale + (__builtin_amdgcn_logf(l) - kLift<DT>)) * kLn2 : -INFINITY;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int v = 0; v < 16; v += 4) store(row, dims(b, v) * inv, 32 * b + 2 * v + 4 * half, lse);
    return;
  }

  // The block's parts meet in the workspace; the workgroup that completes
  // them joins them in order.
  const auto rs = __builtin_amdgcn_make_buffer_rsrc(parts, (short)0, part_bytes, 0x00020000);
  const auto part_at = [&](int part, int r) {  // byte offset of a row's part
    return (kvh * part_rows + blk.part_row + part * all_rows + r) * (D + 4) * 4;
  };
  if (is_row && team == 0) {
    const int at = part_at(blk.part, row);
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int v = 0; v < 16; v += 4) store_partials4(dims(b, v), rs, at + 4 * (32 * b + 2 * v + 4 * half));
    if (half == 0) store_partials4(f32x4_t{m, l, 0.f, 0.f}, rs, at + 4 * D);
  }
  publish_wait();
  lds_barrier();
  uint32_t *counter = counters + blk.block * d.Hkv + kvh;
  if (threadIdx.x == 0)
    s_flags[0][0][0] = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                    (uint32_t)blk.parts - 1;
  lds_barrier();
  if (!s_flags[0][0][0]) return;
  if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  // First each row's weights of the parts, w_s = 2^((m_s - M) scale) / L, and
  // M and L; then the sums, with many loads in flight.  LDS is free by now.
  const int rows = min(kRows, all_rows - blk.row0);
  float *w_of = (float *)s_all;               // [kMaxParts][kRows]
  float *lse_of = w_of + kMaxParts * kRows;   // [kRows]
  for (int r = threadIdx.x; r < rows; r += THREADS) {
    float M = kNoMax, L = 0.f;
    for (int k0 = 0; k0 < blk.parts; k0 += 8) {
      f32x4_t ml[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        ml[u] = load_partials4(rs, part_at(min(k0 + u, blk.parts - 1), blk.row0 + r) + 4 * D);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (k0 + u >= blk.parts) continue;
        const float M2 = fmaxf(M, ml[u][0]);
        L = L * __builtin_amdgcn_exp2f((M - M2) * scale) + ml[u][1] * __builtin_amdgcn_exp2f((ml[u][0] - M2) * scale);
        M = M2;
        w_of[(k0 + u) * kRows + r] = ml[u][0];
      }
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    for (int k = 0; k < blk.parts; ++k)
      w_of[k * kRows + r] = inv * __builtin_amdgcn_exp2f((w_of[k * kRows + r] - M) * scale);
    lse_of[r] = L != 0.f ? (M * scale + (__builtin_amdgcn_logf(L) - kLift<DT>)) * kLn2 : -INFINITY;
  }
  lds_barrier();
  constexpr int AT_ONCE = 4, Q4 = D / 4;
  for (int i0 = threadIdx.x; i0 < rows * Q4; i0 += AT_ONCE * THREADS) {
    f32x4_t o[AT_ONCE];
    int r[AT_ONCE], at[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {  // (past the last row: the last row again, not stored)
      const int i = min(i0 + j * THREADS, rows * Q4 - 1);
      r[j] = i / Q4;
      at[j] = 16 * (i % Q4);
      o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    for (int k0 = 0; k0 < blk.parts; k0 += 8) {
      f32x4_t x[AT_ONCE][8];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
#pragma unroll
        for (int u = 0; u < 8; ++u)
          x[j][u] = load_partials4(rs, part_at(min(k0 + u, blk.parts - 1), blk.row0 + r[j]) + at[j]);
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (k0 + u < blk.parts) o[j] += w_of[(k0 + u) * kRows + r[j]] * x[j][u];
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j)
      if (i0 + j * THREADS < rows * Q4) store(blk.row0 + r[j], o[j], at[j] / 4, lse_of[r[j]]);
  }
}

// Rows of partial sums per head that a call may need: as many as the parts of
// two rounds of workgroups hold, or all rows in kMaxParts parts.
int part_rows_of(int Hq, int Hkv, int n_tokens) {
  return (int)std::min<int64_t>(std::max(2 * kSlots / Hkv, 1) * kRows,
                                (int64_t)kMaxParts * n_tokens * (Hq / Hkv));
}

}  // namespace

size_t attn_prefill_workspace(int D, int Hq, int Hkv, int n_seqs, int n_tokens) {
  return kAttnDataOff + (size_t)part_rows_of(Hq, Hkv, n_tokens) * Hkv * (D + 4) * sizeof(float);
}

namespace {

template <int DT, int D, int GROUPS>
hipError_t launch(const AttnDesc &d, void *ws, hipStream_t s) {
  // Every block of whole rows, and the items that cutting some may add: up to
  // a full round of workgroups, or a round more where sequences may differ in
  // length; none from four rounds on, whose end is short anyway.
  const int64_t blocks = (int64_t)d.n_tokens * d.G / kRows + d.n_seqs;
  const int slots = std::max(kSlots / GROUPS / d.Hkv, 1), part_rows = part_rows_of(d.Hq, d.Hkv, d.n_tokens);
  const int extra = blocks < slots ? slots - (int)blocks : blocks < 4 * slots && d.n_seqs > 1 ? slots : 0;
  const int64_t items = blocks + extra;
  hipLaunchKernelGGL((attn_prefill_kernel<DT, D, GROUPS>), dim3((unsigned)(items * d.Hkv)),
                     dim3(64 * kWaves * GROUPS), 0, s, d, part_rows, extra > 0 ? (int)items : 0, (uint32_t *)ws,
                     (float *)((char *)ws + kAttnDataOff),
                     (int)((size_t)part_rows * d.Hkv * (D + 4) * sizeof(float)));
  return hipGetLastError();
}

// Two groups of waves a workgroup where one workgroup a CU takes all whole
// blocks: what bounds such a call is a block's chain of tiles, which two groups
// halve without partial sums in memory.  In us with two groups, one, and one with
// no block cut: 1024 tokens of 32 / 8 heads over 1024 keys 28, 53, 30 (what is
// gained there is that no block is cut); over 4096 78, 99, 89; over 16384 272, 278,
// 305; 256 of 32 heads over 4096 48, 72, 82; 16 of 64 / 8 heads over 16384 57, 64,
// 301.
// One group with more blocks, where two of them on a CU hide each other's waits
// (2048 tokens of 32 heads over 2048 keys 57 us, with two groups 70), with
// blocks that are half empty (4 x 33..64 tokens of 32 heads, D = 64, over 4096
// keys 35 and 39) and on short tables (16 tokens 7.3 and 8.3).
// The rule sees what the host knows: the table's width and not the lengths in it,
// and the rows of all sequences together.  A short cache in a wide table takes two
// groups too, and more time for it (first chunks of 128 and 256 tokens 11.9 and
// 13.9 us, with one group 10.4 and 12.9).
template <int DT, int D>
hipError_t launch(const AttnDesc &d, void *ws, hipStream_t s) {
  const int64_t rows = (int64_t)d.n_tokens * d.G, blocks = (rows + (int64_t)(kRows - 1) * d.n_seqs) / kRows;
  const int64_t room = (int64_t)d.width * d.page_size;
  const int64_t keys = d.window > 0 ? std::min<int64_t>(room, (int64_t)d.window + d.sinks) : room;
  return 2 * rows > (int64_t)kRows * d.n_seqs && blocks * d.Hkv <= kSlots / 2 && keys >= 8 * kKeys
             ? launch<DT, D, 2>(d, ws, s)
             : launch<DT, D, 1>(d, ws, s);
}

}  // namespace

hipError_t launch_attn_prefill(const AttnDesc &d, void *ws, hipStream_t s) {
  if (d.D == 64)
    return d.dtype == DT_F16 ? launch<DT_F16, 64>(d, ws, s) : launch<DT_BF16, 64>(d, ws, s);
  return d.dtype == DT_F16 ? launch<DT_F16, 128>(d, ws, s) : launch<DT_BF16, 128>(d, ws, s);
}

}  // namespace spear
