// y = x w^T on microscaled operands for many tokens: LDS-tiled, bound by the
// matrix units.
//
// WN x WM waves make 16 NW rows of w times 16 MW tokens each with 32x32x64
// products.  Both matrices lie in memory as the products take them (1 KB a
// wave), so that a 128-column step goes from memory to LDS in loads of 16
// bytes a lane without passing registers, and from LDS to operands in reads of
// 16 bytes a lane, 16 lanes side by side: no conflicts.  STAGES buffers in turn,
// one barrier a step: the loads of step t + STAGES - 1 are in flight while step
// t is multiplied.
//
// Measured (MI355X): 2048 tokens 4096 -> 11008 with e4m3 tokens 81 us (2.3
// PFLOP/s; products alone, of random numbers, reach 4.2 to 4.6, a large fp8
// product of the library 2.7), 28672 -> 8192 with e2m1 tokens 245 us (3.9
// PFLOP/s; 6.8 alone).  Without the loads the first would take 25 us less,
// without the LDS reads 8 less; the products' clock falls under their load.
// Tried: a half step's operands read while the half before is multiplied (82 ->
// 95 us: the waves of a SIMD cover the reads for one another), loads sent
// between the products (92), 256 x 256 tiles of four waves (133) and of eight
// (115), three and four buffers for the large tiles (106, one workgroup a CU).
#include <algorithm>

#include "mx_mfma.h"

namespace spear {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// D += A B for one 32x32x64 block: A 32 rows of w, B 32 rows of x.  Lane l
// holds row l % 32 of either and the scale byte of its block l / 32; its 32
// codes are that block (e2m1) or the columns 32 j + 16 (l / 32) .. + 15,
// j = 0, 1 (e4m3).  D lands as rows of w 8 (v / 4) + 4 (l / 32) + v % 4, row of
// x l % 32.  (16x16x128 products take as long with e4m3, but reach 6.5 instead
// of 9.4 PFLOP/s with e2m1 on both sides.)
//
// EXACT: e4m3 codes in two products, as in mx_mfma.  Only fp32 results have
// them: the products are what bounds this kernel (2048 tokens 4096 -> 11008 83 us
// with one, 157 with two, 128 tokens 4096 -> 4096 12 and 17), and what one drops,
// less than a 2^-12th of the largest product of eight columns each, is 1.3e-5 of
// a typical sum; rounding it to fp16 or bf16 is off by up to 4.9e-4 or 3.9e-3.
template <int XF, bool EXACT>
__device__ __forceinline__ f32x16_t mx_mfma32(u32x4_t w, const u32x4_t (&x)[2], int ws, int xs, f32x16_t c) {
  const i32x8_t a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8_t b = {(int)x[0][0], (int)x[0][1], (int)x[0][2], (int)x[0][3],
                     (int)x[1][0], (int)x[1][1], (int)x[1][2], (int)x[1][3]};
  if constexpr (EXACT && XF == SPEAR_MXFP8) {
    const i32x8_t big = codes_of_2_and_more(b);
    c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b & ~big, c, 4, 0, 0, ws, 0, xs);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, big, c, 4, 0, 0, ws, 0, xs);
  }
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, XF == SPEAR_MXFP4 ? 4 : 0, 0, ws, 0, xs);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A buffer from p on, wave-uniform, as its descriptor words; offsets are the
// caller's to hold in range.
__device__ __forceinline__ u32x4_t buffer_words(const void *p) {
  const uint64_t a = (uint64_t)p;
  return u32x4_t{(uint32_t)uniform((int)a), (uint32_t)uniform((int)(a >> 32)) & 0xFFFFu, 0xFFFFFFFFu, 0x00020000u};
}

// 16 bytes a lane from byte `at` (a lane's) + step (uniform) of a buffer to
// LDS byte lds + 16 lane.  Written out because the compiler waits for such a
// load before any later LDS read.  The block writes no register but m0; the
// wait states are those of a scalar register that a vector instruction may
// have written just before.
__device__ __forceinline__ void load_piece(u32x4_t buffer, uint32_t lds, int at, int step) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 4\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(at), "s"(buffer), "s"(step)
      : "memory", "m0");
}

// At most N of this wave's loads are still in flight, then a barrier; LDS
// reads and loads stay on their side of it.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);  // vmcnt(N)
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Workgroup `b` of `blocks`: workgroups go to the 8 XCDs in turn, so each XCD
// takes a run of tiles, the token tiles of one weight tile after another,
// whose weights its L2 then serves.
__device__ __forceinline__ int tile_of(int b, int blocks) {
  const int x = b & 7, each = blocks >> 3, more = blocks & 7;
  return x * each + min(x, more) + (b >> 3);
}

// Blocks of 32 rows of w that are turned at once, and the bytes that takes at
// most (fp32; rows 16 bytes longer than their values, against bank conflicts).
template <int NB>
constexpr int kTurn = NB > 1 ? 2 : 1;
template <int NB>
constexpr int kTurnBytes = 32 * (kTurn<NB> * 32 * 4 + 16);

template <int YT, int NB, int MB>
__device__ __forceinline__ void turn_out(const MxLinearDesc &d, uint8_t *lds, const f32x16_t (*acc)[MB], int j, int m,
                                         int n, int lane) {
  typedef typename MxType<YT>::T T;
  constexpr int kCols = 32 * kTurn<NB>, kRow = kCols * sizeof(T) + 16, kPiece = 16 / sizeof(T);
  if (n >= d.w.rows || m >= d.x.rows) return;
  const int row = lane & 31, g = lane >> 5;
#pragma unroll
  for (int i = 0; i < kTurn<NB>; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      T o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = MxType<YT>::store(acc[i][j][4 * v + e]);
      __builtin_memcpy(lds + row * kRow + (32 * i + 8 * v + 4 * g) * sizeof(T), o, sizeof o);
    }
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
#pragma unroll
  for (int k = 0; k < 32 * kCols / kPiece / 64; ++k) {
    const int p = lane + 64 * k, r = p / (kCols / kPiece), c = p % (kCols / kPiece) * kPiece;
    const u32x4_t v = *(const u32x4_t *)(lds + r * kRow + c * sizeof(T));
    if (m + r >= d.x.rows) continue;
    T *to = (T *)d.y + (int64_t)(m + r) * d.y_stride + n + c;
    if (d.y_vec16 && n + c + kPiece <= d.w.rows) {
      *(u32x4_t *)to = v;
    } else {
      T o[kPiece];
      __builtin_memcpy(o, &v, 16);
#pragma unroll
      for (int e = 0; e < kPiece; ++e)
        if (n + c + e < d.w.rows) to[e] = o[e];
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
}

template <int XF, bool EXACT, int WN, int WM, int NW, int MW, int STAGES, int PERSIMD>
__global__ __launch_bounds__(64 * WN * WM, PERSIMD) void mx_gemm_kernel(MxLinearDesc d, int mt) {
  constexpr int kWaves = WN * WM;
  constexpr int kXPieces = XF == SPEAR_MXFP4 ? 1 : 2;          // of 1 KB a tile
  constexpr int PN = WN * NW, PM = WM * MW;                    // row blocks of w and x
  constexpr int PW = PN, PX = PM * kXPieces;                   // a step's pieces
  constexpr int WP = PW / kWaves, XP = PX / kWaves;            // a wave's share of them
  constexpr int kStage = (PW + PX) * 1024, kScales = (PN + PM) * 256;
  constexpr int kSlots = STAGES > 5 ? 4 : 2;                   // of scales: 4 steps each
  static_assert(PW % kWaves == 0 && PX % kWaves == 0 && PN % 4 == 0 && PM % 4 == 0, "shares");
  constexpr int kSteps = STAGES * kStage + kSlots * kScales, kOut = kWaves * kTurnBytes<NW / 2>;
  __shared__ __align__(1024) uint8_t lds[kSteps > kOut ? kSteps : kOut];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int tile = tile_of(blockIdx.x, gridDim.x), tn = tile / mt, tm = tile - tn * mt;
  const int n0 = tn * PN, m0 = tm * PM;                        // first row blocks
  const int KT = d.w.kt, KQ = d.w.kq;

  // what this wave loads: pieces of w and x, and of their scales 4 row blocks
  // a load (past the last row block the last one: its results are not stored)
  const u32x4_t wb = buffer_words(d.w.codes + (size_t)n0 * KT * 1024);
  const u32x4_t xb = buffer_words(d.x.codes + (size_t)m0 * KT * (1024 * kXPieces));
  const u32x4_t wsb = buffer_words(d.w.scales + (size_t)n0 * KQ * 256);
  const u32x4_t xsb = buffer_words(d.x.scales + (size_t)m0 * KQ * 256);
  const int n_last = d.w.rb - 1 - n0, m_last = d.x.rb - 1 - m0;
  int w_at[WP], x_at[XP];
#pragma unroll
  for (int i = 0; i < WP; ++i) w_at[i] = min(wave * WP + i, n_last) * KT * 1024 + 16 * lane;
#pragma unroll
  for (int i = 0; i < XP; ++i) {
    const int p = wave * XP + i;
    x_at[i] = min(p / kXPieces, m_last) * KT * (1024 * kXPieces) + (p % kXPieces) * 1024 + 16 * lane;
  }
  // the scales' loads: PN / 4 of w's, then PM / 4 of x's
  constexpr int SW = PN / 4, SX = PM / 4, SL = (SW + SX + kWaves - 1) / kWaves;
  int s_at[SL];
  bool s_x[SL], s_has[SL];
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int j = wave + kWaves * i;
    s_has[i] = j < SW + SX;
    s_x[i] = j >= SW;
    const int block = 4 * (s_x[i] ? j - SW : j) + (lane >> 4);
    s_at[i] = min(block, s_x[i] ? m_last : n_last) * KQ * 256 + 16 * (lane & 15);
  }
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  // piece i of this wave's share of step t
  auto load = [&](int t, int i) {
    const uint32_t to = base + (uint32_t)(t % STAGES) * kStage;
    if (i < WP) load_piece(wb, to + (uint32_t)(wave * WP + i) * 1024, w_at[i], t * 1024);
    else load_piece(xb, to + (uint32_t)(PW + wave * XP + i - WP) * 1024, x_at[i - WP], t * (1024 * kXPieces));
  };
  auto load_scales = [&](int t) {
    const uint32_t at = base + STAGES * kStage + (uint32_t)((t >> 2) & (kSlots - 1)) * kScales;
#pragma unroll
    for (int i = 0; i < SL; ++i)
      if (s_has[i]) load_piece(s_x[i] ? xsb : wsb, at + (uint32_t)(wave + kWaves * i) * 1024, s_at[i], (t >> 2) * 256);
  };
  const int wn = wave / WM, wm = wave % WM;
  constexpr int NB = NW / 2, MB = MW / 2;  // blocks of 32
  f32x16_t acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  // a lane's place in a pair of row blocks: row lane % 32, block lane / 32
  const int row = lane & 15, upper = (lane >> 4) & 1, g = lane >> 5;
  const int w_from = upper * 1024 + 256 * g + 16 * row, x_from = upper * (1024 * kXPieces) + 256 * g + 16 * row;
  const int s_from = upper * 256 + 64 * g + 4 * row;
  auto send = [&](int t) {
    if ((t & 3) == 0) load_scales(t);
#pragma unroll
    for (int i = 0; i < WP + XP; ++i) load(t, i);
  };
#pragma unroll
  for (int t = 0; t < STAGES - 1; ++t)
    if (t < KT) send(t);
  // A step's halves, blocks 2 h and 2 h + 1.
  struct Half {
    u32x4_t x[MB][2], w[NB];
    int xs[MB], ws[NB];
  } half[2];
  auto read = [&](int t, int h) {
    Half &o = half[h];
    const uint8_t *at = lds + (t % STAGES) * kStage;
    const uint8_t *sc = lds + STAGES * kStage + ((t >> 2) & (kSlots - 1)) * kScales + s_from;
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int p = wm * MW + 2 * j;
      o.xs[j] = *(const int *)(sc + (PN + p) * 256 + 128 * h);
      const uint8_t *from = at + (PW + p * kXPieces) * 1024 + x_from;
      if constexpr (XF == SPEAR_MXFP4) {
        o.x[j][0] = *(const u32x4_t *)(from + 512 * h);
        o.x[j][1] = u32x4_t{0u, 0u, 0u, 0u};
      } else {
        o.x[j][0] = *(const u32x4_t *)(from + 1024 * h);
        o.x[j][1] = *(const u32x4_t *)(from + 1024 * h + 512);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int p = wn * NW + 2 * i;
      o.ws[i] = *(const int *)(sc + p * 256 + 128 * h);
      o.w[i] = *(const u32x4_t *)(at + p * 1024 + w_from + 512 * h);
    }
  };
  auto multiply = [&](int t, int h) {
    const Half &o = half[h];
    const int shift = 8 * (t & 3);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j)
        acc[i][j] = mx_mfma32<XF, EXACT>(o.w[i], o.x[j], o.ws[i] >> shift, o.xs[j] >> shift, acc[i][j]);
  };
  for (int t = 0; t < KT; ++t) {
    // step t has landed, and all waves are done with the step before
    if (STAGES > 2 && t + STAGES - 2 < KT) wait_and_meet<(STAGES - 2) * (WP + XP)>();
    else wait_and_meet<0>();
    if (t + STAGES - 1 < KT) send(t + STAGES - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      read(t, h);
      __builtin_amdgcn_s_setprio(1);  // (97 -> 94 us, 248 -> 243 us)
      multiply(t, h);
      __builtin_amdgcn_s_setprio(0);
    }
  }
  // Outputs leave by rows: a wave turns 32 tokens x 64 (or 32) rows of w at a
  // time in a part of LDS of its own.
  wait_and_meet<0>();
  uint8_t *mine = lds + wave * kTurnBytes<NB>;
#pragma unroll
  for (int j = 0; j < MB; ++j)
#pragma unroll
    for (int i = 0; i < NB; i += kTurn<NB>) {
      const int n = 16 * (n0 + wn * NW) + 32 * i, m = 16 * (m0 + wm * MW) + 32 * j;
      if (d.y_dtype == SPEAR_F16) turn_out<0, NB>(d, mine, &acc[i], j, m, n, lane);
      else if (d.y_dtype == SPEAR_BF16) turn_out<1, NB>(d, mine, &acc[i], j, m, n, lane);
      else turn_out<2, NB>(d, mine, &acc[i], j, m, n, lane);
    }
}

template <int XF, bool EXACT, int WN, int WM, int NW, int MW, int STAGES, int PERSIMD>
hipError_t launch_tiles(const MxLinearDesc &d, hipStream_t s) {
  const int nt = (d.w.rb + WN * NW - 1) / (WN * NW), mt = (d.x.rb + WM * MW - 1) / (WM * MW);
  mx_gemm_kernel<XF, EXACT, WN, WM, NW, MW, STAGES, PERSIMD><<<dim3((unsigned)nt * mt), dim3(64 * WN * WM), 0, s>>>(d, mt);
  return hipGetLastError();
}

template <int XF, bool EXACT>
hipError_t launch_as(const MxLinearDesc &d, hipStream_t s) {
  // Large tiles read less from LDS and L2 for each product, small ones fill
  // the chip and end together.  us for 64 x 64 / 128 x 64 / 128 x 128 / 256 x 128
  // (rows of w x e4m3 tokens): 128 tokens 4096 -> 4096 12 / 15 / 20 / 29, 1024
  // tokens 28 / 22 / 23 / 30, 2048 tokens 62 / 42 / 34 / 36, 512 tokens 8192 ->
  // 28672 172 / 145 / 120 / 110; three and four buffers where a CU has one
  // workgroup or two, two where it has more.
  const int units = ((d.w.rb + 3) / 4) * ((d.x.rb + 3) / 4);  // of 64 x 64 outputs
  if (units <= 512) return launch_tiles<XF, EXACT, 2, 2, 2, 2, 4, 1>(d, s);
  if (units <= 1024) return launch_tiles<XF, EXACT, 2, 2, 4, 2, 3, 1>(d, s);
  if (units <= 3200) return launch_tiles<XF, EXACT, 2, 2, 4, 4, 2, 2>(d, s);
  return launch_tiles<XF, EXACT, 4, 2, 4, 4, 2, 4>(d, s);
}

}  // namespace

hipError_t launch_mx_gemm(const MxLinearDesc &d, hipStream_t s) {
  if (d.x_format == SPEAR_MXFP4) return launch_as<SPEAR_MXFP4, false>(d, s);
  return d.y_dtype == SPEAR_F32 ? launch_as<SPEAR_MXFP8, true>(d, s) : launch_as<SPEAR_MXFP8, false>(d, s);
}

}  // namespace spear
