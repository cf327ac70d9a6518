// y = x w^T on microscaled operands for many tokens: LDS-tiled, bound by the
// matrix units.
//
// A workgroup of four waves makes 32 NW rows of w times 32 MW tokens, a wave
// 16 NW x 16 MW of them with 16x16x128 products.  Both matrices lie in memory
// as the products take them (1 KB a wave), so that a 128-column step goes from
// memory to LDS in loads of 16 bytes a lane without passing registers, and from
// LDS to operands in reads of 16 bytes a lane, lanes side by side: no
// conflicts.  STAGES buffers in turn, one barrier a step: the loads of step
// t + STAGES - 1 are in flight while step t is multiplied.
#include <algorithm>

#include "mx_mfma.h"

namespace spear {
namespace {

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A buffer from p on, wave-uniform, as its descriptor words; offsets are the
// caller's to hold in range.
__device__ __forceinline__ u32x4_t buffer_words(const void *p) {
  const uint64_t a = (uint64_t)p;
  return u32x4_t{(uint32_t)uniform((int)a), (uint32_t)uniform((int)(a >> 32)) & 0xFFFFu, 0xFFFFFFFFu, 0x00020000u};
}

// 16 bytes a lane from byte `at` (a lane's) + step (uniform) of a buffer to
// LDS byte lds + 16 lane, N times to LDS 1 KB further on each.  Written out
// because the compiler waits for such a load before any later LDS read.  The
// block writes no register but m0, which nothing else in these kernels uses;
// the first wait states are those of a scalar register that a vector
// instruction may have written just before.
template <int N>
__device__ __forceinline__ void load_pieces(u32x4_t buffer, uint32_t lds, const int (&at)[N], int step) {
  asm volatile("s_nop 4" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(lds + 1024 * i), "v"(at[i]), "s"(buffer), "s"(step)
        : "memory");
}

// At most N of this wave's loads are still in flight, then a barrier; LDS
// reads and loads stay on their side of it.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);  // vmcnt(N), lgkmcnt(0)
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

template <int XF, bool EXACT, int NW, int MW, int STAGES>
__global__ __launch_bounds__(256, NW * MW > 32 ? 1 : 2) void mx_gemm_kernel(MxLinearDesc d, int mt) {
  constexpr int kXPieces = XF == SPEAR_MXFP4 ? 1 : 2;          // of 1 KB a tile
  constexpr int PW = 2 * NW, PX = 2 * MW * kXPieces;           // a step's pieces
  constexpr int WP = PW / 4, XP = PX / 4;                      // a wave's share of them
  constexpr int kStage = (PW + PX) * 1024, kScales = (2 * NW + 2 * MW) * 256;
  static_assert(PW % 4 == 0 && PX % 4 == 0, "shares");
  __shared__ __align__(1024) uint8_t lds[STAGES * kStage + 2 * kScales];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int tile = tile_of(blockIdx.x, gridDim.x), tn = tile / mt, tm = tile - tn * mt;
  const int n0 = tn * 2 * NW, m0 = tm * 2 * MW;                // first row blocks
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
  // the scales' loads: 2 NW / 4 of w's, then 2 MW / 4 of x's
  constexpr int SW = (2 * NW + 3) / 4, SX = (2 * MW + 3) / 4;
  int s_at[2];
  bool s_x[2], s_has[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = wave + 4 * i;
    s_has[i] = j < SW + SX;
    s_x[i] = j >= SW;
    const int block = 4 * (s_x[i] ? j - SW : j) + (lane >> 4);
    s_at[i] = min(block, s_x[i] ? m_last : n_last) * KQ * 256 + 16 * (lane & 15);
  }
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  auto load = [&](int t) {
    const uint32_t to = base + (uint32_t)(t % STAGES) * kStage;
    if ((t & 3) == 0) {
      const uint32_t at = base + STAGES * kStage + (uint32_t)((t >> 2) & 1) * kScales;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (s_has[i]) {
          const int one[1] = {s_at[i]};
          load_pieces<1>(s_x[i] ? xsb : wsb, at + (uint32_t)(wave + 4 * i) * 1024, one, (t >> 2) * 256);
        }
    }
    load_pieces<WP>(wb, to + (uint32_t)(wave * WP) * 1024, w_at, t * 1024);
    load_pieces<XP>(xb, to + (uint32_t)(PW + wave * XP) * 1024, x_at, t * (1024 * kXPieces));
  };

  const int wn = wave >> 1, wm = wave & 1;
  f32x4_t acc[NW][MW];
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int j = 0; j < MW; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < STAGES - 1; ++t)
    if (t < KT) load(t);
  for (int t = 0; t < KT; ++t) {
    // step t has landed, and all waves are done with the step before
    if (STAGES > 2 && t + STAGES - 2 < KT) wait_and_meet<(STAGES - 2) * (WP + XP)>();
    else wait_and_meet<0>();
    if (t + STAGES - 1 < KT) load(t + STAGES - 1);
    const uint8_t *at = lds + (t % STAGES) * kStage + 16 * lane;
    const uint8_t *sc = lds + STAGES * kStage + ((t >> 2) & 1) * kScales + 4 * lane;
    u32x4_t x[MW][2];
    int xs[MW], ws[NW];
#pragma unroll
    for (int j = 0; j < MW; ++j) {
      const int p = wm * MW + j;
#pragma unroll
      for (int h = 0; h < kXPieces; ++h) x[j][h] = *(const u32x4_t *)(at + (PW + p * kXPieces + h) * 1024);
      if (kXPieces == 1) x[j][1] = u32x4_t{0u, 0u, 0u, 0u};
      xs[j] = *(const int *)(sc + (2 * NW + p) * 256) >> (8 * (t & 3));
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) ws[i] = *(const int *)(sc + (wn * NW + i) * 256) >> (8 * (t & 3));
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const u32x4_t w = *(const u32x4_t *)(at + (wn * NW + i) * 1024);
#pragma unroll
      for (int j = 0; j < MW; ++j) acc[i][j] = mx_mfma<XF, EXACT>(w, x[j], ws[i], xs[j], acc[i][j]);
    }
  }
  const int n = 16 * (n0 + wn * NW) + 4 * (lane >> 4), m = 16 * (m0 + wm * MW) + (lane & 15);
#pragma unroll
  for (int j = 0; j < MW; ++j)
#pragma unroll
    for (int i = 0; i < NW; ++i) store_y(d, m + 16 * j, n + 16 * i, acc[i][j]);
}

template <int XF, bool EXACT, int NW, int MW, int STAGES>
hipError_t launch_tiles(const MxLinearDesc &d, hipStream_t s) {
  const int nt = (d.w.rb + 2 * NW - 1) / (2 * NW), mt = (d.x.rb + 2 * MW - 1) / (2 * MW);
  mx_gemm_kernel<XF, EXACT, NW, MW, STAGES><<<dim3((unsigned)nt * mt), dim3(256), 0, s>>>(d, mt);
  return hipGetLastError();
}

template <int XF, bool EXACT>
hipError_t launch_as(const MxLinearDesc &d, hipStream_t s) {
  return launch_tiles<XF, EXACT, 8, 4, 2>(d, s);
}

}  // namespace

hipError_t launch_mx_gemm(const MxLinearDesc &d, hipStream_t s) {
  if (d.x_format == SPEAR_MXFP4) return launch_as<SPEAR_MXFP4, false>(d, s);
  return d.y_dtype == SPEAR_F32 ? launch_as<SPEAR_MXFP8, true>(d, s) : launch_as<SPEAR_MXFP8, false>(d, s);
}

}  // namespace spear
