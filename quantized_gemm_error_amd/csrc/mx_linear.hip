// y = x w^T on microscaled operands for few tokens: bound by the weights'
// stream from memory.
//
// A workgroup makes 16 NT rows of w times 16 MT tokens; its waves take units
// of PER 128-column steps in turn, a wave's operands straight from memory (1 KB
// a load: the matrices lie in memory as the products take them), and their
// sums meet in LDS, always in the same order.  A few tokens that come in 16 bits
// are quantized by the waves that use them, while their weights are on the way:
// four lanes hold a token's 128 columns.
#include "mx_mfma.h"

namespace spear {
namespace {

// Where the tokens come from: a microscaled matrix, or 16-bit rows.
constexpr int kFromMx = -1;

// A token's operand of one step from its 16-bit values: lane (r, g) = (lane %
// 16, lane / 16) has columns 32 g .. (e2m1, its block) or 16 g .. and 64 +
// 16 g .. (e4m3, halves of blocks g / 2 and 2 + g / 2) in four pieces of 8.
// bytes: the scales, e2m1's own block's, e4m3's of the two halves.
template <int DT, int XF>
__device__ __forceinline__ void quantize_step(const u16x8_t (&raw)[4], u32x4_t (&x)[2], uint32_t &bytes) {
  float v[4][8];
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = to_f32<DT>(raw[i][j]);
      m[i] = max(m[i], bitcast<uint32_t>(v[i][j]) & 0x7FFFFFFFu);
    }
  }
  if constexpr (XF == SPEAR_MXFP4) {
    bytes = mx_scale_byte<XF>(max(max(m[0], m[1]), max(m[2], m[3])));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t q[2];
      mx_codes<XF>(v[i], bytes, q);
      x[0][i] = q[0];
      x[1][i] = 0u;
    }
  } else {
    bytes = 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t half = max(m[2 * h], m[2 * h + 1]);
      const auto both = __builtin_amdgcn_permlane16_swap(half, half, false, false);  // with lane ^ 16
      const uint32_t byte = mx_scale_byte<XF>(max((uint32_t)both[0], (uint32_t)both[1]));
      bytes |= byte << (8 * h);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t q[2];
        mx_codes<XF>(v[2 * h + i], byte, q);
        x[h][2 * i] = q[0];
        x[h][2 * i + 1] = q[1];
      }
    }
  }
}

template <int XF, int NT, int MT, int WAVES, int PER, int FROM>
__global__ __launch_bounds__(64 * WAVES) void mx_decode_kernel(MxLinearDesc d) {
  constexpr int kXPieces = XF == SPEAR_MXFP4 ? 1 : 2;
  static_assert(FROM == kFromMx || MT == 1, "one block of tokens is quantized in place");
  __shared__ f32x4_t part[WAVES][NT * MT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * NT, KT = d.w.kt, KQ = d.w.kq;
  f32x4_t acc[NT][MT];
  const uint8_t *w[NT], *x[MT];
  const int *ws[NT], *xs[MT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const size_t b = min(n0 + i, d.w.rb - 1);  // (past the last block its results are not stored)
    w[i] = d.w.codes + b * KT * 1024 + 16 * lane;
    ws[i] = (const int *)d.w.scales + b * KQ * 64 + lane;
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const size_t b = min(j, d.x.rb - 1);
    x[j] = d.x.codes + b * KT * (1024 * kXPieces) + 16 * lane;
    xs[j] = (const int *)d.x.scales + b * KQ * 64 + lane;
  }
  const int r = lane & 15, g = lane >> 4;
  const uint16_t *row = d.x16 + (int64_t)r * d.x16_stride + (XF == SPEAR_MXFP4 ? 32 : 16) * g;

  for (int t0 = wave * PER; t0 < KT; t0 += WAVES * PER) {
    u32x4_t a[PER][NT], b[PER][MT][2];
    int sa[NT], sb[MT];
    uint32_t bytes[PER];
#pragma unroll
    for (int i = 0; i < NT; ++i) sa[i] = __builtin_nontemporal_load(ws[i] + (size_t)(t0 >> 2) * 64);
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int t = min(t0 + p, KT - 1);  // (a step past the last is not multiplied)
#pragma unroll
      for (int i = 0; i < NT; ++i) a[p][i] = __builtin_nontemporal_load((const u32x4_t *)(w[i] + (size_t)t * 1024));
    }
    if constexpr (FROM == kFromMx) {
#pragma unroll
      for (int j = 0; j < MT; ++j) sb[j] = xs[j][(size_t)(t0 >> 2) * 64];
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const int t = min(t0 + p, KT - 1);
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            b[p][j][h] = h < kXPieces ? *(const u32x4_t *)(x[j] + (size_t)t * (1024 * kXPieces) + 1024 * h)
                                      : u32x4_t{0u, 0u, 0u, 0u};
      }
    } else {
      u16x8_t raw[PER][4];
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const int t = min(t0 + p, KT - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = 128 * t + (XF == SPEAR_MXFP4 ? 8 * i : 64 * (i >> 1) + 8 * (i & 1));
          raw[p][i] = r < d.x.rows ? *(const u16x8_t *)(row + at) : u16x8_t{0, 0, 0, 0, 0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int p = 0; p < PER; ++p) quantize_step<FROM, XF>(raw[p], b[p][0], bytes[p]);
    }
    // all of the unit's loads go out before its first product (the compiler
    // would let them wait for registers that it does not need: 28 -> 26 us)
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      if (t0 + p >= KT) break;
      const int shift = 8 * ((t0 + p) & 3);
      int xscale[MT];
      if constexpr (FROM == kFromMx) {
#pragma unroll
        for (int j = 0; j < MT; ++j) xscale[j] = sb[j] >> shift;
      } else if constexpr (XF == SPEAR_MXFP4) {
        xscale[0] = (int)bytes[p];
      } else {
        // block g's byte is half g / 2 of the lanes 2 (g % 2) and the one after
        xscale[0] = __shfl((int)bytes[p], r + 32 * (g & 1)) >> (8 * (g >> 1));
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
          acc[i][j] = mx_mfma<XF>(a[p][i], b[p][j], sa[i] >> shift, xscale[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[wave][i * MT + j][lane] = acc[i][j];
  __syncthreads();
  for (int o = tid; o < NT * MT * 64; o += 64 * WAVES) {
    const int tile = o >> 6, l = o & 63;
    f32x4_t v = part[0][tile][l];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) v += part[k][tile][l];
    store_y(d, 16 * (tile % MT) + (l & 15), 16 * (n0 + tile / MT) + 4 * (l >> 4), v);
  }
}

template <int XF, int NT, int MT, int WAVES, int PER>
hipError_t launch_from(const MxLinearDesc &d, hipStream_t s) {
  const dim3 grid((d.w.rb + NT - 1) / NT), block(64 * WAVES);
  if constexpr (MT == 1) {
    if (d.x16) {
      if (d.x16_dtype == SPEAR_F16) mx_decode_kernel<XF, NT, MT, WAVES, PER, DT_F16><<<grid, block, 0, s>>>(d);
      else mx_decode_kernel<XF, NT, MT, WAVES, PER, DT_BF16><<<grid, block, 0, s>>>(d);
      return hipGetLastError();
    }
  }
  mx_decode_kernel<XF, NT, MT, WAVES, PER, kFromMx><<<grid, block, 0, s>>>(d);
  return hipGetLastError();
}

template <int XF, int MT>
hipError_t launch_rows(const MxLinearDesc &d, hipStream_t s) {
  // As many blocks of 16 rows a workgroup (which share what it reads of x, and
  // quantizes) as leave one to a CU, 4 at most, and then as few waves as keep
  // enough loads in flight.  us in a graph, e4m3 tokens of a matrix, with 1 / 2 /
  // 4 blocks and 4 blocks of 4 waves: one token, 4096 rows of 4096 4.6 / 5.2 / 6.6 /
  // 7.2, 6144 rows 6.7 / 5.6 / 6.9 / 7.7, 11008 rows 9.5 / 8.2 / 8.2 / 8.9, 28672
  // rows of 8192 35 / 25.0 / 27 / 25.1; 32 tokens 5.7 / 6.4 / 7.8 / 10, 9.0 / 6.7 / 8.2 /
  // 10, 12.9 / 10.2 / 9.8 / 11 and 48 / 33 / 31 / 28.8.
  constexpr int PER = MT == 1 ? 4 : MT == 2 ? 2 : 1;
  if (d.w.rb <= 256) return launch_from<XF, 1, MT, 16, PER>(d, s);
  if (d.w.rb <= 512) return launch_from<XF, 2, MT, 8, PER>(d, s);
  if (d.w.rb <= 1024) return launch_from<XF, 4, MT, 8, PER>(d, s);
  return launch_from<XF, 4, MT, 4, PER>(d, s);
}

template <int XF>
hipError_t launch_tokens(const MxLinearDesc &d, hipStream_t s) {
  return d.x.rows <= 16   ? launch_rows<XF, 1>(d, s)
         : d.x.rows <= 32 ? launch_rows<XF, 2>(d, s)
                          : launch_rows<XF, 4>(d, s);
}

}  // namespace

// Every workgroup quantizes the tokens anew, so a launch that does it once pays
// from longer rows or more tokens on.  us in a graph, in place / apart, with 1, 4
// and 8 e4m3 tokens: 2048 -> 1024 4.7 / 5.6, 5.2 / 6.0, 5.5 / 6.0; 2048 -> 11008 7.4 /
// 8.1, 7.6 / 8.4, 8.0 / 8.6; 4096 -> 4096 7.6 / 7.0, 7.6 / 7.4, 7.9 / 7.5; 4096 ->
// 28672 17.3 / 18.2, 18.0 / 18.9, 19.0 / 19.2; 8192 -> 4096 10.9 / 9.1, 10.6 / 9.6,
// 11.2 / 9.5; 8192 -> 28672 29.7 / 28.0, 30.2 / 29.0, 31.9 / 29.1.  (e2m1: 4096 ->
// 4096 6.0 / 6.4, 6.1 / 6.9, 6.7 / 6.8, -> 28672 16.5 / 15.9, 17.7 / 16.8, 18.9 / 17.0.)
// As calls of their own a launch less spares 2 up to 4096 columns: 4096 -> 4096
// 7.9 / 10.6.  So in place where calls gain and a graph loses no more than it gains.
bool mx_linear_quantizes(int tokens, int cols) { return tokens <= 4 && cols <= 4096 && cols % 128 == 0; }

// Streaming makes 64 tokens at most, and up to there is the faster but for the
// widest layers.  us in a graph, streamed / tiled, 33, 48 and 64 e4m3 tokens: 4096 ->
// 4096 8.0 / 11.9, 7.9 / 11.9, 8.4 / 11.9; 4096 -> 11008 11.6 / 12.0, 11.8 / 11.9, 12.1 /
// 12.0; 11008 -> 4096 16 / 28 each; 8192 -> 28672 35 / 32, 37 / 32, 39 / 35 (where the
// tiled product is the inexact one; e2m1 27 / 28, 28 / 28, 30 / 29).
hipError_t launch_mx_linear(const MxLinearDesc &d, hipStream_t s) {
  if (d.x.rows > 64) return launch_mx_gemm(d, s);
  return d.x_format == SPEAR_MXFP4 ? launch_tokens<SPEAR_MXFP4>(d, s) : launch_tokens<SPEAR_MXFP8>(d, s);
}

}  // namespace spear
