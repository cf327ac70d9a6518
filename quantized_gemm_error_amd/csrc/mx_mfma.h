// Device code shared by the products on microscaled operands.
#pragma once

#include "mx_device.h"

namespace spear {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// D += A B for one 16x16x128 block: A 16 rows of w (e2m1), B 16 rows of x.
// Lane l holds row l % 16 of either and the scale byte of its block l / 16;
// its 32 codes are block l / 16 (e2m1, 16 bytes) or the columns
// 64 h + 16 (l / 16) .. + 15, h = 0, 1 (e4m3, 32 bytes).  D lands as rows of w
// 4 * (l / 16) + v, row of x l % 16.  The scales are the words' low bytes.
//
// With e4m3 the unit drops product bits about 16 places below the largest
// product, which leaves an error of 1.3e-5 of a typical sum: nothing beside a
// 16-bit result's rounding, but much beside an fp32 one's.  EXACT takes the
// codes of 2 and more and those below 2 in two products of their own, none of
// which loses a bit (4e-8 over 8192 columns, as an fp32 chain).
template <int XF, bool EXACT>
__device__ __forceinline__ f32x4_t mx_mfma(u32x4_t w, const u32x4_t (&x)[2], int ws, int xs, f32x4_t c) {
  const i32x8_t a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8_t b = {(int)x[0][0], (int)x[0][1], (int)x[0][2], (int)x[0][3],
                     (int)x[1][0], (int)x[1][1], (int)x[1][2], (int)x[1][3]};
  if constexpr (EXACT && XF == SPEAR_MXFP8) {
    const i32x8_t big = ((b >> 6) & 0x01010101) * 255;  // bytes whose exponent field is 8 or more
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b & ~big, c, 4, 0, 0, ws, 0, xs);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b & big, c, 4, 0, 0, ws, 0, xs);
  }
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, XF == SPEAR_MXFP4 ? 4 : 0,
                                                          0, ws, 0, xs);
}

// Four neighbouring outputs of token m, from weight row n on.
template <int YT>
__device__ __forceinline__ void store_as(const MxLinearDesc &d, int m, int n, f32x4_t v) {
  typedef typename MxType<YT>::T T;
  T *p = (T *)d.y + (int64_t)m * d.y_stride + n;
  if (d.y_vec && n + 4 <= d.w.rows) {
    if constexpr (YT == SPEAR_F32) {
      *(f32x4_t *)p = v;
    } else {
      typedef uint16_t u16x4_t __attribute__((ext_vector_type(4)));
      u16x4_t o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = MxType<YT>::store(v[j]);
      *(u16x4_t *)p = o;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < d.w.rows) p[j] = MxType<YT>::store(v[j]);
  }
}
__device__ __forceinline__ void store_y(const MxLinearDesc &d, int m, int n, f32x4_t v) {
  if (m >= d.x.rows || n >= d.w.rows) return;
  if (d.y_dtype == SPEAR_F16) store_as<0>(d, m, n, v);
  else if (d.y_dtype == SPEAR_BF16) store_as<1>(d, m, n, v);
  else store_as<2>(d, m, n, v);
}

}  // namespace spear
