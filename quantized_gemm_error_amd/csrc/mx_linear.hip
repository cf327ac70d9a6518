// y = x w^T on microscaled operands.
#include "mx_device.h"

namespace spear {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// D += A B for one 16x16x128 block: A 16 rows of w (e2m1), B 16 rows of x.
// Lane l holds row l % 16 of either and the scale byte of its block l / 16;
// its 32 codes are block l / 16 (e2m1, 16 bytes) or the columns
// 64 h + 16 (l / 16) .. + 15, h = 0, 1 (e4m3, 32 bytes).  D lands as rows of w
// 4 * (l / 16) + v, row of x l % 16.  BYTE: the scale's place in its word.
//
// With e4m3 the unit drops product bits about 16 places below the largest
// product, which leaves an error of 1.3e-5 of a typical sum: nothing beside a
// 16-bit result's rounding, but much beside an fp32 one's.  EXACT takes the
// codes of 2 and more and those below 2 in two products of their own, none of
// which loses a bit (4e-8 over 8192 columns, as an fp32 chain).
template <int XF, int BYTE, bool EXACT>
__device__ __forceinline__ f32x4_t mx_mfma(u32x4_t w, const u32x4_t (&x)[2], int ws, int xs, f32x4_t c) {
  const i32x8_t a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8_t b = {(int)x[0][0], (int)x[0][1], (int)x[0][2], (int)x[0][3],
                     (int)x[1][0], (int)x[1][1], (int)x[1][2], (int)x[1][3]};
  if constexpr (EXACT && XF == SPEAR_MXFP8) {
    const i32x8_t big = ((b >> 6) & 0x01010101) * 255;  // bytes whose exponent field is 8 or more
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b & ~big, c, 4, 0, BYTE, ws, BYTE, xs);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b & big, c, 4, 0, BYTE, ws, BYTE, xs);
  }
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, XF == SPEAR_MXFP4 ? 4 : 0,
                                                          BYTE, ws, BYTE, xs);
}

template <int YT>
__device__ __forceinline__ void store_y(const MxLinearDesc &d, int m, int n, f32x4_t v) {
  typedef typename MxType<YT>::T T;
  if (m >= d.x.rows) return;
  T *p = (T *)d.y + (int64_t)m * d.y_stride + n;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < d.w.rows) p[j] = MxType<YT>::store(v[j]);
}

// One wave makes 16 x 16 outputs, straight from memory.
template <int XF, int YT>
__global__ __launch_bounds__(64) void mx_linear_simple_kernel(MxLinearDesc d) {
  constexpr int kXTile = XF == SPEAR_MXFP4 ? 1024 : 2048;
  const int nb = blockIdx.x % d.w.rb, mb = blockIdx.x / d.w.rb;
  const int lane = threadIdx.x;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  const uint8_t *w = d.w.codes + (size_t)nb * d.w.kt * 1024 + 16 * lane;
  const uint8_t *x = d.x.codes + (size_t)mb * d.x.kt * kXTile + 16 * lane;
  const int *ws = (const int *)d.w.scales + (size_t)nb * d.w.kq * 64 + lane;
  const int *xs = (const int *)d.x.scales + (size_t)mb * d.x.kq * 64 + lane;
  auto tile = [&](int t, int sw, int sx, auto byte) {
    const u32x4_t a = *(const u32x4_t *)(w + (size_t)t * 1024);
    u32x4_t b[2] = {*(const u32x4_t *)(x + (size_t)t * kXTile), {0u, 0u, 0u, 0u}};
    if constexpr (XF == SPEAR_MXFP8) b[1] = *(const u32x4_t *)(x + (size_t)t * kXTile + 1024);
    acc = mx_mfma<XF, decltype(byte)::value, YT == SPEAR_F32>(a, b, sw, sx, acc);
  };
  for (int q = 0; q < d.w.kq; ++q) {
    const int sw = ws[(size_t)q * 64], sx = xs[(size_t)q * 64], n = d.w.kt - 4 * q;
    tile(4 * q, sw, sx, std::integral_constant<int, 0>());
    if (n > 1) tile(4 * q + 1, sw, sx, std::integral_constant<int, 1>());
    if (n > 2) tile(4 * q + 2, sw, sx, std::integral_constant<int, 2>());
    if (n > 3) tile(4 * q + 3, sw, sx, std::integral_constant<int, 3>());
  }
  store_y<YT>(d, 16 * mb + (lane & 15), 16 * nb + 4 * (lane >> 4), acc);
}

template <int XF, int YT>
hipError_t launch_as(const MxLinearDesc &d, hipStream_t s) {
  mx_linear_simple_kernel<XF, YT><<<dim3((unsigned)d.w.rb * d.x.rb), dim3(64), 0, s>>>(d);
  return hipGetLastError();
}

template <int XF>
hipError_t launch_for(const MxLinearDesc &d, hipStream_t s) {
  return d.y_dtype == SPEAR_F16    ? launch_as<XF, 0>(d, s)
         : d.y_dtype == SPEAR_BF16 ? launch_as<XF, 1>(d, s)
                                   : launch_as<XF, 2>(d, s);
}

}  // namespace

size_t mx_linear_workspace(int, int, int) { return 0; }

hipError_t launch_mx_linear(const MxLinearDesc &d, void *, void *, hipStream_t s) {
  return d.x_format == SPEAR_MXFP4 ? launch_for<SPEAR_MXFP4>(d, s) : launch_for<SPEAR_MXFP8>(d, s);
}

}  // namespace spear
