// Quantizing to and from the microscaled formats, and the root-mean-square
// norm.  All three are bound by memory.
#include "mx_device.h"

namespace spear {
namespace {

constexpr int kConvThreads = 256;

// One workgroup makes the 16 rows x 512 columns of a scale group.  A wave's
// load is 512 columns of one row (16 bytes a lane; four lanes hold a block of
// 32 and share its maximum through DPP); the codes go through LDS, so that
// tiles leave in 16-byte pieces one after the other.
template <int DT, int FMT>
__global__ __launch_bounds__(kConvThreads) void mx_quantize_kernel(
    const typename MxType<DT>::T *x, int64_t stride, bool vec, MxDesc out) {
  constexpr int kTile = FMT == SPEAR_MXFP4 ? 1024 : 2048;
  __shared__ __align__(16) uint8_t codes[4 * kTile];
  __shared__ __align__(16) uint8_t scales[256];
  const int rb = blockIdx.x / out.kq, q = blockIdx.x - rb * out.kq;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int col = 512 * q + 8 * lane;
  MxDesc one{};  // the group in LDS
  one.kt = 4;
  one.kq = 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * wave + i, row = 16 * rb + r;
    float v[8];
    const int n = row < out.rows ? out.cols - col : 0;
    if (n > 0) {
      load8<DT>(x + (int64_t)row * stride + col, n, vec, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
    const uint32_t byte = mx_scale_byte<FMT>(block_max_bits(v));
    uint32_t c[2];
    mx_codes<FMT>(v, byte, c);
    uint32_t *to = (uint32_t *)(codes + mx_code_at<FMT>(one, r, lane));
    to[0] = c[0];
    if constexpr (FMT == SPEAR_MXFP8) to[1] = c[1];
    if ((lane & 3) == 0)
      scales[mx_scale_at(one, r, lane >> 2)] = (uint8_t)(32 * (16 * q + (lane >> 2)) < out.cols ? byte : 127u);
  }
  __syncthreads();
  uint8_t *to = out.codes + ((size_t)rb * out.kt + 4 * q) * kTile;
  const int bytes = min(4, out.kt - 4 * q) * kTile;
  for (int i = 16 * threadIdx.x; i < bytes; i += 16 * kConvThreads) *(u32x4_t *)(to + i) = *(u32x4_t *)(codes + i);
  if (threadIdx.x < 64)
    ((uint32_t *)out.scales)[((size_t)rb * out.kq + q) * 64 + threadIdx.x] = ((uint32_t *)scales)[threadIdx.x];
}

__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const uint32_t m = code & 7u;
  const float v = m < 2u ? 0.5f * (float)m : bitcast<float>(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  return code & 8u ? -v : v;
}
// Codes 2 h and 2 h + 1 of a word, NaN for those of NaN.
__device__ __forceinline__ void e4m3_values(uint32_t word, int h, float *v) {
  const auto t = h ? __builtin_amdgcn_cvt_pk_f32_fp8((int)word, true) : __builtin_amdgcn_cvt_pk_f32_fp8((int)word, false);
  v[0] = t[0];
  v[1] = t[1];
}

// The reverse: codes by 16-byte pieces into LDS, rows out of it.
template <int DT, int FMT>
__global__ __launch_bounds__(kConvThreads) void mx_dequantize_kernel(
    MxDesc x, typename MxType<DT>::T *out, int64_t stride, bool vec) {
  constexpr int kTile = FMT == SPEAR_MXFP4 ? 1024 : 2048;
  __shared__ __align__(16) uint8_t codes[4 * kTile];
  __shared__ __align__(16) uint8_t scales[256];
  const int rb = blockIdx.x / x.kq, q = blockIdx.x - rb * x.kq;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int col = 512 * q + 8 * lane;
  const uint8_t *from = x.codes + ((size_t)rb * x.kt + 4 * q) * kTile;
  const int bytes = min(4, x.kt - 4 * q) * kTile;
  for (int i = 16 * threadIdx.x; i < bytes; i += 16 * kConvThreads) *(u32x4_t *)(codes + i) = *(u32x4_t *)(from + i);
  if (threadIdx.x < 64)
    ((uint32_t *)scales)[threadIdx.x] = ((const uint32_t *)x.scales)[((size_t)rb * x.kq + q) * 64 + threadIdx.x];
  __syncthreads();
  MxDesc one{};
  one.kt = 4;
  one.kq = 1;
  if (col >= x.cols) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * wave + i, row = 16 * rb + r;
    if (row >= x.rows) break;
    const uint32_t byte = scales[mx_scale_at(one, r, lane >> 2)];
    const uint32_t *c = (const uint32_t *)(codes + mx_code_at<FMT>(one, r, lane));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      if constexpr (FMT == SPEAR_MXFP4) v[j] = e2m1_value(c[0] >> (4 * j)), v[j + 1] = e2m1_value(c[0] >> (4 * j + 4));
      else e4m3_values(c[j >> 2], j >> 1 & 1, v + j);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = byte == 255u ? bitcast<float>(0x7FC00000u) : __builtin_amdgcn_ldexpf(v[j], (int)byte - 127);
    store8<DT>(out + (int64_t)row * stride + col, x.cols - col, vec, v);
  }
}

constexpr int kNormThreads = 256;

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// A microscaled row's codes are pieces of 4 or 8 bytes in lines that 16 rows
// share.  Workgroups go to the 8 XCDs in turn, so of each 128 rows an XCD takes
// a block of 16, whose lines its L2 then puts together (2047 rows of 4096 bf16
// with a residual to e4m3: 16.0 -> 14.7 us).
template <int OUT>
__device__ __forceinline__ int norm_row(int i, int rows) {
  if (OUT < 0 || (i | 127) >= rows) return i;
  return (i & ~127) + 16 * (i & 7) + ((i >> 3) & 15);
}

// A workgroup a row.  The row stays in registers (CH pieces of eight values a
// thread); its squares are summed in 64 bits, so that the mean, and with it
// every rounding that follows, does not depend on the split.
// OUT: -1 for the 16-bit type, else the microscaled format.
template <int DT, int OUT, int CH>
__global__ __launch_bounds__(kNormThreads) void rms_norm_kernel(NormDesc d, bool vec) {
  __shared__ double part[kNormThreads / 64];
  const int tid = threadIdx.x;
  for (int i = blockIdx.x; i < d.rows; i += gridDim.x) {
    const int row = norm_row<OUT>(i, d.rows);
    float h[CH][8];
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = 8 * (tid + kNormThreads * c), n = d.hidden - col;
      if (n > 0) {
        load8<DT>(d.x + (int64_t)row * d.x_stride + col, n, vec, h[c]);
        if (d.residual) {
          float r[8];
          load8<DT>(d.residual + (int64_t)row * d.residual_stride + col, n, vec, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] += r[j];
          store8<DT>(d.residual_out + (int64_t)row * d.residual_out_stride + col, n, vec, h[c]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)h[c][j], (double)h[c][j], sum);
      }
    }
    sum = wave_sum(sum);
    __syncthreads();
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    sum = part[0];
#pragma unroll
    for (int i = 1; i < kNormThreads / 64; ++i) sum += part[i];
    const float r = (float)(1.0 / __builtin_sqrt(sum / d.hidden + d.eps));
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = 8 * (tid + kNormThreads * c), n = d.hidden - col;
      if (OUT < 0 ? n <= 0 : col >= 512 * d.mx.kq) break;
      float y[8];
      if (n > 0) {
        float w[8];
        load8<DT>(d.weight + col, n, vec, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = h[c][j] * r * w[j];
        if (n < 8) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = j < n ? y[j] : 0.f;  // (0 r is no number for an infinite r)
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.f;
      }
      if constexpr (OUT < 0) {
        store8<DT>(d.out + (int64_t)row * d.out_stride + col, n, vec, y);
      } else {
        const uint32_t byte = mx_scale_byte<OUT>(block_max_bits(y));
        uint32_t q[2];
        mx_codes<OUT>(y, byte, q);
        if (col < 128 * d.mx.kt) {
          uint32_t *to = (uint32_t *)(d.mx.codes + mx_code_at<OUT>(d.mx, row, col >> 3));
          to[0] = q[0];
          if constexpr (OUT == SPEAR_MXFP8) to[1] = q[1];
        }
        if ((tid & 3) == 0)
          d.mx.scales[mx_scale_at(d.mx, row, col >> 5)] = (uint8_t)(n > 0 ? byte : 127u);
      }
    }
  }
}

template <int DT, int OUT>
hipError_t norm_by_size(const NormDesc &d, bool vec, hipStream_t s) {
  const int cols = OUT < 0 ? d.hidden : 512 * d.mx.kq;
  const int ch = (cols + 8 * kNormThreads - 1) / (8 * kNormThreads);
  const dim3 grid(min(d.rows, 1 << 16)), block(kNormThreads);
  if (ch <= 1) rms_norm_kernel<DT, OUT, 1><<<grid, block, 0, s>>>(d, vec);
  else if (ch <= 2) rms_norm_kernel<DT, OUT, 2><<<grid, block, 0, s>>>(d, vec);
  else if (ch <= 4) rms_norm_kernel<DT, OUT, 4><<<grid, block, 0, s>>>(d, vec);
  else if (ch <= 8) rms_norm_kernel<DT, OUT, 8><<<grid, block, 0, s>>>(d, vec);
  else if (ch <= 16) rms_norm_kernel<DT, OUT, 16><<<grid, block, 0, s>>>(d, vec);
  else rms_norm_kernel<DT, OUT, 32><<<grid, block, 0, s>>>(d, vec);
  return hipGetLastError();
}

bool rows_aligned(const void *p, int64_t stride, int elem) {
  return (uintptr_t)p % 16 == 0 && stride * elem % 16 == 0;
}

template <int DT>
hipError_t quantize_as(const void *x, int64_t stride, int format, const MxDesc &out, hipStream_t s) {
  typedef typename MxType<DT>::T T;
  const bool vec = rows_aligned(x, stride, sizeof(T));
  const dim3 grid((unsigned)out.rb * out.kq), block(kConvThreads);
  if (format == SPEAR_MXFP4) mx_quantize_kernel<DT, SPEAR_MXFP4><<<grid, block, 0, s>>>((const T *)x, stride, vec, out);
  else mx_quantize_kernel<DT, SPEAR_MXFP8><<<grid, block, 0, s>>>((const T *)x, stride, vec, out);
  return hipGetLastError();
}

template <int DT>
hipError_t dequantize_as(const MxDesc &x, int format, void *out, int64_t stride, hipStream_t s) {
  typedef typename MxType<DT>::T T;
  const bool vec = rows_aligned(out, stride, sizeof(T));
  const dim3 grid((unsigned)x.rb * x.kq), block(kConvThreads);
  if (format == SPEAR_MXFP4) mx_dequantize_kernel<DT, SPEAR_MXFP4><<<grid, block, 0, s>>>(x, (T *)out, stride, vec);
  else mx_dequantize_kernel<DT, SPEAR_MXFP8><<<grid, block, 0, s>>>(x, (T *)out, stride, vec);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, int dtype, int64_t stride, int format,
                              const MxDesc &out, hipStream_t s) {
  return dtype == SPEAR_F16    ? quantize_as<0>(x, stride, format, out, s)
         : dtype == SPEAR_BF16 ? quantize_as<1>(x, stride, format, out, s)
                               : quantize_as<2>(x, stride, format, out, s);
}

hipError_t launch_mx_dequantize(const MxDesc &x, int format, void *out, int dtype, int64_t stride,
                                hipStream_t s) {
  return dtype == SPEAR_F16    ? dequantize_as<0>(x, format, out, stride, s)
         : dtype == SPEAR_BF16 ? dequantize_as<1>(x, format, out, stride, s)
                               : dequantize_as<2>(x, format, out, stride, s);
}

hipError_t launch_rms_norm(const NormDesc &d, int dtype, int out_format, hipStream_t s) {
  const bool vec = rows_aligned(d.x, d.x_stride, 2) && rows_aligned(d.weight, 0, 2) &&
                   (!d.residual || (rows_aligned(d.residual, d.residual_stride, 2) &&
                                    rows_aligned(d.residual_out, d.residual_out_stride, 2))) &&
                   (out_format >= 0 || rows_aligned(d.out, d.out_stride, 2));
  if (dtype == SPEAR_F16)
    return out_format < 0              ? norm_by_size<DT_F16, -1>(d, vec, s)
           : out_format == SPEAR_MXFP4 ? norm_by_size<DT_F16, SPEAR_MXFP4>(d, vec, s)
                                       : norm_by_size<DT_F16, SPEAR_MXFP8>(d, vec, s);
  return out_format < 0              ? norm_by_size<DT_BF16, -1>(d, vec, s)
         : out_format == SPEAR_MXFP4 ? norm_by_size<DT_BF16, SPEAR_MXFP4>(d, vec, s)
                                     : norm_by_size<DT_BF16, SPEAR_MXFP8>(d, vec, s);
}

}  // namespace spear
