// Host-side interface between the C ABI of microscaled matrices and sampling
// and their kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/spear_sample.h"
#include "internal.h"

namespace spear {

// A microscaled matrix: kt tiles of 128 columns, kq groups of 4 tiles.
struct MxDesc {
  uint8_t *codes, *scales;
  int rows, cols, rb, kt, kq;
};
inline MxDesc mx_desc(const spear_mx_t &m) {
  return {(uint8_t *)m.codes, (uint8_t *)m.scales, m.rows, m.cols, (m.rows + 15) / 16,
          (m.cols + 127) / 128, (m.cols + 511) / 512};
}

hipError_t launch_mx_quantize(const void *x, int dtype, int64_t stride, int format,
                              const MxDesc &out, hipStream_t s);
hipError_t launch_mx_dequantize(const MxDesc &x, int format, void *out, int dtype, int64_t stride,
                                hipStream_t s);

struct NormDesc {
  int rows, hidden;
  const uint16_t *x, *residual, *weight;
  int64_t x_stride, residual_stride, residual_out_stride, out_stride;
  uint16_t *residual_out, *out;
  MxDesc mx;
  double eps;
};
hipError_t launch_rms_norm(const NormDesc &d, int dtype, int out_format, hipStream_t s);

struct MxLinearDesc {
  MxDesc w, x;
  int x_format;
  void *y;
  int y_dtype;
  int64_t y_stride;
  // Tokens that the product quantizes itself, or null (then x has them):
  // 16-byte aligned rows, mx_linear_quantizes.
  const uint16_t *x16;
  int x16_dtype;
  int64_t x16_stride;
  bool y_vec, y_vec16;  // outputs from a fourth one on are aligned for stores of four, for 16 bytes
};
hipError_t launch_mx_gemm(const MxLinearDesc &d, hipStream_t s);
bool mx_linear_quantizes(int tokens, int cols);
hipError_t launch_mx_linear(const MxLinearDesc &d, hipStream_t s);

size_t sample_workspace(int rows, int vocab);
hipError_t launch_sample(const spear_sample_args_t &a, void *workspace, hipStream_t s);

}  // namespace spear
