// Device helpers of the microscaled formats.
#pragma once

#include "device_common.h"
#include "mx_internal.h"

namespace spear {

constexpr int kMxTop[2] = {2, 8};  // floor(log2) of the largest e2m1 and e4m3 number
constexpr uint32_t kInfBits = 0x7F800000u;

// The scale byte of a block whose largest magnitude has these bits: the power
// 2^(floor(log2 max) - top) by its exponent field (a subnormal maximum has
// field 0 and gives byte 0 like every one below 2^(top - 126)).
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t max_bits) {
  if (max_bits >= kInfBits) return 255u;
  const int e = (int)(max_bits >> 23) - kMxTop[FMT];
  return (uint32_t)(e < 0 ? 0 : e);
}

// Eight values over the scale, to nearest even and saturated: 4 bytes of e2m1
// in q[0], or 8 of e4m3.  The conversions take the scale's exponent field, so
// a byte is a scale as it stands (field 0 is 2^-127); the one to e4m3
// gives NaN above 448, so values are held to that first.
template <int FMT>
__device__ __forceinline__ void mx_codes(const float (&v)[8], uint32_t byte, uint32_t (&q)[2]) {
  if (byte == 255u) {
    q[0] = q[1] = 0u;
    return;
  }
  const float s = bitcast<float>(byte << 23);
  if constexpr (FMT == SPEAR_MXFP4) {
    uint32_t r = 0u;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
    q[0] = r;
    q[1] = 0u;
  } else {
    typedef short s16x2_t __attribute__((ext_vector_type(2)));
    const float most = __builtin_amdgcn_ldexpf(448.f, (int)byte - 127);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = __builtin_amdgcn_fmed3f(v[4 * i + j], -most, most);
      s16x2_t r = {0, 0};
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[0], c[1], s, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[2], c[3], s, true);
      q[i] = bitcast<uint32_t>(r);
    }
  }
}

// Where the eight codes of row r, columns 8 c8 .. lie (c8 = column / 8).
template <int FMT>
__device__ __forceinline__ size_t mx_code_at(const MxDesc &m, int r, int c8) {
  const int tile = c8 >> 4, c = c8 & 15;
  const size_t t = (size_t)(r >> 4) * m.kt + tile;
  if constexpr (FMT == SPEAR_MXFP4) {
    return t * 1024 + 16 * (16 * (c >> 2) + (r & 15)) + 4 * (c & 3);
  } else {
    return t * 2048 + 1024 * (c >> 3) + 16 * (16 * ((c >> 1) & 3) + (r & 15)) + 8 * (c & 1);
  }
}
// Where the scale byte of row r, block c32 (= column / 32) lies.
__device__ __forceinline__ size_t mx_scale_at(const MxDesc &m, int r, int c32) {
  const int tile = c32 >> 2;
  return (((size_t)(r >> 4) * m.kq + (tile >> 2)) * 64 + 16 * (c32 & 3) + (r & 15)) * 4 + (tile & 3);
}

// A value of the types that matrices come in, and its index of spear_dtype.
template <int DT>
struct MxType;
template <>
struct MxType<0> {
  typedef uint16_t T;
  static __device__ __forceinline__ float load(T v) { return to_f32<DT_F16>(v); }
  static __device__ __forceinline__ T store(float v) { return from_f32<DT_F16>(v); }
};
template <>
struct MxType<1> {
  typedef uint16_t T;
  static __device__ __forceinline__ float load(T v) { return to_f32<DT_BF16>(v); }
  static __device__ __forceinline__ T store(float v) { return from_f32<DT_BF16>(v); }
};
template <>
struct MxType<2> {
  typedef float T;
  static __device__ __forceinline__ float load(T v) { return v; }
  static __device__ __forceinline__ T store(float v) { return v; }
};

// Eight values from p, of which the first n count (the others are 0).  vec: p
// is 16-byte aligned.
template <int DT>
__device__ __forceinline__ void load8(const typename MxType<DT>::T *p, int n, bool vec, float (&v)[8]) {
  typedef typename MxType<DT>::T T;
  if (vec && n >= 8) {
    T t[8];
    if constexpr (sizeof(T) == 2) {
      const u16x8_t a = *(const u16x8_t *)p;
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = a[j];
    } else {
      const f32x4_t a = ((const f32x4_t *)p)[0], b = ((const f32x4_t *)p)[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = a[j], t[4 + j] = b[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = MxType<DT>::load(t[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? MxType<DT>::load(p[j]) : 0.f;
  }
}
template <int DT>
__device__ __forceinline__ void store8(typename MxType<DT>::T *p, int n, bool vec, const float (&v)[8]) {
  typedef typename MxType<DT>::T T;
  if (vec && n >= 8) {
    if constexpr (sizeof(T) == 2) {
      u16x8_t a;
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = MxType<DT>::store(v[j]);
      *(u16x8_t *)p = a;
    } else {
      ((f32x4_t *)p)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
      ((f32x4_t *)p)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = MxType<DT>::store(v[j]);
  }
}

// The bits of the largest magnitude of eight values, then over the four lanes
// of a block of 32.
__device__ __forceinline__ uint32_t block_max_bits(const float (&v)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, bitcast<uint32_t>(v[j]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
  return m;
}

}  // namespace spear
