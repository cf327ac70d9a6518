// Device helpers shared by the attention kernels.
#pragma once

#include "attn_internal.h"
#include "device_common.h"

namespace spear {

// What the query at position p of a sequence of `len` cached tokens sees:
// positions [0, sink) and [lo, p], where sink <= lo; without a window sink is
// 0 and lo is 0.
struct Seen {
  int sink, lo;
};
__device__ __forceinline__ Seen seen_by(int p, int window, int sinks) {
  Seen s{0, 0};
  if (window > 0 && p >= window) {
    s.lo = p - window + 1;
    s.sink = min(sinks, s.lo);
  }
  return s;
}

// The table column of the 16-token group i (< 2^31) of a sequence.
__device__ __forceinline__ int column_of(const AttnDesc &d, int i) {
  return d.p16_mul ? (int)(__umulhi((uint32_t)i, d.p16_mul) >> d.p16_shift) : i;
}

// Cached tokens of sequence b, within what its table row can hold.
__device__ __forceinline__ int cached_len(const AttnDesc &d, int b) {
  return max(0, min(d.kv_lens[b], d.width * d.page_size));
}

// Scores are kept times log2(e), so that the softmax is in powers of two; a
// row's maximum starts at the lowest finite number, so that any score passes it
// and one of -infinity (a hidden key) weighs exactly 0.
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.402823466e38f;

// Weights are rounded to the type for the second product.  In fp16 a row's weights
// lie around 2^kLift: around 1 its tail would be lost to what fp16 holds below 2^-14
// (of 32767 keys 17.5 below one in the exponent of e, 2^-25.2 each, nothing would
// reach the output, while l has them).  So a weight keeps fp16's precision down to
// 2^-27 of the row's largest and is at most 2^-38 of it off below.  bf16 has fp32's
// range.
template <int DT>
constexpr float kLift = DT == DT_F16 ? 13.f : 0.f;

// Every lane gets op over its own value and the values of the lanes 16 and
// 32 places away: the four lanes that hold one column of a 16-wide MFMA.
// (permlane swaps of a register with itself put both halves side by side.)
template <typename Op>
__device__ __forceinline__ float over_columns(float v, Op op) {
  const uint32_t u = bitcast<uint32_t>(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float w = op(bitcast<float>((uint32_t)a[0]), bitcast<float>((uint32_t)a[1]));
  const uint32_t x = bitcast<uint32_t>(w);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return op(bitcast<float>((uint32_t)b[0]), bitcast<float>((uint32_t)b[1]));
}
__device__ __forceinline__ float columns_max(float v) {
  return over_columns(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float columns_sum(float v) {
  return over_columns(v, [](float a, float b) { return a + b; });
}

// Inclusive prefix sum over a wave, in six adds with shifted operands.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31
  return v;
}
__device__ __forceinline__ int wave_total(int v) {
  return __builtin_amdgcn_readlane(wave_scan(v), 63);
}

__device__ __forceinline__ int wave_max(int v) {  // of non-negative values
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
  return __builtin_amdgcn_readlane(v, 63);
}

// Two fp32 values rounded to nearest even into a packed pair.
template <int DT>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  if constexpr (DT == DT_F16) {
    return bitcast<uint32_t>(f16x2_t{(_Float16)a, (_Float16)b});
  } else {
    return bitcast<uint32_t>(bf16x2_t{(__bf16)a, (__bf16)b});
  }
}

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// D = A * B + C for one 32x32x16 block.  Lane l supplies row l % 32 of A and
// column l % 32 of B, eight contraction places of half l / 32 each.  D lands
// as rows 8 * (v / 4) + 4 * (l / 32) + v % 4, column l % 32, v = 0..15.
template <int DT>
__device__ __forceinline__ f32x16_t mfma_32x32x16(u32x4_t a, u32x4_t b, f32x16_t c) {
  if constexpr (DT == DT_F16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(bitcast<f16x8_t>(a), bitcast<f16x8_t>(b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(bitcast<bf16x8_t>(a), bitcast<bf16x8_t>(b), c, 0, 0, 0);
  }
}

// op over a lane's value and that of the lane 32 places away.
template <typename Op>
__device__ __forceinline__ float over_halves(float v, Op op) {
  const uint32_t u = bitcast<uint32_t>(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return op(bitcast<float>((uint32_t)a[0]), bitcast<float>((uint32_t)a[1]));
}

// Pairs of the type's exponent bits, and one of each: a half of
// (x & kExp) + kExpOne has its top bit set where x is infinite or no number.
template <int DT>
constexpr uint32_t kExp = DT == DT_F16 ? 0x7C007C00u : 0x7F807F80u;
template <int DT>
constexpr uint32_t kExpOne = DT == DT_F16 ? 0x04000400u : 0x00800080u;
template <int DT>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return ((x & kExp<DT>) + kExpOne<DT>) & 0x80008000u;
}

// This wave's loads to LDS have landed (vmcnt(0)); no LDS read moves before it.
__device__ __forceinline__ void wait_for_lds_loads() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A buffer of `bytes` bytes at p, both wave-uniform, as its descriptor words.
__device__ __forceinline__ u32x4_t buffer_words(const void *p, int bytes) {
  const uint64_t a = (uint64_t)p;
  return u32x4_t{(uint32_t)uniform((int)a), (uint32_t)uniform((int)(a >> 32)) & 0xFFFFu,
                 (uint32_t)uniform(bytes), 0x00020000u};
}

// 16 bytes per lane from a buffer to LDS, N times: load j brings lane i's, at
// byte j step + (j odd ? odd : even), to LDS byte lds + 1024 j + 16 i (lds and
// step are wave-uniform).  Bytes past the buffer's range read as zeros.
// Written out because the compiler waits for every such load before any later
// LDS read; the caller waits (wait_for_lds_loads) before a barrier instead.  The block
// writes no register but m0; the wait states are those of a scalar register
// that a vector instruction may have written just before (the first load) and
// of m0.
template <int N>
__device__ __forceinline__ void load_to_lds(u32x4_t buffer, uint32_t lds, int even, int odd, int step) {
  static_assert(N == 2 || N == 4, "loads");
  if constexpr (N == 2) {
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 4\n\t"
        "buffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
        "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, %4 offen lds"
        :
        : "s"(lds), "v"(even), "v"(odd), "s"(buffer), "s"(step)
        : "memory", "scc", "m0");
  } else {
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 4\n\t"
        "buffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
        "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, %4 offen lds\n\t"
        "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %1, %3, %5 offen lds\n\t"
        "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, %6 offen lds"
        :
        : "s"(lds), "v"(even), "v"(odd), "s"(buffer), "s"(step), "s"(2 * step), "s"(3 * step)
        : "memory", "scc", "m0");
  }
}

// Two fp32 values published by another workgroup (as load_partials4).
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f32x2_t load_partials2(__amdgpu_buffer_rsrc_t r, int byte_off) {
  return bitcast<f32x2_t>(__builtin_amdgcn_raw_buffer_load_b64(r, byte_off, 0, 16));
}

// Read-only words at wave-uniform addresses, through the scalar cache: their
// wait (lgkmcnt) does not drain the vector loads in flight.
typedef const __attribute__((address_space(4))) int32_t *scalar_i32;
__device__ __forceinline__ int scalar_load(const int32_t *p, int64_t i) {
  return ((scalar_i32)(uintptr_t)p)[i];
}

// The header of an attention workspace: counters that every call leaves at
// zero, at the same place for calls of any size.  The data that a call
// writes before it reads it lies past it.
constexpr int kAttnCounters = 4096;
constexpr size_t kAttnDataOff = kAttnCounters * sizeof(uint32_t);
static_assert(kAttnDataOff == SPEAR_ATTN_HEADER_BYTES, "the header that the caller zeroes");

}  // namespace spear
