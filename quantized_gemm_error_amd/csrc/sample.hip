// Drawing tokens from logits.
//
// A row's tokens in descending order are its bins one after the other: bin b
// holds the tokens with 16 (max - l) / T in [b, b + 1), so a bin is e^(1/16)
// wide in weight, and the tokens past the last bin weigh less than e^-64.
// Every limit (the first k, the first whose weight passes p, the first that
// passes u) is a place in that order.  Prefix sums over the bins' counts and
// weights give the few bins in which those places can lie; the tokens of
// these bins are gathered, sorted, and the places found among them.  In rows so
// flat that they are too many, a place's bin is counted again in finer ranges.
//
// A token's weight is held relative to its bin's upper edge as a whole number
// of 2^-32, so that the sums do not depend on the order of the atomics; a row
// is counted in runs of less than 2^16 tokens, so that a bin's count and weight
// fit one 64-bit LDS atomic.
//
// Measured (MI355X): one row of 32000 fp32 logits under k and p 22 us, 64 rows of
// 131072 bf16 logits under limits of their own 45 to 93 (rows at T = 1.3 under p
// alone have more tokens in p's bin than LDS lists), 256 rows of 100003 fp32
// logits without limits 68.  The last reads its 102 MB three times, once from
// memory (16 us) and twice from the cache (counting, bound by the 64-bit
// arithmetic, 25 us; gathering, 15 us); the first is a chain of short steps of
// one workgroup, each fetched and waited for once.  Equal logits of a bin are
// sorted by comparing each with all: one row of 32000 with 500, 1000, 2000 and 3000
// tokens in p's bin takes 26, 27, 30 and 47 us where they differ, 34, 61, 161 and
// 85 where they are equal (past 2048 they are counted, not listed).
#include <algorithm>

#include "mx_device.h"

namespace spear {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 1024;  // one a thread
constexpr double kPerNat = 16.0;
constexpr int kCountShift = 48;                  // kRun tokens of at most 2^32 stay below it
constexpr int kRun = (1 << 16) - 16;             // tokens in one run: their number fits 16 bits
constexpr int kList = 2048;                      // tokens that are gathered at once
static_assert(kBins == kThreads, "a thread has one bin");

struct SampleDesc {
  const void *logits;
  int rows, vocab, parts;
  int64_t stride;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
  float *logprobs;
  uint32_t *arrived;  // [rows], 0 between calls (parts > 1)
  uint64_t *best;     // [rows][parts]: the largest logit's key and its index, inverted
  uint64_t *bins;     // [rows][parts][kBins]
};

// A float's bits in an order that rises with its value.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = bitcast<uint32_t>(l);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return bitcast<float>(key ^ (((key >> 31) - 1u) | 0x80000000u));
}

// Logits from l0 to l1: none as it stands.
struct Span {
  float l0 = __builtin_inff(), l1 = -__builtin_inff();
  __device__ __forceinline__ bool has(float l) const { return l >= l0 && l <= l1; }
  __device__ __forceinline__ void add(const Span &o) {
    l0 = fminf(l0, o.l0);
    l1 = fmaxf(l1, o.l1);
  }
};

// A row's logits in vectors of 16 bytes at their aligned places: element 0 is
// place `skew` of vector 0; vectors first .. end - 1 lie inside the row whole.
template <int DT>
struct Row {
  typedef typename MxType<DT>::T T;
  static constexpr int kVec = 16 / sizeof(T);
  const T *p;
  int n, skew, vecs, first, end;
  float floor, cap;     // what is below is never drawn, what is above counts as cap
  float top;            // the largest logit
  double scale, width;  // 16 / T, and a bin's width in logits

  __device__ Row(const SampleDesc &d, int r) {
    p = (const T *)d.logits + (int64_t)r * d.stride;
    n = d.vocab;
    skew = (int)((uintptr_t)p % 16 / sizeof(T));
    vecs = (n + skew + kVec - 1) / kVec;
    first = skew ? 1 : 0;
    end = (n + skew) / kVec;
    floor = top = -__builtin_inff();
    cap = __builtin_inff();
  }
  // A row that has logits of +infinity draws from these alone: the others
  // become -infinity, and they the largest number.
  __device__ __forceinline__ void set(float best, float T) {
    if (best == __builtin_inff()) floor = best;
    cap = 3.402823466e38f;
    top = fminf(best, cap);
    scale = kPerNat / (double)T;
    width = (double)T * (1.0 / kPerNat);
  }
  // f(values, index of the first) for the whole vectors of [v0, v1), a
  // thread's in ascending order, and f1(value, index) for those of vectors that
  // reach over the row's ends: the row's first before, its last after them.
  // Four loads are in flight a thread.  The loop stays as small as one vector's
  // code: a row passes each of its parts a few times only, and code that is
  // fetched for the first time costs more than it does (unrolled four times,
  // a gather of 131072 logits took up to 35 us).
  template <typename F, typename F1>
  __device__ __forceinline__ void visit_raw(int v0, int v1, F f, F1 f1) const {
    const int a = max(v0, first), b = min(v1, end), tid = threadIdx.x;
    if (v0 < first && tid < kVec) {
      const int i = tid - skew;
      if (i >= 0 && i < n) f1(p[i], i);
    }
    const T *at = p - skew;
    u32x4_t t[4];
    if (a < b) {
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = *(const u32x4_t *)(at + min(a + tid + j * kThreads, b - 1) * kVec);
    }
#pragma nounroll
    for (int v = a + tid; v < b; v += kThreads) {
      T e[kVec];
      __builtin_memcpy(e, &t[0], 16);
      t[0] = t[1], t[1] = t[2], t[2] = t[3];
      t[3] = *(const u32x4_t *)(at + min(v + 4 * kThreads, b - 1) * kVec);
      f(e, v * kVec - skew);
    }
    if (v1 == vecs && vecs > max(end, first) && tid < kVec) {
      const int i = (vecs - 1) * kVec - skew + tid;
      if (i < n) f1(p[i], i);
    }
  }
  // f(logit, index) for the logits of vectors [v0, v1), a thread's in ascending order.
  template <typename F>
  __device__ __forceinline__ void visit(int v0, int v1, F f) const {
    visit_raw(
        v0, v1,
        [&](const T(&e)[kVec], int i0) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) f(clean(e[i]), i0 + i);
        },
        [&](T v, int i) { f(clean(v), i); });
  }
  // f(logit, index) for the row's logits in either of two spans (as set() has
  // them), which few are: one after the other.
  template <typename F>
  __device__ __forceinline__ void visit_few(Span a, Span b, F f) const {
    if (a.l1 == cap) a.l1 = __builtin_inff();
    if (b.l1 == cap) b.l1 = __builtin_inff();
    const auto either = [&](T v) {
      const float l = MxType<DT>::load(v);
      return a.has(l) || b.has(l);
    };
    visit_raw(
        0, vecs,
        [&](const T(&e)[kVec], int i0) {
          uint32_t in = 0, w[4];
          __builtin_memcpy(w, e, 16);
#pragma unroll
          for (int i = 0; i < kVec; ++i) in |= either(e[i]) ? 1u << i : 0u;
#pragma nounroll
          for (; in; in &= in - 1) {
            const int i = __builtin_ctz(in), word = i * (int)sizeof(T) / 4;
            uint32_t bits = word & 2 ? (word & 1 ? w[3] : w[2]) : (word & 1 ? w[1] : w[0]);
            if (sizeof(T) == 2 && (i & 1)) bits >>= 16;
            T v;
            __builtin_memcpy(&v, &bits, sizeof v);
            f(clean(v), i0 + i);
          }
        },
        [&](T v, int i) {
          if (either(v)) f(clean(v), i);
        });
  }
  // NaN (of which no comparison holds) counts as -infinity.
  __device__ __forceinline__ float clean(T v) const {
    const float l = MxType<DT>::load(v);
    return fminf(l >= floor ? l : -__builtin_inff(), cap);
  }
  // 16 (top - l) / T, exactly 0 for the largest; infinite or NaN where the
  // logit is never drawn.
  __device__ __forceinline__ double depth(float l) const {
    return ((double)top - (double)l) * scale;
  }
};

__device__ __forceinline__ int bin_of(double t) { return t < (double)kBins ? (int)t : kBins; }

// The weight of a token in its bin, e^(-f / 16) with f = t - b in [0, 1), in
// units of 2^-32: six terms of the series leave 2^-33, and adding 2^52
// rounds to a whole number in the mantissa.
__device__ __forceinline__ uint64_t mass_of(double t, int b) {
  constexpr double x = -1.0 / kPerNat, unit = 0x1p32;
  const double f = t - (double)b;
  double e = unit * x * x * x * x * x / 120;
  e = __builtin_fma(e, f, unit * x * x * x * x / 24);
  e = __builtin_fma(e, f, unit * x * x * x / 6);
  e = __builtin_fma(e, f, unit * x * x / 2);
  e = __builtin_fma(e, f, unit * x);
  e = __builtin_fma(e, f, unit + 0x1p52);
  return bitcast<uint64_t>(e) & 0xFFFFFFFFFFFFFull;
}
__device__ __forceinline__ double edge_of(int b) { return exp((double)b * (-1.0 / kPerNat)); }
__device__ __forceinline__ double mass_value(uint64_t m, double edge) { return (double)m * 0x1p-32 * edge; }

struct Shared {
  uint64_t run[kBins];        // a run's bins: count and weight in one word
  int count[kBins], count_before[kBins];
  double mass[kBins], mass_before[kBins], edge[kBins];
  uint64_t list[kList];       // tokens: key << 32 | index inverted, so that they rise against the order
  int fine_count[kBins];      // finer ranges of a bin's tokens
  union {
    struct {
      uint64_t fine_mass[kBins], fine_token[kBins];
    };
    uint64_t buckets[kList];
  };
  uint64_t words[2][kWaves];  // what waves tell one another, every other time here and there
  double sums[2][kWaves];
  double found_mass, found_weight;
  uint64_t found_token;       // the row's first token until another one is found
  int found_count, listed, is_last;
};

__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  return bitcast<double>(lane_value(bitcast<uint64_t>(v), lane));
}

// Inclusive prefix sums over a wave in six adds with shifted operands, and
// the value of the lane before.
template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double v) {
  const uint64_t u = bitcast<uint64_t>(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, false);
  return bitcast<double>((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan(double v) {
  v += shifted<0x111, 0xF>(v);  // row_shr:1
  v += shifted<0x112, 0xF>(v);
  v += shifted<0x114, 0xF>(v);
  v += shifted<0x118, 0xF>(v);
  v += shifted<0x142, 0xA>(v);  // row_bcast:15
  v += shifted<0x143, 0xC>(v);  // row_bcast:31
  return v;
}
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}
__device__ __forceinline__ double lane_before(double v) { return shifted<0x138, 0xF>(v); }  // wave_shr:1

// A workgroup's threads tell one another through s.words and s.sums, whose
// halves take turns: a half is written again only after the barrier of the
// exchange between, which every thread reaches after it has read.
struct Turn {
  Shared &s;
  int half = 0;

  // Sums before each thread's values, in thread order, and the totals.  (A
  // sum before is the inclusive one of the thread before: they never fall.)
  __device__ __forceinline__ void scan(int c, double m, int &c_before, double &m_before, int &c_all, double &m_all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int cs = wave_scan(c);
    const double ms = wave_scan(m);
    if (lane == 63) s.words[half][wave] = (uint64_t)cs, s.sums[half][wave] = ms;
    __syncthreads();
    const int ct = wave_scan(lane < kWaves ? (int)s.words[half][lane] : 0);
    const double mt = wave_scan(lane < kWaves ? s.sums[half][lane] : 0.0);
    c_before = cs - c + (wave ? __builtin_amdgcn_readlane(ct, uniform_wave() - 1) : 0);
    m_before = lane_before(ms) + (wave ? lane_value(mt, uniform_wave() - 1) : 0.0);
    c_all = __builtin_amdgcn_readlane(ct, kWaves - 1);
    m_all = lane_value(mt, kWaves - 1);
    half ^= 1;
  }
  // The first and the last thread for which `pass` holds, -1 for none.
  __device__ __forceinline__ int first(bool pass) {
    const uint64_t x = gather(pass), some = __ballot(x != 0);
    if (!some) return -1;
    const int w = __builtin_ctzll(some);
    return 64 * w + __builtin_ctzll(lane_value(x, w));
  }
  __device__ __forceinline__ int last(bool pass) {
    const uint64_t x = gather(pass), some = __ballot(x != 0);
    if (!some) return -1;
    const int w = 63 - __builtin_clzll(some);
    return 64 * w + 63 - __builtin_clzll(lane_value(x, w));
  }

 private:
  __device__ __forceinline__ uint64_t gather(bool pass) {
    const int lane = threadIdx.x & 63;
    const uint64_t mine = __ballot(pass);
    if (lane == 0) s.words[half][threadIdx.x >> 6] = mine;
    __syncthreads();
    const uint64_t x = lane < kWaves ? s.words[half][lane] : 0;
    half ^= 1;
    return x;
  }
  static __device__ __forceinline__ int uniform_wave() {
    return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  }
};

// A token of the order by its number there (from 1), with the weight up to it.
struct Place {
  int count;
  double mass, weight;
  uint64_t token;
};

enum Want { kCount, kMassAtLeast, kMassAbove };

__device__ __forceinline__ bool passes(Want want, double target, int count, double mass) {
  return want == kCount ? (double)count >= target : want == kMassAtLeast ? mass >= target : mass > target;
}

// The first bin with tokens whose sums pass; `end`, the last one with tokens, if none does.
__device__ __forceinline__ int first_bin(Shared &s, Turn &turn, Want want, double target, int end) {
  const int b = threadIdx.x, c = s.count[b];
  const int first = turn.first(c && passes(want, target, s.count_before[b] + c, s.mass_before[b] + s.mass[b]));
  return first < 0 ? end : first;
}

// (adding 0 makes one logit of 0 and -0)
__device__ __forceinline__ uint64_t token_of(float l, int i) { return (uint64_t)key_of(l + 0.f) << 32 | (uint32_t)~i; }
__device__ __forceinline__ float logit_of(uint64_t token) { return value_of((uint32_t)(token >> 32)); }

// Those of bins b0 .. b1 and perhaps a few more: all l whose depth() falls
// into them.  A depth is 16 (top - l) / T to 2^-51 of itself (a difference, 16 / T
// and a product, each rounded to 2^-53), so an l that is small beside top may
// lie on either side of a border by as much: around a border at 0 this is far
// more than a step of l's type.  2^-50 of |top| and of the depth's logits cover
// it and what is rounded here (b width is exact); the step of one number after
// that covers the rounding to fp32.  (An infinite T leaves hi NaN and top in l1.)
template <int DT>
__device__ __forceinline__ Span logits_of_bins(const Row<DT> &row, int b0, int b1) {
  Span s;
  const double top = (double)row.top, past = (double)(b1 + 1) * row.width;
  const double margin = 0x1p-50 * (__builtin_fabs(top) + past);
  const float lo = (float)(top - past - margin);
  s.l0 = lo > -__builtin_inff() ? value_of(key_of(lo) - 1u) : -__builtin_inff();
  s.l1 = row.top;
  if (b0) {
    const float hi = (float)(top - (double)b0 * row.width + margin);
    const float up = value_of(key_of(hi) + 1u);
    if (up < s.l1) s.l1 = up;
  }
  return s;
}

// The first token of a bin whose sums pass (the bin's last one if none does):
// its tokens are counted in 1024 equal ranges of their words, then those of
// the range that passes in as many again, until that holds one; from the row
// until few enough are left for LDS.
template <int DT>
__device__ __forceinline__ Place find_place(Shared &s, Turn &turn, const Row<DT> &row, Want want, double target, int bin) {
  const int tid = threadIdx.x;
  const double edge = s.edge[bin];
  Span span = logits_of_bins(row, bin, bin);
  uint64_t low = (uint64_t)key_of(span.l0) << 32, high = (uint64_t)key_of(span.l1) << 32 | 0xFFFFFFFFull;
  Place at{};
  at.token = s.found_token;
  at.weight = 1.0;
  at.count = s.count_before[bin];
  at.mass = s.mass_before[bin];
  int listed = -1;  // tokens left, in s.list; none there yet
  for (;;) {
    if (low >> 32 == high >> 32) low = max(low, (low >> 32) << 32 | (uint32_t)~(row.n - 1));
    const uint64_t width = high - low;
    const int shift = max(0, 64 - (width ? __builtin_clzll(width) : 63) - 10);
    __syncthreads();
    s.fine_count[tid] = 0;
    s.fine_mass[tid] = 0;
    __syncthreads();
    auto count = [&](uint64_t token) {
      if (token < low || token > high) return;
      const double t = row.depth(logit_of(token));
      if (bin_of(t) != bin) return;
      const int c = (int)((high - token) >> shift);
      atomicAdd(&s.fine_count[c], 1);
      atomicAdd((unsigned long long *)&s.fine_mass[c], (unsigned long long)mass_of(t, bin));
      s.fine_token[c] = token;
    };
    if (listed < 0) {
      row.visit_few(span, Span(), [&](float l, int i) { count(token_of(l, i)); });
    } else {
      for (int j = tid; j < listed; j += kThreads) count(s.list[j]);
    }
    __syncthreads();
    const int c = s.fine_count[tid];
    const double m = mass_value(s.fine_mass[tid], edge);
    int c0, c_all;
    double m0, m_all;
    turn.scan(c, m, c0, m0, c_all, m_all);
    int b = turn.first(c && passes(want, target, at.count + c0 + c, at.mass + (m0 + m)));
    if (b < 0) b = turn.last(c != 0);
    if (b < 0) return at;  // (no token of the bin, which has one: the row's first)
    // the sums before range b, from the thread that has it (s.sums was last
    // read before the barrier of first())
    if (tid == b) s.sums[0][0] = (double)c0, s.sums[1][0] = m0;
    __syncthreads();
    at.count += (int)s.sums[0][0];
    at.mass += s.sums[1][0];
    if (s.fine_count[b] == 1) {
      at.token = s.fine_token[b];
      at.weight = mass_value(s.fine_mass[b], edge);
      at.count += 1;
      at.mass += at.weight;
      __syncthreads();
      return at;
    }
    high -= (uint64_t)b << shift;
    const uint64_t rest = (1ull << shift) - 1;
    low = high - low > rest ? high - rest : low;
    if (listed < 0 && s.fine_count[b] <= kList) {
      listed = s.fine_count[b];
      if (tid == 0) s.listed = 0;
      span.l0 = logit_of(low);
      span.l1 = logit_of(high);
      __syncthreads();
      row.visit_few(span, Span(), [&](float l, int i) {
        const uint64_t token = token_of(l, i);
        if (token < low || token > high || bin_of(row.depth(l)) != bin) return;
        const int j = atomicAdd(&s.listed, 1);
        if (j < kList) s.list[j] = token;
      });
    }
  }
}

// The bins of vectors [v0, v1) of the row, added up over runs of kRun tokens:
// a thread's own bin; or, for a part of a row, its only run in s.run.
template <int DT>
__device__ __forceinline__ void count_bins(Shared &s, const Row<DT> &row, int v0, int v1, bool part, int &count,
                                           uint64_t &mass) {
  const int tid = threadIdx.x;
  constexpr int kStep = kRun / Row<DT>::kVec;
  for (int a = v0; a < v1; a += kStep) {
    s.run[tid] = 0;
    __syncthreads();
    row.visit(a, min(v1, a + kStep), [&](float l, int) {
      const double t = row.depth(l);
      const int b = bin_of(t);
      if (b < kBins)
        atomicAdd((unsigned long long *)&s.run[b], (unsigned long long)(mass_of(t, b) + (1ull << kCountShift)));
    });
    __syncthreads();
    if (part) return;
    count += (int)(s.run[tid] >> kCountShift);
    mass += s.run[tid] & ((1ull << kCountShift) - 1);
  }
}

struct Limits {
  float u, T, p, m;
  int k;
};

__device__ __forceinline__ void answer(const SampleDesc &d, int r, uint64_t token, double weight, double kept) {
  d.tokens[r] = (int)~(uint32_t)token;
  if (d.logprobs) d.logprobs[r] = (float)log(weight / kept);
}

// The row's last token kept and the token drawn, from its bins: a thread's own
// bin has my_count tokens of my_mass.
template <int DT>
__device__ __forceinline__ void finish(Shared &s, const SampleDesc &d, const Row<DT> &row, int r, const Limits &lim, int my_count,
                       uint64_t my_mass) {
  const int tid = threadIdx.x, lane = tid & 63;
  Turn turn{s};
  int n_all;
  double z_all;
  {
    const double mass = mass_value(my_mass, s.edge[tid]);
    int c0;
    double m0;
    turn.scan(my_count, mass, c0, m0, n_all, z_all);
    s.count[tid] = my_count;
    s.mass[tid] = mass;
    s.count_before[tid] = c0;
    s.mass_before[tid] = m0;
  }
  const double u = lim.u > 0.f ? (double)lim.u : 0.0, p = (double)lim.p;
  const bool to_end = lim.u >= 1.f;  // the last token kept
  const int k = lim.k;
  bool by_k = k > 0 && k < n_all, by_p = lim.p < 1.f;
  // the depth within which weights are at least m
  const double deep = lim.m > 0.f ? -kPerNat * log((double)fminf(lim.m, 1.f)) : (double)kBins;
  bool by_m = deep < (double)kBins;
  const int bm = by_m ? (int)deep : 0;
  const int end = turn.last(my_count != 0);  // (and the arrays above are written)

  // The bins in which the last token kept can lie, [lo, hi], and what is kept
  // at least and at most: a limit on weights is known to the bins of the
  // limit before it (and to the sums' rounding).  `wanted`: all bins in which
  // a place is looked for.
  constexpr double kLess = 1.0 - 0x1p-40, kMore = 1.0 + 0x1p-40;
  int lo = end, hi = end;
  double z_lo = z_all, z_hi = z_all;
  bool wanted = false;
  Span limits, drawn;  // of logits: the bins of k, p and m, and of the draw
  if (by_k) {
    lo = hi = first_bin(s, turn, kCount, (double)k, end);
    wanted = tid == hi;
    limits.add(logits_of_bins(row, hi, hi));
    z_lo = s.mass_before[hi];
    z_hi = z_lo + s.mass[hi];
  }
#pragma nounroll
  for (int step = by_p ? 0 : 1; step < 2; ++step) {  // p, then the draw
    const double f = step ? u : p;
    const Want want = step ? kMassAbove : kMassAtLeast;
    if (step && bm > hi) by_m = false;  // the limits before end the row sooner
    if (step && by_m) {
      if (bm < lo) {  // and here later, wherever they lie in their bins
        by_k = by_p = wanted = false;
        limits = Span();
      }
      wanted |= tid == bm;
      limits.add(logits_of_bins(row, bm, bm));
      lo = min(lo, bm);
      hi = min(hi, bm);
      z_lo = min(z_lo, s.mass_before[bm]);
      z_hi = min(z_hi, s.mass_before[bm] + s.mass[bm]);
    }
    int a = lo, b = hi;
    if (step && to_end) {  // (and where m's bin has no token that is kept, in the last bin before)
      const int before = by_m ? turn.last(my_count != 0 && tid < bm) : -1;
      if (before >= 0) a = min(a, before);
    } else {
      a = first_bin(s, turn, want, f * z_lo * kLess, end);
      b = min(first_bin(s, turn, want, f * z_hi * kMore, end), hi);
    }
    wanted |= tid >= a && tid <= b;
    const Span span = logits_of_bins(row, a, b);
    if (step) drawn = span;
    else limits.add(span);
    if (!step) {
      lo = min(lo, a);
      hi = min(hi, b);
      z_lo = s.mass_before[lo];
      z_hi = s.mass_before[hi] + s.mass[hi];
    }
  }
  wanted = wanted && my_count;
  int place, n;
  double none;
  turn.scan(wanted ? my_count : 0, 0.0, place, none, n, none);
  if (n <= kList) {
    // gather: logits of the two spans, then by their bins
    uint32_t *bits = (uint32_t *)s.run;  // a bit for each bin
    {
      const uint64_t who = __ballot(wanted);
      if (lane == 0) s.run[tid >> 6] = who;
      if (tid == 0) s.listed = 0;
    }
    s.fine_count[tid] = 0;
    __syncthreads();
    if (wanted) s.count[tid] = place;  // where the bin's tokens begin in the sorted list
    auto list = [&](float l, int i) {
      const int b = bin_of(row.depth(l));
      if (b < kBins && (bits[b >> 5] >> (b & 31) & 1u)) {
        const int j = atomicAdd(&s.listed, 1);
        if (j < kList) s.list[j] = token_of(l, i);
      }
    };
    row.visit_few(limits, drawn, list);
    __syncthreads();
    const int half = n > kBins;  // (ranges in pairs)
    n = min(n, s.listed);        // (as many as were counted)
    // sort: a bin's tokens spread over as many ranges as they are by their
    // depth in it, then by comparing with the others of the same range
    uint64_t e[2];
    int range[2], slot[2];
    bool has[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = tid + kThreads * i;
      has[i] = j < n;
      e[i] = has[i] ? s.list[j] : 0;
      range[i] = 0;
      if (has[i]) {
        const double t = row.depth(logit_of(e[i]));
        const int b = bin_of(t), c = (b + 1 < kBins ? s.count_before[b + 1] : n_all) - s.count_before[b];
        range[i] = (s.count[b] + min((int)((t - b) * c), c - 1)) >> half;
      }
      slot[i] = has[i] ? atomicAdd(&s.fine_count[range[i]], 1) : 0;
    }
    __syncthreads();
    int *start = (int *)s.run;  // (the bits have been read)
    {
      int c0, c_all;
      turn.scan(s.fine_count[tid], 0.0, c0, none, c_all, none);
      start[tid] = c0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      slot[i] += start[range[i]];
      if (has[i]) s.buckets[slot[i]] = e[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int from = start[range[i]], to = has[i] ? from + s.fine_count[range[i]] : from;
      int at = from;
#pragma unroll 8
      for (int j = from; j < to; ++j) at += s.buckets[j] > e[i];
      if (has[i]) s.list[at] = e[i];
    }
    __syncthreads();
    // two neighbours a thread: their numbers in the order, their weights and the sums up to them
    double t[2], w[2], upto[2];
    int bin[2], first[2], count[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = 2 * tid + i;
      has[i] = j < n;
      e[i] = has[i] ? s.list[j] : 0;
      t[i] = has[i] ? row.depth(logit_of(e[i])) : 0.0;
      bin[i] = bin_of(t[i]);
      first[i] = has[i] ? s.count[bin[i]] : 0;
      count[i] = s.count_before[bin[i]] + j - first[i] + 1;
      w[i] = has[i] ? mass_value(mass_of(t[i], bin[i]), s.edge[bin[i]]) : 0.0;
    }
    double sum, *sums = (double *)s.buckets;
    int c0, c_all;
    turn.scan(0, w[0] + w[1], c0, sum, c_all, none);
    sums[2 * tid] = sum;
    sums[2 * tid + 1] = sum + w[0];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      upto[i] = s.mass_before[bin[i]] + ((i ? sum + w[0] : sum) - sums[first[i]]) + w[i];
    int kept_count = n_all;
    double kept = z_all;
    // the first or last thread with a token for which `pass` holds tells it
    auto tell = [&](bool is_first, bool a, bool b) {
      a = a && has[0], b = b && has[1];
      const int j = is_first ? turn.first(a || b) : turn.last(a || b);
      if (tid == j) {
        const int i = is_first ? !a : b;
        s.found_count = count[i];
        s.found_mass = upto[i];
        s.found_weight = w[i];
        s.found_token = e[i];
      }
      __syncthreads();
      return j >= 0;
    };
    auto keep = [&](int c, double m) {
      if (c < kept_count) kept_count = c, kept = m;
    };
    if (by_k && tell(true, count[0] >= k, count[1] >= k)) keep(k, s.found_mass);
    if (by_p && tell(true, upto[0] >= p * kept, upto[1] >= p * kept)) keep(s.found_count, s.found_mass);
    if (by_m) {
      // deep enough in the bins around the limit; none: what lies before them
      const bool any = tell(false, bin[0] >= bm && t[0] <= deep, bin[1] >= bm && t[1] <= deep);
      keep(any ? s.found_count : s.count_before[bm], any ? s.found_mass : s.mass_before[bm]);
    }
    if (to_end) tell(true, count[0] >= kept_count, count[1] >= kept_count);
    else if (!tell(true, upto[0] > u * kept, upto[1] > u * kept)) tell(false, true, true);
    if (tid == 0) answer(d, r, s.found_token, s.found_weight, kept);
    return;
  }
  Place at{n_all, z_all, s.found_weight, s.found_token};
  int kept_count = n_all;
  double kept = z_all;
#pragma nounroll
  for (int step = 0; step < 4; ++step) {
    double target;
    Want want = kCount;
    if (step == 0) {
      if (!by_k) continue;
      target = (double)k;
    } else if (step == 1) {
      if (!by_p) continue;
      target = p * kept;
      want = kMassAtLeast;
    } else if (step == 2) {
      if (!by_m) continue;
      int c = 0, c0;
      row.visit(0, row.vecs, [&](float l, int) { c += row.depth(l) <= deep; });
      turn.scan(c, 0.0, c0, none, c, none);
      target = (double)c;
    } else if (to_end) {
      target = (double)kept_count;
    } else {
      target = u * kept;
      want = kMassAbove;
    }
    if (step < 3 && want == kCount && target >= (double)kept_count) continue;
    at = find_place(s, turn, row, want, target, first_bin(s, turn, want, target, end));
    if (step < 3 && at.count < kept_count) kept_count = at.count, kept = at.mass;
  }
  if (tid == 0) answer(d, r, at.token, at.weight, kept);
}

__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

// The largest logit of vectors [v0, v1) and the lowest index that has it.
template <int DT>
__device__ __forceinline__ uint64_t best_of(uint64_t *wave_best, const Row<DT> &row, int v0, int v1) {
  float top = -__builtin_inff();
  int at = 0;
  row.visit(v0, v1, [&](float l, int i) {
    at = l > top ? i : at;
    top = l > top ? l : top;
  });
  uint64_t best = token_of(top, at);
#pragma unroll
  for (int o = 32; o; o >>= 1) best = larger(best, __shfl_xor((unsigned long long)best, o));
  if ((threadIdx.x & 63) == 0) wave_best[threadIdx.x >> 6] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) best = larger(best, wave_best[w]);
  return best;
}

// The vectors of a part: even shares.
__device__ __forceinline__ int part_begin(int vecs, int part, int parts) {
  return (int)((int64_t)vecs * part / parts);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void best_kernel(SampleDesc d) {
  __shared__ uint64_t wave_best[kWaves];
  const int r = blockIdx.y, part = blockIdx.x;
  const Row<DT> row(d, r);
  const uint64_t best = best_of(wave_best, row, part_begin(row.vecs, part, d.parts), part_begin(row.vecs, part + 1, d.parts));
  if (threadIdx.x == 0) d.best[r * d.parts + part] = best;
}

// A workgroup a row, or one for each of its parts, of which the last to
// arrive goes on with all their bins.
template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleDesc d) {
  __shared__ Shared s;
  const int r = blockIdx.y, part = blockIdx.x, tid = threadIdx.x;
  Row<DT> row(d, r);
  const Limits lim{d.u[r], d.temperature ? d.temperature[r] : 1.f, d.top_p ? d.top_p[r] : 1.f,
                   d.min_p ? d.min_p[r] : 0.f, d.top_k ? d.top_k[r] : 0};
  s.edge[tid] = edge_of(tid);
  if (tid == 0) s.found_weight = 1.0;
  uint64_t best = 0;
  if (d.best) {
    const int i = tid & 15;
    best = i < d.parts ? d.best[r * d.parts + i] : 0;
#pragma unroll
    for (int o = 8; o; o >>= 1) best = larger(best, __shfl_xor((unsigned long long)best, o));
  } else {
    best = best_of(s.words[0], row, 0, row.vecs);
  }
  const float top = logit_of(best);
  const bool none = top == -__builtin_inff();
  if (none || !(lim.T > 0.f) || lim.k == 1) {
    if (tid == 0 && part == 0) {
      d.tokens[r] = none ? -1 : (int)~(uint32_t)best;
      if (d.logprobs) d.logprobs[r] = none ? -__builtin_inff() : 0.f;
    }
    return;
  }
  row.set(top, lim.T);
  if (tid == 0) s.found_token = best;
  int count = 0;
  uint64_t mass = 0;
  if (d.parts > 1) {
    count_bins(s, row, part_begin(row.vecs, part, d.parts), part_begin(row.vecs, part + 1, d.parts), true, count, mass);
    uint64_t *all = d.bins + (size_t)r * d.parts * kBins + tid;
    __hip_atomic_store(&all[(size_t)part * kBins], s.run[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    publish_wait();
    __syncthreads();
    if (tid == 0)
      s.is_last = __hip_atomic_fetch_add(&d.arrived[r], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                  (uint32_t)d.parts - 1;
    __syncthreads();
    if (!s.is_last) return;
    if (tid == 0) __hip_atomic_store(&d.arrived[r], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll 8
    for (int i = 0; i < d.parts; ++i) {
      const uint64_t v = __hip_atomic_load(&all[(size_t)i * kBins], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      count += (int)(v >> kCountShift);
      mass += v & ((1ull << kCountShift) - 1);
    }
  } else {
    count_bins(s, row, 0, row.vecs, false, count, mass);
  }
  finish(s, d, row, r, lim, count, mass);
}

// Parts a row is cut into: one for each CU that would be idle otherwise, of
// 2048 tokens at least, and at most 8; more where one would be longer than a
// run.
int parts_of(int rows, int vocab) {
  const int idle = (256 + rows - 1) / rows, fine = (vocab + 2047) / 2048;
  if (idle < 2 || fine < 2) return 1;
  // (a run less what a row's skew and the parts' rounding to vectors may add)
  const int runs = (vocab + kRun - 33) / (kRun - 32);
  return std::max(std::min({idle, fine, 8}), runs);
}

// Whether the row's largest logit is found in a launch of its own: a
// workgroup of each part reads the whole row for it otherwise.
bool best_apart(int parts, int vocab, int size) { return parts > 1 && (int64_t)vocab * size > (128 << 10); }

template <int DT>
hipError_t launch_as(const SampleDesc &d, hipStream_t s) {
  // (the grid's second extent holds 65535 rows)
  for (int r0 = 0; r0 < d.rows; r0 += 65535) {
    SampleDesc e = d;
    e.rows = min(d.rows - r0, 65535);
    typedef typename MxType<DT>::T T;
    e.logits = (const T *)d.logits + (int64_t)r0 * d.stride;
    e.u += r0;
    if (e.temperature) e.temperature += r0;
    if (e.top_k) e.top_k += r0;
    if (e.top_p) e.top_p += r0;
    if (e.min_p) e.min_p += r0;
    e.tokens += r0;
    if (e.logprobs) e.logprobs += r0;
    const dim3 grid(e.parts, e.rows), block(kThreads);
    if (e.best) best_kernel<DT><<<grid, block, 0, s>>>(e);
    sample_kernel<DT><<<grid, block, 0, s>>>(e);
  }
  return hipGetLastError();
}

}  // namespace

// Of all calls of at most these sizes: fewer rows have more parts.
size_t sample_workspace(int rows, int vocab) {
  size_t most = 0;
  for (int r = 1; r <= min(rows, 255); ++r) most = std::max(most, (size_t)r * parts_of(r, vocab));
  return SPEAR_SAMPLE_HEADER_BYTES + (most * 8 + 255) / 256 * 256 + most * kBins * 8;
}

hipError_t launch_sample(const spear_sample_args_t &a, void *workspace, hipStream_t s) {
  SampleDesc d{a.logits, a.rows, a.vocab, parts_of(a.rows, a.vocab), a.stride, a.u, a.temperature, a.top_p,
               a.min_p, a.top_k, a.tokens, a.logprobs, nullptr, nullptr, nullptr};
  const size_t n = (size_t)a.rows * d.parts;
  d.arrived = (uint32_t *)workspace;
  d.bins = (uint64_t *)((char *)workspace + SPEAR_SAMPLE_HEADER_BYTES);
  const bool apart = best_apart(d.parts, a.vocab, a.dtype == SPEAR_F32 ? 4 : 2);
  d.best = apart ? d.bins + n * kBins : nullptr;
  return a.dtype == SPEAR_F16 ? launch_as<0>(d, s) : a.dtype == SPEAR_BF16 ? launch_as<1>(d, s) : launch_as<2>(d, s);
}

}  // namespace spear
