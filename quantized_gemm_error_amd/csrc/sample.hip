// Drawing tokens from logits.
//
// A row's tokens in descending order are its bins one after the other: bin b
// holds the tokens with 32 (max - l) / T in [b, b + 1), so a bin is e^(1/32)
// wide in weight, and the tokens past the last bin weigh less than e^-64.
// Every limit (the first k, the first whose weight passes p, the first that
// passes u) is a place in that order: the bin comes from a prefix sum over the
// bins' counts and weights, the place inside it from a radix descent over the
// logits' bits, and among equal logits from the index.
//
// A token's weight is held relative to its bin's upper edge as a whole number
// of 2^-45, so that the LDS sums do not depend on the order of the atomics.
#include "mx_device.h"

namespace spear {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048, kBinsPerThread = kBins / kThreads;
constexpr float kPerNat = 32.f;
constexpr int kMassBits = 45;  // (a row's 2^18 tokens of at most 1 stay below 2^63)

struct SampleDesc {
  const void *logits;
  int rows, vocab;
  int64_t stride;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
  float *logprobs;
};

// A float's bits in an order that rises with its value.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = bitcast<uint32_t>(l);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return bitcast<float>(key ^ ((key >> 31) - 1u | 0x80000000u));
}

// A row's logits, a number for all, and where they lie in the order.
template <int DT>
struct Row {
  const typename MxType<DT>::T *p;
  int n;
  float top;     // the largest logit
  double scale;  // 32 / T
  __device__ __forceinline__ float at(int i) const {
    const float l = MxType<DT>::load(p[i]);
    return l != l ? -__builtin_inff() : l + 0.f;  // (-0 and 0 are one logit)
  }
  // 32 (top - l) / T; infinite where the logit is never drawn.
  __device__ __forceinline__ double depth(float l) const {
    if (l == top) return 0.0;
    if (l == -__builtin_inff() || top == __builtin_inff()) return (double)__builtin_inff();
    return ((double)top - (double)l) * scale;
  }
};

__device__ __forceinline__ int bin_of(double t) { return t < (double)kBins ? (int)t : kBins; }

// The weight of a token in its bin, e^-(t - b) / 32, in units of 2^-45.
__device__ __forceinline__ uint64_t mass_of(double t, int b) {
  return (uint64_t)__builtin_rint(exp(((double)b - t) * (1.0 / kPerNat)) * (double)(1ull << kMassBits));
}
__device__ __forceinline__ double edge_of(int b) { return exp((double)b * (-1.0 / kPerNat)); }
__device__ __forceinline__ double mass_value(uint64_t m, double edge) {
  return (double)m * (1.0 / (double)(1ull << kMassBits)) * edge;
}

struct Shared {
  uint32_t count[kBins];
  uint64_t mass[kBins];
  int count_before[kBins];     // of the bins before, then prefix sums of a descent
  double mass_before[kBins];
  double wave_mass[kWaves];
  int wave_count[kWaves];
  uint64_t best[kWaves];
  int found;
  int total_count;
  double total_mass;
};

// count_before and mass_before of the first `bins` bins, weights times
// edge(b); every thread has n / kThreads neighbouring bins.
template <typename Edge>
__device__ void scan_bins(Shared &s, int bins, Edge edge) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int c[kBinsPerThread], csum = 0;
  double m[kBinsPerThread], msum = 0.0;
#pragma unroll
  for (int i = 0; i < kBinsPerThread; ++i) {
    const int b = kBinsPerThread * tid + i;
    c[i] = b < bins ? (int)s.count[b] : 0;
    m[i] = b < bins ? mass_value(s.mass[b], edge(b)) : 0.0;
    csum += c[i];
    msum += m[i];
  }
  int cs = csum;
  double ms = msum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int cu = __shfl_up(cs, o);
    const double mu = __shfl_up(ms, o);
    if (lane >= o) cs += cu, ms += mu;
  }
  if (lane == 63) s.wave_count[wave] = cs, s.wave_mass[wave] = ms;
  __syncthreads();
  int c0 = 0;
  double m0 = 0.0;
  for (int w = 0; w < wave; ++w) c0 += s.wave_count[w], m0 += s.wave_mass[w];
  c0 += cs - csum;
  // (the exclusive sum as the inclusive one of the thread before: monotone)
  double before = __shfl_up(ms, 1);
  m0 += lane ? before : 0.0;
#pragma unroll
  for (int i = 0; i < kBinsPerThread; ++i) {
    const int b = kBinsPerThread * tid + i;
    if (b < bins) s.count_before[b] = c0, s.mass_before[b] = m0;
    c0 += c[i];
    m0 += m[i];
  }
  if (tid == kThreads - 1) s.total_count = c0, s.total_mass = m0;
  __syncthreads();
}

// The place of a token in the order, and the sums up to it, itself included.
struct Place {
  uint32_t key;
  int index;
  int count;
  double mass, weight;
};

enum Want { kCount, kMassAtLeast, kMassAbove };

// The smallest bin for which `pass` holds, or the last bin that is not empty.
template <typename Pass>
__device__ int first_bin(Shared &s, int bins, Pass pass) {
  const int tid = threadIdx.x;
  if (tid == 0) s.found = kBins;
  __syncthreads();
  int first = kBins, last = -1;
#pragma unroll
  for (int i = kBinsPerThread - 1; i >= 0; --i) {
    const int b = kBinsPerThread * tid + i;
    if (b < bins && s.count[b]) {
      if (pass(b)) first = b;
      last = max(last, b);
    }
  }
  if (first < kBins) atomicMin(&s.found, first);
  __syncthreads();
  int found = s.found;
  __syncthreads();
  if (found < kBins) return found;
  if (tid == 0) s.found = -1;
  __syncthreads();
  if (last >= 0) atomicMax(&s.found, last);
  __syncthreads();
  found = s.found;
  __syncthreads();
  return found;
}

// The first token of the order whose sums pass: whose count reaches `target`
// or whose weight reaches or passes it; the row's last token in the bins if
// none does.  The bins' sums are those of the whole row and are taken again
// at the end.
template <int DT>
__device__ Place find_place(Shared &s, const Row<DT> &row, Want want, double target, int bin, int count0,
                            double mass0) {
  const int tid = threadIdx.x;
  const double edge = edge_of(bin);
  uint32_t prefix = 0;
  Place at{};
  at.count = count0;
  at.mass = mass0;
  for (int level = 3; level >= 0; --level) {
    const int shift = 8 * level;
    __syncthreads();
    for (int i = tid; i < 256; i += kThreads) s.count[i] = 0u, s.mass[i] = 0ull;
    __syncthreads();
    for (int i = tid; i < row.n; i += kThreads) {
      const float l = row.at(i);
      const uint32_t key = key_of(l);
      if (level < 3 && (key >> (shift + 8)) != prefix) continue;
      const double t = row.depth(l);
      if (bin_of(t) != bin) continue;
      const int b = 255 - (int)((key >> shift) & 255u);
      atomicAdd(&s.count[b], 1u);
      atomicAdd((unsigned long long *)&s.mass[b], (unsigned long long)mass_of(t, bin));
    }
    __syncthreads();
    scan_bins(s, 256, [&](int) { return edge; });
    const int c0 = at.count;
    const double m0 = at.mass;
    const int b = first_bin(s, 256, [&](int b) {
      if (want == kCount) return (double)(c0 + s.count_before[b] + (int)s.count[b]) >= target;
      const double m = m0 + (s.mass_before[b] + mass_value(s.mass[b], edge));
      return want == kMassAtLeast ? m >= target : m > target;
    });
    at.count = c0 + s.count_before[b];
    at.mass = m0 + s.mass_before[b];
    prefix = prefix << 8 | (uint32_t)(255 - b);
  }
  // all that is left are equal logits: the n-th of them by index
  const int equal = (int)s.count[255 - (int)(prefix & 255u)];
  at.key = prefix;
  const double t = row.depth(value_of(prefix));
  at.weight = mass_value(mass_of(t, bin), edge);
  int nth = equal;
  if (want == kCount) {
    nth = (int)target - at.count;
  } else {
    // the least n with mass + n weight passing
    int lo = 1, hi = equal;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      const double m = at.mass + mid * at.weight;
      if (want == kMassAtLeast ? m >= target : m > target) hi = mid;
      else lo = mid + 1;
    }
    nth = lo;
  }
  nth = max(1, min(nth, equal));
  at.count += nth;
  at.mass += nth * at.weight;
  const int lane = tid & 63, wave = tid >> 6;
  int seen = 0;
  __syncthreads();
  if (tid == 0) s.found = -1;
  for (int i0 = 0; i0 < row.n; i0 += kThreads) {
    const int i = i0 + tid;
    const bool same = i < row.n && key_of(row.at(min(i, row.n - 1))) == prefix;
    const uint64_t who = __ballot(same);
    __syncthreads();
    if (lane == 0) s.wave_count[wave] = __popcll(who);
    __syncthreads();
    int before = seen;
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) before = seen;
      seen += s.wave_count[w];
    }
    if (same && before + __popcll(who & ((1ull << lane) - 1)) == nth - 1) s.found = i;
    if (seen >= nth) break;
  }
  __syncthreads();
  at.index = s.found;
  __syncthreads();
  return at;
}

// Whether a lies before b in the order, or is it.
__device__ __forceinline__ bool not_after(const Place &a, const Place &b) {
  return a.key > b.key || (a.key == b.key && a.index <= b.index);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleDesc d) {
  __shared__ Shared s;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Row<DT> row;
  row.p = (const typename MxType<DT>::T *)d.logits + (int64_t)r * d.stride;
  row.n = d.vocab;
  // the first token: largest key, then lowest index
  uint64_t best = 0;
  for (int i = tid; i < row.n; i += kThreads) {
    const uint64_t k = (uint64_t)key_of(row.at(i)) << 32 | (uint32_t)~i;
    best = k > best ? k : best;
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const uint64_t k = __shfl_xor((unsigned long long)best, o);
    best = k > best ? k : best;
  }
  if (lane == 0) s.best[wave] = best;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w) best = s.best[w] > best ? s.best[w] : best;
  row.top = value_of((uint32_t)(best >> 32));
  const int first = (int)~(uint32_t)best;
  const float T = d.temperature ? d.temperature[r] : 1.f;
  const int k = d.top_k ? d.top_k[r] : 0;
  const float p = d.top_p ? d.top_p[r] : 1.f;
  const float m = d.min_p ? d.min_p[r] : 0.f;
  if (row.top == -__builtin_inff()) {
    if (tid == 0) {
      d.tokens[r] = -1;
      if (d.logprobs) d.logprobs[r] = -__builtin_inff();
    }
    return;
  }
  if (!(T > 0.f) || k == 1) {
    if (tid == 0) {
      d.tokens[r] = first;
      if (d.logprobs) d.logprobs[r] = 0.f;
    }
    return;
  }
  row.scale = (double)kPerNat / (double)T;
  auto histogram = [&]() {
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0u, s.mass[i] = 0ull;
    __syncthreads();
    for (int i = tid; i < row.n; i += kThreads) {
      const double t = row.depth(row.at(i));
      const int b = bin_of(t);
      if (b == kBins) continue;
      atomicAdd(&s.count[b], 1u);
      atomicAdd((unsigned long long *)&s.mass[b], (unsigned long long)mass_of(t, b));
    }
    __syncthreads();
    scan_bins(s, kBins, [](int b) { return edge_of(b); });
  };
  // the last token kept, and what is kept
  Place last{0u, d.vocab, 0, 0.0, 0.0};
  histogram();
  last.count = s.total_count;
  last.mass = s.total_mass;
  auto cut = [&](Want want, double target) {
    const int b = first_bin(s, kBins, [&](int b) {
      if (want == kCount) return (double)(s.count_before[b] + (int)s.count[b]) >= target;
      const double mass = s.mass_before[b] + mass_value(s.mass[b], edge_of(b));
      return want == kMassAtLeast ? mass >= target : mass > target;
    });
    const Place at = find_place(s, row, want, target, b, s.count_before[b], s.mass_before[b]);
    return at;
  };
  if (k > 0 && k < last.count) {
    const Place at = cut(kCount, (double)k);
    if (not_after(at, last)) last = at;
    histogram();
  }
  if (p < 1.f) {
    const Place at = cut(kMassAtLeast, (double)p * last.mass);
    if (not_after(at, last)) last = at;
    histogram();
  }
  if (m > 0.f) {
    // how many tokens weigh at least m
    const double most = -(double)kPerNat * log((double)fminf(m, 1.f));
    int n = 0;
    for (int i = tid; i < row.n; i += kThreads) n += row.depth(row.at(i)) <= most;
#pragma unroll
    for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o);
    __syncthreads();
    if (lane == 0) s.wave_count[wave] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kWaves; ++w) n += s.wave_count[w];
    __syncthreads();
    if (n < last.count) {
      const Place at = cut(kCount, (double)n);
      last = at;
      histogram();
    }
  }
  const float u0 = d.u[r];
  const double u = u0 > 0.f ? (double)fminf(u0, 0x1.fffffep-1f) : 0.0;
  Place at = cut(kMassAbove, u * last.mass);
  if (!not_after(at, last)) at = last;
  if (tid == 0) {
    d.tokens[r] = at.index;
    if (d.logprobs) d.logprobs[r] = (float)log(at.weight / last.mass);
  }
}

}  // namespace

size_t sample_workspace(int, int) { return SPEAR_SAMPLE_HEADER_BYTES; }

hipError_t launch_sample(const spear_sample_args_t &a, void *, hipStream_t s) {
  const SampleDesc d{a.logits, a.rows, a.vocab, a.stride, a.u, a.temperature, a.top_p,
                     a.min_p, a.top_k, a.tokens, a.logprobs};
  const dim3 grid(a.rows), block(kThreads);
  if (a.dtype == SPEAR_F16) sample_kernel<0><<<grid, block, 0, s>>>(d);
  else if (a.dtype == SPEAR_BF16) sample_kernel<1><<<grid, block, 0, s>>>(d);
  else sample_kernel<2><<<grid, block, 0, s>>>(d);
  return hipGetLastError();
}

}  // namespace spear
