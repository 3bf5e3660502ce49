// One token of every row of logits: temperature, top-k, top-p, min-p.
//
// An entry's place in the order (logit descending, index ascending) is one 64-bit number,
// smaller first; each of the rules keeps a run from the start, so what is left is known by
// the place of its last entry.  That place, and the token by its index, are found by
// histograms over ranges that shrink by 2^10 a time.  Weights are integers of 2^-43, so
// that sums by atomics do not depend on their order.

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

typedef unsigned long long u64;
constexpr int kThreads = 1024, kBins = 1024;
constexpr uint32_t kNegInf = 0x007fffffu, kPosInf = 0xff800000u;   // keys of -inf and +inf

// floats as integers of the same order; NaN below everything, -0 as 0
__device__ inline uint32_t key_of(float v) {
  if (v != v) return 0;
  const uint32_t b = __float_as_uint(v + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ inline float of_key(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }

struct Row {
  const void *p;
  int f32, vocab;
  double inv_t, top;   // 1 / T and the largest logit
  bool top_inf;
  __device__ uint32_t key(int i) const {
    return key_of(f32 ? static_cast<const float *>(p)[i] : bf16f(static_cast<const uint16_t *>(p)[i]));
  }
  __device__ u64 place(int i) const { return (u64)~key(i) << 32 | (uint32_t)i; }
  __device__ double weight(uint32_t k) const {
    if (k <= kNegInf) return 0.;
    if (top_inf) return k == kPosInf ? 1. : 0.;
    return exp(((double)of_key(k) - top) * inv_t);
  }
  __device__ u64 mass(uint32_t k) const { return (u64)(weight(k) * 0x1p43 + 0.5); }
};

// ceil(f * total) for a positive float f < 1 and total < 2^63
__device__ inline u64 share(float f, u64 total, bool up) {
  const uint32_t b = __float_as_uint(f);
  const int e = b >> 23;
  const u64 m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int s = 150 - (e ? e : 1);   // f = m * 2^-s
  const unsigned __int128 p = (unsigned __int128)m * total;
  if (s >= 128) return up && p ? 1 : 0;
  const u64 q = (u64)(p >> s);
  return up && ((unsigned __int128)q << s) != p ? q + 1 : q;
}

struct Shared {
  u64 bin[kBins];
  u64 wave[kThreads / 64];
  u64 a, b, lo;
};

// The smallest place in [lo, hi] up to which amounts add up to `target` or more (hi if they never do), and
// what they add up to there.
template <typename Place, typename Amount>
__device__ u64 find(Shared &sm, int count, u64 lo, u64 hi, u64 target, Place place, Amount amount, u64 &reached) {
  u64 before = 0;
  for (;;) {
    const u64 range = hi - lo;
    const int bits = range ? 64 - __clzll(range) : 0, shift = bits > 10 ? bits - 10 : 0;
    sm.bin[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const u64 c = place(i);
      if (c < lo || c > hi) continue;
      const u64 v = amount(i);
      if (v) atomicAdd(&sm.bin[(c - lo) >> shift], v);
    }
    __syncthreads();
    // inclusive scan
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const u64 own = sm.bin[threadIdx.x];
    u64 sum = own;
    for (int d = 1; d < 64; d <<= 1) {
      const u64 up = __shfl_up(sum, d, 64);
      if (lane >= d) sum += up;
    }
    if (lane == 63) sm.wave[wave] = sum;
    if (threadIdx.x == 0) sm.lo = ~0ull;
    __syncthreads();
    for (int w = 0; w < wave; ++w) sum += sm.wave[w];
    const u64 end = before + sum, start = end - own;
    if (start < target && end >= target) {
      sm.lo = threadIdx.x;
      sm.a = start;
      sm.b = end;
    }
    __syncthreads();
    const u64 bin = sm.lo, a = sm.a, b = sm.b;
    u64 all = before;
    for (int w = 0; w < kThreads / 64; ++w) all += sm.wave[w];
    __syncthreads();
    if (bin == ~0ull) {
      reached = all;
      return hi;
    }
    lo += bin << shift;
    if (shift == 0) {
      reached = b;
      return lo;
    }
    hi = min(hi, lo + (1ull << shift) - 1);
    before = a;
  }
}

__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
  __shared__ Shared sm;
  const int t = blockIdx.x;
  Row row;
  row.p = a.f32 ? (const void *)(static_cast<const float *>(a.logits) + t * a.row) : (const void *)(static_cast<const uint16_t *>(a.logits) + t * a.row);
  row.f32 = a.f32;
  row.vocab = a.vocab;
  const float temp = a.temperature ? a.temperature[t] : 1.f, p = a.top_p ? a.top_p[t] : 1.f, u = a.u[t];
  float least = a.min_p ? a.min_p[t] : 0.f;
  const int k = a.top_k ? a.top_k[t] : 0;
  // the first of the order
  u64 first = ~0ull;
  for (int i = threadIdx.x; i < a.vocab; i += kThreads) first = min(first, row.place(i));
  for (int d = 32; d; d >>= 1) first = min(first, (u64)__shfl_xor(first, d, 64));
  if ((threadIdx.x & 63) == 0) sm.wave[threadIdx.x >> 6] = first;
  __syncthreads();
  for (int w = 0; w < kThreads / 64; ++w) first = min(first, sm.wave[w]);
  __syncthreads();
  const uint32_t top = ~(uint32_t)(first >> 32);
  if (top <= kNegInf || !(temp > 0.f)) {
    if (threadIdx.x == 0) {
      a.ids[t] = top <= kNegInf ? -1 : (int)(uint32_t)first;
      if (a.logprob) a.logprob[t] = top <= kNegInf ? -INFINITY : 0.f;
    }
    return;
  }
  row.inv_t = 1. / (double)temp;
  row.top = of_key(top);
  row.top_inf = top == kPosInf;
  auto place = [&](int i) { return row.place(i); };
  u64 last = (u64)~(kNegInf + 1) << 32 | 0xffffffffu, total = 0;   // behind it: -inf and NaN
  if (k > 0 && k < a.vocab) {
    u64 n;
    last = find(sm, a.vocab, first, last, k, place, [&](int) { return 1ull; }, n);
  }
  if (p < 1.f) {
    find(sm, a.vocab, first, last, ~0ull, place, [&](int i) { return row.mass(row.key(i)); }, total);
    u64 n;
    last = find(sm, a.vocab, first, last, p > 0.f ? max(share(p, total, true), 1ull) : 1ull, place, [&](int i) { return row.mass(row.key(i)); }, n);
  }
  least = least > 1.f ? 1.f : least;
  auto kept = [&](int i) {
    const uint32_t key = row.key(i);
    if (((u64)~key << 32 | (uint32_t)i) > last || (least > 0.f && row.weight(key) < (double)least)) return 0ull;
    return row.mass(key);
  };
  auto index = [](int i) { return (u64)i; };
  find(sm, a.vocab, 0, a.vocab - 1, ~0ull, index, kept, total);
  const float uc = u >= 0.f ? u : 0.f;   // NaN too
  const u64 target = uc < 1.f ? share(uc, total, false) + 1 : total;
  u64 n;
  const u64 id = find(sm, a.vocab, 0, a.vocab - 1, min(target, total), index, kept, n);
  if (threadIdx.x == 0) {
    a.ids[t] = (int)id;
    if (a.logprob) {
      const uint32_t key = row.key((int)id);
      a.logprob[t] = (float)((row.top_inf ? 0. : ((double)of_key(key) - row.top) * row.inv_t) - log((double)total * 0x1p-43));
    }
  }
}

}  // namespace

int64_t sample_workspace_bytes(int n, int vocab) { return 16; }

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
  hipLaunchKernelGGL(sample_kernel, dim3(a.n), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace oes
