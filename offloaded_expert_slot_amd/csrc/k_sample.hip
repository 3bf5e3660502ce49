// One token of every row of logits: temperature, top-k, top-p, min-p.
//
// An entry's place in the order (logit descending, index ascending) is one integer, smaller first; each of the rules
// keeps a run from the start, so what is left is known by the place of its last entry.  Two launches:
//   weigh   a workgroup per slice of a row: its largest logit, the sum of its weights, and (as far as the row's settings
//           ask for them) numbers and weights of its entries by bins of 1 / 8 in logit / T
//   choose  a workgroup per row: from the slices' bins the bin in which the last entry stands; if no more than kList
//           entries stand up to there, they are gathered in LDS and everything is decided among them; otherwise the
//           entries of that bin alone are gathered, and the token is looked for in the slice that the bins' sums name
// Weights are formed in fp64 and are integers of 2^-43 of the largest weight of the slice (or row), so that sums by
// atomics do not depend on their order.  fp32 would not do: over 100000 entries its sums are off by more than the
// share of many tokens.

#include <algorithm>

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

typedef unsigned long long u64;
constexpr int kBins = 256, kPer = 16;        // bins below the largest logit; entries of a thread of `weigh`
constexpr int kList = 4096, kThreads = 1024;  // `choose`
constexpr int kPairs = 512;                  // entries that are compared with one another, each with each
constexpr int kCopies = 4;                   // of the bins in LDS, for lanes side by side
constexpr uint32_t kNegInf = 0x007fffffu, kPosInf = 0xff800000u;   // keys of -inf and +inf
constexpr int kIndexBits = 20;
constexpr u64 kNowhere = ~0ull;

// floats as integers of the same order; NaN below everything, -0 as 0
__device__ inline uint32_t key_of(float v) {
  if (v != v) return 0;
  const uint32_t b = __float_as_uint(v + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ inline float of_key(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }
__device__ inline u64 place_of(uint32_t key, int index) { return (u64)~key << kIndexBits | (uint32_t)index; }
__device__ inline uint32_t key_at(u64 place) { return ~(uint32_t)(place >> kIndexBits); }
__device__ inline int index_at(u64 place) { return (int)(place & ((1u << kIndexBits) - 1)); }

// exp(x) for x <= 0: x = n ln 2 + rest (ln 2 in two parts, so that n times the first is exact), |rest| <= ln 2 / 2, and
// the Taylor series of exp(rest) to its 11th power: the next term is below 2^-47
__device__ inline double exp_of(double x) {
  if (!(x > -40.)) return 0.;   // below 2^-57
  const double n = rint(x * 1.4426950408889634);
  const double r = fma(n, -1.9082149292705877e-10, fma(n, -0.6931471803691238, x));
  double s = 1. / 39916800;
  const double c[] = {1. / 3628800, 1. / 362880, 1. / 40320, 1. / 5040, 1. / 720, 1. / 120, 1. / 24, 1. / 6, 0.5, 1., 1.};
#pragma unroll
  for (int i = 0; i < 11; ++i) s = fma(s, r, c[i]);
  return ldexp(s, (int)n);
}

// A row's logits and how they weigh against a largest one.
struct Row {
  const void *p;
  int f32;
  double inv_t;
  __device__ uint32_t key(int i) const {
    return key_of(f32 ? static_cast<const float *>(p)[i] : bf16f(static_cast<const uint16_t *>(p)[i]));
  }
  // the bin's number as a whole number in fp64: exact however large, and ascending with the key
  __device__ double bin(uint32_t k) const { return k == kPosInf ? 1e300 : floor((double)of_key(k) * inv_t * 8.); }
  __device__ double weight(uint32_t k, uint32_t top) const {
    if (top == kPosInf || k <= kNegInf) return k == top && k > kNegInf ? 1. : 0.;
    return exp_of(((double)of_key(k) - (double)of_key(top)) * inv_t);
  }
  __device__ u64 mass(uint32_t k, uint32_t top) const { return (u64)(weight(k, top) * 0x1p43 + 0.5); }
};

// Settings of a row.
struct Rules {
  float t, p, least, u;
  int k;
  bool by_k, by_p, by_min;
  __device__ Rules(const SampleArgs &a, int row) {
    t = a.temperature ? a.temperature[row] : 1.f;
    p = a.top_p ? a.top_p[row] : 1.f;
    least = a.min_p ? a.min_p[row] : 0.f;
    least = least > 1.f ? 1.f : least;   // NaN stays, and counts as none
    k = a.top_k ? a.top_k[row] : 0;
    u = a.u[row];
    by_k = k > 0 && k < a.vocab;
    by_p = p < 1.f;
    by_min = least > 0.f;
  }
  __device__ bool greedy() const { return !(t > 0.f); }
  // up to half a list the entries by k and those beside the last one nearly always fit, and no bin's weight is needed
  __device__ bool counts() const { return !greedy() && (by_k || by_p || by_min); }
  __device__ bool masses() const { return counts() && !(by_k && k <= kList / 2); }
};

// Workspace: per row and slice the first place, the sum of weights, numbers and weights by bins.
struct Slices {
  int count, size;
  u64 *first, *sum, *mass;
  uint32_t *number;
};
__host__ __device__ inline Slices slices_of(const SampleArgs &a, int count, int size) {
  Slices s;
  const int64_t all = (int64_t)a.n * count;
  s.count = count;
  s.size = size;
  s.first = reinterpret_cast<u64 *>(a.ws);
  s.sum = s.first + all;
  s.mass = s.sum + all;
  s.number = reinterpret_cast<uint32_t *>(s.mass + all * kBins);
  return s;
}
// Slices of 4096, or up to 16384 entries where there would be more than 2048 of them.
inline int slice_threads(int n, int vocab) {
  int threads = 256;
  while (threads < 1024 && (int64_t)n * ((vocab + threads * kPer - 1) / (threads * kPer)) > 2048) threads *= 2;
  return threads;
}

__device__ inline u64 wave_min(u64 v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = min(v, (u64)__shfl_xor(v, d, 64));
  return v;
}
__device__ inline u64 wave_sum(u64 v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += (u64)__shfl_xor(v, d, 64);
  return v;
}

__device__ inline Row row_of(const SampleArgs &a, int t, const Rules &r) {
  Row row;
  row.p = a.f32 ? (const void *)(static_cast<const float *>(a.logits) + t * a.row) : (const void *)(static_cast<const uint16_t *>(a.logits) + t * a.row);
  row.f32 = a.f32;
  row.inv_t = 1. / (double)r.t;
  return row;
}

// Entries as they stand in memory, 16 bytes a load; rows may start at any entry, whatever its alignment.
struct __attribute__((packed, aligned(4))) Words32 {
  float v[4];
  static constexpr int n = 4;
  __device__ uint32_t key(int e) const { return key_of(v[e]); }
  __device__ void none(int e) { v[e] = -INFINITY; }
  __device__ void one(const void *p, int i, int e) { v[e] = static_cast<const float *>(p)[i]; }
  static __device__ const Words32 *at(const void *p, int i) { return reinterpret_cast<const Words32 *>(static_cast<const float *>(p) + i); }
};
struct __attribute__((packed, aligned(2))) Words16 {
  uint16_t v[8];
  static constexpr int n = 8;
  __device__ uint32_t key(int e) const { return key_of(bf16f(v[e])); }
  __device__ void none(int e) { v[e] = 0xff80; }
  __device__ void one(const void *p, int i, int e) { v[e] = static_cast<const uint16_t *>(p)[i]; }
  static __device__ const Words16 *at(const void *p, int i) { return reinterpret_cast<const Words16 *>(static_cast<const uint16_t *>(p) + i); }
};
// entries i ...; -inf from `to` on
template <typename W>
__device__ inline W load_words(const void *p, int i, int to) {
  W w;
#pragma unroll
  for (int e = 0; e < W::n; ++e) w.none(e);
  if (i + W::n <= to) {
    w = *W::at(p, i);
  } else {
#pragma unroll
    for (int e = 0; e < W::n; ++e)
      if (i + e < to) w.one(p, i + e, e);
  }
  return w;
}
// f(index, key) for all entries of a row
template <typename W, int T, typename F>
__device__ inline void each_word(const void *p, int to, F f) {
  constexpr int AHEAD = 4;
  for (int i = W::n * (int)threadIdx.x; i < to; i += W::n * T * AHEAD) {
    W w[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) w[j] = load_words<W>(p, i + j * W::n * T, to);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
#pragma unroll
      for (int e = 0; e < W::n; ++e) f(i + j * W::n * T + e, w[j].key(e));
  }
}
template <int T, typename F>
__device__ inline void each_entry(const Row &row, int to, F f) {
  if (row.f32)
    each_word<Words32, T>(row.p, to, f);
  else
    each_word<Words16, T>(row.p, to, f);
}

// ---------------------------------------------------------------- weigh
template <int T>
__global__ __launch_bounds__(T) void weigh_kernel(SampleArgs a, int count) {
  __shared__ u64 mass[kBins][kCopies], wave_first[T / 64], wave_total[T / 64];
  __shared__ uint32_t number[kBins][kCopies];
  const int t = blockIdx.y, slice = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Slices s = slices_of(a, count, T * kPer);
  const int64_t at = (int64_t)t * count + slice;
  const Rules rules(a, t);
  const Row row = row_of(a, t, rules);
  const int from = slice * s.size, to = min(a.vocab, from + s.size);
  const bool counts = rules.counts(), masses = rules.masses();
  if (counts) {
    for (int i = threadIdx.x; i < kBins * kCopies; i += T) {
      mass[i / kCopies][i % kCopies] = 0;
      number[i / kCopies][i % kCopies] = 0;
    }
  }
  uint32_t key[kPer];
  auto load = [&](auto W) {
    typedef decltype(W) Words;
    Words w[kPer / Words::n];
#pragma unroll
    for (int j = 0; j < kPer / Words::n; ++j) w[j] = load_words<Words>(row.p, from + Words::n * ((int)threadIdx.x + j * T), to);
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = w[i / Words::n].key(i % Words::n);
  };
  if (row.f32)
    load(Words32());
  else
    load(Words16());
  u64 first = kNowhere;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int per = a.f32 ? 4 : 8;
    const int index = from + per * ((int)threadIdx.x + (i / per) * T) + i % per;
    if (key[i] > kNegInf) first = min(first, place_of(key[i], index));
  }
  first = wave_min(first);
  if (lane == 0) wave_first[wave] = first;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64; ++w) first = min(first, wave_first[w]);
  if (threadIdx.x == 0) s.first[at] = first;
  if (first == kNowhere || rules.greedy()) return;   // the same for the whole workgroup
  const uint32_t top = key_at(first);
  const double top_bin = row.bin(top);
  u64 total = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (key[i] <= kNegInf) continue;
    if (!counts) {
      total += row.mass(key[i], top);
      continue;
    }
    const double d = top_bin - row.bin(key[i]);
    if (!(d < kBins)) continue;
    atomicAdd(&number[(int)d][lane % kCopies], 1u);
    if (masses) atomicAdd(&mass[(int)d][lane % kCopies], row.mass(key[i], top));
  }
  if (!counts) {
    total = wave_sum(total);
    if (lane == 0) wave_total[wave] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < T / 64; ++w) total += wave_total[w];
      s.sum[at] = total;
    }
    return;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += T) {
    u64 m = 0;
    uint32_t c = 0;
#pragma unroll
    for (int g = 0; g < kCopies; ++g) m += mass[i][g], c += number[i][g];
    s.number[at * kBins + i] = c;
    if (masses) s.mass[at * kBins + i] = m;
  }
}

// ---------------------------------------------------------------- choose
// f * total for 0 <= f < 1 and total < 2^63, rounded down or up
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
  u64 place[kList], mass[kList];
  u64 bin[kThreads];
  u64 row_mass[kBins];
  uint32_t row_number[kBins];
  u64 slice_mass[kBins];          // at most 2^20 / 4096 slices
  double slice_share[kBins];      // a slice's weights in those of the row
  int slice_shift[kBins];         // bins between the row's largest logit and the slice's
  u64 wave[kThreads / 64];
  u64 a, b, at;
  int listed;
};

// Sum, or minimum, over the workgroup.
__device__ inline u64 all_sum(Shared &sm, u64 v) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v += sm.wave[w];
  return v;
}
__device__ inline u64 all_min(Shared &sm, u64 v) {
  v = wave_min(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm.wave[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v = min(v, sm.wave[w]);
  return v;
}

// The thread whose amount `own` takes the running sum over threads, from `before` on, to target or more leaves its
// number in sm.at and the sums before and after it in sm.a and sm.b; sm.at is kNowhere if there is none.  Returns
// the sum of all.
__device__ inline u64 cross(Shared &sm, u64 own, u64 before, u64 target) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  u64 sum = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const u64 up = __shfl_up(sum, d, 64);
    if (lane >= d) sum += up;
  }
  __syncthreads();
  if (lane == 63) sm.wave[wave] = sum;
  if (threadIdx.x == 0) sm.at = kNowhere;
  __syncthreads();
  u64 all = before;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) sum += sm.wave[w];
    all += sm.wave[w];
  }
  const u64 end = before + sum, start = end - own;
  if (start < target && end >= target) {
    sm.at = threadIdx.x;
    sm.a = start;
    sm.b = end;
  }
  __syncthreads();
  return all;
}

// The smallest number in [lo, hi] up to which amounts add up to `target` or more, `before` counted in (hi if they never
// do): over(f) calls f(number, amount) for the entries of the thread, and the range shrinks to 2^-10 a time.
template <typename Over>
__device__ u64 find(Shared &sm, u64 lo, u64 hi, u64 before, u64 target, Over over) {
  for (;;) {
    const u64 range = hi - lo;
    const int bits = range ? 64 - __clzll(range) : 0, shift = bits > 10 ? bits - 10 : 0;
    __syncthreads();
    sm.bin[threadIdx.x] = 0;
    __syncthreads();
    over([&](u64 number, u64 amount) {
      if (number >= lo && number <= hi && amount) atomicAdd(&sm.bin[(number - lo) >> shift], amount);
    });
    __syncthreads();
    cross(sm, sm.bin[threadIdx.x], before, target);
    const u64 bin = sm.at, start = sm.a;
    if (bin == kNowhere) return hi;
    lo += bin << shift;
    if (shift == 0) return lo;
    hi = min(hi, lo + (1ull << shift) - 1);
    before = start;
  }
}

__global__ __launch_bounds__(kThreads) void choose_kernel(SampleArgs a, int count, int size) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  Shared &sm = *reinterpret_cast<Shared *>(lds);
  const int t = blockIdx.x;
  const Slices s = slices_of(a, count, size);
  const int64_t at = (int64_t)t * count;
  const Rules rules(a, t);
  const Row row = row_of(a, t, rules);
  const u64 first = all_min(sm, (int)threadIdx.x < count ? s.first[at + threadIdx.x] : kNowhere);
  const uint32_t top = key_at(first);
  auto answer = [&](int id, float logprob) {
    if (threadIdx.x == 0) {
      a.ids[t] = id;
      if (a.logprob) a.logprob[t] = logprob;
    }
  };
  if (first == kNowhere) return answer(-1, -INFINITY);
  if (rules.greedy()) return answer(index_at(first), 0.f);
  const double top_bin = row.bin(top);
  auto found = [&](int id, u64 total) {
    const uint32_t k = row.key(id);
    const double z = top == kPosInf ? 0. : ((double)of_key(k) - (double)of_key(top)) * row.inv_t;
    answer(id, (float)(z - log((double)total * 0x1p-43)));
  };
  auto aim = [&](u64 total) {   // the running sum that the token's must reach
    const float u = rules.u >= 0.f ? rules.u : 0.f;   // NaN too
    return u < 1.f ? share(u, total, false) + 1 : total;
  };
  if ((int)threadIdx.x < count) {
    const u64 f = s.first[at + threadIdx.x];
    double d = f == kNowhere ? kBins : top_bin - row.bin(key_at(f));
    d = d < kBins ? d : kBins;
    sm.slice_shift[threadIdx.x] = (int)d;
    sm.slice_share[threadIdx.x] = d < kBins ? row.weight(key_at(f), top) : 0.;
  }
  __syncthreads();
  // the smallest key of bins 0 ... j, by 64 places at a time
  auto key_from = [&](int j) {
    if (j < 0) return top + 1;
    uint32_t lo = kNegInf + 1, hi = top;   // the answer is in [lo, hi]
    while (lo < hi) {
      const uint32_t step = (hi - lo + 63) / 64, mine = lo + step * (threadIdx.x & 63);
      const u64 in = __ballot(mine >= hi || mine < lo || top_bin - row.bin(mine) <= j);
      const int at = __ffsll(in) - 1;   // the first place that is in; -1: behind all of them
      const uint32_t below = at < 0 ? lo + step * 63 + 1 : at == 0 ? lo : lo + step * (at - 1) + 1;
      if (at >= 0) hi = min(hi, lo + step * at);
      lo = min(below, hi);
    }
    return lo;
  };
  // what bin j of the row has from slice i, in the row's weights
  auto part = [&](int i, int j) {
    const int from = j - sm.slice_shift[i];
    return from < 0 ? 0ull : (u64)((double)s.mass[(at + i) * kBins + from] * sm.slice_share[i] + 0.5);
  };
  const bool masses = rules.masses();
  u64 last = kNowhere, all = 0;   // the last place by k and p, the weight of all
  int edge = kBins;               // the bin of the last place; entries of the bins before it stay whole
  if (rules.counts()) {
    if (threadIdx.x < kBins) {
      sm.row_mass[threadIdx.x] = 0;
      sm.row_number[threadIdx.x] = 0;
    }
    __syncthreads();
    const int j = threadIdx.x % kBins;
    u64 m = 0;
    uint32_t c = 0;
    for (int i = threadIdx.x / kBins; i < count; i += kThreads / kBins) {
      const int from = j - sm.slice_shift[i];
      if (from >= 0) c += s.number[(at + i) * kBins + from];
      if (masses) m += part(i, j);
    }
    if (c) atomicAdd(&sm.row_number[j], c);
    if (m) atomicAdd(&sm.row_mass[j], m);
    __syncthreads();
    if (masses) all = all_sum(sm, threadIdx.x < kBins ? sm.row_mass[threadIdx.x] : 0);
    // the bin up to which an amount is reached (the last one if it is not)
    auto bin_of = [&](bool mass, u64 target) {
      __syncthreads();
      cross(sm, threadIdx.x >= kBins ? 0 : mass ? sm.row_mass[threadIdx.x] : sm.row_number[threadIdx.x], 0, target);
      return sm.at == kNowhere ? kBins - 1 : (int)sm.at;
    };
    const int k_bin = rules.by_k ? bin_of(false, rules.k) : kBins - 1;
    int upto = k_bin;
    if (rules.by_p && !rules.by_k) {
      // a little further, since a bin's weight and its entries' are rounded apart
      const u64 want = rules.p > 0.f ? share(rules.p, all, true) : 1;
      upto = bin_of(true, min(all, want + (want >> 36)));
    }
    int min_bin = kBins;   // one bin further than the smallest weight's, which is off by less
    if (rules.by_min) {
      const double d = top == kPosInf ? 0. : top_bin - floor(((double)of_key(top) * row.inv_t + log((double)rules.least)) * 8.) + 1.;
      min_bin = d < kBins ? (int)d : kBins;
      if (!(rules.by_k && rules.by_p)) upto = min(upto, min_bin);   // p takes its share of all that k leaves
    }
    __syncthreads();
    const u64 listed = all_sum(sm, threadIdx.x <= (uint32_t)upto && threadIdx.x < kBins ? sm.row_number[threadIdx.x] : 0);
    auto gather = [&](int low, int high) {   // places of the entries of bins low ... high, and their weights, into LDS
      if (threadIdx.x == 0) sm.listed = 0;
      __syncthreads();
      const uint32_t from = key_from(high), to = key_from(low - 1);
      each_entry<kThreads>(row, a.vocab, [&](int i, uint32_t k) {
        if (k >= from && k < to) {
          const int slot = atomicAdd(&sm.listed, 1);
          if (slot < kList) {
            sm.place[slot] = place_of(k, i);
            sm.mass[slot] = row.mass(k, top);
          }
        }
      });
      __syncthreads();
      return min(sm.listed, kList);
    };
    if (listed <= kList) {
      const int m = gather(0, upto);
      if (m <= kPairs) {
        // each with each: g threads an entry
        int g = 2;
        while (g < 16 && kThreads / g / 2 >= m) g *= 2;
        const int i = threadIdx.x / g, sub = threadIdx.x % g;
        const bool live = i < m;
        const u64 me = live ? sm.place[i] : kNowhere, own = live ? sm.mass[i] : 0;
        u64 before = 0;
        int rank = 0;
        for (int o = sub; o < m; o += g)
          if (sm.place[o] < me) before += sm.mass[o], ++rank;
        for (int d = 1; d < g; d <<= 1) before += (u64)__shfl_xor(before, d, 64), rank += __shfl_xor(rank, d, 64);
        const bool in_k = live && (!rules.by_k || rank < rules.k);
        bool stays = in_k;
        if (rules.by_p) {
          const u64 sum = rules.by_k ? all_sum(sm, in_k && sub == 0 ? own : 0) : all;
          stays &= before < (rules.p > 0.f ? max(share(rules.p, sum, true), 1ull) : 1ull);
        }
        if (rules.by_min) stays &= live && row.weight(key_at(me), top) >= (double)rules.least;
        const u64 total = all_sum(sm, stays && sub == 0 ? own : 0);
        if (live && !stays && sub == 0) sm.mass[i] = 0;
        __syncthreads();
        u64 sum = 0;
        for (int o = sub; o < m; o += g)
          if (index_at(sm.place[o]) <= index_at(me)) sum += sm.mass[o];
        for (int d = 1; d < g; d <<= 1) sum += (u64)__shfl_xor(sum, d, 64);
        const u64 id = all_min(sm, stays && sum >= aim(total) ? (u64)index_at(me) : kNowhere);
        return found((int)id, total);
      }
      auto each = [&](auto f) {
        for (int i = threadIdx.x; i < m; i += kThreads) f(sm.place[i], sm.mass[i]);
      };
      auto sum_to = [&](u64 border) {
        u64 v = 0;
        each([&](u64 place, u64 mass) { v += place <= border ? mass : 0; });
        return all_sum(sm, v);
      };
      const u64 end = place_of(kNegInf + 1, 0) | ((1u << kIndexBits) - 1);
      last = end;
      if (rules.by_k) last = find(sm, first, last, 0, rules.k, [&](auto f) { each([&](u64 place, u64) { f(place, 1ull); }); });
      if (rules.by_p) {
        const u64 sum = rules.by_k ? sum_to(last) : all;
        last = find(sm, first, last, 0, rules.p > 0.f ? max(share(rules.p, sum, true), 1ull) : 1ull, [&](auto f) { each(f); });
      }
      for (int i = threadIdx.x; i < m; i += kThreads)
        if (sm.place[i] > last || (rules.by_min && row.weight(key_at(sm.place[i]), top) < (double)rules.least)) sm.mass[i] = 0;
      const u64 total = sum_to(end);
      const u64 id = find(sm, 0, a.vocab - 1, 0, aim(total), [&](auto f) { each([&](u64 place, u64 mass) { f((u64)index_at(place), mass); }); });
      return found((int)id, total);
    }

    // Too many entries.  The last place by k, and then by p, among the entries of its bin: gathered if they fit, read
    // from the row each time if not.
    auto over_row = [&](bool mass) {
      return [&, mass](auto f) { each_entry<kThreads>(row, a.vocab, [&](int i, uint32_t k) {
        if (k > kNegInf) f(place_of(k, i), mass ? row.mass(k, top) : 1ull);
      }); };
    };
    auto border = [&](int bin, bool mass, u64 target) {
      u64 before = 0;
      if ((int)threadIdx.x < bin && threadIdx.x < kBins) before = mass ? sm.row_mass[threadIdx.x] : sm.row_number[threadIdx.x];
      before = all_sum(sm, before);
      const u64 end = place_of(kNegInf + 1, 0) | ((1u << kIndexBits) - 1);
      if (sm.row_number[bin] <= kList) {
        const int m = gather(bin, bin);
        if (m == 0) return kNowhere;   // the amount is not reached
        u64 lo = kNowhere, hi = 0;
        for (int i = threadIdx.x; i < m; i += kThreads) lo = min(lo, sm.place[i]), hi = max(hi, sm.place[i]);
        lo = all_min(sm, lo);
        hi = ~all_min(sm, ~hi);
        return find(sm, lo, hi, before, target, [&](auto f) {
          for (int i = threadIdx.x; i < m; i += kThreads) f(sm.place[i], mass ? sm.mass[i] : 1ull);
        });
      }
      return mass ? find(sm, first, end, 0, target, over_row(true)) : find(sm, first, end, 0, target, over_row(false));
    };
    if (rules.by_k) last = border(k_bin, false, rules.k);
    if (rules.by_p) {
      u64 sum = all;
      if (rules.by_k) {
        sum = 0;
        each_entry<kThreads>(row, a.vocab, [&](int i, uint32_t k) { sum += k > kNegInf && place_of(k, i) <= last ? row.mass(k, top) : 0; });
        sum = all_sum(sm, sum);
      }
      const u64 want = rules.p > 0.f ? max(share(rules.p, sum, true), 1ull) : 1ull;
      if (masses) {
        last = min(last, border(bin_of(true, want), true, want));
      } else {
        last = min(last, find(sm, first, last, 0, want, over_row(true)));
      }
    }
    edge = last == kNowhere ? kBins : min(upto, (int)fmin(top_bin - row.bin(key_at(last)), (double)kBins));
    if (rules.by_min) edge = min(edge, max(0, min_bin - 2));
  }

  // The slices' sums: whole bins, and what stays of the others' entries.
  auto stays = [&](int i, uint32_t k) {
    return k > kNegInf && place_of(k, i) <= last && !(rules.by_min && row.weight(k, top) < (double)rules.least);
  };
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads) sm.slice_mass[i] = 0;
  __syncthreads();
  if (!rules.counts()) {
    if ((int)threadIdx.x < count) sm.slice_mass[threadIdx.x] = s.first[at + threadIdx.x] == kNowhere ? 0 : (u64)((double)s.sum[at + threadIdx.x] * sm.slice_share[threadIdx.x] + 0.5);
  } else {
    const int whole = masses ? edge : 0;
    for (int u = threadIdx.x; u < count * kBins; u += kThreads) {
      const int i = u / kBins, j = u % kBins;
      const u64 v = j < whole ? part(i, j) : 0;
      if (v) atomicAdd(&sm.slice_mass[i], v);
    }
    if (whole < kBins) {
      const uint32_t below = key_from(whole - 1);
      each_entry<kThreads>(row, a.vocab, [&](int i, uint32_t k) {
        if (k >= below || !stays(i, k)) return;
        const u64 v = row.mass(k, top);
        if (v) atomicAdd(&sm.slice_mass[i / s.size], v);
      });
    }
  }
  __syncthreads();
  const u64 of_slice = (int)threadIdx.x < count ? sm.slice_mass[threadIdx.x] : 0;
  const u64 total = all_sum(sm, of_slice), target = aim(total);
  __syncthreads();
  cross(sm, of_slice, 0, target);
  const int slice = (int)min(sm.at, (u64)count - 1);
  u64 before = sm.a;
  __syncthreads();
  // within the slice, entries side by side; their sum may miss the slice's by what was rounded: then the last one
  const int per = s.size / kThreads, from = slice * s.size + per * threadIdx.x;
  u64 own = 0, end_id = kNowhere;
  for (int i = from; i < min(from + per, a.vocab); ++i) {
    const uint32_t k = row.key(i);
    const u64 v = stays(i, k) ? row.mass(k, top) : 0;
    own += v;
    if (v) end_id = ~(u64)i;
  }
  end_id = ~all_min(sm, end_id);
  __syncthreads();
  cross(sm, own, before, target);
  if (sm.at == kNowhere) return found(end_id == ~kNowhere ? index_at(first) : (int)end_id, total);
  if (sm.at == threadIdx.x) {
    u64 sum = sm.a;
    int id = from;
    for (int i = from; i < min(from + per, a.vocab); ++i) {
      const uint32_t k = row.key(i);
      sum += stays(i, k) ? row.mass(k, top) : 0;
      if (sum >= target) {
        id = i;
        break;
      }
    }
    sm.b = id;
  }
  __syncthreads();
  found((int)sm.b, total);
}

}  // namespace

int64_t sample_workspace_bytes(int n, int vocab) {
  const int size = slice_threads(n, vocab) * kPer;
  const int64_t all = (int64_t)n * ((vocab + size - 1) / size);
  return (all * (16 + kBins * 12) + 15) / 16 * 16;
}

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
  const int threads = slice_threads(a.n, a.vocab), size = threads * kPer, count = (a.vocab + size - 1) / size;
  const dim3 g(count, a.n);
  if (threads == 256)
    hipLaunchKernelGGL(weigh_kernel<256>, g, dim3(256), 0, s, a, count);
  else if (threads == 512)
    hipLaunchKernelGGL(weigh_kernel<512>, g, dim3(512), 0, s, a, count);
  else
    hipLaunchKernelGGL(weigh_kernel<1024>, g, dim3(1024), 0, s, a, count);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(choose_kernel, dim3(a.n), dim3(kThreads), sizeof(Shared), s, a, count, size);
  return hipGetLastError();
}

}  // namespace oes
