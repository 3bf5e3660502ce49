// One token of every row of logits: temperature, top-k, top-p, min-p.
//
// An entry's place in the order (logit descending, index ascending) is one integer, smaller first; each of the rules
// keeps a run from the start, so what is left is known by the place of its last entry.  Two launches:
//   weigh   a workgroup per slice of a row: its largest logit, the sum of its weights, and (as far as the row's settings
//           ask for them) numbers and weights of its entries by bins of 1 / 8 in logit / T
//   choose  a workgroup per row: from the slices' bins the bin in which the last entry stands; if no more than kList
//           entries stand up to there, they are gathered in LDS and everything is decided among them;
//           otherwise the entries of that bin alone are, and the token is looked for in the slice that the bins' sums
//           name
// Nothing is sorted.  A row is read twice where at most kList entries stand up to the last one's bin (and with no rule
// but u, once and one slice of it again).  Where more do, further passes read it: one for the list of each border, k's and then
// p's, and one before for every 2^-9 of a bin that holds more than kList entries; one for the weight of what k left; one for the last
// bin's entries where two rules meet in it.  Of one row of 100003 that takes 148 us for k = 30000 and p = 0.7 of logits spread by
// 2, 184 us for p = 0.9 of logits spread by 0.05, and 310 us where all are equal.
// Weights are formed in fp64 and are integers of 2^-43 of the largest weight of the slice (or row), so that sums by
// atomics do not depend on their order.  fp32 would not do: over 100000 entries its sums are off by more than the
// share of many tokens.
//
// Measured, both launches replayed in a graph: one row of 100003 fp32 by k = 64 and p = 0.95 28.5 us, 4.0 of them weigh and
// about 11 the gather (latency: what a workgroup's few instructions and trips to memory take one after the other); 48
// rows of 100003 bf16, settings mixed, 56 us; 160 rows of 200003 fp32 by p 107 us: weigh 46 (2.8 TB/s; the weights'
// fp64 and the bins' atomics, vector units busy for 0.8 of it), the gather about 30, the searches about 20.

#include <algorithm>
#include <type_traits>

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

typedef unsigned long long u64;
// Functions of the kernel below have barriers and take much of the workgroup's state: no calls, no stack.
#define INLINE __attribute__((always_inline))
constexpr int kBins = 256, kPer = 16;        // bins below the largest logit; entries of a thread of `weigh`
constexpr int kList = 8192, kThreads = 512, kDigit = 9;   // `choose`: entries in LDS, threads, and their logarithm
constexpr uint32_t kNegInf = 0x007fffffu, kPosInf = 0xff800000u;   // keys of -inf and +inf
constexpr int kIndexBits = 20;
constexpr u64 kNowhere = ~0ull;

// A value that is the same in all lanes, kept in scalar registers.
__device__ INLINE inline uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ INLINE inline u64 uniform(u64 v) { return (u64)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v); }
__device__ INLINE inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ INLINE inline float uniform(float v) { return __uint_as_float(uniform(__float_as_uint(v))); }
__device__ INLINE inline double uniform(double v) { return __builtin_bit_cast(double, uniform(__builtin_bit_cast(u64, v))); }

// floats as integers of the same order; NaN below everything, -0 as 0
__device__ INLINE inline uint32_t key_of(float v) {
  if (v != v) return 0;
  const uint32_t b = __float_as_uint(v + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ INLINE inline float of_key(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }
__device__ INLINE inline u64 place_of(uint32_t key, int index) { return (u64)~key << kIndexBits | (uint32_t)index; }
__device__ INLINE inline uint32_t key_at(u64 place) { return ~(uint32_t)(place >> kIndexBits); }
__device__ INLINE inline int index_at(u64 place) { return (int)(place & ((1u << kIndexBits) - 1)); }

// A constant in scalar registers, where an fma takes it as its third operand; as a literal it would be moved into vector
// registers before each (18 of 70 instructions for an entry's weight and bin).
__device__ INLINE inline double held(double v) {
  asm("" : "+s"(v));
  return v;
}
// 2^y for -45 <= y <= 0 as s 2^n, s within [0.7, 1.42]: y = n + f, and s = 2^f by a polynomial 1 + f q(f) whose q goes
// through the values of (2^f - 1) / f at the nine Chebyshev nodes of [-1/2, 1/2]; off by 4e-14 at most, and 1 for f = 0.
struct Exp2 {
  double magic, c[9], unit, least;
  __device__ INLINE Exp2() {
    const double q[] = {0.6931471805599453, 0.2402265069581299, 0.055504108664760424, 0.009618129159402558, 0.0013333558179043112,
                        0.00015403455852453838, 1.525268684626772e-05, 1.3255224878668817e-06, 1.0203121063391729e-07};
#pragma unroll
    for (int i = 0; i < 9; ++i) c[i] = held(q[i]);
    magic = held(0x1.8p52), unit = held(0x1p52), least = held(-45.);
  }
  __device__ INLINE double parts(double y, int &n) const {
    const double t = y + magic;   // rounds y to a whole number, and leaves it in the low bits
    n = (int)(uint32_t)__builtin_bit_cast(u64, t);
    const double f = y - (t - magic);
    double s = fma(c[8], f, c[7]);
#pragma unroll
    for (int i = 6; i >= 0; --i) s = fma(s, f, c[i]);
    return fma(s, f, 1.);
  }
};

// Logits in memory: rows may start at any entry, whatever its alignment, and are read by 16 bytes that are aligned.
struct F32 {
  typedef float elem;
  static constexpr int n = 4;   // entries of 16 bytes
  static __device__ INLINE float value(u32x4 w, int e) { return __uint_as_float(w[e]); }
  static __device__ INLINE float value(float v) { return v; }
  static __device__ INLINE float pick(u32x4 w, int e) { return __uint_as_float(e & 2 ? (e & 1 ? w.w : w.z) : e & 1 ? w.y : w.x); }
  static __device__ INLINE void put(u32x4 &w, int e, float v) { w[e] = __float_as_uint(v); }
};
struct B16 {
  typedef uint16_t elem;
  static constexpr int n = 8;
  static __device__ INLINE float value(u32x4 w, int e) { return e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]); }
  static __device__ INLINE float value(uint16_t v) { return bf16f(v); }
  static __device__ INLINE float pick(u32x4 w, int e) {
    const uint32_t two = e & 4 ? (e & 2 ? w.w : w.z) : e & 2 ? w.y : w.x;
    return e & 1 ? bf16_hi(two) : bf16_lo(two);
  }
  static __device__ INLINE void put(u32x4 &w, int e, uint16_t v) { w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | (uint32_t)v << 16 : (w[e / 2] & 0xffff0000u) | v; }
};

// A row, and how its logits weigh against a largest one.
template <typename L>
struct Row {
  const typename L::elem *p;
  int vocab, off;      // entries; those of the first 16 bytes that stand before the row
  double inv_t, per;   // 1 / T, and what makes a difference of logits a power of 2
  float bins;          // bins of a logit's 1: 8 / T
  Exp2 exp2;
  __device__ INLINE Row(const SampleArgs &a, int t) {
    p = static_cast<const typename L::elem *>(a.logits) + t * a.row;
    vocab = a.vocab;
    off = (int)(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(typename L::elem));
  }
  __device__ INLINE void heat(float temperature) {
    inv_t = uniform(1. / (double)temperature);
    per = uniform(inv_t * 1.4426950408889634);
    bins = uniform((float)fmin(inv_t * 8., (double)__FLT_MAX__));
  }
  __device__ INLINE uint32_t key(int i) const { return key_of(L::value(p[i])); }
  // The entries from i + j * step on, which are 16-byte aligned; NaN outside of the row.  All are asked for at once: the
  // words that the row has in part only are put together afterwards, since a load that hangs on a condition has the
  // next one wait (a row of 100003 at 14.8 in place of 6.7 us).
  template <int COUNT>
  __device__ INLINE void words(int i, int step, u32x4 (&w)[COUNT]) const {
    const int some = off ? L::n - off : 0;   // a word that is whole, in rows of two words and more
#pragma unroll
    for (int j = 0; j < COUNT; ++j) {
      const int at = i + j * step;
      w[j] = u32x4{~0u, ~0u, ~0u, ~0u};
      if (vocab >= 2 * L::n) w[j] = *reinterpret_cast<const u32x4 *>(p + (at >= 0 && at + L::n <= vocab ? at : some));
    }
#pragma unroll
    for (int j = 0; j < COUNT; ++j) {
      const int at = i + j * step;
      if (vocab >= 2 * L::n && at >= 0 && at + L::n <= vocab) continue;
      w[j] = u32x4{~0u, ~0u, ~0u, ~0u};
      if (at + L::n <= 0 || at >= vocab) continue;
#pragma unroll
      for (int e = 0; e < L::n; ++e)
        if (at + e >= 0 && at + e < vocab) L::put(w[j], e, p[at + e]);
    }
  }
  // The number of a value's bin, a whole number that ascends with the value.  Numbers whose difference is below kBins are
  // subtracted without rounding, however large they are.
  __device__ INLINE float bin(float v) const {
    const float m = __FLT_MAX__;
    return floorf(__builtin_amdgcn_fmed3f(__builtin_amdgcn_fmed3f(v, -m, m) * bins, -m, m));
  }
  __device__ INLINE double weight(uint32_t k, uint32_t top) const {
    if (top == kPosInf || k <= kNegInf) return k == top && k > kNegInf ? 1. : 0.;
    const double y = ((double)of_key(k) - (double)of_key(top)) * per;
    int n;
    const double s = exp2.parts(fmax(y, exp2.least), n);
    return y < -45. ? 0. : ldexp(s, n);
  }
  // the weight of v against the largest logit, which is finite, in units of 2^-43, to the nearest: 2^52 more, it is the
  // low bits of its fp64; 0 for -inf, NaN and whatever is below 2^-44
  __device__ INLINE u64 mass_of(float v, double top) const {
    int n;
    const double s = exp2.parts(fmax(((double)v - top) * per, exp2.least), n);
    const double m = fma(s, __builtin_bit_cast(double, (u64)(n + 43 + 1023) << 52), exp2.unit);
    return __builtin_bit_cast(u64, m) & ((1ull << 52) - 1);
  }
  __device__ INLINE u64 mass(uint32_t k, uint32_t top) const {
    const u64 m = mass_of(of_key(k), (double)of_key(top));
    return top == kPosInf ? (k == top ? 1ull << 43 : 0) : m;
  }
};

// Settings of a row.
struct Rules {
  float t, p, least, u;
  int k;
  bool by_k, by_p, by_min;
  __device__ INLINE Rules(const SampleArgs &a, int row) {
    t = uniform(a.temperature ? a.temperature[row] : 1.f);
    p = uniform(a.top_p ? a.top_p[row] : 1.f);
    least = uniform(a.min_p ? a.min_p[row] : 0.f);
    least = least > 1.f ? 1.f : least;   // NaN stays, and counts as none
    k = uniform(a.top_k ? a.top_k[row] : 0);
    u = uniform(a.u[row]);
    by_k = k > 0 && k < a.vocab;
    by_p = p < 1.f;
    by_min = least > 0.f;
  }
  __device__ INLINE bool greedy() const { return !(t > 0.f); }
  __device__ INLINE bool counts() const { return !greedy() && (by_k || by_p || by_min); }
  // up to a quarter of a list the entries by k and those beside the last one nearly always fit, and no bin's weight is
  // needed
  __device__ INLINE bool masses() const { return counts() && !(by_k && k <= kList / 4); }
};

// Workspace: per row and slice the first place, the sum of weights, numbers and weights by bins.
struct Slices {
  int count, size;
  u64 *first, *sum, *mass;
  uint32_t *number;
};
__device__ INLINE inline Slices slices_of(const SampleArgs &a, int count, int size) {
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
// Slices of 4096, or of 8192 entries where there would be more than 2048 of them; a row may begin with up to 7 entries of
// another one's.
constexpr int kShortSlices = 2048;
inline int slice_threads(int n, int vocab) {
  return (int64_t)n * ((vocab + 7 + 256 * kPer - 1) / (256 * kPer)) > kShortSlices ? 512 : 256;
}
inline int slice_count(int threads, int vocab) { return (vocab + 7 + threads * kPer - 1) / (threads * kPer); }

__device__ INLINE inline u64 wave_min(u64 v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = min(v, (u64)__shfl_xor(v, d, 64));
  return v;
}
__device__ INLINE inline u64 wave_sum(u64 v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += (u64)__shfl_xor(v, d, 64);
  return v;
}

// ---------------------------------------------------------------- weigh
template <typename L, int T>
__global__ __launch_bounds__(T) void weigh_kernel(SampleArgs a, int count) {
  __shared__ u64 mass[kBins], wave_first[T / 64], wave_total[T / 64];
  __shared__ uint32_t number[kBins];
  const int t = blockIdx.x / count, slice = blockIdx.x % count, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Slices s = slices_of(a, count, T * kPer);
  const int64_t at = (int64_t)t * count + slice;
  Row<L> row(a, t);
  constexpr int N = L::n, WORDS = kPer / N;
  const int from = slice * s.size - row.off + N * (int)threadIdx.x;
  u32x4 w[WORDS];
  row.words(from, N * T, w);
  const Rules rules(a, t);
  row.heat(rules.t);
  const bool counts = rules.counts(), masses = rules.masses();
  if (counts)
    for (int i = threadIdx.x; i < kBins; i += T) mass[i] = 0, number[i] = 0;
  float v[WORDS][N], largest = -INFINITY;
#pragma unroll
  for (int j = 0; j < WORDS; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      v[j][e] = L::value(w[j], e);
      largest = fmaxf(largest, v[j][e]);
    }
  // of the largest values the first one
  u64 first = kNowhere;
#pragma unroll
  for (int j = WORDS - 1; j >= 0; --j)
#pragma unroll
    for (int e = N - 1; e >= 0; --e)
      if (v[j][e] == largest) first = from + j * N * T + e;
  first = largest > -INFINITY ? place_of(key_of(largest), (int)first) : kNowhere;
  first = wave_min(first);
  if (lane == 0) wave_first[wave] = first;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64; ++w) first = min(first, wave_first[w]);
  first = uniform(first);
  if (threadIdx.x == 0) s.first[at] = first;
  if (first == kNowhere || rules.greedy()) return;   // the same for the whole workgroup
  float top = of_key(key_at(first));
  if (top == INFINITY) {   // beside it nothing weighs
    top = 0.f;
#pragma unroll
    for (int j = 0; j < WORDS; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) v[j][e] = v[j][e] == INFINITY ? 0.f : -INFINITY;
  }
  const float top_bin = row.bin(top);
  if (!counts) {
    u64 total = 0;
#pragma unroll
    for (int j = 0; j < WORDS; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) total += row.mass_of(v[j][e], (double)top);
    total = wave_sum(total);
    if (lane == 0) wave_total[wave] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < T / 64; ++w) total += wave_total[w];
      s.sum[at] = total;
    }
    return;
  }
  auto put = [&](auto by_mass) INLINE {
#pragma unroll
    for (int j = 0; j < WORDS; ++j) {
      u64 m[N];
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (by_mass) m[e] = row.mass_of(v[j][e], (double)top);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = top_bin - row.bin(v[j][e]);
        if (v[j][e] > -INFINITY && d < kBins) {
          atomicAdd(&number[(int)d], 1u);
          if (by_mass && m[e]) atomicAdd(&mass[(int)d], m[e]);
        }
      }
    }
  };
  if (masses)
    put(std::true_type{});
  else
    put(std::false_type{});
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += T) {
    s.number[at * kBins + i] = number[i];
    if (masses) s.mass[at * kBins + i] = mass[i];
  }
}

// ---------------------------------------------------------------- choose
// f * total for 0 <= f < 1 and total < 2^63, rounded down or up
__device__ INLINE inline u64 share(float f, u64 total, bool up) {
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
  u64 list[kList];                // places
  u64 mass[kList];                // and weights
  u64 bin[kThreads];
  uint32_t bin_number[kThreads];
  u64 row_mass[kBins];
  uint32_t row_number[kBins];
  u64 slice_mass[kBins + 1];      // at most 2^20 / 4096 slices and one
  double slice_share[kBins + 1];  // a slice's weights in those of the row
  int slice_shift[kBins + 1];     // bins between the row's largest logit and the slice's
  u64 wave[kThreads / 64];
  u64 before, at;
  uint32_t key;
  int listed;
};

__device__ INLINE inline u64 all_sum(Shared &sm, u64 v) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v += sm.wave[w];
  return uniform(v);
}
__device__ INLINE inline u64 all_min(Shared &sm, u64 v) {
  v = wave_min(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm.wave[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v = min(v, sm.wave[w]);
  return uniform(v);
}

// Where a running sum over threads reaches `target`: the thread whose amount `own` takes it there gets its number into
// sm.at and the sum before it into sm.before; sm.at is kNowhere if none does.
__device__ INLINE inline void cross(Shared &sm, u64 own, u64 before, u64 target) {
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
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w)
    if (w < wave) sum += sm.wave[w];
  const u64 end = before + sum, start = end - own;
  if (start < target && end >= target) {
    sm.at = threadIdx.x;
    sm.before = start;
  }
  __syncthreads();
}

// The first of `count` entries at which the running sum of amount(i), from `before` on, reaches `target`; count - 1 if none.
template <typename F>
__device__ INLINE inline int locate(Shared &sm, int count, u64 before, u64 target, F amount) {
  const int per = (count + kThreads - 1) / kThreads, from = per * (int)threadIdx.x, to = min(from + per, count);
  u64 own = 0;
  for (int i = from; i < to; ++i) own += amount(i);
  cross(sm, own, before, target);
  if (uniform(sm.at) == kNowhere) return count - 1;
  if (sm.at == threadIdx.x) {
    u64 sum = sm.before;
    int i = from;
    for (; i < to - 1; ++i) {
      sum += amount(i);
      if (sum >= target) break;
    }
    sm.listed = i;
  }
  __syncthreads();
  return uniform(sm.listed);
}

// The smallest number among the list's m entries up to which amounts add up to `target`, `before` counted in (the largest
// one if they never do); numbers are places, or indices, and lie in [lo, hi].  Histograms over the range, which shrinks
// to 2^-9 a time, until one entry is left in it.
enum { BY_NUMBER, BY_WEIGHT, BY_INDEX };   // one each by place, weights by place, weights by index
__device__ INLINE inline u64 find(Shared &sm, int m, int by, u64 lo, u64 hi, u64 before, u64 target) {
  const int tid = threadIdx.x;
  for (;;) {
    const u64 range = hi - lo;
    const int bits = range ? 64 - __clzll(range) : 0, shift = bits > kDigit ? bits - kDigit : 0;
    __syncthreads();
    sm.bin[tid] = 0, sm.bin_number[tid] = 0;
    __syncthreads();
    for (int i = tid; i < m; i += kThreads) {
      const u64 number = by == BY_INDEX ? (u64)index_at(sm.list[i]) : sm.list[i], amount = by == BY_NUMBER ? 1 : sm.mass[i];
      if (number < lo || number > hi || !amount) continue;
      const int bin = (int)((number - lo) >> shift);
      atomicAdd(&sm.bin_number[bin], 1u);
      if (by != BY_NUMBER) atomicAdd(&sm.bin[bin], amount);
    }
    __syncthreads();
    cross(sm, by == BY_NUMBER ? sm.bin_number[tid] : sm.bin[tid], before, target);
    const u64 bin = uniform(sm.at);
    if (bin == kNowhere) return hi;
    lo += bin << shift;
    if (shift == 0) return lo;
    hi = min(hi, lo + (1ull << shift) - 1);
    before = uniform(sm.before);
    if (uniform(sm.bin_number[bin]) == 1) {
      __syncthreads();
      for (int i = tid; i < m; i += kThreads) {
        const u64 number = by == BY_INDEX ? (u64)index_at(sm.list[i]) : sm.list[i];
        if (number >= lo && number <= hi && (by == BY_NUMBER || sm.mass[i])) sm.at = number;
      }
      __syncthreads();
      return uniform(sm.at);
    }
  }
}

// the sum over a wave's lanes up to each, all of which are active: four shifts within rows of 16, two across them
__device__ INLINE inline int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}

// A pass over a row's entries with places in [from, to].  A thread has a round of words, 32 entries, asked for together;
// take(in, index, w) gets those to be taken as the bits of `in`, of which bit j * N + e is entry e of word j and has the
// index index + j * N * kThreads + e.  The entries before the first and behind the last whole word come as a round of
// their own, each as a word's first.  take is called by all lanes of a wave.
template <typename L, typename F>
__device__ INLINE inline void scan(const Row<L> &row, u64 from, u64 to, F take) {
  constexpr int N = L::n, AHEAD = 32 / N;
  constexpr u64 index_mask = (1ull << kIndexBits) - 1;
  constexpr uint32_t none = 0x7fffffffu;   // no value has the key of -0, which compares as 0
  if (key_at(from) == none) from = place_of(none - 1, 0);
  if (key_at(to) == none) to = place_of(none + 1, 0) | index_mask;
  const float low = of_key(key_at(to)), high = of_key(key_at(from));
  const int from_index = index_at(from), to_index = index_at(to);
  const bool ragged = from_index != 0 || to_index != (int)index_mask;
  const int head = min(row.off ? N - row.off : 0, row.vocab), whole = (row.vocab - head) / N, behind = head + whole * N;
  const int rounds = (whole + kThreads * AHEAD - 1) / (kThreads * AHEAD), tid = threadIdx.x;
#pragma unroll 1
  for (int r = 0; r <= rounds; ++r) {
    const int word = r * kThreads * AHEAD + tid;   // the thread's first one
    u32x4 w[AHEAD];
    int i = head + word * N;
    uint32_t mine = 0;   // which bits are of the row
    if (r < rounds) {
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) w[j] = *reinterpret_cast<const u32x4 *>(row.p + head + (int64_t)min(word + j * kThreads, whole - 1) * N);
      const int words = (whole - word + kThreads - 1) / kThreads;
      mine = words <= 0 ? 0u : words >= AHEAD ? ~0u : (1u << words * N) - 1;
    } else {
      i = tid < head ? tid : behind + tid - head;
      w[0] = u32x4{0, 0, 0, 0};
      if (i < row.vocab) L::put(w[0], 0, row.p[i]), mine = 1;
    }
    uint32_t in = 0;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float v = L::value(w[j], e);
        in |= v >= low && v <= high ? 1u << (j * N + e) : 0u;
      }
    in &= mine;
    if (ragged) {
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float v = L::value(w[j], e);
          const int index = i + j * N * kThreads + e;
          in &= ~((v == high && index < from_index) || (v == low && index > to_index) ? 1u << (j * N + e) : 0u);
        }
    }
    if (__ballot(in != 0)) take(in, i, w);
  }
}
// The same by entry: f(index, key).
template <typename L, typename F>
__device__ INLINE inline void scan_each(const Row<L> &row, u64 from, u64 to, F f) {
  constexpr int N = L::n;
  scan(row, from, to, [&](uint32_t in, int i, u32x4 (&w)[32 / N]) INLINE {
#pragma unroll
    for (int j = 0; j < 32 / N; ++j) {
      uint32_t left = in >> (j * N) & ((1u << N) - 1);
#pragma unroll 1
      while (left) {
        const int e = __ffs(left) - 1;
        left &= left - 1;
        f(i + j * N * kThreads + e, key_of(L::pick(w[j], e)));
      }
    }
  });
}

template <typename L>
__global__ __launch_bounds__(kThreads) void choose_kernel(SampleArgs a, int count, int size) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  Shared &sm = *reinterpret_cast<Shared *>(lds);
  const int t = blockIdx.x, tid = threadIdx.x;
  const Slices s = slices_of(a, count, size);
  const int64_t at = (int64_t)t * count;
  const u64 of_mine = tid < count ? s.first[at + tid] : kNowhere;
  const Rules rules(a, t);
  const u64 first = all_min(sm, of_mine);
  const uint32_t top = key_at(first);
  if (first == kNowhere || rules.greedy()) {
    if (tid == 0) {
      a.ids[t] = first == kNowhere ? -1 : index_at(first);
      if (a.logprob) a.logprob[t] = first == kNowhere ? -INFINITY : 0.f;
    }
    return;
  }
  Row<L> row(a, t);
  row.heat(rules.t);
  const float top_bin = row.bin(of_key(top));
  auto bin_at = [&](uint32_t k) INLINE { return k >= top ? 0.f : top == kPosInf ? (float)kBins : top_bin - row.bin(of_key(k)); };
  const u64 end = place_of(kNegInf + 1, (1 << kIndexBits) - 1);   // the last place that counts
  const u64 index_mask = (1ull << kIndexBits) - 1, start = first & ~index_mask;   // the largest logit's first place
  auto found = [&](int id, uint32_t k, u64 total) INLINE {
    if (tid != 0) return;
    const double z = top == kPosInf ? 0. : ((double)of_key(k) - (double)of_key(top)) * row.inv_t;
    a.ids[t] = id;
    if (a.logprob) a.logprob[t] = (float)(z - log((double)total * 0x1p-43));
  };
  auto aim = [&](u64 total) INLINE {   // the running sum that the token's must reach
    const float u = rules.u > 0.f ? rules.u : 0.f;   // NaN and -0 too: `share` takes no sign
    return u < 1.f ? share(u, total, false) + 1 : total;
  };
  auto by_p = [&](u64 total) INLINE { return rules.p > 0.f ? max(share(rules.p, total, true), 1ull) : 1ull; };
  if (tid < count) {
    const u64 f = of_mine;
    const float d = f == kNowhere ? (float)kBins : fminf(bin_at(key_at(f)), (float)kBins);
    sm.slice_shift[tid] = (int)d;
    // a slice whose largest entry counts as 0 has nothing to choose, whatever its entries add up to
    sm.slice_share[tid] = d < kBins && row.mass(key_at(f), top) ? row.weight(key_at(f), top) : 0.;
  }
  if (tid < kBins) sm.row_mass[tid] = 0, sm.row_number[tid] = 0;
  if (tid <= kBins) sm.slice_mass[tid] = 0;
  __syncthreads();
  // The smallest key of bins 0 ... j: the first wave looks at 64 places at a time.
  auto key_from = [&](int j) INLINE {
    __syncthreads();
    if (tid < 64) {
      uint32_t lo = kNegInf + 1, hi = top;   // the answer is in [lo, hi]
      while (lo < hi) {
        const uint32_t step = (hi - lo + 63) / 64, mine = lo + step * tid;
        const u64 in = __ballot(mine >= hi || bin_at(mine) <= (float)j);
        const int n = __ffsll(in) - 1;   // the first place that is in; -1: behind all of them
        const uint32_t below = n < 0 ? lo + step * 63 + 1 : n == 0 ? lo : lo + step * (n - 1) + 1;
        if (n >= 0) hi = min(hi, lo + step * n);
        lo = min(below, hi);
      }
      if (tid == 0) sm.key = j < 0 ? top + 1 : lo;
    }
    __syncthreads();
    return uniform(sm.key);
  };
  // a weight of slice i in those of the row
  auto in_row = [&](u64 v, int i) INLINE { return (u64)((double)v * sm.slice_share[i] + 0.5); };
  auto heavy = [&](u64 place) INLINE { return !rules.by_min || row.weight(key_at(place), top) >= (double)rules.least; };
  // The places in [lo, hi] into the list, in no order, and their weights; returns how many.
  auto gather = [&](u64 lo, u64 hi) INLINE {
    __syncthreads();
    if (tid == 0) sm.listed = 0;
    __syncthreads();
    scan(row, lo, hi, [&](uint32_t in, int i, u32x4 (&)[32 / L::n]) INLINE {
      const int n = __popc(in), upto = wave_scan(n);
      int slot = 0;
      if ((tid & 63) == 63) slot = atomicAdd(&sm.listed, upto);
      slot = __builtin_amdgcn_readlane(slot, 63) + upto - n;
#pragma unroll 1
      for (; in; in &= in - 1, ++slot) {
        const int bit = __ffs(in) - 1;
        if (slot < kList) sm.list[slot] = i + bit / L::n * (L::n * kThreads) + bit % L::n;
      }
    });
    __syncthreads();
    const int m = uniform(min(sm.listed, kList));
#pragma unroll 4
    for (int i = tid; i < m; i += kThreads) {
      const int index = (int)sm.list[i];
      const uint32_t k = row.key(index);
      sm.list[i] = place_of(k, index);
      sm.mass[i] = row.mass(k, top);
    }
    __syncthreads();
    return m;
  };
  auto listed_sum = [&](int m, u64 border) INLINE {
    u64 v = 0;
    for (int i = tid; i < m; i += kThreads) v += sm.list[i] <= border ? sm.mass[i] : 0;
    return all_sum(sm, v);
  };

  const bool masses = rules.masses();
  u64 last = end;        // the last place by k and p
  int edge = kBins;      // entries of the bins before it stay whole
  int edge_listed = -1;  // entries of the list, if it has all of bin `edge`
  if (rules.counts()) {
    {
      const int j = tid % kBins, group = tid / kBins;
      u64 m = 0;
      uint32_t c = 0;
      constexpr int GROUPS = kThreads / kBins, AHEAD = 8;
      for (int i0 = group; i0 < count; i0 += GROUPS * AHEAD) {
        u64 mv[AHEAD];
        uint32_t cv[AHEAD];
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) {
          const int i = i0 + GROUPS * b, from = i < count ? j - sm.slice_shift[i] : -1;
          mv[b] = cv[b] = 0;
          if (from >= 0) {
            cv[b] = s.number[(at + i) * kBins + from];
            if (masses) mv[b] = s.mass[(at + i) * kBins + from];
          }
        }
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) {
          c += cv[b];
          if (mv[b]) m += in_row(mv[b], i0 + GROUPS * b);
        }
      }
      if (c) atomicAdd(&sm.row_number[j], c);
      if (m) atomicAdd(&sm.row_mass[j], m);
    }
    __syncthreads();
    const u64 all = masses ? all_sum(sm, tid < kBins ? sm.row_mass[tid] : 0) : 0;
    // the bin up to which a number or a weight is reached (kBins if it is not)
    auto bin_of = [&](bool mass, u64 target) INLINE {
      cross(sm, tid >= kBins ? 0 : mass ? sm.row_mass[tid] : sm.row_number[tid], 0, target);
      return uniform((int)min(sm.at, (u64)kBins));
    };
    int upto = rules.by_k ? bin_of(false, rules.k) : kBins;
    if (rules.by_p && !rules.by_k) {
      // a little further, since a bin's weight and its entries' are rounded apart
      const u64 want = by_p(all);
      upto = bin_of(true, min(all, want + (want >> 36)));
    }
    int min_bin = kBins;   // one bin further than that of the smallest weight's logit, which is rounded
    if (rules.by_min) {
      const double z = (double)of_key(top) + log((double)rules.least) / row.inv_t;
      float v = (float)z;
      if ((double)v > z) v = of_key(key_of(v) - 1);
      min_bin = (int)fminf(bin_at(key_of(v)) + 1.f, (float)kBins);
      if (!(rules.by_k && rules.by_p)) upto = min(upto, min_bin);   // p takes its share of all that k leaves
    }
    if (all_sum(sm, tid <= upto && tid < kBins ? sm.row_number[tid] : 0) <= kList) {
      last = place_of(key_from(min(upto, kBins - 1)), index_mask);   // of the list: the searches' ranges end with it
      const int m = gather(start, last);
      u64 total = all;
#pragma unroll 1
      for (int by = rules.by_k ? BY_NUMBER : rules.by_p ? BY_WEIGHT : BY_INDEX;; ++by) {
        if (by == BY_WEIGHT && !rules.by_p) continue;
        u64 lo = first, hi = last, target = rules.k;
        if (by == BY_WEIGHT) {
          if (rules.by_k) total = listed_sum(m, last);
          target = by_p(total);
        } else if (by == BY_INDEX) {
          for (int i = tid; i < m; i += kThreads)
            if (sm.list[i] > last || !heavy(sm.list[i])) sm.mass[i] = 0;
          __syncthreads();
          total = listed_sum(m, kNowhere);
          target = aim(total);
          lo = 0, hi = a.vocab - 1;
        }
        const u64 border = find(sm, m, by, lo, hi, 0, target);
        if (by == BY_INDEX) return found((int)border, row.key((int)border), total);
        last = border;
      }
    }

    // Too many entries.  The last place by k, and then by p, among those of its bin; if they do not fit into the list
    // either, their places are narrowed down to 2^-9 a time by their numbers and weights.
    auto border = [&](u64 lo, u64 hi, u64 before, u64 number, bool one, u64 target) INLINE {
      while (number > kList) {
        const u64 range = hi - lo;
        const int bits = 64 - __clzll(range), shift = bits > kDigit ? bits - kDigit : 0;
        __syncthreads();
        sm.bin[tid] = 0, sm.bin_number[tid] = 0;
        __syncthreads();
        scan_each(row, lo, hi, [&](int i, uint32_t k) INLINE {
          const u64 place = place_of(k, i);
          atomicAdd(&sm.bin_number[(place - lo) >> shift], 1u);
          if (!one) atomicAdd(&sm.bin[(place - lo) >> shift], row.mass(k, top));
        });
        __syncthreads();
        cross(sm, one ? sm.bin_number[tid] : sm.bin[tid], before, target);
        const u64 bin = uniform(sm.at);
        if (bin == kNowhere) return hi;   // not reached
        before = uniform(sm.before);
        number = uniform(sm.bin_number[bin]);
        lo += bin << shift;
        hi = min(hi, lo + (1ull << shift) - 1);
      }
      const int m = gather(lo, hi);
      edge_listed = m;
      return find(sm, m, one ? BY_NUMBER : BY_WEIGHT, lo, hi, before, target);
    };
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      const bool one = pass == 0;
      if (!(one ? rules.by_k : rules.by_p)) continue;
      u64 target = rules.k;
      if (!one) {
        u64 sum = all;
        if (rules.by_k) {
          u64 v = 0;
          scan_each(row, start, last, [&](int, uint32_t k) INLINE { v += row.mass(k, top); });
          sum = all_sum(sm, v);
        }
        target = by_p(sum);
      }
      u64 lo = start, hi = last, before = 0, number = kNowhere;
      if (one || masses) {
        const int bin = bin_of(!one, target);
        if (bin == kBins) continue;   // not reached: all stay
        before = all_sum(sm, tid >= bin ? 0 : one ? sm.row_number[tid] : sm.row_mass[tid]);
        lo = place_of(key_from(bin - 1) - 1, 0);
        hi = place_of(key_from(bin), index_mask);
        number = uniform(sm.row_number[bin]);
      }
      last = min(last, border(lo, hi, before, number, one, target));
      if (number > kList) edge_listed = -1;
    }
    edge = last >= end ? kBins : (int)fminf(bin_at(key_at(last)), (float)kBins);
    if (rules.by_min) edge = min(edge, max(0, min_bin - 2)), edge_listed = -1;
    // (the list is that of the smaller of two borders, or has been given up)
    if (rules.by_k && rules.by_p) edge_listed = -1;
  }

  // The slices' sums: whole bins, and what stays of the others' entries.
  __syncthreads();
  if (!rules.counts()) {
    if (tid < count && sm.slice_share[tid] > 0.) sm.slice_mass[tid] = in_row(s.sum[at + tid], tid);
  } else {
    const int whole = masses ? edge : 0;
    constexpr int AHEAD = 4;   // a wave takes a slice's bins, and asks for those of four slices together
    for (int i0 = tid / 64; i0 < count && whole; i0 += kThreads / 64 * AHEAD) {
      u64 v[AHEAD][kBins / 64];
#pragma unroll
      for (int b = 0; b < AHEAD; ++b)
#pragma unroll
        for (int c = 0; c < kBins / 64; ++c) {
          const int i = i0 + kThreads / 64 * b, from = tid % 64 + 64 * c;
          v[b][c] = i < count && from + sm.slice_shift[i] < whole ? s.mass[(at + i) * kBins + from] : 0;
        }
#pragma unroll
      for (int b = 0; b < AHEAD; ++b) {
        const int i = i0 + kThreads / 64 * b;
        if (i >= count) break;   // the same for the whole wave
        u64 sum = 0;
#pragma unroll
        for (int c = 0; c < kBins / 64; ++c) sum += v[b][c] ? in_row(v[b][c], i) : 0;
        sum = wave_sum(sum);
        if (tid % 64 == 0) sm.slice_mass[i] = sum;
      }
    }
    __syncthreads();
    if (masses && edge_listed >= 0) {
      for (int i = tid; i < edge_listed; i += kThreads)
        if (sm.list[i] <= last) atomicAdd(&sm.slice_mass[(index_at(sm.list[i]) + row.off) / s.size], sm.mass[i]);
    } else if (whole < kBins) {
      const uint32_t to = key_from(whole - 1) - 1;
      if (to > kNegInf) scan_each(row, place_of(to, 0), last, [&](int i, uint32_t k) INLINE {
        if (heavy(place_of(k, i))) atomicAdd(&sm.slice_mass[(i + row.off) / s.size], row.mass(k, top));
      });
    }
  }
  __syncthreads();
  const u64 total = all_sum(sm, tid < count ? sm.slice_mass[tid] : 0), target = aim(total);
  cross(sm, tid < count ? sm.slice_mass[tid] : 0, 0, target);
  const int slice = uniform((int)min(sm.at, (u64)count - 1));
  const u64 before = uniform(sm.before);
  __syncthreads();
  // Within the slice; its entries' sum may miss the slice's by what was rounded: then the last one that weighs something
  // (there is one: the slice's largest is kept where any of its entries is), which is the one that u >= 1 asks for anyway.
  const int from = slice * s.size - row.off, to = min(from + s.size, a.vocab);
#pragma unroll 4
  for (int i = tid; i < to - from; i += kThreads) {
    const uint32_t k = from + i < 0 ? 0u : row.key(from + i);
    const u64 place = place_of(k, from + i);
    sm.mass[i] = k > kNegInf && place <= last && heavy(place) ? row.mass(k, top) : 0;
  }
  __syncthreads();
  int id = from + locate(sm, to - from, before, rules.u >= 1.f ? kNowhere : target, [&](int i) INLINE { return sm.mass[i]; });
  if (uniform(sm.at) == kNowhere) {
    u64 behind = kNowhere;
    for (int i = tid; i < to - from; i += kThreads)
      if (sm.mass[i]) behind = ~(u64)(from + i);
    behind = all_min(sm, behind);
    id = behind == kNowhere ? index_at(first) : (int)~behind;
  }
  found(id, row.key(id), total);
}

template <typename L>
hipError_t launch_logits(const SampleArgs &a, hipStream_t s) {
  const int threads = slice_threads(a.n, a.vocab), count = slice_count(threads, a.vocab);
  const dim3 g((uint32_t)count * (uint32_t)a.n);
  if (threads == 256)
    hipLaunchKernelGGL((weigh_kernel<L, 256>), g, dim3(256), 0, s, a, count);
  else
    hipLaunchKernelGGL((weigh_kernel<L, 512>), g, dim3(512), 0, s, a, count);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(choose_kernel<L>, dim3(a.n), dim3(kThreads), sizeof(Shared), s, a, count, threads * kPer);
  return hipGetLastError();
}

}  // namespace

bool sample_fits(int n, int vocab) {
  const int threads = slice_threads(n, vocab);
  return launch_fits((int64_t)n * slice_count(threads, vocab), threads) && launch_fits(n, kThreads);
}

// Beyond kShortSlices at least what they take, so that a call's workspace is enough for every smaller one.
int64_t sample_workspace_bytes(int n, int vocab) {
  const int threads = slice_threads(n, vocab);
  const int64_t count = (int64_t)n * slice_count(threads, vocab), all = threads == 256 ? count : std::max<int64_t>(count, kShortSlices);
  return (all * (16 + kBins * 12) + 15) / 16 * 16;
}

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) { return a.f32 ? launch_logits<F32>(a, s) : launch_logits<B16>(a, s); }

}  // namespace oes
