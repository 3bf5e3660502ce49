// y = res + scale * act(x . W^T + bias) for bf16 weights.
//
// A workgroup makes a tile of BN rows of W times BM tokens by v_mfma_f32_16x16x32_bf16 (A = weights, B =
// tokens: a lane's accumulators are 4 rows of W for one token).  WK groups of WN x WM waves take every WK-th
// step of 64 of K; each has S buffers of a step in LDS, filled by loads that go there directly, up to S steps
// ahead.  A group of one wave waits for its own loads alone; others meet at a barrier a step.  The groups' sums
// are joined in LDS, in order.
//
// Few tokens are bound by reading W: 16 tokens of 100003 x 4096 128 us, 6.5 TB/s; 24 tokens of SwiGLU 2 x 2048 x 7168 16.4
// us (3.6 TB/s; 11.4 where W is still in the memory-side cache).  Small tiles with K cut over a workgroup's waves then keep
// all CUs reading.  Many are bound by the matrix units: 4096 tokens of 7168 x 7168 364 us in a graph, 1.15 PFLOP/s (368 - 386 by
// calls and traces), by tiles of 256 x 256, each of whose operand values in LDS feeds 8 or 4 products a wave.  Between them
// (333 tokens of 2880 x 2880 18.4 us, 23.2 from memory) there are fewer tiles than CUs, and the time is that of one tile's 45
// steps.
//
// In LDS a row of a step is 8 pieces of 16 bytes, piece c at c ^ f(row), f such that the 16 rows that a read takes
// spread over all banks.  Where a wave has 32 rows of W, block i = 2 p + b takes rows 32 p + 8 (r / 4) + 4 b + r % 4, so
// that a lane holds 8 adjacent columns of y.  SwiGLU puts rows of g where b = 0 and the same rows of u where b = 1; of
// 16 rows the first 8 are of g and the others of u, and lane i finds its u in lane i + 32's sums.

#include <algorithm>
#include <utility>

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __attribute__((aligned(16))) const uint32_t nothing[4] = {0, 0, 0, 0};

// Until all but N loads have arrived and the wave's reads of LDS are done; then, BARRIER, until every wave has come here.
template <int N, bool BARRIER>
__device__ inline void wait_loads() {
  if (BARRIER)
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
  else
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ inline float activate(int act, float v) {
  switch (act) {
    case OES_ACT_SIGMOID: return sigmoid(v);
    case OES_ACT_SILU: return v * sigmoid(v);
    // v / 2 (1 + tanh(t)) = v / (1 + exp(-2 t))
    case OES_ACT_GELU: return v * sigmoid(1.5957691216057308f * fmaf(0.044715f * v * v, v, v));
    default: return v;
  }
}

template <int V>
struct __attribute__((packed, aligned(4))) Columns32 { float v[V]; };
template <int V>
struct __attribute__((packed, aligned(2))) Columns16 { uint32_t v[V / 2]; };

// V adjacent columns of the residual of one token; 0 where there is none
template <int V>
__device__ inline void residual(const DenseArgs &a, int64_t t, int col, float (&v)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = 0.f;
  const int count = min(V, a.N - col);
  if (!a.res || t >= a.n || count <= 0) return;
  if (a.y_f32) {
    const float *res = static_cast<const float *>(a.res) + t * a.res_row + col;
    if (count == V) {
      const Columns32<V> r = *reinterpret_cast<const Columns32<V> *>(res);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = r.v[e];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < count) v[e] = res[e];
    }
  } else {
    const uint16_t *res = static_cast<const uint16_t *>(a.res) + t * a.res_row + col;
    if (count == V) {
      const Columns16<V> r = *reinterpret_cast<const Columns16<V> *>(res);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) v[2 * e] = bf16_lo(r.v[e]), v[2 * e + 1] = bf16_hi(r.v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < count) v[e] = bf16f(res[e]);
    }
  }
}

// the epilogue of V adjacent columns of one token
template <int V, bool SWIGLU>
__device__ inline void finish(const DenseArgs &a, int64_t t, int col, const float (&z)[V], const float (&up)[V], const float (&res)[V]) {
  const int count = min(V, a.N - col);
  if (t >= a.n || count <= 0) return;
  float v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float s = z[e], w = up[e];
    if (a.bias && e < count) {
      s += bf16f(a.bias[col + e]);
      if (SWIGLU) w += bf16f(a.bias[a.N + col + e]);
    }
    v[e] = fmaf(a.scale, SWIGLU ? s * sigmoid(s) * w : activate(a.act, s), res[e]);
  }
  if (a.y_f32) {
    float *y = static_cast<float *>(a.y) + t * a.y_row + col;
    if (count == V) {
      Columns32<V> o;
#pragma unroll
      for (int e = 0; e < V; ++e) o.v[e] = v[e];
      *reinterpret_cast<Columns32<V> *>(y) = o;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < count) y[e] = v[e];
    }
  } else {
    uint16_t *y = static_cast<uint16_t *>(a.y) + t * a.y_row + col;
    if (count == V) {
      Columns16<V> o;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) o.v[e] = f2bf16_pair(v[2 * e], v[2 * e + 1]);
      *reinterpret_cast<Columns16<V> *>(y) = o;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < count) y[e] = (uint16_t)f2bf16(v[e]);
    }
  }
}

template <int... I, typename F>
__device__ inline void each_step(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ inline void step_loop(F f) {   // f(0) ... f(N - 1), each known to the compiler
  each_step(std::make_integer_sequence<int, N>{}, f);
}

// What a launch is cut into: tiles_n x tiles_m tiles, `band` of tokens side by side.
struct Tiles {
  int tiles_n, tiles_m, band;
};

// Workgroup ids go round the 8 XCDs; each takes a run of adjacent tiles, so that its L2 holds what they share.
__device__ inline void tile_of(const Tiles &p, int &tn, int &tm) {
  const int id = blockIdx.x, count = gridDim.x, xcd = id & 7, each = count >> 3, more = count & 7;
  const int at = xcd * each + min(xcd, more) + (id >> 3);
  const int per = p.band * p.tiles_n, b = at / per, left = at - b * per, wide = min(p.band, p.tiles_m - b * p.band);
  tn = left / wide;
  tm = b * p.band + left - tn * wide;
}

template <int BM_, int BN_, int WM_, int WN_, int WK_, int S_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, WK = WK_, S = S_;
  static constexpr int G = WM * WN, threads = 64 * G * WK;
  static constexpr int TM = BM / WM, TN = BN / WN;   // a wave's tokens and rows
  static constexpr int groups = (BM + BN) / 8;       // of 8 rows, one load each
  static constexpr int loads = (groups + G - 1) / G; // a wave's loads of a step
  static constexpr int step_bytes = (BM + BN) * 128;
  static constexpr int join_bytes = WK > 1 ? WK * BM * BN * 4 : 0;
  static constexpr int lds = WK * S * step_bytes > join_bytes ? WK * S * step_bytes : join_bytes;
  static constexpr bool wide = TN % 32 == 0;         // 8 adjacent columns a lane
  static_assert(TM % 16 == 0 && TN % 16 == 0 && lds <= 160 << 10 && threads <= 1024 && S >= 2 && (S - 1) * WK * 128 < 4096, "shape");
};

// ONCE: there is one tile of tokens, so that each row of W is read once, and caches need not keep it.  us with and without
// the hint, weights from memory: 16 tokens 512 x 2048 4.5 and 5.3, 7168 x 7168 18.8 and 23.2, 100003 x 4096 125 and 149; 64
// tokens 7168 x 7168 28.8 and 32.6.
template <typename P, bool SWIGLU, bool ONCE>
__global__ __launch_bounds__(P::threads) void dense_kernel(DenseArgs a, Tiles tiles) {
  extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
  constexpr int NW = P::TN / 16, NX = P::TM / 16;   // a wave's blocks
  static_assert(!SWIGLU || P::wide || P::WK > 1, "g and u of 16 rows meet in LDS");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  const int wk = wave / P::G, wg = P::G > 1 ? wave % P::G : 0, wn = wg % P::WN, wm = wg / P::WN;
  int tn, tm;
  tile_of(tiles, tn, tm);
  const int n0 = tn * P::BN, t0 = tm * P::BM, steps = (a.K + 63) / 64;

  // A wave's load j takes 8 rows: W's first, then x's; past the last row the last one again (and past the last
  // group, so that every wave has as many loads to wait for).
  const uint8_t *src[P::loads];
  uint32_t whole = 0;   // bit j: the lane's piece of the last step is within K
#pragma unroll
  for (int j = 0; j < P::loads; ++j) {
    const int g = min(wg * P::loads + j, P::groups - 1), lr = lane >> 3, h = (lr >> 1 & 1) << 2;
    int piece;
    if (g < P::BN / 8) {
      piece = (lane & 7) ^ (h | (P::wide ? g >> 1 & 1 : g & 1) * 3);
      int64_t row;
      if (SWIGLU && P::wide)
        row = min((n0 >> 1) + 4 * g + (lr & 3), a.N - 1) + (lr >> 2) * (int64_t)a.N;
      else if (SWIGLU)
        row = min((n0 >> 1) + 8 * (g >> 1) + lr, a.N - 1) + (g & 1) * (int64_t)a.N;
      else
        row = min(n0 + 8 * g + lr, a.N - 1);
      src[j] = reinterpret_cast<const uint8_t *>(a.w + row * a.w_row);
    } else {
      const int gx = g - P::BN / 8;
      piece = (lane & 7) ^ (h | (gx & 1) * 3);
      src[j] = reinterpret_cast<const uint8_t *>(a.x + (int64_t)min(t0 + 8 * gx + lr, a.n - 1) * a.x_row);
    }
    src[j] += wk * 128 + piece * 16;
    whole |= (uint32_t)(64 * (steps - 1) + 8 * piece < a.K) << j;
  }
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds_addr(sm) + wk * P::S * P::step_bytes);
  auto to = [&](int buf, int j) { return ring + buf * P::step_bytes + min(wg * P::loads + j, P::groups - 1) * 1024; };
  auto load = [&](int i) {   // the group's i-th step, src at it
    const bool last = i * P::WK + wk == steps - 1;
    step_loop<P::loads>([&](auto J) {
      constexpr int j = J;
      const uint8_t *from = src[j];
      if (last && !(whole >> j & 1)) from = reinterpret_cast<const uint8_t *>(nothing);
      if (ONCE && wg * P::loads + j < P::BN / 8)
        load_to_lds<0, true>(from, to(i % P::S, j));
      else
        load_to_lds<0>(from, to(i % P::S, j));
      src[j] += P::WK * 128;
    });
  };

  f32x4 acc[NW][NX];
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int j = 0; j < NX; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // where the lane's rows of block 0 start, and its piece of the step's first half (the second's is 64 bytes off)
  const int f = (r >> 1 & 1) << 2 | (r >> 3) * 3, p0 = (q ^ f) * 16;
  const uint8_t *mine = sm + wk * P::S * P::step_bytes;
  const int w_at = (wn * P::TN + (P::wide ? 8 * (r >> 2) + (r & 3) : r)) * 128 + p0;
  const int x_at = (P::BN + wm * P::TM + r) * 128 + p0;
  struct Half { bf16x8 w[NW], x[NX]; };
  auto read = [&](int buf, int h, Half &v) {
    const uint8_t *wb = mine + buf * P::step_bytes + (w_at ^ 64 * h), *xb = mine + buf * P::step_bytes + (x_at ^ 64 * h);
#pragma unroll
    for (int j = 0; j < NX; ++j) v.x[j] = *reinterpret_cast<const bf16x8 *>(xb + 16 * j * 128);
#pragma unroll
    for (int k = 0; k < NW; ++k)
      v.w[k] = *reinterpret_cast<const bf16x8 *>(wb + (P::wide ? 32 * (k / 2) + 4 * (k & 1) : 16 * k) * 128);
  };
  auto multiply = [&](const Half &v) {
#pragma unroll
    for (int k = 0; k < NW; ++k)
#pragma unroll
      for (int j = 0; j < NX; ++j) acc[k][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v.w[k], v.x[j], acc[k][j], 0, 0, 0);
  };

  // The first half of a step is in registers when its products begin, and the second is read under them; then, all
  // being read, its buffer takes the step S further on, and the next step's first half is read under the second half's
  // products.
  constexpr int S = P::S;
  constexpr bool meet = P::G > 1;
  const int rounds = (steps + P::WK - 1) / P::WK, own = (steps - wk + P::WK - 1) / P::WK, all = steps / P::WK;
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (i < own) load(i);
  if (S <= own)
    wait_loads<(S - 1) * P::loads, meet>();
  else
    wait_loads<0, meet>();
  Half a0, a1;
  if (own > 0) read(0, 0, a0);
  int i = 0;
  for (; i + 2 * S <= all - 1; i += S) {   // no last step among the ones that these S load
    step_loop<S>([&](auto U) {
      constexpr int u = U;
      read(u, 1, a1);
      multiply(a0);
      __builtin_amdgcn_sched_barrier(0);
      wait_loads<(S - 2) * P::loads, meet>();
      step_loop<P::loads>([&](auto J) {
        constexpr int j = J;
        if (ONCE && wg * P::loads + j < P::BN / 8)
          load_to_lds<u * P::WK * 128, true>(src[j], to(u, j));
        else
          load_to_lds<u * P::WK * 128>(src[j], to(u, j));
      });
      read((u + 1) % S, 0, a0);
      multiply(a1);
    });
#pragma unroll
    for (int j = 0; j < P::loads; ++j) src[j] += S * P::WK * 128;
  }
  for (; i < rounds; ++i) {
    if (i < own) {
      read(i % S, 1, a1);
      multiply(a0);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (i + S - 1 < own)
      wait_loads<(S - 2) * P::loads, meet>();
    else
      wait_loads<0, meet>();
    if (i + S < own) load(i + S);
    if (i + 1 < own) read((i + 1) % S, 0, a0);
    if (i < own) multiply(a1);
  }

  // Units of one token block and 32 (16) rows: V adjacent columns a lane.
  constexpr int UW = P::wide ? NW / 2 : NW, B = P::wide || SWIGLU ? 2 : 1, V = SWIGLU || !P::wide ? 4 : 8;
  auto token = [&](int j) { return (int64_t)t0 + wm * P::TM + 16 * j + r; };
  auto column = [&](int p) {
    const int row = n0 + wn * P::TN + (P::wide ? 32 : 16) * p;
    if (!SWIGLU) return row + V * q;
    // g and u of 16 rows: lanes from 32 on have sums of u, which lane - 32 takes
    return !P::wide && lane >= 32 ? a.N : (row >> 1) + 4 * q;
  };
  auto put = [&](int p, int j, const f32x4 (&v)[B], const float (&res)[V]) {
    float z[V], up[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      z[e] = v[SWIGLU ? 0 : e / 4][e % 4];
      up[e] = v[B - 1][e % 4];
    }
    finish<V, SWIGLU>(a, token(j), column(p), z, up, res);
  };
  if (P::WK == 1) {
#pragma unroll
    for (int p = 0; p < UW; ++p) {
      float res[NX][V];   // all asked for before the first store, which they may not pass (y may be res)
#pragma unroll
      for (int j = 0; j < NX; ++j) residual(a, token(j), column(p), res[j]);
#pragma unroll
      for (int j = 0; j < NX; ++j) {
        f32x4 v[B];
#pragma unroll
        for (int k = 0; k < B; ++k) v[k] = acc[(NW / UW) * p + k][j];
        put(p, j, v, res[j]);
      }
    }
  } else {
    f32x4 *part = reinterpret_cast<f32x4 *>(sm);   // [WK][G][NX][NW][64]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NX; ++j)
#pragma unroll
      for (int k = 0; k < NW; ++k) part[((wave * NX + j) * NW + k) * 64 + lane] = acc[k][j];
    __syncthreads();
    for (int u = wk; u < UW * NX; u += P::WK) {
      const int p = u % UW, j = u / UW;
      float res[V];
      residual(a, token(j), column(p), res);
      f32x4 v[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int block = P::wide ? 2 * p + k : p, from = SWIGLU && !P::wide ? (lane & 31) + 32 * k : lane;
        v[k] = part[((wg * NX + j) * NW + block) * 64 + from];
        for (int g = 1; g < P::WK; ++g) v[k] += part[(((g * P::G + wg) * NX + j) * NW + block) * 64 + from];
      }
      put(p, j, v, res);
    }
  }
}

// One token.  Two columns of y a workgroup (four rows of W for SwiGLU), 4 waves that take every fourth piece of 512 of K:
// all of a small matrix is asked for at once, and no product waits for x to be in LDS.  us, weights from memory, and by
// tiles (for 3 tokens): 512 x 2048 3.1 and 4.2, 5120 x 2048 6.0 and 6.6, 7168 x 7168 17.6 and 17.3, 100003 x 4096 111 (7.35
// TB/s) and 120.  Two tokens so were no faster than the tiles: 5120 x 2048 7.2, 100003 x 4096 125.
template <bool SWIGLU>
__global__ __launch_bounds__(256) void row_kernel(DenseArgs a) {
  constexpr int R = SWIGLU ? 4 : 2;   // rows of g and u in turn
  __shared__ float part[4][R];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = 2 * blockIdx.x;
  const uint16_t *w[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    w[i] = a.w + (min(col + (SWIGLU ? i >> 1 : i), a.N - 1) + (SWIGLU && (i & 1) ? (int64_t)a.N : 0)) * a.w_row;
  float sum[R];
#pragma unroll
  for (int i = 0; i < R; ++i) sum[i] = 0.f;
  constexpr int AHEAD = 2;
  for (int k0 = wave * 512; k0 < a.K; k0 += 2048 * AHEAD) {
    u32x4 wv[AHEAD][R], xv[AHEAD];
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) {
      const int k = k0 + 2048 * s + 8 * lane;
      xv[s] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < R; ++i) wv[s][i] = u32x4{0, 0, 0, 0};
      if (k < a.K) {
#pragma unroll
        for (int i = 0; i < R; ++i) wv[s][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(w[i] + k));
        xv[s] = *reinterpret_cast<const u32x4 *>(a.x + k);
      }
    }
#pragma unroll
    for (int s = 0; s < AHEAD; ++s)
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[i] = fmaf(bf16_lo(wv[s][i][e]), bf16_lo(xv[s][e]), sum[i]);
          sum[i] = fmaf(bf16_hi(wv[s][i][e]), bf16_hi(xv[s][e]), sum[i]);
        }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
#pragma unroll
    for (int d = 32; d; d >>= 1) sum[i] += __shfl_xor(sum[i], d, 64);
    if (lane == 0) part[wave][i] = sum[i];
  }
  __syncthreads();
  if (threadIdx.x > 0) return;
  float z[2], up[2], res[2];
  residual(a, 0, col, res);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int i = SWIGLU ? 2 * c : c, u = SWIGLU ? i + 1 : i;
    z[c] = part[0][i] + part[1][i] + part[2][i] + part[3][i];
    up[c] = part[0][u] + part[1][u] + part[2][u] + part[3][u];
  }
  finish<2, SWIGLU>(a, 0, col, z, up, res);
}

template <typename P>
Tiles tiles_of(const DenseArgs &a) {
  Tiles t;
  t.tiles_n = (int)(((a.act == OES_ACT_SWIGLU ? 2ll : 1ll) * a.N + P::BN - 1) / P::BN);
  t.tiles_m = (a.n + P::BM - 1) / P::BM;
  t.band = std::min(4, t.tiles_m);
  return t;
}

template <typename P>
hipError_t launch_shape(const DenseArgs &a, hipStream_t s) {
  const Tiles t = tiles_of<P>(a);
  const dim3 g((uint32_t)t.tiles_n * (uint32_t)t.tiles_m), b(P::threads);
  const bool swiglu = a.act == OES_ACT_SWIGLU;
  // (32 x 16 is not taken for one tile of tokens: 16 x 32 makes as many workgroups then, and theirs cost less.)
  if constexpr (P::BM <= 64 && !(P::BM == 32 && P::BN == 16)) {
    if (t.tiles_m == 1) {
      if (swiglu)
        hipLaunchKernelGGL((dense_kernel<P, true, true>), g, b, P::lds, s, a, t);
      else
        hipLaunchKernelGGL((dense_kernel<P, false, true>), g, b, P::lds, s, a, t);
      return hipGetLastError();
    }
  }
  if (swiglu)
    hipLaunchKernelGGL((dense_kernel<P, true, false>), g, b, P::lds, s, a, t);
  else
    hipLaunchKernelGGL((dense_kernel<P, false, false>), g, b, P::lds, s, a, t);
  return hipGetLastError();
}

// The shapes, and what a round of 256 workgroups of each costs, in us at K = 7168 (4096 rows of W, or as many tokens as
// make 224 - 256 tiles; the smallest read W from memory).  A call takes the shape whose rounds cost least.  Over 146 sizes
// (512 ... 20000 rows, K 2048 ... 7168, 4 ... 4096 tokens) that takes 0.9 % more than the fastest of fifteen shapes, in the
// geometric mean; 5 % more at nine of them, and the most where shapes of other proportions would need fewer rounds: 384 x
// 20000 x 4096 84 us (128 x 256: 71), 192 x 7168 x 7168 54 (128 x 64: 46), 192 x 2 * 2880 x 2880 23.5 (128 x 64: 20.5).
template <typename F>
auto with_shape(const DenseArgs &a, F f) {
  const int cost[] = {130, 145, 155, 190, 245, 360, 515, 690, 1040, 1750};
  const auto rounds = [&](Tiles t) { return ((int64_t)t.tiles_n * t.tiles_m + 255) / 256; };
  typedef Shape<16, 16, 1, 1, 8, 3> P0;
  typedef Shape<16, 32, 1, 1, 4, 3> P1;
  typedef Shape<32, 16, 1, 1, 4, 3> P2;
  typedef Shape<32, 32, 1, 1, 4, 3> P3;
  typedef Shape<64, 32, 2, 1, 4, 3> P4;
  typedef Shape<64, 64, 2, 2, 2, 3> P5;
  typedef Shape<64, 128, 2, 4, 1, 4> P6;
  typedef Shape<128, 128, 2, 4, 1, 3> P7;
  typedef Shape<256, 128, 4, 2, 1, 3> P8;
  typedef Shape<256, 256, 2, 4, 1, 2> P9;
  const int64_t r[] = {rounds(tiles_of<P0>(a)), rounds(tiles_of<P1>(a)), rounds(tiles_of<P2>(a)), rounds(tiles_of<P3>(a)),
                       rounds(tiles_of<P4>(a)), rounds(tiles_of<P5>(a)), rounds(tiles_of<P6>(a)), rounds(tiles_of<P7>(a)),
                       rounds(tiles_of<P8>(a)), rounds(tiles_of<P9>(a))};
  int best = 0;
  for (int i = 1; i < 10; ++i)
    if (r[i] * cost[i] < r[best] * cost[best]) best = i;
  switch (best) {
    case 0: return f(P0{});
    case 1: return f(P1{});
    case 2: return f(P2{});
    case 3: return f(P3{});
    case 4: return f(P4{});
    case 5: return f(P5{});
    case 6: return f(P6{});
    case 7: return f(P7{});
    case 8: return f(P8{});
    default: return f(P9{});
  }
}

}  // namespace

bool linear_bf16_fits(const DenseArgs &a) {
  if (a.n == 1) return true;   // 2^21 workgroups at most
  return with_shape(a, [&](auto p) {
    const Tiles t = tiles_of<decltype(p)>(a);
    return launch_fits((int64_t)t.tiles_n * t.tiles_m, decltype(p)::threads);
  });
}

hipError_t launch_linear_bf16(const DenseArgs &a, hipStream_t s) {
  if (a.n == 1) {
    const dim3 g((a.N + 1) / 2), b(256);
    if (a.act == OES_ACT_SWIGLU)
      hipLaunchKernelGGL(row_kernel<true>, g, b, 0, s, a);
    else
      hipLaunchKernelGGL(row_kernel<false>, g, b, 0, s, a);
    return hipGetLastError();
  }
  return with_shape(a, [&](auto p) { return launch_shape<decltype(p)>(a, s); });
}

}  // namespace oes
