// Norms between the blocks: r = res + scale * act(gate) * post(x), y = pre(r).
//
// Bound by memory (8192 x 4096 with a bf16 residual 50.5 us, 5.3 TB/s; 3001 x 7168 with both norms, a gate and an fp32
// residual 55.5 us, 4.7 TB/s; one row of 2048 2.7 us in a graph, latency): a row is read once into registers, 8 values a piece
// of 16 (fp32: 32) bytes, and stays there through both norms.  Up to 64 lanes of a wave have a row, whose sums meet by lane
// exchanges, or a workgroup of just as many waves as it takes, whose sums meet in LDS (in order, so that a row's result
// depends on nothing else).  Squares are taken of differences from the mean, which a sum of squares less the
// squared mean would lose for rows far from 0.

#include <algorithm>

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

// 8 values as they stand in memory: bf16, or (F32, and f32 says so) fp32
template <bool F32>
struct Piece {
  u32x4 w[F32 ? 2 : 1];
  __device__ void load(const void *p, int64_t at, bool f32) {
    const u32x4 *q = reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(p) + at * (F32 && f32 ? 4 : 2));
    w[0] = q[0];
    if (F32 && f32) w[F32] = q[1];
  }
  __device__ float value(int e, bool f32) const {
    return F32 && f32 ? __uint_as_float(w[F32 ? e / 4 : 0][e % 4]) : (e & 1 ? bf16_hi(w[0][e / 2]) : bf16_lo(w[0][e / 2]));
  }
};

__device__ inline u32x4 packed(const float (&v)[8]) {
  return u32x4{f2bf16_pair(v[0], v[1]), f2bf16_pair(v[2], v[3]), f2bf16_pair(v[4], v[5]), f2bf16_pair(v[6], v[7])};
}

__device__ inline float opened(int act, float g) {   // act(g)
  if (act == OES_GATE_PLAIN) return g;
  const float p = sigmoid(g);
  return act == OES_GATE_SIGMOID ? p : g * p;
}

// L lanes a row (64 and MANY: the whole workgroup), P pieces each.  ANY: x, the gains and the residual may be fp32;
// otherwise x and the gains are bf16 and the residual is fp32 if RF.  PAST: stores go past the caches.
template <int L, bool MANY, int P, bool ANY, bool RF, bool PAST>
__global__ __launch_bounds__(MANY ? (P == 1 ? 256 : 1024) : 256) void norm_kernel(NormArgs a) {
  constexpr int per = MANY ? 1 : 256 / L;   // rows of a workgroup
  __shared__ float sm[2][16];
  int turn = 0;
  // the sum over the row's threads; one barrier, since the next sum uses the other words
  auto row_sum = [&](float v) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) v += __shfl_xor(v, d, 64);
    if (MANY) {
      if ((threadIdx.x & 63) == 0) sm[turn][threadIdx.x >> 6] = v;
      __syncthreads();
      v = sm[turn][0];
      for (int w = 1; w < (int)(blockDim.x >> 6); ++w) v += sm[turn][w];
      turn ^= 1;
    }
    return v;
  };
  auto store = [&](u32x4 w, u32x4 *to) {
    if (PAST)
      __builtin_nontemporal_store(w, to);
    else
      *to = w;
  };
  const bool xf = ANY && a.x_f32, rf = ANY ? a.res_f32 : RF;
  const int me = MANY ? threadIdx.x : threadIdx.x % L, step = MANY ? blockDim.x : L;
  const float share = 1.f / a.dim;
  float v[P][8];
  bool in[P];
#pragma unroll
  for (int i = 0; i < P; ++i) in[i] = 8 * (me + i * step) < a.dim;
  // v becomes its norm; v is 0 past the row's end
  auto norm = [&](const NormSpec &s) {
    if (!s.on) return;
    const bool gf = ANY && s.f32;
    Piece<ANY> w[P], b[P];   // asked for ahead of the sum that they wait for
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) {
        if (s.w) w[i].load(s.w, 8 * (me + i * step), gf);
        if (s.b) b[i].load(s.b, 8 * (me + i * step), gf);
      }
    if (s.layer) {
      // Half the mean and half the differences, neither of which overflows for finite values (an infinite difference times
      // an inverse of 0 would be NaN): v - m over the root of its mean square and eps is (v / 2 - m / 2) over the root of
      // its own and eps / 4, which s.eps is here.
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(v[i][e], 0.5f * share, sum);
      const float half = row_sum(sum);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = in[i] ? fmaf(v[i][e], 0.5f, -half) : 0.f;
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(v[i][e], v[i][e], sq);
    const float inv = 1.f / sqrtf(row_sum(sq) * share + s.eps);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= inv;
    if (s.w) {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= s.offset + w[i].value(e, gf);
    }
    if (s.b) {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] += b[i].value(e, gf);
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = in[i] ? v[i][e] : 0.f;
  };
  const int64_t rows = (int64_t)a.n * a.heads;
  for (int64_t first = (int64_t)blockIdx.x * per; first < rows; first += (int64_t)gridDim.x * per) {
    const int64_t row = MANY ? first : min(first + threadIdx.x / L, rows - 1);
    const bool live = MANY || first + threadIdx.x / L < rows;
    const uint32_t t = a.heads == 1 ? (uint32_t)row : (uint32_t)row / (uint32_t)a.heads, h = (uint32_t)row - t * (uint32_t)a.heads;
    const int64_t x0 = t * a.x_row + h * a.x_head, r0 = t * a.res_row + h * a.res_head, g0 = t * a.gate_row + h * a.gate_head;
    const int64_t o0 = t * a.ro_row + h * a.ro_head, y0 = t * a.y_row + h * a.y_head;
    Piece<ANY> x[P];
    Piece<ANY || RF> res[P];
    Piece<false> gate[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = 8 * (me + i * step);
      if (MANY) gate[i].w[0] = u32x4{0, 0, 0, 0};
      if (!in[i]) continue;
      x[i].load(a.x, x0 + c, xf);
      if (a.res) res[i].load(a.res, r0 + c, rf);
      if (a.gate && a.gate_col) gate[i].load(a.gate, g0 + c, false);
    }
    // Behind the row's end a gate must open to a number, so that v stays 0 there: registers of 0, or 0 where it is used.  us,
    // the first and the second way: 8192 x 32 heads of 128 without a gate 31.9 and 29.4; 4096 x 2880 with one 28.7 and 29.1;
    // 8192 x 4096 with fp32 gains and no gate 70.3 and 78.9.
    const uint32_t one = a.gate && !a.gate_col ? static_cast<const uint16_t *>(a.gate)[g0] : 0u;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = in[i] ? x[i].value(e, xf) : 0.f;
    norm(a.post);
    if (a.gate && a.gate_col) {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= a.scale * opened(a.gate_act, MANY || in[i] ? gate[i].value(e, false) : 0.f);
    } else {
      const float s = a.gate ? a.scale * opened(a.gate_act, bf16f(one)) : a.scale;
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= s;
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] += in[i] ? res[i].value(e, rf) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!in[i]) continue;
      if (a.res_out && live) {
        u32x4 *to = reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(a.res_out) + (o0 + 8 * (me + i * step)) * (rf ? 4 : 2));
        if (rf) {
          store(u32x4{__float_as_uint(v[i][0]), __float_as_uint(v[i][1]), __float_as_uint(v[i][2]), __float_as_uint(v[i][3])}, to);
          store(u32x4{__float_as_uint(v[i][4]), __float_as_uint(v[i][5]), __float_as_uint(v[i][6]), __float_as_uint(v[i][7])}, to + 1);
        } else {
          const u32x4 w = packed(v[i]);
          store(w, to);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
        }
      }
    }
    if (!a.y) continue;
    norm(a.pre);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i] && live) store(packed(v[i]), reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.y) + y0 + 8 * (me + i * step)));
  }
}

template <int L, bool MANY, int P, bool PAST>
hipError_t launch_types(const NormArgs &a, dim3 g, dim3 b, hipStream_t s) {
  if (a.x_f32 || a.post.f32 || a.pre.f32)
    hipLaunchKernelGGL((norm_kernel<L, MANY, P, true, true, PAST>), g, b, 0, s, a);
  else if (a.res_f32)
    hipLaunchKernelGGL((norm_kernel<L, MANY, P, false, true, PAST>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((norm_kernel<L, MANY, P, false, false, PAST>), g, b, 0, s, a);
  return hipGetLastError();
}

template <int L, bool MANY, int P>
hipError_t launch_shape(const NormArgs &a, hipStream_t s) {
  constexpr int per = MANY ? 1 : 256 / L;
  const int64_t rows = (int64_t)a.n * a.heads;
  const int threads = MANY ? ((a.dim / 8 + P - 1) / P + 63) / 64 * 64 : 256;
  const dim3 g((uint32_t)std::min<int64_t>((rows + per - 1) / per, 1 << 21)), b(threads);

  // From 2^24 values on, what is stored would push itself out of the caches before it is read.  us of a norm and the
  // product behind it, with stores past the caches and without: 8192 x 4096 274 and 280, 4096 x 7168 231 and 237, 2048 x
  // 4096 113 both; 512 x 7168 53 and 46, 64 x 7168 22.1 and 19.3.
  if (MANY && rows * a.dim >= 1 << 24) return launch_types<L, MANY, P, MANY>(a, g, b, s);
  return launch_types<L, MANY, P, false>(a, g, b, s);
}

}  // namespace

// us with one piece a thread and with two: 2048 x 2880 13.0 and 10.8, 8192 x 4096 53.4 and 49.9, 3001 x 7168 44.0 and 35.3; four
// took 37.8 there, and 128 x 4096 is 0.4 slower with two than with one.  A wave of its own for a row of 4096 took 62.5.
hipError_t launch_norm(const NormArgs &a, hipStream_t s) {
  const int pieces = a.dim / 8;
  if (pieces <= 4) return launch_shape<4, false, 1>(a, s);
  if (pieces <= 8) return launch_shape<8, false, 1>(a, s);
  if (pieces <= 16) return launch_shape<16, false, 1>(a, s);
  if (pieces <= 32) return launch_shape<32, false, 1>(a, s);
  if (pieces <= 64) return launch_shape<64, false, 1>(a, s);
  if (pieces <= 256) return launch_shape<64, true, 1>(a, s);
  return launch_shape<64, true, 2>(a, s);
}

}  // namespace oes
