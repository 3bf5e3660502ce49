// Rotary positions on q and k, with k and v written into the paged cache.
//
// Bound by reading and writing the rows once.  A wave takes one token and a part of its
// heads; the token's rot_dim / 2 sines and cosines are formed once per wave, in LDS: the
// angle pos * freq in fp64, reduced to an eighth of a turn, sine and cosine by their series in
// fp64 and rounded to fp32 once, with mscale (a position of a million keeps 2^-30 of a turn,
// where an fp32 product would lose 0.06 radians).  Products are fp32; but for keys of an e4m3
// cache an error of 2^-24 now and then crosses a border and costs 2^-4, so where one is near
// they are formed anew in fp64 and rounded to fp32 once (of 4.5 million entries some 2 come
// out on another side than in 64 bits, in place of 5; all in fp64 8740 tokens took 94 us in
// place of 83).  An item is 16 values of a head: two 16-byte pieces that hold 8
// pairs (values i .. i + 7 and their partners, half a rotation away or next to them), or that
// are copied.  A lane reads both pieces before it writes them, and no other lane touches
// them, so a call in place is safe.  Where the pairs of the half layout do not fall into whole
// pieces (rot_dim no multiple of 16), a lane takes single pairs.
//
// The number of workgroups is bounded, since starting one costs some 4 ns of the launch: with
// one for each of 8740 tokens of 80 heads, pair by pair, the launch took 182 us; it takes 83 (4.1 TB/s), and 5.2 for 32
// decoded tokens.

#include <algorithm>

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

constexpr int kWaves = 4, kUnroll = 2;

// Where a token's k and v go: sequence (-1: a row of none), and page (-1: no entry).  Wave-wide.
struct Place {
  int seq, page, in_page;
};

__device__ inline Place find_place(const RopeArgs &a, int t, int shift) {
  const int lane = threadIdx.x & 63;
  Place p = {-1, -1, 0};
  for (int b0 = 0; b0 < a.kv.batch && p.seq < 0; b0 += 64) {
    const int b = b0 + lane;
    bool bad = false;
    int first = 0, rows = 0, len = 0;
    if (b < a.kv.batch) {
      rows = kv_rows(a.q_start[b], a.q_start[b + 1], a.n, &first, &bad);
      len = kv_len(a.kv, a.kv.len[b], &bad);
    }
    if (bad) raise_status(a.kv);
    const uint64_t hit = __ballot(t >= first && t < first + rows);
    if (hit) {
      const int w = __builtin_amdgcn_readfirstlane(__builtin_ctzll(hit));
      p.seq = b0 + w;
      const int entry = __builtin_amdgcn_readlane(len - rows + t - first, w);
      if (entry >= 0) {
        p.page = kv_page(a.kv, a.kv.table + p.seq * a.kv.table_stride, shift, entry, &p.in_page);
        if (p.page < 0 && lane == 0) raise_status(a.kv);
      }
    }
  }
  return p;
}

// Head `hh` of a token's q, k and v heads: where it is read and written.
struct Head {
  const uint16_t *src;
  void *dst;
  float scale;   // e4m3: values are divided by it; 0: bf16
  bool turn;
};
__device__ inline Head head_at(const RopeArgs &a, const Place &p, int t, int hh) {
  Head h;
  h.scale = 0.f;
  h.turn = true;
  if (hh < a.heads) {
    h.src = a.x.p + t * a.x.row + hh * a.x.head;
    h.dst = a.y.p + t * a.y.row + hh * a.y.head;
    return h;
  }
  const int k = hh - a.heads, v = k - a.kv.kv_heads;
  const bool is_v = v >= 0, fp8 = a.kv.elem == OES_ELEM_E4M3;
  h.src = is_v ? a.v.p + t * a.v.row + v * a.v.head : a.k.p + t * a.k.row + k * a.k.head;
  const int64_t off = is_v ? kv_v_off(a.kv, p.page, p.in_page) + a.kv.v_head * v : kv_k_off(a.kv, p.page, p.in_page) + a.kv.k_head * k;
  h.dst = static_cast<uint8_t *>(is_v ? a.kv.v : a.kv.k) + off * (fp8 ? 1 : 2);
  if (fp8) h.scale = is_v ? a.kv.v_scale : a.kv.k_scale;
  h.turn = !is_v;
  return h;
}

// 8 values of a piece to where they go.
__device__ inline void put8(const Head &h, int at, const float *v, u32x4 raw, bool turned) {
  if (h.scale > 0.f) {
    u32x2 w;
    if (!turned)
      for (int i = 0; i < 4; ++i) const_cast<float *>(v)[2 * i] = bf16_lo(raw[i]), const_cast<float *>(v)[2 * i + 1] = bf16_hi(raw[i]);
    w.x = f2e4m3_pair(v[0] / h.scale, v[1] / h.scale) | f2e4m3_pair(v[2] / h.scale, v[3] / h.scale) << 16;
    w.y = f2e4m3_pair(v[4] / h.scale, v[5] / h.scale) | f2e4m3_pair(v[6] / h.scale, v[7] / h.scale) << 16;
    *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(h.dst) + at) = w;
  } else {
    if (turned) raw = u32x4{f2bf16_pair(v[0], v[1]), f2bf16_pair(v[2], v[3]), f2bf16_pair(v[4], v[5]), f2bf16_pair(v[6], v[7])};
    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(h.dst) + at) = raw;
  }
}

// Cosine and sine of `turns` turns.  |x| <= pi / 4 after the reduction: the first terms left out are x^13 / 13! < 7e-12
// and x^14 / 14! < 4e-13.
__device__ inline void turn_by(double turns, double *c, double *s) {
  const double quarter = rint(4. * turns), x = (turns - 0.25 * quarter) * 6.283185307179586477, y = x * x;
  const double sx = x * fma(y, fma(y, fma(y, fma(y, fma(y, -1. / 39916800., 1. / 362880.), -1. / 5040.), 1. / 120.), -1. / 6.), 1.);
  const double cx = fma(y, fma(y, fma(y, fma(y, fma(y, fma(y, 1. / 479001600., -1. / 3628800.), 1. / 40320.), -1. / 720.), 1. / 24.), -0.5), 1.);
  const int k = (int)(quarter - 4. * floor(0.25 * quarter));   // quarter turns on top: 0 .. 3
  *c = k == 0 ? cx : (k == 1 ? -sx : (k == 2 ? -cx : sx));
  *s = k == 0 ? sx : (k == 1 ? cx : (k == 2 ? -sx : -cx));
}

// Whether a value's e4m3 rounding (20 bits below the last one kept) depends on its last three bits.
__device__ inline bool near_border(float v) { return (__float_as_uint(v) & 0xfffffu) - 0x7fff8u < 16u; }

template <bool INTERLEAVED, bool PIECES, bool FP8>
__global__ __launch_bounds__(kWaves * 64, 3) void rope_kernel(RopeArgs a, int parts, int shift) {
  __shared__ __attribute__((aligned(16))) float cs[kWaves][128], sn[kWaves][128];
  __shared__ float cs_low[FP8 ? kWaves : 1][128], sn_low[FP8 ? kWaves : 1][128];   // what fp32 leaves of them
  const float per_scale = FP8 ? 1.f / a.kv.k_scale : 0.f;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, D = a.head_dim, half = a.rot_dim / 2;
  const int per = PIECES ? D / 16 : D / 2;         // items (or pairs) of a head
  const int heads = a.heads + (a.append ? 2 * a.kv.kv_heads : 0);
  const int per_pass = PIECES ? 64 / per : 1;      // heads that the wave takes at once
  const int hl = PIECES ? lane / per : 0, j = PIECES ? lane - hl * per : lane;
  const int passes = (heads + per_pass - 1) / per_pass;
  for (int64_t it = (int64_t)blockIdx.x * kWaves + wave; it < (int64_t)a.n * parts; it += (int64_t)gridDim.x * kWaves) {
    const int t = (int)(it / parts), part = (int)(it - (int64_t)t * parts);
    Place p = {0, -1, 0};
    if (a.append) p = find_place(a, t, shift);
    if (p.seq < 0) continue;
    const int live_heads = p.page >= 0 ? heads : a.heads;
    const double pos = a.pos[t];
    __builtin_amdgcn_wave_barrier();   // the last token's tables have been read
    for (int i = lane; i < half; i += 64) {
      double c, s;
      turn_by(pos * a.freq[i] * 0.15915494309189533577, &c, &s);
      c *= a.mscale;
      s *= a.mscale;
      cs[wave][i] = (float)c;
      sn[wave][i] = (float)s;
      if (FP8) {
        cs_low[wave][i] = (float)(c - (float)c);
        sn_low[wave][i] = (float)(s - (float)s);
      }
    }
    __builtin_amdgcn_wave_barrier();   // one wave's LDS operations run in order
    const int pass0 = (int)((int64_t)passes * part / parts), pass1 = (int)((int64_t)passes * (part + 1) / parts);
    if (PIECES) {
      // this lane's item: pieces at p0 and p1, pairs i0 .. i0 + 7
      const bool turns = INTERLEAVED ? 16 * j < a.rot_dim : 8 * j < half;
      const int p0 = INTERLEAVED || !turns ? 16 * j : 8 * j, p1 = INTERLEAVED || !turns ? 16 * j + 8 : 8 * j + half;
      float c8[8], s8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pr = turns ? 8 * j + i : 0;
        c8[i] = pr < half ? cs[wave][pr] : 0.f;
        s8[i] = pr < half ? sn[wave][pr] : 0.f;
      }
      for (int ps = pass0; ps < pass1; ps += kUnroll) {
        Head h[kUnroll];
        u32x4 r0[kUnroll], r1[kUnroll];
        bool in[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int hh = (ps + u) * per_pass + hl;
          in[u] = ps + u < pass1 && hl < per_pass && hh < live_heads;
          if (in[u]) {
            h[u] = head_at(a, p, t, hh);
            r0[u] = *reinterpret_cast<const u32x4 *>(h[u].src + p0);
            r1[u] = *reinterpret_cast<const u32x4 *>(h[u].src + p1);
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (!in[u]) continue;
          const bool turn = turns && h[u].turn;
          float y0[8], y1[8];
          if (turn) {
            // pair i: INTERLEAVED, the two halves of word i of the 16 values; else value i of either piece
            auto pair = [&](int i, float *x0, float *x1) {
              const uint32_t w0 = INTERLEAVED ? (i < 4 ? r0[u][i] : r1[u][i - 4]) : r0[u][i / 2], w1 = r1[u][i / 2];
              *x0 = INTERLEAVED ? bf16_lo(w0) : (i & 1 ? bf16_hi(w0) : bf16_lo(w0));
              *x1 = INTERLEAVED ? bf16_hi(w0) : (i & 1 ? bf16_hi(w1) : bf16_lo(w1));
            };
            auto put = [&](int i, float v0, float v1) {
              if (INTERLEAVED) {
                (i < 4 ? y0 : y1)[2 * (i & 3)] = v0;
                (i < 4 ? y0 : y1)[2 * (i & 3) + 1] = v1;
              } else {
                y0[i] = v0;
                y1[i] = v1;
              }
            };
            bool close = false;   // to a border of e4m3 rounding
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x0, x1;
              pair(i, &x0, &x1);
              float v0 = x0 * c8[i] - x1 * s8[i], v1 = x0 * s8[i] + x1 * c8[i];
              if (INTERLEAVED && 8 * j + i >= half) v0 = x0, v1 = x1;   // rot_dim ends within the item
              if (FP8) close |= near_border(v0 * per_scale) | near_border(v1 * per_scale);
              put(i, v0, v1);
            }
            if (FP8 && close && h[u].scale > 0.f) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                int pr = 8 * j + i;
                asm volatile("" : "+v"(pr));   // (or the tables are read before the branch)
                if (INTERLEAVED && pr >= half) continue;
                float x0, x1;
                pair(i, &x0, &x1);
                const double c = (double)cs[wave][pr] + cs_low[wave][pr], s = (double)sn[wave][pr] + sn_low[wave][pr];
                put(i, (float)(x0 * c - x1 * s), (float)(x0 * s + x1 * c));
              }
            }
          }
          put8(h[u], p0, y0, r0[u], turn);
          put8(h[u], p1, y1, r1[u], turn);
        }
      }
    } else {
      for (int hh = pass0; hh < min(pass1, live_heads); ++hh) {
        const Head h = head_at(a, p, t, hh);
        for (int i = j; i < per; i += 64) {
          // pair i of the half layout for i < half, else two values that are copied
          const int e0 = i < half ? i : 2 * i, e1 = i < half ? i + half : 2 * i + 1;
          const float x0 = bf16f(h.src[e0]), x1 = bf16f(h.src[e1]);
          float v0 = x0, v1 = x1;
          if (i < half && h.turn) {
            if (FP8 && h.scale > 0.f) {
              const double c = (double)cs[wave][i] + cs_low[wave][i], s = (double)sn[wave][i] + sn_low[wave][i];
              v0 = (float)(x0 * c - x1 * s);
              v1 = (float)(x0 * s + x1 * c);
            } else {
              const float c = cs[wave][i], s = sn[wave][i];
              v0 = x0 * c - x1 * s;
              v1 = x0 * s + x1 * c;
            }
          }
          if (h.scale > 0.f) {
            const uint32_t w = f2e4m3_pair(v0 / h.scale, v1 / h.scale);
            static_cast<uint8_t *>(h.dst)[e0] = (uint8_t)w;
            static_cast<uint8_t *>(h.dst)[e1] = (uint8_t)(w >> 8);
          } else {
            static_cast<uint16_t *>(h.dst)[e0] = (uint16_t)f2bf16(v0);
            static_cast<uint16_t *>(h.dst)[e1] = (uint16_t)f2bf16(v1);
          }
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, hipStream_t s) {
  const bool inter = a.layout == OES_ROPE_INTERLEAVED, pieces = inter || a.rot_dim % 16 == 0;
  const int heads = a.heads + (a.append ? 2 * a.kv.kv_heads : 0), per_pass = pieces ? 64 / (a.head_dim / 16) : 1;
  const int passes = (heads + per_pass - 1) / per_pass;
  // with few tokens, a wave to a pass of each; with many, a token to a wave, and several to each of 2048 workgroups
  const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(passes, 4096 / a.n));
  const int64_t blocks = std::min<int64_t>(2048, ((int64_t)a.n * parts + kWaves - 1) / kWaves);
  const int shift = a.append ? kv_shift(a.kv.page_size) : 0;
  const dim3 g((uint32_t)blocks), b(kWaves * 64);
  const bool fp8 = a.append && a.kv.elem == OES_ELEM_E4M3;
  if (inter && fp8)
    hipLaunchKernelGGL((rope_kernel<true, true, true>), g, b, 0, s, a, parts, shift);
  else if (inter)
    hipLaunchKernelGGL((rope_kernel<true, true, false>), g, b, 0, s, a, parts, shift);
  else if (pieces && fp8)
    hipLaunchKernelGGL((rope_kernel<false, true, true>), g, b, 0, s, a, parts, shift);
  else if (pieces)
    hipLaunchKernelGGL((rope_kernel<false, true, false>), g, b, 0, s, a, parts, shift);
  else if (fp8)
    hipLaunchKernelGGL((rope_kernel<false, false, true>), g, b, 0, s, a, parts, shift);
  else
    hipLaunchKernelGGL((rope_kernel<false, false, false>), g, b, 0, s, a, parts, shift);
  return hipGetLastError();
}

}  // namespace oes
