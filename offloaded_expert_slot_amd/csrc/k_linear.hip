// y = x . W^T for 4-bit weights with group scales, in the layouts of the expert banks.
//
// Bound by reading the weights (4.5 bits each) up to some 16 tokens: nvfp4 100003 x 7168 at 16 tokens 100 - 110 us a
// call, 3.7 - 4.0 TB/s (114 - 127 in a kernel trace, 100 at best; it asks memory for 1.14 times its operands); with more
// tokens widening the codes and the products add to it: 164 us at 40.  Small ones are bound by latency: q4_0 5120 x 2048
// for one token 5.4 us.  A workgroup reads its weights once for 16 NT tokens (16, or up to 64 from 1536 row tiles on),
// so a call of more tokens reads and widens them again.  A
// wave takes R tiles of 16 weight rows and multiplies them with up to 16 NT tokens by
// v_mfma_f32_16x16x32_bf16 (A = tokens, B = weights: a lane's accumulators are 4 tokens of
// one weight row).  A step covers 256 of K: two 16-byte loads per lane and tile, into one of
// RD sets of registers, so that RD - 1 steps' loads are under way.  They are buffer loads,
// which return 0 past the end without a fetch, so the loop's loads hang on no condition
// (where they do, the compiler has to wait for all of them).
//
// A product wants lane (r, q) to hold codes of row r.  Rows of q4_0 and nvfp4 are loaded as
// 8 rows x 128 bytes per instruction and brought there through LDS: read directly, 16 rows x
// 64 bytes, every line is asked for twice, and 100003 x 7168 did not pass 2.9 TB/s.  mxfp4_t's
// rows are adjacent as they are.  Then word b of the lane's block goes to product b with the
// matching x; q4_0's lanes first exchange words within a row (a 4 x 4 transpose by lane swaps),
// after which a product covers one block: one scale per product.
//
// x stands in LDS, a chunk of K at a time for all waves of the workgroup (read from global
// memory by every wave it takes more address cycles than the weights: 100003 x 7168 at 16
// tokens 168 us at best, at 64 tokens 424 us).  WR waves take different rows, WK waves
// different steps of the same rows, whose sums are joined in LDS in order.
//
// The weights are used exactly:
//   nvfp4    e2m1 * e4m3 has at most 6 significant bits: formed in fp32, it is a bf16; the
//            fp16 of the row multiplies the finished sum
//   mxfp4_t  e2m1 * 2^e: the conversion instruction takes the scale
//   q4_0     (q - 8) d has up to 15 bits, so d multiplies the product of its block; a code
//            counts as the exact bf16 2^-14 (128 + q), and the product starts from
//            -136 sum(x) 2^-14, so that with any finite x it stays within fp32
//            (32 (143 + 136) 2^-14 < 1); the finished sum counts 2^14-fold.  An x that is not
//            finite (inf - inf would be NaN) is 0 there and meets its weights at the end

#include <algorithm>
#include <type_traits>

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int B>
__device__ inline uint32_t fp4_bf16_pair(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
}
template <int B>
__device__ inline uint32_t fp4_scaled_pair(uint32_t w, float scale) {  // exact products (see above)
  const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, B);
  return f2bf16_pair(v.x * scale, v.y * scale);
}
__device__ inline float e8m0_scale(uint32_t e) {
  return e == 255 ? __uint_as_float(0x7fc00000u) : (e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23));
}

// Codes and scales of a step of one tile.  q4_0 and nvfp4: w[h] is chunk l % 8 of row 8 h + l / 8; mxfp4_t: block 4 h + q
// of row r.  sc: q4_0 fp16 of the row's 8 blocks (two a word, !TAIL); nvfp4 the two e4m3 of block 4 h + q; mxfp4_t its e8m0.
template <int FMT, bool TAIL>
struct Chunk {
  u32x4 w[2];
  uint32_t sc[FMT == OES_Q4_0 ? (TAIL ? 8 : 4) : 2];
};

constexpr uint32_t kNowhere = 0x7ffffff0u;   // a buffer offset past every end
constexpr int kPad = 8;                      // values behind a row of x in LDS: 16 rows spread over the banks

// `bytes` from p on; none if there are none left (bytes <= 0).  kNowhere is past the end of any.
__device__ inline __amdgpu_buffer_rsrc_t buffer(const void *p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)max((int64_t)0, min(bytes, (int64_t)0x7fffffe0)), 0x00027000);
}

// TAIL: K is no multiple of 256, the last step has fewer than eight blocks.
template <int FMT, int R, int NT, int WR, int WK, int RD, bool TAIL>
__global__ __launch_bounds__(WR * WK * 64) void linear_kernel(LinearArgs a, int KC, int per) {
  constexpr int W = WR * WK;
  typedef Chunk<FMT, TAIL> C;
  extern __shared__ __attribute__((aligned(16))) uint16_t xs[];   // [buffers][16 NT][KC + kPad]
  __shared__ __attribute__((aligned(16))) u32x4 swap[FMT == OES_MXFP4_T ? 1 : W][FMT == OES_MXFP4_T ? 1 : 128];
  __shared__ int odd_sm[FMT == OES_Q4_0 ? W : 1];   // whether a wave has stored x that is not finite
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  const int wk = wave % WK, wr = wave / WK;
  const int KB = a.K / 32, steps = (KB + 7) / 8;
  const int t0 = blockIdx.y * 16 * NT, tokens = min(16 * NT, a.n - t0);
  // `per` row tiles of a workgroup, shared out over its WR waves: at most R each
  const int tile0 = wr * per / WR, tiles = (wr + 1) * per / WR - tile0;
  const int64_t row0 = ((int64_t)blockIdx.x * per + tile0) * 16;
  const int rows_left = (int)max((int64_t)0, min((int64_t)16 * tiles, a.N - row0));
  const int64_t codes_bytes = (int64_t)KB * 16;

  // Offsets of the lane's codes and scales from a step's first ones; the step is in the buffer's start and size (the
  // range check is of the vector offset alone).
  const uint32_t w_off = ((lane >> 3) * KB + (lane & 7)) * 16, s_off = FMT == OES_MXFP4_T ? q * a.N + r : (r * KB + (FMT == OES_NVFP4 ? q : 0)) * 2;
  auto load = [&](C(&c)[R], int step) {
    const bool any = step < steps;
    if (FMT == OES_MXFP4_T) {
      // blocks of K are N rows apart
      const int64_t at = any ? 8ll * step * a.N + row0 : 0, left = any ? (int64_t)KB * a.N - at : 0;
      const __amdgpu_buffer_rsrc_t wt = buffer(a.w0 + at * 16, left * 16), st = buffer(a.w1 + at, left);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = 16 * i + r < rows_left && (!TAIL || 8 * step + 4 * h + q < KB);
          const uint32_t off = s_off + 16 * i + 4 * h * a.N;
          c[i].w[h] = __builtin_amdgcn_raw_buffer_load_b128(wt, in ? off * 16 : kNowhere, 0, 0);
          c[i].sc[h] = __builtin_amdgcn_raw_buffer_load_b8(st, in ? off : kNowhere, 0, 0);
        }
    } else {
      const int64_t w_at = any ? step * 128ll : 0, s_at = any ? step * 16ll : 0;
      const __amdgpu_buffer_rsrc_t wt = buffer(a.w0 + row0 * codes_bytes + w_at, any ? rows_left * codes_bytes - w_at : 0);
      const __amdgpu_buffer_rsrc_t st = buffer(a.w1 + row0 * KB * 2 + s_at, any ? (int64_t)rows_left * KB * 2 - s_at : 0);
      const bool in = !TAIL || 8 * step + (lane & 7) < KB;
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          c[i].w[h] = __builtin_amdgcn_raw_buffer_load_b128(wt, in ? w_off + (16 * i + 8 * h) * KB * 16 : kNowhere, 0, 0);
          if (FMT == OES_NVFP4)
            c[i].sc[h] = __builtin_amdgcn_raw_buffer_load_b16(st, !TAIL || 8 * step + 4 * h + q < KB ? s_off + 16 * i * KB * 2 + 8 * h : kNowhere, 0, 0);
        }
        if (FMT == OES_Q4_0 && !TAIL) {
          const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(st, s_off + 16 * i * KB * 2, 0, 0));
#pragma unroll
          for (int b = 0; b < 4; ++b) c[i].sc[b] = v[b];
        }
        if (FMT == OES_Q4_0 && TAIL) {
#pragma unroll
          for (int b = 0; b < 8; ++b)
            c[i].sc[b] = __builtin_amdgcn_raw_buffer_load_b16(st, 8 * step + b < KB ? s_off + 16 * i * KB * 2 + 2 * b : kNowhere, 0, 0);
        }
      }
    }
  };
  f32x4 acc[R][NT];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // x of product (h, b) for token 16 j + r: values 128 h + 32 q + 8 b .. + 7 of the step (word b of block 4 h + q);
  // q4_0: of block 4 h + b, 4 q .. + 3 and 16 + 4 q .. + 3 (a word's low and high codes); `at`: the step's first
  // value in the chunk
  auto multiply = [&](C(&c)[R], const uint16_t *chunk, int at) {
    u32x4 w[R][2];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (FMT == OES_MXFP4_T) {
        w[i][0] = c[i].w[0];
        w[i][1] = c[i].w[1];
      } else {  // chunk of a row at (chunk ^ row % 8)
        u32x4 *sw = swap[wave];
        sw[(lane & ~7) | ((lane & 7) ^ (lane >> 3))] = c[i].w[0];
        sw[64 + ((lane & ~7) | ((lane & 7) ^ (lane >> 3)))] = c[i].w[1];
#pragma unroll
        for (int h = 0; h < 2; ++h) w[i][h] = sw[r * 8 + ((4 * h + q) ^ (r & 7))];
      }
      if (FMT == OES_Q4_0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // word b of lane q of a row <-> word q of lane b
          u32x4 &v = w[i][h];
          auto p = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
          v.x = p[0], v.z = p[1];
          p = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
          v.y = p[0], v.w = p[1];
          p = __builtin_amdgcn_permlane16_swap(v.x, v.y, false, false);
          v.x = p[0], v.y = p[1];
          p = __builtin_amdgcn_permlane16_swap(v.z, v.w, false, false);
          v.z = p[0], v.w = p[1];
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x2 sc2[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (FMT == OES_NVFP4) sc2[i] = e4m3_pair<false>(c[i].sc[h]);
        if (FMT == OES_MXFP4_T) sc2[i].x = sc2[i].y = e8m0_scale(c[i].sc[h]);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        u32x4 xv[NT];
        f32x4 start[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint16_t *xb = chunk + (16 * j + r) * (KC + kPad) + at + 128 * h + (FMT == OES_Q4_0 ? 32 * b : 32 * q + 8 * b);
          if (FMT == OES_Q4_0) {
            const u32x2 lo = *reinterpret_cast<const u32x2 *>(xb + 4 * q), hi = *reinterpret_cast<const u32x2 *>(xb + 16 + 4 * q);
            xv[j] = u32x4{lo.x, lo.y, hi.x, hi.y};
            // -136 sum(x) of the block for the lane's 4 tokens: one product with bf16 -136 2^-14
            const u32x4 m136 = {0xbc08bc08u, 0xbc08bc08u, 0xbc08bc08u, 0xbc08bc08u};
            start[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[j]), __builtin_bit_cast(bf16x8, m136),
                                                                f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
          } else {
            xv[j] = *reinterpret_cast<const u32x4 *>(xb);
          }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const uint32_t v = w[i][h][b];
          u32x4 wv;
          if (FMT == OES_Q4_0) {
            const uint32_t lo = v & 0x0f0f0f0fu, hi = (v >> 4) & 0x0f0f0f0fu;
            // bytes 2 p, 2 p + 1 under 0x3c: the pair (128 + q, 128 + q') 2^-14
            wv = u32x4{__builtin_amdgcn_perm(0x3c3c3c3cu, lo, 0x04010400u), __builtin_amdgcn_perm(0x3c3c3c3cu, lo, 0x04030402u),
                       __builtin_amdgcn_perm(0x3c3c3c3cu, hi, 0x04010400u), __builtin_amdgcn_perm(0x3c3c3c3cu, hi, 0x04030402u)};
          } else if (FMT == OES_NVFP4) {
            const float s = b < 2 ? sc2[i].x : sc2[i].y;   // words 0, 1: a block's first 16
            wv = u32x4{fp4_scaled_pair<0>(v, s), fp4_scaled_pair<1>(v, s), fp4_scaled_pair<2>(v, s), fp4_scaled_pair<3>(v, s)};
          } else {
            const float s = sc2[i].x;
            wv = u32x4{fp4_bf16_pair<0>(v, s), fp4_bf16_pair<1>(v, s), fp4_bf16_pair<2>(v, s), fp4_bf16_pair<3>(v, s)};
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (FMT == OES_Q4_0) {
              const f32x4 p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[j]),
                                                                      __builtin_bit_cast(bf16x8, wv), start[j], 0, 0, 0);
              const uint32_t d16 = TAIL ? c[i].sc[(4 * h + b) % (TAIL ? 8 : 4)] : c[i].sc[2 * h + b / 2] >> (16 * (b & 1));
              const float d = (float)__builtin_bit_cast(_Float16, (uint16_t)d16);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], d, acc[i][j][e]);
            } else {
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[j]),
                                                                  __builtin_bit_cast(bf16x8, wv), acc[i][j], 0, 0, 0);
            }
          }
        }
      }
    }
  };

  // x chunks (past K, 0): one chunk, all of K, token by token; or several of RD steps of every wave, cut into
  // kPieces pieces of 16 bytes a token
  const int chunks = (a.K + KC - 1) / KC;
  constexpr int T = W * 64, kPieces = 32 * RD * WK, kHold = (16 * NT * kPieces + T - 1) / T;
  auto x_load = [&](int tk, int k) {
    u32x4 v = {0, 0, 0, 0};
    if (tk < tokens && k < a.K) v = *reinterpret_cast<const u32x4 *>(a.x + (int64_t)(t0 + tk) * a.x_stride + k);
    return v;
  };
  auto x_piece = [&](int chunk, int p) { return x_load(p / kPieces, chunk * KC + (p % kPieces) * 8); };
  auto x_put = [&](int chunk, int p, u32x4 v) {
    if (p / kPieces < tokens)
      *reinterpret_cast<u32x4 *>(xs + ((chunk & 1) * 16 * NT + p / kPieces) * (KC + kPad) + (p % kPieces) * 8) = v;
  };
  bool odd = false;   // q4_0: the thread has met x that is not finite, and put 0 in its place
  auto finite = [&](auto &v, int pieces) {
    if (FMT != OES_Q4_0) return;
    uint32_t any = 0;
#pragma unroll
    for (int h = 0; h < pieces; ++h) any |= (odd_bits(v[h].x) | odd_bits(v[h].y)) | (odd_bits(v[h].z) | odd_bits(v[h].w));
    if (__builtin_expect(__any(any != 0), 0)) {
      odd = true;
#pragma unroll
      for (int h = 0; h < pieces; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[h][i] &= ~((odd_bits(v[h][i]) >> 15) * 0xffffu);
    }
  };

  // steps of a wave: wk, wk + WK, ...; spc of them in a chunk (RD if there are several)
  const int spc = (KC / 256 + WK - 1) / WK;
  C c[RD][R];
#pragma unroll
  for (int d = 0; d + 1 < RD; ++d) load(c[d], wk + d * WK);
  if (chunks == 1) {
    for (int tk = 0; tk < tokens; ++tk)
      for (int k = threadIdx.x * 8; k < KC; k += T * 8) {
        u32x4 v[1] = {x_load(tk, k)};
        finite(v, 1);
        *reinterpret_cast<u32x4 *>(xs + tk * (KC + kPad) + k) = v[0];
      }
  } else {
    u32x4 v[kHold];
#pragma unroll
    for (int h = 0; h < kHold; ++h) v[h] = x_piece(0, threadIdx.x + h * T);
    finite(v, kHold);
#pragma unroll
    for (int h = 0; h < kHold; ++h) x_put(0, threadIdx.x + h * T, v[h]);
  }
  __syncthreads();
  int s = wk;
  for (int chunk = 0; chunk < chunks; ++chunk) {
    u32x4 hold[kHold];
    if (chunk + 1 < chunks) {
#pragma unroll
      for (int h = 0; h < kHold; ++h) hold[h] = x_piece(chunk + 1, threadIdx.x + h * T);
    }
    const uint16_t *xc = xs + (chunk & 1) * 16 * NT * (KC + kPad);
    const int k0 = chunk * KC;
    for (int i = 0; i < spc; i += RD) {
#pragma unroll
      for (int d = 0; d < RD; ++d) {
        load(c[(d + RD - 1) % RD], s + (d + RD - 1) * WK);
        if (s + d * WK < steps && i + d < spc) multiply(c[d], xc, (s + d * WK) * 256 - k0);
      }
      s += RD * WK;
    }
    if (chunk + 1 < chunks) {
      finite(hold, kHold);
#pragma unroll
      for (int h = 0; h < kHold; ++h) x_put(chunk + 1, threadIdx.x + h * T, hold[h]);
      __syncthreads();
    }
  }

  // join the WK waves of a row tile in order; lane (r, q) has tokens 4 q .. of row r
  f32x4 *part = reinterpret_cast<f32x4 *>(xs);   // [WR][WK][NT][64]
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (WK > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NT; ++j) part[((wr * WK + wk) * NT + j) * 64 + lane] = acc[i][j];
      __syncthreads();
    }
    for (int j = wk; j < NT; j += WK) {
      f32x4 sum;
      if (WK > 1) {
        sum = part[(wr * WK * NT + j) * 64 + lane];
        for (int w = 1; w < WK; ++w) sum += part[((wr * WK + w) * NT + j) * 64 + lane];
      } else {
        sum = acc[i][0];
#pragma unroll
        for (int jj = 1; jj < NT; ++jj)
          if (jj == j) sum = acc[i][jj];
      }
      const int64_t rr = row0 + 16 * i + r;
      if (16 * i + r < rows_left) {
        float scale = 1.f, bias = 0.f;
        if (FMT == OES_NVFP4) scale = (float)__builtin_bit_cast(_Float16, reinterpret_cast<const uint16_t *>(a.w2)[rr]);
        if (FMT == OES_MXFP4_T && a.w2) bias = bf16f(reinterpret_cast<const uint16_t *>(a.w2)[rr]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = t0 + 16 * j + 4 * q + e;
          if (t < a.n)
            a.y[t * a.y_stride + rr] = (uint16_t)f2bf16(FMT == OES_Q4_0 ? sum[e] * 0x1p14f : (FMT == OES_NVFP4 ? sum[e] * scale : sum[e] + bias));
        }
      }
    }
  }

  if (FMT == OES_Q4_0) {
    const bool mine = __any(odd);
    if (lane == 0) odd_sm[wave] = mine;
    __syncthreads();
    bool any = false;
#pragma unroll
    for (int w = 0; w < W; ++w) any |= odd_sm[w] != 0;
    if (!any) return;
    // x that is not finite: its products with the row's weights, added to what the lane has stored.  (The looking for it
    // costs up to 5 % of a call without any; a token with one in 16 of 100003 x 7168 takes 1.2 ms in place of 96 us.)
#pragma unroll 1
    for (int i = 0; i < R; ++i)
#pragma unroll 1
      for (int at = wk * 4; at < NT * 4; at += at % 4 < 3 ? 1 : 4 * WK - 3) {
        const int t = t0 + 16 * (at / 4) + 4 * q + at % 4;
        const int64_t rr = row0 + 16 * i + r;
        if (16 * i + r >= rows_left || t >= a.n) continue;
        float sum = 0.f;
#pragma unroll 1
        for (int k8 = 0; k8 < a.K; k8 += 8) {
          const uint16_t *xp = a.x + t * a.x_stride + k8;
          const u32x4 x8 = *reinterpret_cast<const u32x4 *>(xp);
          if (!(odd_bits(x8.x) | odd_bits(x8.y) | odd_bits(x8.z) | odd_bits(x8.w))) continue;
#pragma unroll 1
          for (int k = k8; k < k8 + 8; ++k) {
            const float x = bf16f(xp[k - k8]);
            if (fabsf(x) < INFINITY) continue;
            const int64_t block = rr * KB + k / 32;
            const uint32_t two = a.w0[block * 16 + k % 16], code = k % 32 < 16 ? two & 15 : two >> 4;
            sum += (float)((int)code - 8) * (float)__builtin_bit_cast(_Float16, reinterpret_cast<const uint16_t *>(a.w1)[block]) * x;
          }
        }
        uint16_t *y = a.y + t * a.y_stride + rr;
        if (!(sum == 0.f)) *y = (uint16_t)f2bf16(bf16f(*y) + sum);
      }
  }
}

// Whether 16 NT tokens' x stands in LDS whole (32 KiB where many workgroups are to share a CU).
int x_whole(const LinearArgs &a) { return (a.K + 255) / 256 * 256; }
bool x_fits(const LinearArgs &a, int NT, int most = 32 << 10) { return 16ll * NT * (x_whole(a) + kPad) * 2 <= most; }

template <int FMT, int R, int NT, int WR, int WK, int RD, int MOST = 32 << 10>
hipError_t launch_shape(const LinearArgs &a, hipStream_t s) {
  constexpr int W = WR * WK;
  const int64_t groups = (a.n + 16 * NT - 1) / (16 * NT), tiles = (a.N + 15) / 16;
  // with several tiles a wave, a whole number of workgroups to a CU, of equal numbers of tiles
  int64_t blocks = (tiles + R * WR - 1) / (R * WR);
  if (R > 1) blocks = (blocks + 255) / 256 * 256;
  const int per = R > 1 ? (int)((tiles + blocks - 1) / blocks) : WR;
  blocks = (tiles + per - 1) / per;
  if (groups > 65535) return hipErrorInvalidConfiguration;
  // the chunk of x: all of K if it fits into LDS, else RD steps of every wave, twice
  const int kp = x_whole(a), KC = x_fits(a, NT, MOST) ? kp : 256 * RD * WK, buffers = KC == kp ? 1 : 2;
  const int lds = std::max(buffers * 16 * NT * (KC + kPad) * 2, WK > 1 ? W * NT * 64 * 16 : 0);
  if (lds + (FMT == OES_MXFP4_T ? 16 : W * 2048) > 160 << 10) return hipErrorInvalidConfiguration;
  const dim3 g((uint32_t)blocks, (uint32_t)groups), b(W * 64);
  if (a.K % 256)
    hipLaunchKernelGGL((linear_kernel<FMT, R, NT, WR, WK, RD, true>), g, b, lds, s, a, KC, per);
  else
    hipLaunchKernelGGL((linear_kernel<FMT, R, NT, WR, WK, RD, false>), g, b, lds, s, a, KC, per);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_format(const LinearArgs &a, hipStream_t s) {
  const int64_t tiles = (a.N + 15) / 16;
  // From 1536 row tiles on: two tiles a wave, 8 waves of rows share x, up to 64 tokens at a time (100003 x 7168 a call,
  // us, at 16 and 40 tokens: nvfp4 102 - 113 and 164, q4_0 96 - 115 and 221, mxfp4 72 and 129; with one tile a wave
  // nvfp4 took 114 at 16 where two took 102).
  if (tiles >= 1536) {
    if (a.n <= 16) return launch_shape<FMT, 2, 1, 8, 1, 2>(a, s);
    if (a.n <= 32) return launch_shape<FMT, 2, 2, 8, 1, 2>(a, s);
    return launch_shape<FMT, 2, 4, 8, 1, 2>(a, s);
  }
  // Fewer: 16 tokens at a time (the weights come from caches again), and as many of the 8 waves on K as
  // leave no more than about one workgroup to a CU.  Measured, us, K split 8 / 4 / 2 / 1: q4_0 2048 x 4096
  // (128 tiles) 4.7 / 6.4 / 9.4 / 15.6; q4_0 5120 x 2048 (320) 6.7 / 4.5 / 5.7 / 8.2; mxfp4 10000 x 2880 (625)
  // 23 / 16.8 / 8.7 / 11.6; nvfp4 20000 x 2048 (1250) 25 / 17 / 13.3 / 10.2.
  const int64_t work = tiles * ((a.n + 15) / 16);
  if (work <= 256 && x_fits(a, 1, 128 << 10)) return launch_shape<FMT, 1, 1, 1, 8, 2, 128 << 10>(a, s);
  if (work <= 512) return launch_shape<FMT, 1, 1, 2, 4, 2>(a, s);
  if (work <= 1024) return launch_shape<FMT, 1, 1, 4, 2, 2>(a, s);
  return launch_shape<FMT, 1, 1, 8, 1, 2>(a, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
  if (a.format == OES_Q4_0) return launch_format<OES_Q4_0>(a, s);
  if (a.format == OES_NVFP4) return launch_format<OES_NVFP4>(a, s);
  return launch_format<OES_MXFP4_T>(a, s);
}

}  // namespace oes
