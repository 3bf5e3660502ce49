// y = x . W^T for 4-bit weights with group scales, in the layouts of the expert banks.
//
// Bound by reading the weights (4.5 bits each and nothing twice) up to some 64 tokens.  A
// wave takes R tiles of 16 weight rows over its share of K and multiplies them with up to
// 16 NT tokens by v_mfma_f32_16x16x32_bf16 (A = tokens, B = weights: a lane's accumulators
// are 4 tokens of one weight row).  A step covers 128 of K: lane (r, q) loads 16 bytes, the
// 32 codes of block 4 t + q of row r, so a load instruction reads 64 contiguous bytes of
// 16 rows (256 of MXFP4_T's).  The next step's loads are issued before this one's products.
// The waves of a workgroup share a tile and split K; their sums are joined in LDS, in
// order, and rounded once.
//
// The weights are used exactly:
//   nvfp4    e2m1 * e4m3 has at most 6 significant bits: formed in fp32, it is a bf16; the
//            fp16 of the row multiplies the finished sum
//   mxfp4_t  e2m1 * 2^e: the conversion instruction takes the scale
//   q4_0     (q - 8) d has up to 15 bits, so d has to multiply the sum of its block of 32.
//            Four blocks' codes are exchanged between the four lanes of a row (a 4 x 4
//            transpose of words, by two lane swaps each), after which one product covers
//            one block; a code counts as the exact bf16 128 + q, and the product starts
//            from -136 sum(x) of the block

#include <algorithm>
#include <type_traits>

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ inline float dot2_ones(uint32_t x, float acc) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x), __builtin_bit_cast(bf16x2, 0x3f803f80u), acc, false);
}
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

// What a lane holds of a step of one tile.
template <int FMT>
struct Chunk {
  u32x4 w;
  u32x2 sc;   // q4_0: fp16 scales of blocks 4 t .. 4 t + 3; nvfp4: the block's two e4m3; mxfp4_t: its e8m0
};

template <int FMT, int R, int NT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void linear_kernel(LinearArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  const int KB = a.K / 32, steps = (KB + 3) / 4;
  const int t0 = blockIdx.y * 16 * NT;
  const int64_t row0 = (int64_t)blockIdx.x * 16 * R;
  // rows past the end read the last one
  int64_t row[R];
#pragma unroll
  for (int i = 0; i < R; ++i) row[i] = min(row0 + 16 * i + r, (int64_t)a.N - 1);
  const uint16_t *x[NT];
  bool token[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    token[j] = t0 + 16 * j + r < a.n;
    x[j] = a.x + (int64_t)min(t0 + 16 * j + r, a.n - 1) * a.x_stride;
  }

  auto load = [&](Chunk<FMT>(&c)[R], int step) {
    const int kb = min(4 * step + q, KB - 1);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (FMT == OES_MXFP4_T) {
        c[i].w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(a.w0) + kb * (int64_t)a.N + row[i]);
        c[i].sc.x = a.w1[kb * (int64_t)a.N + row[i]];
      } else {
        c[i].w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(a.w0) + row[i] * KB + kb);
        const uint16_t *s = reinterpret_cast<const uint16_t *>(a.w1) + row[i] * KB;
        if (FMT == OES_NVFP4) {
          c[i].sc.x = s[kb];
        } else if (KB % 4 == 0) {
          c[i].sc = *reinterpret_cast<const u32x2 *>(s + 4 * step);
        } else {
          uint32_t h[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) h[b] = 4 * step + b < KB ? s[4 * step + b] : 0;
          c[i].sc.x = h[0] | h[1] << 16;
          c[i].sc.y = h[2] | h[3] << 16;
        }
      }
      if (FMT != OES_Q4_0 && 4 * step + q >= KB) c[i].sc.x = 0;   // past K: 0 * 0, whatever the last block holds
    }
  };
  f32x4 acc[R][NT];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto multiply = [&](Chunk<FMT>(&c)[R], int step) {
    if (FMT == OES_Q4_0) {
#pragma unroll
      for (int i = 0; i < R; ++i) {  // word b of lane q of a row <-> word q of lane b
        auto p = __builtin_amdgcn_permlane32_swap(c[i].w.x, c[i].w.z, false, false);
        c[i].w.x = p[0], c[i].w.z = p[1];
        p = __builtin_amdgcn_permlane32_swap(c[i].w.y, c[i].w.w, false, false);
        c[i].w.y = p[0], c[i].w.w = p[1];
        p = __builtin_amdgcn_permlane16_swap(c[i].w.x, c[i].w.y, false, false);
        c[i].w.x = p[0], c[i].w.y = p[1];
        p = __builtin_amdgcn_permlane16_swap(c[i].w.z, c[i].w.w, false, false);
        c[i].w.z = p[0], c[i].w.w = p[1];
      }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      // x of this product: q4_0: block 4 step + b, values 4 q .. + 3 and 16 + 4 q .. + 3 (a word's low
      // and high codes); else block 4 step + q, values 8 b .. + 7 (word b)
      const int kb = FMT == OES_Q4_0 ? 4 * step + b : 4 * step + q;
      u32x4 xv[NT];
      f32x4 start[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        xv[j] = u32x4{0, 0, 0, 0};
        if (token[j] && kb < KB) {
          if (FMT == OES_Q4_0) {
            const u32x2 lo = *reinterpret_cast<const u32x2 *>(x[j] + kb * 32 + 4 * q);
            const u32x2 hi = *reinterpret_cast<const u32x2 *>(x[j] + kb * 32 + 16 + 4 * q);
            xv[j] = u32x4{lo.x, lo.y, hi.x, hi.y};
          } else {
            xv[j] = *reinterpret_cast<const u32x4 *>(x[j] + kb * 32 + 8 * b);
          }
        }
        if (FMT == OES_Q4_0) {  // -136 sum(x) of the block for the lane's 4 tokens: one product with ones
          const u32x4 ones = {0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u};  // bf16 -136
          start[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[j]), __builtin_bit_cast(bf16x8, ones),
                                                              f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t w = c[i].w[b];
        u32x4 wv;
        if (FMT == OES_Q4_0) {
          const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
          // bytes 2 p, 2 p + 1 under 0x43: the pair (128 + q, 128 + q')
          wv = u32x4{__builtin_amdgcn_perm(0x43434343u, lo, 0x04010400u), __builtin_amdgcn_perm(0x43434343u, lo, 0x04030402u),
                     __builtin_amdgcn_perm(0x43434343u, hi, 0x04010400u), __builtin_amdgcn_perm(0x43434343u, hi, 0x04030402u)};
        } else if (FMT == OES_NVFP4) {
          const f32x2 sc = e4m3_pair<false>(c[i].sc.x);
          const float s = b < 2 ? sc.x : sc.y;
          wv = u32x4{fp4_scaled_pair<0>(w, s), fp4_scaled_pair<1>(w, s), fp4_scaled_pair<2>(w, s), fp4_scaled_pair<3>(w, s)};
        } else {
          const float s = e8m0_scale(c[i].sc.x);
          wv = u32x4{fp4_bf16_pair<0>(w, s), fp4_bf16_pair<1>(w, s), fp4_bf16_pair<2>(w, s), fp4_bf16_pair<3>(w, s)};
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (FMT == OES_Q4_0) {
            const f32x4 p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[j]),
                                                                    __builtin_bit_cast(bf16x8, wv), start[j], 0, 0, 0);
            const uint32_t d16 = (b < 2 ? c[i].sc.x : c[i].sc.y) >> (16 * (b & 1));
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
  };

  // steps wave, wave + WAVES, ...; two sets of registers, the loads one step ahead
  Chunk<FMT> c0[R], c1[R];
  int s = wave;
  if (s < steps) load(c0, s);
  while (s < steps) {
    if (s + WAVES < steps) load(c1, s + WAVES);
    multiply(c0, s);
    s += WAVES;
    if (s >= steps) break;
    if (s + WAVES < steps) load(c0, s + WAVES);
    multiply(c1, s);
    s += WAVES;
  }

  // join the waves in order; the lane (r, q) of wave 0 .. has tokens 4 q .. of row r
  __shared__ f32x4 part[WAVES > 1 ? WAVES : 1][NT][64];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (WAVES > 1) {
      if (i) __syncthreads();
#pragma unroll
      for (int j = 0; j < NT; ++j) part[wave][j][lane] = acc[i][j];
      __syncthreads();
    }
    for (int j = wave; j < NT; j += WAVES) {
      f32x4 sum = WAVES > 1 ? part[0][j][lane] : acc[i][j];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) sum += part[w][j][lane];
      const int64_t rr = row0 + 16 * i + r;
      if (rr < a.N) {
        float scale = 1.f, bias = 0.f;
        if (FMT == OES_NVFP4) scale = (float)__builtin_bit_cast(_Float16, reinterpret_cast<const uint16_t *>(a.w2)[rr]);
        if (FMT == OES_MXFP4_T && a.w2) bias = bf16f(reinterpret_cast<const uint16_t *>(a.w2)[rr]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = t0 + 16 * j + 4 * q + e;
          if (t < a.n) a.y[t * a.y_stride + rr] = (uint16_t)f2bf16(FMT == OES_NVFP4 ? sum[e] * scale : sum[e] + bias);
        }
      }
    }
  }
}

template <int FMT, int NT>
hipError_t launch_format(const LinearArgs &a, hipStream_t s) {
  const int tiles = (a.N + 15) / 16, groups = (a.n + 16 * NT - 1) / (16 * NT);
  const dim3 b4(256), b16(1024);
  if (groups > 65535) return hipErrorInvalidConfiguration;
  // enough workgroups for every CU come first, then more rows per x value read
  if (tiles * (int64_t)groups >= 4096)
    hipLaunchKernelGGL((linear_kernel<FMT, 4, NT, 4>), dim3((tiles + 3) / 4, groups), b4, 0, s, a);
  else if (tiles * (int64_t)groups >= 256)
    hipLaunchKernelGGL((linear_kernel<FMT, 1, NT, 4>), dim3(tiles, groups), b4, 0, s, a);
  else
    hipLaunchKernelGGL((linear_kernel<FMT, 1, NT, 16>), dim3(tiles, groups), b16, 0, s, a);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_tokens(const LinearArgs &a, hipStream_t s) {
  if (a.n <= 16) return launch_format<FMT, 1>(a, s);
  if (a.n <= 32) return launch_format<FMT, 2>(a, s);
  return launch_format<FMT, 4>(a, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
  if (a.format == OES_Q4_0) return launch_tokens<OES_Q4_0>(a, s);
  if (a.format == OES_NVFP4) return launch_tokens<OES_NVFP4>(a, s);
  return launch_tokens<OES_MXFP4_T>(a, s);
}

}  // namespace oes
