// y = x . W^T for 4-bit weights with group scales, in the layouts of the expert banks.
//
// One wave per (output row, token): lanes take the row's 32-element blocks in turn,
// decode a block to fp32 and sum its products before its scale.

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

__device__ inline float e2m1f(uint32_t c) {
  const uint32_t e = (c >> 1) & 3, m = c & 1;
  const float mag = e ? (float)(2 + m) * (float)(1 << e) * 0.25f : 0.5f * m;
  return (c & 8) ? -mag : mag;
}

template <int FMT>
__global__ __launch_bounds__(256) void linear_kernel(LinearArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= (int64_t)a.N * a.n) return;
  const int t = (int)(item / a.N), r = (int)(item - (int64_t)t * a.N);
  const uint16_t *x = a.x + t * a.x_stride;
  float sum = 0.f;
  for (int b = lane; b < a.K / 32; b += 64) {
    const uint8_t *c = FMT == OES_MXFP4_T ? a.w0 + ((int64_t)b * a.N + r) * 16 : a.w0 + (int64_t)r * (a.K / 2) + b * 16;
    float s0 = 0.f, s1 = 0.f;
    for (int j = 0; j < 16; ++j) {
      if (FMT == OES_Q4_0) {
        s0 += ((int)(c[j] & 15) - 8) * bf16f(x[b * 32 + j]);
        s1 += ((int)(c[j] >> 4) - 8) * bf16f(x[b * 32 + j + 16]);
      } else {
        float &s = j < 8 ? s0 : s1;
        s += e2m1f(c[j] & 15) * bf16f(x[b * 32 + 2 * j]);
        s += e2m1f(c[j] >> 4) * bf16f(x[b * 32 + 2 * j + 1]);
      }
    }
    if (FMT == OES_Q4_0) {
      const uint16_t d = reinterpret_cast<const uint16_t *>(a.w1)[(int64_t)r * (a.K / 32) + b];
      sum += (s0 + s1) * (float)__builtin_bit_cast(_Float16, d);
    } else if (FMT == OES_NVFP4) {
      const uint32_t w = reinterpret_cast<const uint16_t *>(a.w1)[(int64_t)r * (a.K / 32) + b];
      const f32x2 sc = e4m3_pair<false>(w);
      sum += s0 * sc.x + s1 * sc.y;
    } else {
      const uint32_t e = a.w1[(int64_t)b * a.N + r];
      const float sc = e == 255 ? __uint_as_float(0x7fc00000u)
                                : (e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23));
      sum += (s0 + s1) * sc;
    }
  }
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
  if (lane == 0) {
    if (FMT == OES_NVFP4) sum *= (float)__builtin_bit_cast(_Float16, reinterpret_cast<const uint16_t *>(a.w2)[r]);
    if (FMT == OES_MXFP4_T && a.w2) sum += bf16f(reinterpret_cast<const uint16_t *>(a.w2)[r]);
    a.y[t * a.y_stride + r] = (uint16_t)f2bf16(sum);
  }
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
  const int64_t blocks = ((int64_t)a.N * a.n + 3) / 4;
  if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
  const dim3 g((uint32_t)blocks), b(256);
  if (a.format == OES_Q4_0)
    hipLaunchKernelGGL(linear_kernel<OES_Q4_0>, g, b, 0, s, a);
  else if (a.format == OES_NVFP4)
    hipLaunchKernelGGL(linear_kernel<OES_NVFP4>, g, b, 0, s, a);
  else
    hipLaunchKernelGGL(linear_kernel<OES_MXFP4_T>, g, b, 0, s, a);
  return hipGetLastError();
}

}  // namespace oes
