// Norms between the blocks: r = res + scale * act(gate) * post(x), y = pre(r).

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

constexpr int kThreads = 256;

__device__ inline float block_sum(float v, float *sm) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < kThreads / 64; ++w) s += sm[w];
  return s;
}

__device__ inline float value(const void *p, int f32, int64_t i) {
  return f32 ? static_cast<const float *>(p)[i] : bf16f(static_cast<const uint16_t *>(p)[i]);
}

__device__ inline float gated(const NormArgs &a, int64_t at) {
  if (!a.gate) return 1.f;
  const float g = bf16f(static_cast<const uint16_t *>(a.gate)[at]);
  if (a.gate_act == OES_GATE_PLAIN) return g;
  const float s = 1.f / (1.f + expf(-g));
  return a.gate_act == OES_GATE_SILU ? g * s : s;
}

__device__ inline float affine(const NormSpec &s, float v, int c) {
  const float gain = s.w ? s.offset + value(s.w, s.f32, c) : 1.f;
  return v * gain + (s.b ? value(s.b, s.f32, c) : 0.f);
}

// mean (0 for RMS) and 1 / sqrt(mean square + eps) of f(c)
template <typename F>
__device__ inline void stats(const NormSpec &s, int dim, float *sm, F f, float &mean, float &inv) {
  mean = 0.f;
  inv = 1.f;
  if (!s.on) return;
  if (s.layer) {
    float sum = 0.f;
    for (int c = threadIdx.x; c < dim; c += kThreads) sum += f(c);
    mean = block_sum(sum, sm) / dim;
  }
  float sq = 0.f;
  for (int c = threadIdx.x; c < dim; c += kThreads) {
    const float d = f(c) - mean;
    sq = fmaf(d, d, sq);
  }
  inv = 1.f / sqrtf(block_sum(sq, sm) / dim + s.eps);
}

__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a) {
  __shared__ float sm[kThreads / 64];
  extern __shared__ float row[];   // r
  const int t = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
  const int64_t x0 = t * a.x_row + h * a.x_head, g0 = t * a.gate_row + h * a.gate_head, r0 = t * a.res_row + h * a.res_head;
  const int64_t o0 = t * a.ro_row + h * a.ro_head, y0 = t * a.y_row + h * a.y_head;
  float mean, inv;
  stats(a.post, a.dim, sm, [&](int c) { return value(a.x, a.x_f32, x0 + c); }, mean, inv);
  for (int c = threadIdx.x; c < a.dim; c += kThreads) {
    float v = value(a.x, a.x_f32, x0 + c);
    if (a.post.on) v = affine(a.post, (v - mean) * inv, c);
    v = a.scale * gated(a, g0 + c * a.gate_col) * v;
    if (a.res) v += value(a.res, a.res_f32, r0 + c);
    if (a.res_out) {
      if (a.res_f32) {
        static_cast<float *>(a.res_out)[o0 + c] = v;
      } else {
        const uint32_t b = f2bf16(v);
        static_cast<uint16_t *>(a.res_out)[o0 + c] = (uint16_t)b;
        v = bf16f(b);
      }
    }
    row[c] = v;
  }
  if (!a.y) return;
  __syncthreads();
  stats(a.pre, a.dim, sm, [&](int c) { return row[c]; }, mean, inv);
  for (int c = threadIdx.x; c < a.dim; c += kThreads)
    static_cast<uint16_t *>(a.y)[y0 + c] = (uint16_t)f2bf16(a.pre.on ? affine(a.pre, (row[c] - mean) * inv, c) : row[c]);
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, hipStream_t s) {
  const int64_t blocks = (int64_t)a.n * a.heads;
  if (!launch_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(norm_kernel, dim3((uint32_t)blocks), dim3(kThreads), a.dim * 4, s, a);
  return hipGetLastError();
}

}  // namespace oes
