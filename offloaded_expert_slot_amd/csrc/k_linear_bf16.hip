// y = res + scale * act(x . W^T + bias) for bf16 weights.

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

constexpr int kTile = 16, kChunk = 32;

__device__ inline float silu(float v) { return v / (1.f + expf(-v)); }
__device__ inline float activate(int act, float v) {
  switch (act) {
    case OES_ACT_SIGMOID: return 1.f / (1.f + expf(-v));
    case OES_ACT_SILU: return silu(v);
    case OES_ACT_GELU: return 0.5f * v * (1.f + tanhf(0.7978845608028654f * (v + 0.044715f * v * v * v)));
    default: return v;
  }
}

// a thread per value of y, tiles of 16 tokens x 16 columns
__global__ __launch_bounds__(256) void dense_kernel(DenseArgs a) {
  __shared__ float xs[kTile][kChunk + 1], ws[2][kTile][kChunk + 1];
  const int c = threadIdx.x % kTile, r = threadIdx.x / kTile;
  const int64_t col0 = (int64_t)blockIdx.x * kTile;
  const int t0 = blockIdx.y * kTile, parts = a.act == OES_ACT_SWIGLU ? 2 : 1;
  float sum[2] = {0.f, 0.f};
  for (int k0 = 0; k0 < a.K; k0 += kChunk) {
    for (int k = c; k < kChunk; k += kTile) {
      const bool in = k0 + k < a.K;
      xs[r][k] = in && t0 + r < a.n ? bf16f(a.x[(t0 + r) * a.x_row + k0 + k]) : 0.f;
      for (int p = 0; p < parts; ++p)
        ws[p][r][k] = in && col0 + r < a.N ? bf16f(a.w[(p * (int64_t)a.N + col0 + r) * a.w_row + k0 + k]) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < kChunk; ++k)
      for (int p = 0; p < parts; ++p) sum[p] = fmaf(xs[r][k], ws[p][c][k], sum[p]);
    __syncthreads();
  }
  const int64_t col = col0 + c, t = t0 + r;
  if (col >= a.N || t >= a.n) return;
  if (a.bias) sum[0] += bf16f(a.bias[col]);
  if (a.bias && parts == 2) sum[1] += bf16f(a.bias[a.N + col]);
  float v = a.scale * (parts == 2 ? silu(sum[0]) * sum[1] : activate(a.act, sum[0]));
  if (a.y_f32) {
    if (a.res) v += static_cast<const float *>(a.res)[t * a.res_row + col];
    static_cast<float *>(a.y)[t * a.y_row + col] = v;
  } else {
    if (a.res) v += bf16f(static_cast<const uint16_t *>(a.res)[t * a.res_row + col]);
    static_cast<uint16_t *>(a.y)[t * a.y_row + col] = (uint16_t)f2bf16(v);
  }
}

}  // namespace

bool linear_bf16_fits(const DenseArgs &a) {
  const int64_t tiles = (int64_t)((a.N + kTile - 1) / kTile) * ((a.n + kTile - 1) / kTile);
  return (a.n + kTile - 1) / kTile <= 65535 && launch_fits(tiles, 256);
}

hipError_t launch_linear_bf16(const DenseArgs &a, hipStream_t s) {
  hipLaunchKernelGGL(dense_kernel, dim3((a.N + kTile - 1) / kTile, (a.n + kTile - 1) / kTile), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace oes
