// Attention of new tokens over a paged cache, and the weights that its entries receive.
//
//   attn   one wave per (row, head): 64 entries at a time, each lane the score of one
//          entry, then each lane sums four of the output's values over the 64 weights
//          (running maximum and sum, one pass over the cache);
//   weigh  one thread per entry, over all rows and heads that see it.

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

// Sequence that row t belongs to (wave-wide), or -1.
__device__ inline int find_seq(const AttnArgs &a, int t, int *first, int *rows) {
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < a.kv.batch; b0 += 64) {
    const int b = b0 + lane;
    bool bad = false, hit = false;
    int f = 0, r = 0;
    if (b < a.kv.batch) {
      r = kv_rows(a.q_start[b], a.q_start[b + 1], a.n, &f, &bad);
      hit = t >= f && t < f + r;
      if (bad) raise_status(a.kv);
    }
    const uint64_t m = __ballot(hit);
    if (m) {
      const int w = __ffsll((unsigned long long)m) - 1;
      *first = __shfl(f, w, 64);
      *rows = __shfl(r, w, 64);
      return b0 + w;
    }
  }
  return -1;
}

template <bool FP8>
__device__ inline float cache_at(const void *base, int64_t off) {
  if (FP8) return e4m3_pair<false>((uint32_t) static_cast<const uint8_t *>(base)[off]).x;
  return bf16f(static_cast<const uint16_t *>(base)[off]);
}

template <bool FP8>
__device__ inline float dot_key(const AttnArgs &a, const uint16_t *q, int page, int in_page, int g) {
  const int64_t off = kv_k_off(a.kv, page, in_page) + a.kv.k_head * g;
  float s = 0.f;
  for (int d = 0; d < a.kv.head_dim; ++d) s = fmaf(bf16f(q[d]), cache_at<FP8>(a.kv.k, off + d), s);
  return s * a.kv.k_scale * a.scale;
}

template <bool FP8>
__global__ __launch_bounds__(64) void attn_kernel(AttnArgs a) {
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, D = a.kv.head_dim;
  int first = 0, rows = 0;
  const int b = find_seq(a, t, &first, &rows);
  if (b < 0) return;
  bool bad = false;
  const int len = kv_len(a.kv, a.kv.len[b], &bad);
  if (bad) raise_status(a.kv);
  const int g = h / (a.q_heads / a.kv.kv_heads), shift = kv_shift(a.kv.page_size);
  const int32_t *table = a.kv.table + b * a.kv.table_stride;
  const uint16_t *q = a.q.p + t * a.q.row + h * a.q.head;
  int lo, hi;
  kv_seen(len, rows, t - first, a.window, &lo, &hi);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = lo; j0 < hi; j0 += 64) {
    const int j = j0 + lane;
    int page = -1, in_page = 0;
    float s = -INFINITY;
    if (j < hi) {
      page = kv_page(a.kv, table, shift, j, &in_page);
      if (page >= 0)
        s = dot_key<FP8>(a, q, page, in_page, g);
      else
        raise_status(a.kv);
    }
    float mx = s;
    for (int d = 32; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d, 64));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float p = page >= 0 ? expf(s - mn) : 0.f, f = expf(m - mn);
    m = mn;
    float ps = p;
    for (int d = 32; d > 0; d >>= 1) ps += __shfl_xor(ps, d, 64);
    l = l * f + ps;
    for (int c = 0; c < 4; ++c) o[c] *= f;
    for (int w = 0; w < 64 && j0 + w < hi; ++w) {
      const int pg = __shfl(page, w, 64), ip = __shfl(in_page, w, 64);
      const float pw = __shfl(p, w, 64);
      if (pg < 0) continue;
      const int64_t off = kv_v_off(a.kv, pg, ip) + a.kv.v_head * g;
      for (int c = 0; c < 4; ++c)
        if (lane + 64 * c < D) o[c] = fmaf(pw, cache_at<FP8>(a.kv.v, off + lane + 64 * c), o[c]);
    }
  }
  uint16_t *out = a.out.p + t * a.out.row + h * a.out.head;
  for (int c = 0; c < 4; ++c)
    if (lane + 64 * c < D) out[lane + 64 * c] = (uint16_t)f2bf16(l > 0.f ? o[c] * a.kv.v_scale / l : l == 0.f ? 0.f : l);
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.q_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <bool FP8>
__global__ __launch_bounds__(256) void weigh_kernel(AttnArgs a) {
  const int b = blockIdx.z, g = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  const int G = a.q_heads / a.kv.kv_heads;
  bool bad = false;
  const int len = kv_len(a.kv, a.kv.len[b], &bad);
  int first;
  const int rows = kv_rows(a.q_start[b], a.q_start[b + 1], a.n, &first, &bad);
  if (bad) raise_status(a.kv);
  if (j >= len || rows == 0) return;
  int in_page;
  const int page = kv_page(a.kv, a.kv.table + b * a.kv.table_stride, kv_shift(a.kv.page_size), j, &in_page);
  if (page < 0) {
    raise_status(a.kv);
    return;
  }
  float sum = 0.f;
  for (int i = 0; i < rows; ++i) {
    int lo, hi;
    kv_seen(len, rows, i, a.window, &lo, &hi);
    if (j < lo || j >= hi) continue;
    for (int c = 0; c < G; ++c) {
      const int h = g * G + c;
      const float lse = a.lse[(int64_t)(first + i) * a.q_heads + h];
      if (lse == -INFINITY) continue;
      sum += expf(dot_key<FP8>(a, a.q.p + (first + i) * a.q.row + h * a.q.head, page, in_page, g) - lse);
    }
  }
  a.acc[((int64_t)b * a.kv.kv_heads + g) * a.acc_stride + j] += sum;
}

}  // namespace

int64_t attn_workspace_bytes(const oes_kv &, int, int) { return 0; }

hipError_t launch_attn(const AttnArgs &a, hipStream_t s) {
  const dim3 g(a.n, a.q_heads), b(64);
  if (a.kv.elem == OES_ELEM_E4M3)
    hipLaunchKernelGGL(attn_kernel<true>, g, b, 0, s, a);
  else
    hipLaunchKernelGGL(attn_kernel<false>, g, b, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_attn_weigh(const AttnArgs &a, hipStream_t s) {
  const int64_t cap = (int64_t)a.kv.max_pages * a.kv.page_size;
  if (a.kv.batch > 65535) return hipErrorInvalidConfiguration;
  const dim3 g((uint32_t)((cap + 255) / 256), a.kv.kv_heads, a.kv.batch), b(256);
  if (a.kv.elem == OES_ELEM_E4M3)
    hipLaunchKernelGGL(weigh_kernel<true>, g, b, 0, s, a);
  else
    hipLaunchKernelGGL(weigh_kernel<false>, g, b, 0, s, a);
  return hipGetLastError();
}

}  // namespace oes
