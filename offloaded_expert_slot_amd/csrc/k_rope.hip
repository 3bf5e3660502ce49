// Rotary positions on q and k, with k and v written into the paged cache.
//
// One workgroup per token.  Its rot_dim / 2 sines and cosines are formed once, in LDS:
// the angle pos * freq in fp64, reduced to a fraction of a turn in fp64 (a position of
// a million keeps 2^-30 of a turn, where an fp32 product would lose 0.06 radians), the
// sine and cosine of that fraction in fp32.  All heads of the token share them.  Each
// thread then owns whole pairs, so an in-place call never reads what another thread
// wrote.

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

constexpr int kThreads = 256;

// Where a token's k and v go: sequence and entry, or entry -1 (none) / seq -1 (a row of
// no sequence).  All threads of a workgroup call it and get the same answer.
struct Place {
  int seq, entry, page, in_page;
};

__device__ inline Place find_place(const RopeArgs &a, int t) {
  __shared__ int found[2];
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < a.kv.batch; b += kThreads) {
    bool bad = false;
    int first;
    const int rows = kv_rows(a.q_start[b], a.q_start[b + 1], a.n, &first, &bad);
    if (bad) raise_status(a.kv);
    if (t >= first && t < first + rows) atomicMax(&found[0], b);
  }
  __syncthreads();
  Place p;
  p.seq = found[0];
  p.entry = p.page = -1;
  p.in_page = 0;
  if (p.seq < 0) return p;
  bool bad = false;
  int first;
  const int rows = kv_rows(a.q_start[p.seq], a.q_start[p.seq + 1], a.n, &first, &bad);
  const int len = kv_len(a.kv, a.kv.len[p.seq], &bad);
  p.entry = len - rows + (t - first);
  if (p.entry >= 0) {
    p.page = kv_page(a.kv, a.kv.table + p.seq * a.kv.table_stride, kv_shift(a.kv.page_size), p.entry, &p.in_page);
    if (p.page < 0) bad = true;
  }
  if (bad && threadIdx.x == 0) raise_status(a.kv);
  return p;
}

__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
  __shared__ float cs[128], sn[128];
  const int t = blockIdx.x, half = a.rot_dim / 2, D = a.head_dim;
  Place p = {0, -1, -1, 0};
  if (a.append) {
    p = find_place(a, t);
    if (p.seq < 0) return;
  }
  const double pos = a.pos[t];
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double turns = pos * a.freq[i] * 0.15915494309189533577;
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = c * a.mscale;
    sn[i] = s * a.mscale;
  }
  __syncthreads();
  const int kvh = a.append && p.page >= 0 ? a.kv.kv_heads : 0;
  const int pairs = D / 2;
  const bool fp8 = a.kv.elem == OES_ELEM_E4M3;
  for (int it = threadIdx.x; it < (a.heads + 2 * kvh) * pairs; it += kThreads) {
    const int hh = it / pairs, i = it - hh * pairs;
    // pair i: a rotated one for i < half, else two values that are copied
    const bool rot = i < half;
    const int e0 = rot ? (a.layout == OES_ROPE_HALF ? i : 2 * i) : 2 * i;
    const int e1 = rot ? (a.layout == OES_ROPE_HALF ? i + half : 2 * i + 1) : 2 * i + 1;
    const bool is_q = hh < a.heads, is_v = hh >= a.heads + kvh;
    const int h = is_q ? hh : (is_v ? hh - a.heads - kvh : hh - a.heads);
    const Rows &src = is_q ? a.x : (is_v ? a.v : a.k);
    const uint16_t *sp = src.p + t * src.row + h * src.head;
    const uint32_t b0 = sp[e0], b1 = sp[e1];
    float x0 = bf16f(b0), x1 = bf16f(b1);
    if (rot && !is_v) {
      const float c = cs[i], s = sn[i], y0 = x0 * c - x1 * s, y1 = x0 * s + x1 * c;
      x0 = y0;
      x1 = y1;
    }
    if (is_q) {
      uint16_t *dp = a.y.p + t * a.y.row + h * a.y.head;
      dp[e0] = (uint16_t)f2bf16(x0);
      dp[e1] = (uint16_t)f2bf16(x1);
    } else {
      const int64_t off = (is_v ? kv_v_off(a.kv, p.page, p.in_page) + a.kv.v_head * h
                                : kv_k_off(a.kv, p.page, p.in_page) + a.kv.k_head * h);
      void *base = is_v ? a.kv.v : a.kv.k;
      if (fp8) {
        const float sc = is_v ? a.kv.v_scale : a.kv.k_scale;
        const uint32_t pr = f2e4m3_pair(x0 / sc, x1 / sc);
        static_cast<uint8_t *>(base)[off + e0] = (uint8_t)pr;
        static_cast<uint8_t *>(base)[off + e1] = (uint8_t)(pr >> 8);
      } else {
        static_cast<uint16_t *>(base)[off + e0] = (uint16_t)f2bf16(x0);
        static_cast<uint16_t *>(base)[off + e1] = (uint16_t)f2bf16(x1);
      }
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, hipStream_t s) {
  hipLaunchKernelGGL(rope_kernel, dim3(a.n), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace oes
