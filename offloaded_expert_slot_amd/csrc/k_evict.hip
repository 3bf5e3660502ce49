// Eviction by accumulated attention weight: which entries stay, and the cache closed up.
//
//   evict_select  one workgroup per (sequence, head).  Every entry gets a 32-bit key
//                 that orders as its weight does (NaN lowest, -0 as 0); the first and
//                 last ones are always kept.  The smallest kept key is found by a radix
//                 select, 8 bits a pass, then one ordered pass over the entries writes the
//                 kept ones' indices in order (equal keys: the lowest indices) and moves
//                 their weights.
//   evict_move    moves the k and v rows.  Entry i comes from kept[i] >= i, so going up in
//                 batches that are read whole before they are written is safe in place:
//                 a row i in the batch [i0, i1) that is itself kept has a rank <= i, so
//                 it was moved with this batch or before, and later batches read rows
//                 from i1 on only.  Head rows are cut into 16-byte columns, and each
//                 workgroup moves one group of columns of one (sequence, head).

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

constexpr int kSel = 1024;

__device__ inline uint32_t weight_key(float v) {
  if (v != v) return 0u;
  if (v == 0.f) v = 0.f;
  const uint32_t u = __float_as_uint(v);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// ws: per (sequence, head) the first entry that moves (= the new length if none does)
__global__ __launch_bounds__(kSel) void evict_select_kernel(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int wave_gt[16], wave_eq[16], sh[4];
  const int bh = blockIdx.x, b = bh / a.kv.kv_heads, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  bool bad = false;
  const int len = kv_len(a.kv, a.kv.len[b], &bad);
  int32_t *kept = a.kept + (int64_t)bh * a.budget;
  float *acc = a.acc + (int64_t)bh * a.acc_stride;
  // every page that the sequence uses has to be one of the cache
  const int32_t *table = a.kv.table + b * a.kv.table_stride;
  const int cols = (int)(((int64_t)len + a.kv.page_size - 1) / a.kv.page_size);
  if (tid == 0) sh[0] = 0;
  __syncthreads();
  for (int c = tid; c < cols; c += kSel)
    if (table[c] < 0 || table[c] >= a.kv.num_pages) sh[0] = 1;
  __syncthreads();
  const bool no_page = sh[0] != 0;
  if ((bad || no_page) && tid == 0) raise_status(a.kv);
  if (len <= a.budget || no_page) {
    for (int i = tid; i < a.budget; i += kSel) kept[i] = !no_page && i < len ? i : -1;
    if (tid == 0) a.ws[2 * bh] = a.ws[2 * bh + 1] = len;
    return;
  }
  const int mid0 = a.first, mid1 = len - a.last;    // entries that have to earn their place
  int want = a.budget - a.first - a.last;           // of them stay
  uint32_t prefix = 0, mask = 0;
  int left = want;                                  // still wanted among the keys of this prefix
  for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSel) hist[i] = 0;
    __syncthreads();
    for (int j = mid0 + tid; j < mid1; j += kSel) {
      const uint32_t k = weight_key(acc[j]);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255, n = left;
      while (d > 0 && n > hist[d]) n -= hist[d--];
      sh[1] = d;
      sh[2] = n;
    }
    __syncthreads();
    prefix |= (uint32_t)sh[1] << shift;
    mask |= 255u << shift;
    left = sh[2];
    __syncthreads();
  }
  // keys above prefix stay, and the `left` lowest-indexed ones equal to it
  int at = 0, eq_at = 0, moved = a.budget;
  for (int j0 = 0; j0 < len; j0 += kSel) {
    const int j = j0 + tid;
    bool stay = false, eq = false;
    float v = 0.f;
    if (j < len) {
      v = acc[j];
    }
    // a weight still on its way must not be overtaken by the stores of this stretch
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (j < len) {
      if (j < mid0 || j >= mid1) {
        stay = true;
      } else if (want > 0) {
        const uint32_t k = weight_key(v);
        stay = k > prefix;
        eq = k == prefix;
      }
    }
    const uint64_t below = (1ull << lane) - 1;
    const uint64_t meq = __ballot(eq);
    if (lane == 0) wave_eq[wave] = __popcll(meq);
    __syncthreads();
    int eq_rank = eq_at + __popcll(meq & below);
    int eq_all = 0;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) eq_rank += wave_eq[w];
      eq_all += wave_eq[w];
    }
    if (eq && eq_rank < left) stay = true;
    eq_at += eq_all;
    const uint64_t mst = __ballot(stay);
    if (lane == 0) wave_gt[wave] = __popcll(mst);
    __syncthreads();
    int pos = at + __popcll(mst & below), all = 0;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) pos += wave_gt[w];
      all += wave_gt[w];
    }
    // every thread has read its weight of this stretch; places up to here are free
    if (stay) {
      kept[pos] = j;
      if (pos != j) acc[pos] = v;
    }
    if (all < min(kSel, len - j0) && moved == a.budget) {  // the first dropped entry is in here
      if (tid == 0) sh[3] = kSel;
      __syncthreads();
      if (j < len && !stay) atomicMin(&sh[3], tid);
      __syncthreads();
      moved = min(a.budget, j0 + sh[3]);
    }
    at += all;
    __syncthreads();
  }
  if (tid == 0) {
    a.ws[2 * bh] = moved;
    a.ws[2 * bh + 1] = a.budget;
  }
}

// 16-byte columns [c0, c0 + 4) of the head rows of k and v; thread (row, column)
constexpr int kMove = 256, kUnroll = 8;

__global__ __launch_bounds__(kMove) void evict_move_kernel(EvictArgs a, int groups) {
  const int bh = blockIdx.x / groups, grp = blockIdx.x - bh * groups;
  const int b = bh / a.kv.kv_heads, h = bh - b * a.kv.kv_heads;
  const int from = a.ws[2 * bh], to = a.ws[2 * bh + 1];
  if (h == 0 && grp == 0 && threadIdx.x == 0) a.new_len[b] = to;
  if (from >= to) return;
  const int es = a.kv.elem == OES_ELEM_BF16 ? 2 : 1, per_row = a.kv.head_dim * es / 16;
  const int kgroups = (per_row + 3) / 4;
  const bool is_v = grp >= kgroups;
  const int col = (is_v ? grp - kgroups : grp) * 4 + (threadIdx.x & 3);
  const bool live = col < per_row;
  uint8_t *base = static_cast<uint8_t *>(is_v ? a.kv.v : a.kv.k) + (is_v ? a.kv.v_head : a.kv.k_head) * h * es + col * 16;
  const int32_t *table = a.kv.table + b * a.kv.table_stride, *kept = a.kept + (int64_t)bh * a.budget;
  const int shift = kv_shift(a.kv.page_size);
  auto row = [&](int j) {
    int ip = 0;
    const int p = kv_page(a.kv, table, shift, j, &ip);  // >= 0: checked for the whole sequence
    return reinterpret_cast<u32x4 *>(base + es * (is_v ? kv_v_off(a.kv, p, ip) : kv_k_off(a.kv, p, ip)));
  };
  constexpr int kRows = kMove / 4;
  for (int i0 = from; i0 < to; i0 += kRows * kUnroll) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kRows + (threadIdx.x >> 2);
      if (live && i < to) v[u] = *row(kept[i]);
    }
    // the whole batch is in registers before its first row is written
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kRows + (threadIdx.x >> 2);
      if (live && i < to) *row(i) = v[u];
    }
  }
}

}  // namespace

int64_t evict_workspace_bytes(const oes_kv &kv, int) { return ((int64_t)kv.batch * kv.kv_heads * 8 + 255) / 256 * 256; }

hipError_t launch_evict(const EvictArgs &a, hipStream_t s) {
  const int bh = a.kv.batch * a.kv.kv_heads;
  hipLaunchKernelGGL(evict_select_kernel, dim3(bh), dim3(kSel), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int es = a.kv.elem == OES_ELEM_BF16 ? 2 : 1, per_row = a.kv.head_dim * es / 16;
  const int groups = 2 * ((per_row + 3) / 4);
  hipLaunchKernelGGL(evict_move_kernel, dim3(bh * groups), dim3(kMove), 0, s, a, groups);
  return hipGetLastError();
}

}  // namespace oes
