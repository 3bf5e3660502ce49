// Eviction by accumulated attention weight: which entries stay, and the cache closed up.
//
//   evict_select  one workgroup per (sequence, head).  Every entry gets a 32-bit key
//                 that orders as its weight does (NaN lowest, -0 as 0); the first and
//                 last ones are always kept.  The smallest kept key is found by a radix
//                 select, 8 bits a pass, on keys that stay in registers (16 a thread; more
//                 than 16384 entries are read again in each pass).  Then the kept entries'
//                 ranks, from one ordered sum over the waves' counts (equal keys: the
//                 lowest indices stay), place their indices and weights.
//   evict_move    moves the k and v rows.  Entry i comes from kept[i] >= i, so going up in
//                 batches that are read whole before they are written is safe in place:
//                 a row i in the batch [i0, i1) that is itself kept has a rank <= i, so
//                 it was moved with this batch or before, and later batches read rows
//                 from i1 on only (so the next batch's reads go out before this one's
//                 writes).  Head rows are cut into columns of 128 bytes, and each
//                 workgroup moves one column of one (sequence, head); bound by reading and
//                 writing the moved rows once.

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

constexpr int kSel = 1024, kWaves = kSel / 64, kHold = 16, kChunk = kSel * kHold;
constexpr int kCopies = 16;   // of the histogram, by lane: the leading digits of most keys are the same

__device__ inline uint32_t weight_key(float v) {
  if (v != v) return 0u;
  if (v == 0.f) v = 0.f;
  const uint32_t u = __float_as_uint(v);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ inline int scan64(int v) {  // inclusive, over the wave
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}

// ws: per (sequence, head) the first entry that moves and the new length (the same: none moves)
__global__ __launch_bounds__(kSel) void evict_select_kernel(EvictArgs a) {
  __shared__ __attribute__((aligned(16))) int hist[256 * kCopies];
  __shared__ int counts[kHold * kWaves], sh[4];
  const int bh = blockIdx.x, b = bh / a.kv.kv_heads, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  bool bad = false;
  const int len = kv_len(a.kv, a.kv.len[b], &bad);
  int32_t *kept = a.kept + (int64_t)bh * a.budget;
  float *acc = a.acc + (int64_t)bh * a.acc_stride;
  // every page that the sequence uses has to be one of the cache
  const int32_t *table = a.kv.table + b * a.kv.table_stride;
  const int cols = (int)(((int64_t)len + a.kv.page_size - 1) / a.kv.page_size);
  if (tid == 0) {
    sh[0] = 0;
    sh[3] = len;
  }
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
  const int want = a.budget - a.first - a.last;     // of them stay
  float v[kHold];
  auto load = [&](int base) {
#pragma unroll
    for (int x = 0; x < kHold; ++x) {
      if (base + x * kSel >= len) break;
      const int j = base + x * kSel + tid;
      v[x] = j < len ? acc[j] : 0.f;
    }
  };
  if (len <= kChunk) load(0);
  uint32_t prefix = 0, mask = 0;
  int left = want;                                  // still wanted among the keys of this prefix
  for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
    for (int i = tid; i < 256 * kCopies; i += kSel) hist[i] = 0;
    __syncthreads();
    for (int base = 0; base < len; base += kChunk) {
      if (len > kChunk) load(base);
#pragma unroll
      for (int x = 0; x < kHold; ++x) {
        if (base + x * kSel >= len) break;
        const int j = base + x * kSel + tid;
        const uint32_t k = weight_key(v[x]);
        if (j >= mid0 && j < mid1 && (k & mask) == prefix) atomicAdd(&hist[((k >> shift) & 255) * kCopies + (lane & (kCopies - 1))], 1);
      }
    }
    __syncthreads();
    if (wave == 0) {
      // lane l: digits 255 - 4 l down to 252 - 4 l, so that the running sum goes from the largest down
      int n[4], sum = 0;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        n[d] = 0;
        const int4 *h = reinterpret_cast<const int4 *>(hist + (255 - 4 * lane - d) * kCopies);
#pragma unroll
        for (int c = 0; c < kCopies / 4; ++c) n[d] += (h[c].x + h[c].y) + (h[c].z + h[c].w);
        sum += n[d];
      }
      int above = scan64(sum) - sum;   // keys with a larger digit than the lane's
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if (above < left && above + n[d] >= left) {
          sh[1] = 255 - 4 * lane - d;
          sh[2] = left - above;
        }
        above += n[d];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh[1] << shift;
    mask |= 255u << shift;
    left = sh[2];
  }
  // Exclusive sum over (stretch, wave), in the order of the entries, of counts[stretch * waves + wave]; all threads.
  auto ranks = [&](int *total) {
    __syncthreads();
    if (wave == 0) {
      constexpr int kPer = kHold * kWaves / 64;
      int n[kPer], sum = 0;
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        n[x] = counts[lane * kPer + x];
        sum += n[x];
      }
      const int upto = scan64(sum);
      int at = upto - sum;
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        counts[lane * kPer + x] = at;
        at += n[x];
      }
      if (lane == 63) sh[1] = upto;
    }
    __syncthreads();
    *total = sh[1];
  };
  // keys above prefix stay, and the `left` lowest-indexed ones equal to it
  int at = 0, eq_at = 0;
  const uint64_t below = (1ull << lane) - 1;
  for (int base = 0; base < len; base += kChunk) {
    if (len > kChunk) load(base);
    uint32_t stay = 0, eq = 0;   // bit x: the thread's entry of stretch x
#pragma unroll
    for (int x = 0; x < kHold; ++x) {
      if (base + x * kSel >= len) {   // (the same in every thread; the sums go over all stretches)
        if (lane == 0) counts[x * kWaves + wave] = 0;
        continue;
      }
      const int j = base + x * kSel + tid;
      const uint32_t k = weight_key(v[x]);
      const bool in = j < len, mid = j >= mid0 && j < mid1;
      if (in && (!mid || (want > 0 && k > prefix))) stay |= 1u << x;
      const bool same = in && mid && want > 0 && k == prefix;
      if (same) eq |= 1u << x;
      const uint64_t m = __ballot(same);
      if (lane == 0) counts[x * kWaves + wave] = __popcll(m);
    }
    int total;
    ranks(&total);
#pragma unroll
    for (int x = 0; x < kHold; ++x) {
      if (base + x * kSel >= len) break;
      const uint64_t m = __ballot((eq >> x) & 1);
      if (((eq >> x) & 1) && eq_at + counts[x * kWaves + wave] + __popcll(m & below) < left) stay |= 1u << x;
    }
    eq_at += total;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kHold; ++x) {
      const uint64_t m = __ballot((stay >> x) & 1);
      if (lane == 0) counts[x * kWaves + wave] = __popcll(m);
      if (base + x * kSel >= len) continue;
      const uint64_t gone = __ballot(base + x * kSel + tid < len && !((stay >> x) & 1));
      if (lane == 0 && gone) atomicMin(&sh[3], base + x * kSel + wave * 64 + __builtin_ctzll(gone));
    }
    ranks(&total);
    // every thread has the weights of this chunk in registers, and places up to here are free
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kHold; ++x) {
      if (base + x * kSel >= len) break;
      const uint64_t m = __ballot((stay >> x) & 1);
      if ((stay >> x) & 1) {
        const int j = base + x * kSel + tid, pos = at + counts[x * kWaves + wave] + __popcll(m & below);
        kept[pos] = j;
        if (pos != j) acc[pos] = v[x];
      }
    }
    at += total;
    __syncthreads();
  }
  if (tid == 0) {
    a.ws[2 * bh] = min(a.budget, sh[3]);
    a.ws[2 * bh + 1] = a.budget;
  }
}

// 256 rows of 128 bytes in flight per workgroup.  (16 x 4 heads of 2048 bf16 rows, 256 workgroups: 28.9 us; with 512
// threads and 4 rows a thread 37; 64-byte columns, twice the workgroups, 38.)
constexpr int kMove = 1024, kUnroll = 2, kRows = kMove / 8, kBatch = kRows * kUnroll;


__global__ __launch_bounds__(kMove) void evict_move_kernel(EvictArgs a, int columns, int shift) {
  const int bh = blockIdx.x / columns, column = blockIdx.x - bh * columns;
  const int b = bh / a.kv.kv_heads, h = bh - b * a.kv.kv_heads;
  const int from = a.ws[2 * bh], to = a.ws[2 * bh + 1];
  if (h == 0 && column == 0 && threadIdx.x == 0) a.new_len[b] = to;
  if (from >= to) return;
  const int es = a.kv.elem == OES_ELEM_BF16 ? 2 : 1, pieces = a.kv.head_dim * es / 16;
  const bool is_v = column >= columns / 2;
  const int piece = (is_v ? column - columns / 2 : column) * 8 + (threadIdx.x & 7), r0 = threadIdx.x >> 3;
  const bool live = piece < pieces;
  uint8_t *base = static_cast<uint8_t *>(is_v ? a.kv.v : a.kv.k) + (is_v ? a.kv.v_head : a.kv.k_head) * h * es + (live ? piece * 16 : 0);
  const int32_t *table = a.kv.table + b * a.kv.table_stride, *kept = a.kept + (int64_t)bh * a.budget;
  auto row = [&](int j) {
    int ip = 0;
    const int p = kv_page(a.kv, table, shift, j, &ip);  // >= 0: checked for the whole sequence
    return reinterpret_cast<u32x4 *>(base + es * (is_v ? kv_v_off(a.kv, p, ip) : kv_k_off(a.kv, p, ip)));
  };
  // rows past the last one are read again, and not written
  const u32x4 *src[kUnroll];
  u32x4 v[kUnroll], next[kUnroll];
  auto sources = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) src[u] = row(kept[min(i0 + u * kRows + r0, to - 1)]);
  };
  sources(from);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) v[u] = *src[u];
  for (int i0 = from; i0 < to; i0 += kBatch) {
    const bool more = i0 + kBatch < to;
    if (more) sources(i0 + kBatch);
    u32x4 *dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) dst[u] = row(min(i0 + u * kRows + r0, to - 1));
    // the whole batch is in registers before its first row is written
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (more) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) next[u] = *src[u];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (live && i0 + u * kRows + r0 < to) *dst[u] = v[u];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = next[u];
  }
}

}  // namespace

int64_t evict_workspace_bytes(const oes_kv &kv, int) { return ((int64_t)kv.batch * kv.kv_heads * 8 + 255) / 256 * 256; }

hipError_t launch_evict(const EvictArgs &a, hipStream_t s) {
  const int bh = a.kv.batch * a.kv.kv_heads;
  hipLaunchKernelGGL(evict_select_kernel, dim3(bh), dim3(kSel), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int columns = 2 * ((a.kv.head_dim * (a.kv.elem == OES_ELEM_BF16 ? 2 : 1) + 127) / 128);
  hipLaunchKernelGGL(evict_move_kernel, dim3(bh * columns), dim3(kMove), 0, s, a, columns, kv_shift(a.kv.page_size));
  return hipGetLastError();
}

}  // namespace oes
