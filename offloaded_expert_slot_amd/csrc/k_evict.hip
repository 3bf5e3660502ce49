// Eviction by accumulated attention weight: which entries stay, and the cache closed up.
//
//   evict_select  one workgroup per (sequence, head).  Every entry gets a 32-bit key
//                 that orders as its weight does (NaN lowest, -0 as 0); the first and
//                 last ones are always kept.  The smallest kept key is found by a radix
//                 select, 8 bits a pass until a digit's keys all stay, on weights that stay
//                 in LDS (more than 16384 are read again in each pass).  Then the kept
//                 entries' ranks, from one ordered sum over the threads' counts (equal keys:
//                 the lowest indices stay), place their indices and weights.  Short loops: in
//                 a launch of 10 us code that runs once waits for its instructions (with the
//                 weights in registers and 16-fold unrolled loops the ranks alone took 3.6).
//   evict_move    moves the k and v rows.  Entry i comes from kept[i] >= i, so going up in
//                 batches that are read whole before they are written is safe in place:
//                 a row i in the batch [i0, i1) that is itself kept has a rank <= i, so
//                 it was moved with this batch or before, and later batches read rows
//                 from i1 on only (so the next batch's reads go out before this one's
//                 writes).  Head rows are cut into columns of 128 bytes, and each
//                 workgroup moves one column of one (sequence, head); bound by reading and
//                 writing the moved rows once.
// 16 sequences x 4 heads from 2080 to 2048 bf16 rows of 128: select 10.5 us, move 23.7; 4 x 8 heads from 9204 .. 15074
// to 4099: 23.3 + 29.6 (4.6 TB/s of moved rows).

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

constexpr int kSel = 1024, kWaves = kSel / 64, kChunk = 16 * kSel;
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
  __shared__ __attribute__((aligned(16))) int hists[2][256 * kCopies];   // of a pass, and cleared for the next one
  __shared__ __attribute__((aligned(16))) float vals[kChunk];                                         // the weights, a chunk at a time
  __shared__ int sums[kWaves], sh[4];
  const int bh = blockIdx.x, b = bh / a.kv.kv_heads, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  bool bad = false;
  const int len = kv_len(a.kv, a.kv.len[b], &bad);
  int32_t *kept = a.kept + (int64_t)bh * a.budget;
  float *acc = a.acc + (int64_t)bh * a.acc_stride;
  // every page that the sequence uses has to be one of the cache
  const int32_t *table = a.kv.table + b * a.kv.table_stride;
  const int cols = (int)(((int64_t)len + a.kv.page_size - 1) / a.kv.page_size);
  static_assert(256 * kCopies == 4 * kSel, "16 bytes a thread");
  reinterpret_cast<int4 *>(hists[0])[tid] = int4{0, 0, 0, 0};
  if (tid == 0) {
    sh[0] = 0;
    sh[3] = len;
  }
  auto load = [&](int base) {   // a chunk, to LDS
    for (int j = tid; j < min(kChunk, len - base); j += kSel) vals[j] = acc[base + j];
  };
  if (len > a.budget && len <= kChunk) load(0);
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
  uint32_t prefix = 0, mask = 0;
  int left = want;                                  // still wanted among the keys of this prefix
  for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
    int *hist = hists[((shift >> 3) & 1) ^ 1];
    for (int base = 0; base < len; base += kChunk) {
      if (len > kChunk) {
        __syncthreads();
        load(base);
        __syncthreads();
      }
      for (int j0 = base + 4 * tid; j0 < min(mid1, base + kChunk); j0 += 4 * kSel) {
        const float4 v = *reinterpret_cast<const float4 *>(vals + (j0 - base));
        const float v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t k = weight_key(v4[e]);
          if (j0 + e >= mid0 && j0 + e < mid1 && (k & mask) == prefix) atomicAdd(&hist[((k >> shift) & 255) * kCopies + (lane & (kCopies - 1))], 1);
        }
      }
    }
    __syncthreads();
    reinterpret_cast<int4 *>(hists[(shift >> 3) & 1])[tid] = int4{0, 0, 0, 0};
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
          sh[0] = n[d] == left - above;   // all keys of this digit stay: the others' digits are the same to it
        }
        above += n[d];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh[1] << shift;
    mask |= 255u << shift;
    left = sh[2];
    if (sh[0]) break;
  }
  // Keys above prefix (as far as their digits were looked at) stay, and the `left` lowest-indexed ones equal to it.  A
  // thread takes neighbouring entries of the chunk (an odd number: different banks), so that one sum over the threads
  // gives all ranks.
  uint16_t *list = reinterpret_cast<uint16_t *>(hists);   // what stays of a chunk, in order
  static_assert(sizeof(hists) == 2 * kChunk, "an index each");
  int at = 0, eq_at = 0;   // entries that stay, and equal ones, of the chunks before
  for (int base = 0; base < len; base += kChunk) {
    if (len > kChunk) load(base);
    __syncthreads();
    const int n = min(kChunk, len - base), per = ((n + kSel - 1) / kSel) | 1, i0 = tid * per, i1 = min(n, i0 + per);
    uint32_t sure = 0, same = 0;   // bit i - i0: stays, is equal (at most 17 entries)
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
      const int j = base + i;
      const uint32_t k = weight_key(vals[i]) & mask;
      const bool mid = j >= mid0 && j < mid1;
      if (!mid || (want > 0 && k > prefix)) sure |= 1u << (i - i0);
      if (mid && want > 0 && k == prefix) same |= 1u << (i - i0);
    }
    const int mine = __popc(sure) | __popc(same) << 16;   // (of a chunk at most 16384 each)
    const int upto = scan64(mine);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    const int waves = scan64(lane < kWaves ? sums[lane] : 0), all = __builtin_amdgcn_readlane(waves, kWaves - 1);
    const int before = upto - mine + (wave > 0 ? __builtin_amdgcn_readlane(waves, max(wave, 1) - 1) : 0);
    int eq = eq_at + (before >> 16);
    int pos = at + (before & 0xffff) + min(eq, left) - min(eq_at, left);
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      if (((sure >> (i - i0)) & 1) || (((same >> (i - i0)) & 1) && eq++ < left))
        list[pos++ - at] = (uint16_t)i;
      else if (pos == base + i)
        sh[3] = pos;   // the first one that goes
    }
    const int stay = (all & 0xffff) + min(eq_at + (all >> 16), left) - min(eq_at, left);
    __syncthreads();
#pragma unroll 2
    for (int x = tid; x < stay; x += kSel) {
      const int i = list[x];
      kept[at + x] = base + i;
      if (x + at != base + i) acc[at + x] = vals[i];   // (a place before the entry's: that one has been read)
    }
    at += stay;
    eq_at += all >> 16;
    __syncthreads();
  }
  if (tid == 0) {
    a.ws[2 * bh] = min(a.budget, sh[3]);
    a.ws[2 * bh + 1] = a.budget;
  }
}

// 256 rows of 128 bytes in flight per workgroup.  (16 x 4 heads of 2048 bf16 rows, 256 workgroups, before loads were
// asked for ahead: 28.9 us; with 512 threads and 4 rows a thread 37; 64-byte columns, twice the workgroups, 38.)
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
  // An entry's place: its page, as loaded (valid: checked for the whole sequence), and its row in the page.
  struct Place {
    int page, row;
  };
  auto place = [&](int j) {
    const int col = shift >= 0 ? j >> shift : j / a.kv.page_size;
    return Place{table[col], j - col * a.kv.page_size};
  };
  auto at = [&](const Place &p) {
    return reinterpret_cast<u32x4 *>(base + es * (is_v ? kv_v_off(a.kv, p.page, p.row) : kv_k_off(a.kv, p.page, p.row)));
  };
  // Entry u of the thread in the batch from i0 on (past the last one, that one again, which is not written)
  auto entry = [&](int i0, int u) { return (int)min((int64_t)i0 + u * kRows + r0, (int64_t)to - 1); };
  // All that a batch needs is asked for ahead, before the batch before it is written: loads wait for the stores
  // issued before them, so a chain of index, page and row behind the stores took a turn of 2.7 us.
  u32x4 v[kUnroll], next[kUnroll];
  Place src[kUnroll], dst[kUnroll];   // sources of the next batch, places of this one
  int index[kUnroll];                 // sources of the batch after the next
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    v[u] = *at(place(kept[entry(from, u)]));
    src[u] = place(kept[entry(min(from + kBatch, to), u)]);
    index[u] = kept[entry(min(from + 2 * kBatch, to), u)];
    dst[u] = place(entry(from, u));
  }
  for (int i0 = from; i0 < to; i0 += kBatch) {
    // the whole batch is in registers before its first row is written
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) asm volatile("" : "+v"(src[u].page), "+v"(dst[u].page), "+v"(index[u]), "+v"(v[u]));
    __syncthreads();
    Place after[kUnroll], dst_next[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      next[u] = *at(src[u]);
      after[u] = place(index[u]);
      index[u] = kept[entry(i0 + 3 * kBatch, u)];
      dst_next[u] = place(entry(i0 + kBatch, u));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (live && i0 + u * kRows + r0 < to) *at(dst[u]) = v[u];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      v[u] = next[u];
      src[u] = after[u];
      dst[u] = dst_next[u];
    }
  }
}

}  // namespace

namespace {
// columns of 128 bytes of a head's k and v rows
int move_columns(const oes_kv &kv) { return 2 * ((kv.head_dim * (kv.elem == OES_ELEM_BF16 ? 2 : 1) + 127) / 128); }
}  // namespace

bool evict_fits(const oes_kv &kv) {
  const int64_t bh = (int64_t)kv.batch * kv.kv_heads;
  return launch_fits(bh, kSel) && launch_fits(bh * move_columns(kv), kMove);
}

int64_t evict_workspace_bytes(const oes_kv &kv, int) { return ((int64_t)kv.batch * kv.kv_heads * 8 + 255) / 256 * 256; }

hipError_t launch_evict(const EvictArgs &a, hipStream_t s) {
  const int bh = a.kv.batch * a.kv.kv_heads;
  hipLaunchKernelGGL(evict_select_kernel, dim3(bh), dim3(kSel), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int columns = move_columns(a.kv);
  hipLaunchKernelGGL(evict_move_kernel, dim3(bh * columns), dim3(kMove), 0, s, a, columns, kv_shift(a.kv.page_size));
  return hipGetLastError();
}

}  // namespace oes
