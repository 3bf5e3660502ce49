// Index arithmetic of the paged key / value cache, shared by the kernels and the
// host (oes_debug_kv_entry, tests on the CPU).  Offsets are 64-bit: a long cache
// passes 2^32 elements.
#pragma once

#include <stdint.h>

#include "../../include/oes.h"

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define OES_HD __host__ __device__ inline
#else
#define OES_HD inline
#endif

namespace oes {

// Page of entry j, or -1 if j is outside the table or the page outside the cache.
// shift: log2(page_size), or -1 if page_size is no power of two.
OES_HD int32_t kv_page(const oes_kv &kv, const int32_t *table_row, int32_t shift, int32_t j, int32_t *in_page) {
  if (j < 0) return -1;
  const int32_t col = shift >= 0 ? j >> shift : j / kv.page_size;
  *in_page = j - col * kv.page_size;
  if (col >= kv.max_pages) return -1;
  const int32_t p = table_row[col];
  return p >= 0 && p < kv.num_pages ? p : -1;
}

OES_HD int64_t kv_k_off(const oes_kv &kv, int32_t page, int32_t in_page) {
  return kv.k_page * page + kv.k_row * in_page;
}
OES_HD int64_t kv_v_off(const oes_kv &kv, int32_t page, int32_t in_page) {
  return kv.v_page * page + kv.v_row * in_page;
}

OES_HD int32_t kv_shift(int32_t page_size) {
  for (int s = 0; s < 31; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// Length of sequence b within the table's capacity; *bad if it had to be clamped.
OES_HD int32_t kv_len(const oes_kv &kv, int32_t len, bool *bad) {
  const int64_t cap = (int64_t)kv.max_pages * kv.page_size;
  if (len < 0) {
    *bad = true;
    return 0;
  }
  if (len > cap) {
    *bad = true;
    return (int32_t)cap;
  }
  return len;
}

// Rows [*first, *first + return) of a sequence within n rows; *bad if clamped.
OES_HD int32_t kv_rows(int32_t start, int32_t end, int32_t n, int32_t *first, bool *bad) {
  if (start < 0 || end < start || end > n) *bad = true;
  const int32_t a = start < 0 ? 0 : (start > n ? n : start);
  const int32_t e = end < a ? a : (end > n ? n : end);
  *first = a;
  return e - a;
}

// Entries [*lo, *hi) that token i of q_len new ones sees in a cache of len entries.
OES_HD void kv_seen(int32_t len, int32_t q_len, int32_t i, int32_t window, int32_t *lo, int32_t *hi) {
  const int32_t at = len - q_len + i;  // its own entry; < 0: none (0 <= len <= 2^30, 0 <= i < q_len: in 32 bits)
  *hi = at < 0 ? 0 : at + 1;
  *lo = window > 0 && at >= window ? at - window + 1 : 0;
}

}  // namespace oes
