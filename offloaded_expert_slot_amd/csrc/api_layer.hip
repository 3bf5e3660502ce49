// Host side of the operators around the expert step: argument checks and launches of
// the 4-bit linear product, the rotary positions, attention over the paged cache, the
// weights its entries receive, and the eviction by them; of the norms between the
// blocks, the bf16 product with its epilogue, and sampling.

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <utility>

#include "kv_pages.h"
#include "oes_internal.h"

using namespace oes;

namespace {

oes_status fail(oes_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
oes_status fail(oes_status st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_error(st, buf);
}

oes_status launched(hipError_t e, const char *what) {
  if (e == hipSuccess) return OES_OK;
  (void)hipGetLastError();  // clear the runtime's sticky last-error slot
  return fail(OES_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }
inline bool aligned(const void *p, int a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

oes_status check_kv(const oes_kv *kv, bool written) {
  if (!kv) return fail(OES_ERR_ARG, "kv is NULL");
  if (kv->elem != OES_ELEM_BF16 && kv->elem != OES_ELEM_E4M3)
    return fail(OES_ERR_UNSUPPORTED, "cache element %d: bf16 or e4m3", kv->elem);
  if (kv->head_dim < 16 || kv->head_dim > 256 || kv->head_dim % 16)
    return fail(OES_ERR_ARG, "head_dim %d: a multiple of 16 in [16, 256]", kv->head_dim);
  if (kv->kv_heads < 1 || kv->kv_heads > 1024) return fail(OES_ERR_ARG, "kv_heads %d outside [1, 1024]", kv->kv_heads);
  if (kv->page_size < 1 || kv->max_pages < 1 || kv->num_pages < 0 || kv->batch < 0)
    return fail(OES_ERR_ARG, "need page_size >= 1, max_pages >= 1, num_pages >= 0, batch >= 0");
  if (kv->batch > (1 << 20)) return fail(OES_ERR_ARG, "batch %d exceeds 2^20", kv->batch);
  if ((int64_t)kv->page_size * kv->max_pages > (1ll << 30))
    return fail(OES_ERR_ARG, "max_pages * page_size = %lld exceeds 2^30", (long long)kv->page_size * kv->max_pages);
  if (!(kv->k_scale > 0) || !(kv->v_scale > 0) || !isfinite(kv->k_scale) || !isfinite(kv->v_scale))
    return fail(OES_ERR_ARG, "k_scale and v_scale must be positive and finite");
  if (kv->elem == OES_ELEM_BF16 && (kv->k_scale != 1.f || kv->v_scale != 1.f))
    return fail(OES_ERR_ARG, "a bf16 cache has scales of 1");
  if (kv->batch == 0) return OES_OK;
  if (!kv->k || !kv->v || !kv->table || !kv->len) return fail(OES_ERR_ARG, "NULL pointer in kv");
  if (kv->table_stride < kv->max_pages && kv->batch > 1) return fail(OES_ERR_ARG, "table_stride < max_pages");
  if (!aligned(kv->table, 4) || !aligned(kv->len, 4) || !aligned(kv->status, 4))
    return fail(OES_ERR_ARG, "table, len and status must be 4-byte aligned");
  const int per = kv->elem == OES_ELEM_BF16 ? 8 : 16;  // elements of 16 bytes
  const int64_t strides[] = {kv->k_page, kv->k_row, kv->k_head, kv->v_page, kv->v_row, kv->v_head};
  for (int64_t s : strides)
    if (s < 0 || s % per) return fail(OES_ERR_ARG, "cache strides must be >= 0 and keep head rows 16-byte aligned");
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return fail(OES_ERR_ARG, "k and v must be 16-byte aligned");
  if (written) {
    const int D = kv->head_dim;
    if ((kv->num_pages > 1 && (kv->k_page < D || kv->v_page < D)) ||
        (kv->page_size > 1 && (kv->k_row < D || kv->v_row < D)) ||
        (kv->kv_heads > 1 && (kv->k_head < D || kv->v_head < D)))
      return fail(OES_ERR_ARG, "rows of a cache that is written must not overlap");
  }
  return OES_OK;
}

// bf16 [n, heads, head_dim] with 16-byte aligned rows
oes_status check_rows(const char *what, const void *p, int64_t row, int64_t head, int n, int heads, int D, bool written) {
  if (!p) return fail(OES_ERR_ARG, "%s is NULL", what);
  if (!aligned(p, 16) || row % 8 || head % 8 || row < 0 || head < 0)
    return fail(OES_ERR_ARG, "%s: rows must be 16-byte aligned, strides >= 0", what);
  if (written && ((n > 1 && row < D) || (heads > 1 && head < D)))
    return fail(OES_ERR_ARG, "%s: rows that are written must not overlap", what);
  return OES_OK;
}

oes_status check_q_heads(const oes_kv *kv, int32_t q_heads) {
  if (q_heads < 1 || q_heads % kv->kv_heads || q_heads / kv->kv_heads > 128)
    return fail(OES_ERR_ARG, "q_heads %d: a multiple of kv_heads %d, at most 128 per cache head", q_heads, kv->kv_heads);
  return OES_OK;
}

oes_status check_rope(int32_t n, int32_t heads, int32_t head_dim, int32_t rot_dim, int32_t layout, const double *freq,
                      float mscale, const int32_t *pos) {
  if (n < 0) return fail(OES_ERR_ARG, "n < 0");
  if (head_dim < 16 || head_dim > 256 || head_dim % 16)
    return fail(OES_ERR_ARG, "head_dim %d: a multiple of 16 in [16, 256]", head_dim);
  if (heads < 1 || heads > 4096) return fail(OES_ERR_ARG, "heads %d outside [1, 4096]", heads);
  if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
    return fail(OES_ERR_ARG, "rot_dim %d: even, in [2, head_dim]", rot_dim);
  if (layout != OES_ROPE_HALF && layout != OES_ROPE_INTERLEAVED) return fail(OES_ERR_ARG, "unknown layout %d", layout);
  if (!isfinite(mscale)) return fail(OES_ERR_ARG, "mscale must be finite");
  if (n > 0 && (!freq || !pos)) return fail(OES_ERR_ARG, "freq / pos are NULL");
  if (!aligned(freq, 8) || !aligned(pos, 4)) return fail(OES_ERR_ARG, "freq and pos must be aligned to their elements");
  return OES_OK;
}

oes_status check_attn(const oes_kv *kv, int32_t q_heads, int32_t n, float scale, int32_t window) {
  oes_status st = check_q_heads(kv, q_heads);
  if (st != OES_OK) return st;
  if (n < 0 || window < 0) return fail(OES_ERR_ARG, "n < 0 or window < 0");
  // row numbers are added up in 32 bits (a tile's padding rows count as 2^30 on)
  if (n > (1 << 30)) return fail(OES_ERR_UNSUPPORTED, "n = %d: at most 2^30 rows", n);
  const float s = scale * kv->k_scale;  // what the scores are multiplied with
  if (!(scale > 0) || !(s >= 1e-30f) || !(s <= 1e30f)) return fail(OES_ERR_ARG, "scale (and scale * k_scale) must lie in [1e-30, 1e30]");
  return OES_OK;
}

// Larger calls are refused before their first launch.
oes_status too_large() { return fail(OES_ERR_UNSUPPORTED, "more work than one launch holds"); }

Rows rows(const void *p, int64_t row, int64_t head) {
  return Rows{static_cast<uint16_t *>(const_cast<void *>(p)), row, head};
}

}  // namespace

// ============================================================================ linear
extern "C" oes_status oes_linear(int32_t format, const void *w0, const void *w1, const void *w2, int32_t N, int32_t K,
                                 const void *x, int64_t x_stride, void *y, int64_t y_stride, int32_t n, void *stream) {
  if (format != OES_Q4_0 && format != OES_NVFP4 && format != OES_MXFP4_T)
    return fail(OES_ERR_UNSUPPORTED, "format %d has no 4-bit linear product", format);
  if (N < 1 || K < 32 || K % 32 || K > (1 << 20)) return fail(OES_ERR_ARG, "need N >= 1 and K a multiple of 32 up to 2^20");
  if (n < 0) return fail(OES_ERR_ARG, "n < 0");
  if (N > (1 << 23) || n > (1 << 19)) return fail(OES_ERR_UNSUPPORTED, "N = %d, n = %d: at most 2^23 rows and 2^19 tokens", N, n);
  if (n == 0) return OES_OK;
  if (!w0 || !w1 || !x || !y || (format == OES_NVFP4 && !w2)) return fail(OES_ERR_ARG, "NULL input");
  if (format == OES_Q4_0 && w2) return fail(OES_ERR_ARG, "q4_0 has two banks: w2 must be NULL");
  if (!aligned(w0, 16) || !aligned(w1, 16) || !aligned(x, 16) || x_stride % 8)
    return fail(OES_ERR_ARG, "w0, w1 and the rows of x must be 16-byte aligned");
  if (!aligned(w2, 2) || !aligned(y, 2)) return fail(OES_ERR_ARG, "w2 and y must be 2-byte aligned");
  if (n > 1 && (x_stride < K || y_stride < N)) return fail(OES_ERR_ARG, "x_stride < K or y_stride < N");
  LinearArgs a;
  a.format = format;
  a.N = N;
  a.K = K;
  a.n = n;
  a.w0 = static_cast<const uint8_t *>(w0);
  a.w1 = static_cast<const uint8_t *>(w1);
  a.w2 = static_cast<const uint8_t *>(w2);
  a.x = static_cast<const uint16_t *>(x);
  a.x_stride = x_stride;
  a.y = static_cast<uint16_t *>(y);
  a.y_stride = y_stride;
  return launched(launch_linear(a, as_stream(stream)), "oes_linear");
}

// ============================================================================ paged cache, rotary positions
extern "C" oes_status oes_debug_kv_entry(const oes_kv *kv, const int32_t *host_table, int32_t b, int32_t j,
                                         int64_t *k_off, int64_t *v_off) {
  if (!kv || !host_table || !k_off || !v_off) return fail(OES_ERR_ARG, "NULL argument");
  if (b < 0 || b >= kv->batch || kv->page_size < 1) return fail(OES_ERR_ARG, "sequence %d outside the batch", b);
  int32_t in_page = 0;
  const int32_t p = kv_page(*kv, host_table + b * kv->table_stride, kv_shift(kv->page_size), j, &in_page);
  if (p < 0) return fail(OES_ERR_ARG, "entry %d of sequence %d has no page", j, b);
  *k_off = kv_k_off(*kv, p, in_page);
  *v_off = kv_v_off(*kv, p, in_page);
  return OES_OK;
}

extern "C" oes_status oes_rope_freqs(int32_t scaling, int32_t rot_dim, double base, double factor, int32_t trained_len,
                                     double *freq, float *mscale) {
  if (!freq || !mscale) return fail(OES_ERR_ARG, "freq / mscale are NULL");
  if (rot_dim < 2 || rot_dim > 256 || rot_dim % 2) return fail(OES_ERR_ARG, "rot_dim %d: even, in [2, 256]", rot_dim);
  if (scaling < OES_ROPE_NONE || scaling > OES_ROPE_YARN) return fail(OES_ERR_ARG, "unknown scaling %d", scaling);
  if (!(base > 1) || !isfinite(base)) return fail(OES_ERR_ARG, "base must be finite and > 1");
  if (scaling != OES_ROPE_NONE && (!(factor >= 1) || !isfinite(factor))) return fail(OES_ERR_ARG, "factor must be finite and >= 1");
  if (scaling == OES_ROPE_NTK && rot_dim < 4) return fail(OES_ERR_ARG, "NTK scaling needs rot_dim >= 4");
  if (scaling == OES_ROPE_YARN && trained_len < 1) return fail(OES_ERR_ARG, "trained_len must be positive");
  const int half = rot_dim / 2;
  if (scaling == OES_ROPE_NTK) base *= pow(factor, rot_dim / (rot_dim - 2.0));
  double lo = 0, hi = 0;
  if (scaling == OES_ROPE_YARN) {
    // pair i turns trained_len * base^(-2 i / rot_dim) / (2 pi) times over trained_len
    const double two_pi = 6.283185307179586476925;
    const double per = rot_dim / (2 * log(base));
    lo = std::max(0.0, floor(per * log(trained_len / (32 * two_pi))));
    hi = std::min(rot_dim - 1.0, ceil(per * log(trained_len / two_pi)));
  }
  for (int i = 0; i < half; ++i) {
    const double f = pow(base, -2.0 * i / rot_dim);
    if (scaling == OES_ROPE_LINEAR) {
      freq[i] = f / factor;
    } else if (scaling == OES_ROPE_YARN) {
      const double r = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
      freq[i] = f * (1 - r) + f / factor * r;
    } else {
      freq[i] = f;
    }
  }
  *mscale = scaling == OES_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  return OES_OK;
}

extern "C" oes_status oes_rope(const void *x, int64_t x_row, int64_t x_head, void *y, int64_t y_row, int64_t y_head,
                               int32_t n, int32_t heads, int32_t head_dim, int32_t rot_dim, int32_t layout,
                               const double *freq, float mscale, const int32_t *pos, void *stream) {
  oes_status st = check_rope(n, heads, head_dim, rot_dim, layout, freq, mscale, pos);
  if (st != OES_OK || n == 0) return st;
  if ((st = check_rows("x", x, x_row, x_head, n, heads, head_dim, false)) != OES_OK) return st;
  if ((st = check_rows("y", y, y_row, y_head, n, heads, head_dim, true)) != OES_OK) return st;
  if (x == y && (x_row != y_row || x_head != y_head)) return fail(OES_ERR_ARG, "in place, y has the strides of x");
  RopeArgs a = {};
  a.x = rows(x, x_row, x_head);
  a.y = rows(y, y_row, y_head);
  a.heads = heads;
  a.n = n;
  a.head_dim = head_dim;
  a.rot_dim = rot_dim;
  a.layout = layout;
  a.freq = freq;
  a.mscale = mscale;
  a.pos = pos;
  return launched(launch_rope(a, as_stream(stream)), "oes_rope");
}

extern "C" oes_status oes_rope_append(const oes_kv *kv, const void *q, int64_t q_row, int64_t q_head, void *q_out,
                                      int64_t qo_row, int64_t qo_head, int32_t q_heads, const void *k, int64_t k_row,
                                      int64_t k_head, const void *v, int64_t v_row, int64_t v_head, int32_t n,
                                      const int32_t *q_start, int32_t rot_dim, int32_t layout, const double *freq,
                                      float mscale, const int32_t *pos, void *stream) {
  oes_status st = check_kv(kv, true);
  if (st != OES_OK) return st;
  const int D = kv->head_dim;
  if ((st = check_rope(n, q_heads, D, rot_dim, layout, freq, mscale, pos)) != OES_OK) return st;
  if (n == 0 || kv->batch == 0) return OES_OK;
  if (!q_start || !aligned(q_start, 4)) return fail(OES_ERR_ARG, "q_start is NULL or not 4-byte aligned");
  if ((st = check_rows("q", q, q_row, q_head, n, q_heads, D, false)) != OES_OK) return st;
  if ((st = check_rows("q_out", q_out, qo_row, qo_head, n, q_heads, D, true)) != OES_OK) return st;
  if ((st = check_rows("k", k, k_row, k_head, n, kv->kv_heads, D, false)) != OES_OK) return st;
  if ((st = check_rows("v", v, v_row, v_head, n, kv->kv_heads, D, false)) != OES_OK) return st;
  if (q == q_out && (q_row != qo_row || q_head != qo_head)) return fail(OES_ERR_ARG, "in place, q_out has the strides of q");
  RopeArgs a = {};
  a.x = rows(q, q_row, q_head);
  a.y = rows(q_out, qo_row, qo_head);
  a.heads = q_heads;
  a.n = n;
  a.head_dim = D;
  a.rot_dim = rot_dim;
  a.layout = layout;
  a.freq = freq;
  a.mscale = mscale;
  a.pos = pos;
  a.append = 1;
  a.k = rows(k, k_row, k_head);
  a.v = rows(v, v_row, v_head);
  a.kv = *kv;
  a.q_start = q_start;
  return launched(launch_rope(a, as_stream(stream)), "oes_rope_append");
}

// ============================================================================ attention
extern "C" oes_status oes_attn_workspace(const oes_kv *kv, int32_t q_heads, int32_t n, int64_t *bytes) {
  if (!bytes) return fail(OES_ERR_ARG, "bytes is NULL");
  oes_status st = check_kv(kv, false);
  if (st != OES_OK) return st;
  if ((st = check_attn(kv, q_heads, n, 1.f, 0)) != OES_OK) return st;
  *bytes = 0;
  if (n == 0 || kv->batch == 0) return OES_OK;
  if (!attn_fits(*kv, q_heads, n)) return too_large();
  *bytes = attn_workspace_bytes(*kv, q_heads, n);
  return OES_OK;
}

extern "C" oes_status oes_attn(const oes_kv *kv, const void *q, int64_t q_row, int64_t q_head, void *out, int64_t o_row,
                               int64_t o_head, float *lse, int32_t q_heads, int32_t n, const int32_t *q_start,
                               float scale, int32_t window, void *workspace, int64_t workspace_bytes, void *stream) {
  oes_status st = check_kv(kv, false);
  if (st != OES_OK) return st;
  if ((st = check_attn(kv, q_heads, n, scale, window)) != OES_OK) return st;
  if (n == 0 || kv->batch == 0) return OES_OK;
  if (!q_start || !aligned(q_start, 4) || !aligned(lse, 4)) return fail(OES_ERR_ARG, "q_start is NULL, or q_start or lse not aligned");
  if ((st = check_rows("q", q, q_row, q_head, n, q_heads, kv->head_dim, false)) != OES_OK) return st;
  if ((st = check_rows("out", out, o_row, o_head, n, q_heads, kv->head_dim, true)) != OES_OK) return st;
  if (out == q) return fail(OES_ERR_ARG, "out must not be q");
  if (!attn_fits(*kv, q_heads, n)) return too_large();
  const int64_t need = attn_workspace_bytes(*kv, q_heads, n);
  if (workspace_bytes < need)
    return fail(OES_ERR_ARG, "workspace %lld < %lld bytes", (long long)workspace_bytes, (long long)need);
  if (need > 0 && (!workspace || !aligned(workspace, 16))) return fail(OES_ERR_ARG, "workspace is NULL or not 16-byte aligned");
  AttnArgs a = {};
  a.kv = *kv;
  a.q = rows(q, q_row, q_head);
  a.out = rows(out, o_row, o_head);
  a.lse = lse;
  a.q_heads = q_heads;
  a.n = n;
  a.q_start = q_start;
  a.scale = scale;
  a.window = window;
  a.ws = static_cast<float *>(workspace);
  return launched(launch_attn(a, as_stream(stream)), "oes_attn");
}

extern "C" oes_status oes_attn_weigh(const oes_kv *kv, const void *q, int64_t q_row, int64_t q_head, const float *lse,
                                     int32_t q_heads, int32_t n, const int32_t *q_start, float scale, int32_t window,
                                     float *acc, int64_t acc_stride, void *stream) {
  oes_status st = check_kv(kv, false);
  if (st != OES_OK) return st;
  if ((st = check_attn(kv, q_heads, n, scale, window)) != OES_OK) return st;
  if (n == 0 || kv->batch == 0) return OES_OK;
  if (!q_start || !lse || !acc) return fail(OES_ERR_ARG, "q_start / lse / acc are NULL");
  if (!aligned(q_start, 4) || !aligned(lse, 4) || !aligned(acc, 4)) return fail(OES_ERR_ARG, "q_start, lse and acc must be 4-byte aligned");
  if ((st = check_rows("q", q, q_row, q_head, n, q_heads, kv->head_dim, false)) != OES_OK) return st;
  if (acc_stride < (int64_t)kv->max_pages * kv->page_size) return fail(OES_ERR_ARG, "acc_stride < max_pages * page_size");
  if (!attn_weigh_fits(*kv, q_heads, n)) return too_large();
  AttnArgs a = {};
  a.kv = *kv;
  a.q = rows(q, q_row, q_head);
  a.lse = const_cast<float *>(lse);
  a.q_heads = q_heads;
  a.n = n;
  a.q_start = q_start;
  a.scale = scale;
  a.window = window;
  a.acc = acc;
  a.acc_stride = acc_stride;
  return launched(launch_attn_weigh(a, as_stream(stream)), "oes_attn_weigh");
}

// ============================================================================ eviction
extern "C" oes_status oes_kv_evict_workspace(const oes_kv *kv, int32_t budget, int64_t *bytes) {
  if (!bytes) return fail(OES_ERR_ARG, "bytes is NULL");
  oes_status st = check_kv(kv, true);
  if (st != OES_OK) return st;
  if (budget < 1 || budget > (1 << 30)) return fail(OES_ERR_ARG, "budget %d outside [1, 2^30]", budget);
  if (!evict_fits(*kv)) return too_large();
  *bytes = evict_workspace_bytes(*kv, budget);
  return OES_OK;
}

extern "C" oes_status oes_kv_evict(const oes_kv *kv, float *acc, int64_t acc_stride, int32_t budget, int32_t first,
                                   int32_t last, int32_t *kept, int32_t *new_len, void *workspace,
                                   int64_t workspace_bytes, void *stream) {
  oes_status st = check_kv(kv, true);
  if (st != OES_OK) return st;
  if (budget < 1 || budget > (1 << 30) || first < 0 || last < 0 || (int64_t)first + last > budget)
    return fail(OES_ERR_ARG, "need budget in [1, 2^30], first, last >= 0 and first + last <= budget");
  if (kv->batch == 0) return OES_OK;
  if (!acc || !kept || !new_len) return fail(OES_ERR_ARG, "acc / kept / new_len are NULL");
  if (!aligned(acc, 4) || !aligned(kept, 4) || !aligned(new_len, 4)) return fail(OES_ERR_ARG, "acc, kept and new_len must be 4-byte aligned");
  if (acc_stride < (int64_t)kv->max_pages * kv->page_size) return fail(OES_ERR_ARG, "acc_stride < max_pages * page_size");
  const int64_t need = evict_workspace_bytes(*kv, budget);
  if (workspace_bytes < need || !workspace || !aligned(workspace, 16))
    return fail(OES_ERR_ARG, "workspace: %lld bytes, 16-byte aligned, are needed", (long long)need);
  if (!evict_fits(*kv)) return too_large();
  EvictArgs a = {};
  a.kv = *kv;
  a.acc = acc;
  a.acc_stride = acc_stride;
  a.budget = budget;
  a.first = first;
  a.last = last;
  a.kept = kept;
  a.new_len = new_len;
  a.ws = static_cast<int32_t *>(workspace);
  return launched(launch_evict(a, as_stream(stream)), "oes_kv_evict");
}

// ============================================================================ norms between the blocks
namespace {

oes_status check_spec(const char *what, const oes_norm_spec *s, NormSpec &out) {
  out = NormSpec{};
  if (!s) return OES_OK;
  if (s->kind != OES_NORM_RMS && s->kind != OES_NORM_LAYER) return fail(OES_ERR_ARG, "%s: unknown kind %d", what, s->kind);
  if (s->elem != OES_ELEM_BF16 && s->elem != OES_ELEM_F32) return fail(OES_ERR_UNSUPPORTED, "%s: w and b are bf16 or fp32", what);
  if (!(s->eps >= 0) || !isfinite(s->eps) || !isfinite(s->offset)) return fail(OES_ERR_ARG, "%s: eps must be finite and >= 0, offset finite", what);
  if (!aligned(s->w, 16) || !aligned(s->b, 16)) return fail(OES_ERR_ARG, "%s: w and b must be 16-byte aligned", what);
  const bool layer = s->kind == OES_NORM_LAYER;
  out = NormSpec{s->w, s->b, 1, layer, s->elem == OES_ELEM_F32, layer ? 0.25f * s->eps : s->eps, s->offset};
  return OES_OK;
}

// Whether two of n x heads rows of dim elements, at t * row + h * head, share an element
bool rows_overlap(int64_t n, int64_t row, int64_t heads, int64_t head, int64_t dim) {
  if ((n > 1 && row < dim) || (heads > 1 && head < dim)) return true;
  if (n == 1 || heads == 1) return false;
  const auto in_turn = [&](int64_t outer, int64_t inner, int64_t count) { return (outer - dim) / inner >= count - 1; };
  if (in_turn(row, head, heads) || in_turn(head, row, n)) return false;   // all of a token behind the one before, or of a head
  if (n > heads) std::swap(n, heads), std::swap(row, head);
  for (int64_t t = 1; t < n; ++t) {   // fewer than 2^16; the heads next to a row t further on
    const __int128 at = (__int128)t * row, h = at / head, past = at - h * head;
    if ((h < heads && past < dim) || (h + 1 < heads && head - past < dim)) return true;
  }
  return false;
}

// [n, heads, dim] rows of elements of `size` bytes; the stride over a single row or head counts as 0
oes_status check_norm_rows(const char *what, const void *p, int64_t &row, int64_t &head, const oes_norm_args *a, int size, bool written) {
  const int64_t per = 16 / size;
  if (a->n == 1) row = 0;
  if (a->heads == 1) head = 0;
  if (!aligned(p, 16) || row < 0 || head < 0 || row % per || head % per)
    return fail(OES_ERR_ARG, "%s: rows must be 16-byte aligned, strides >= 0", what);
  if (written && rows_overlap(a->n, row, a->heads, head, a->dim))
    return fail(OES_ERR_ARG, "%s: rows that are written must not overlap", what);
  return OES_OK;
}

}  // namespace

extern "C" oes_status oes_norm(const oes_norm_args *a, void *stream) {
  if (!a) return fail(OES_ERR_ARG, "args is NULL");
  if (a->n < 0 || a->heads < 1 || (int64_t)a->n * a->heads > 0x7fffffff) return fail(OES_ERR_ARG, "need n >= 0, heads >= 1 and n * heads < 2^31");
  if (a->dim < 8 || a->dim > 16384 || a->dim % 8) return fail(OES_ERR_ARG, "dim %d: a multiple of 8 in [8, 16384]", a->dim);
  if (a->reserved != 0) return fail(OES_ERR_ARG, "reserved must be 0");
  if (a->x_elem != OES_ELEM_BF16 && a->x_elem != OES_ELEM_F32) return fail(OES_ERR_UNSUPPORTED, "x is bf16 or fp32");
  if ((a->res || a->res_out) && a->res_elem != OES_ELEM_BF16 && a->res_elem != OES_ELEM_F32) return fail(OES_ERR_UNSUPPORTED, "the residual is bf16 or fp32");
  if (!isfinite(a->scale)) return fail(OES_ERR_ARG, "scale must be finite");
  if (a->gate && (a->gate_act < OES_GATE_PLAIN || a->gate_act > OES_GATE_SILU)) return fail(OES_ERR_ARG, "unknown gate_act %d", a->gate_act);
  NormArgs r = {};
  oes_status st;
  if ((st = check_spec("post", a->post, r.post)) != OES_OK) return st;
  if ((st = check_spec("pre", a->pre, r.pre)) != OES_OK) return st;
  if (a->n == 0) return OES_OK;
  if (!a->res_out && !a->y) return fail(OES_ERR_ARG, "neither res_out nor y is given");
  if (a->pre && !a->y) return fail(OES_ERR_ARG, "pre without y");
  if (!a->x) return fail(OES_ERR_ARG, "x is NULL");
  r.x = a->x, r.gate = a->gate, r.res = a->res, r.res_out = a->res_out, r.y = a->y;
  r.x_row = a->x_row, r.x_head = a->x_head, r.gate_row = a->gate_row, r.gate_head = a->gate_head, r.gate_col = a->gate_col;
  r.res_row = a->res_row, r.res_head = a->res_head, r.ro_row = a->ro_row, r.ro_head = a->ro_head, r.y_row = a->y_row, r.y_head = a->y_head;
  const int xs = a->x_elem == OES_ELEM_F32 ? 4 : 2, rs = a->res_elem == OES_ELEM_F32 ? 4 : 2;
  if ((st = check_norm_rows("x", a->x, r.x_row, r.x_head, a, xs, false)) != OES_OK) return st;
  if (a->res && (st = check_norm_rows("res", a->res, r.res_row, r.res_head, a, rs, false)) != OES_OK) return st;
  if (a->res_out && (st = check_norm_rows("res_out", a->res_out, r.ro_row, r.ro_head, a, rs, true)) != OES_OK) return st;
  if (a->y && (st = check_norm_rows("y", a->y, r.y_row, r.y_head, a, 2, true)) != OES_OK) return st;
  if (a->gate) {
    if (a->n == 1) r.gate_row = 0;
    if (a->heads == 1) r.gate_head = 0;
    if (r.gate_row < 0 || r.gate_head < 0 || (r.gate_col != 0 && r.gate_col != 1))
      return fail(OES_ERR_ARG, "gate: strides >= 0, and 0 or 1 over the columns");
    if (r.gate_col ? !aligned(a->gate, 16) || r.gate_row % 8 || r.gate_head % 8 : !aligned(a->gate, 2))
      return fail(OES_ERR_ARG, "gate: rows must be 16-byte aligned (one value a row: 2-byte)");
  }
  if (a->res_out == a->x || (a->res_out && a->res_out == a->y)) return fail(OES_ERR_ARG, "res_out must be neither x nor y");
  if (a->res_out && a->res_out == a->res && (r.ro_row != r.res_row || r.ro_head != r.res_head))
    return fail(OES_ERR_ARG, "in place, res_out has the strides of res");
  if (a->y && a->y == a->x && (a->x_elem != OES_ELEM_BF16 || r.y_row != r.x_row || r.y_head != r.x_head))
    return fail(OES_ERR_ARG, "in place, y has the type and the strides of x");
  if (a->y && (a->y == a->res || a->y == a->gate)) return fail(OES_ERR_ARG, "y must be neither res nor gate");
  if (a->res_out && a->res_out == a->gate) return fail(OES_ERR_ARG, "res_out must not be gate");
  r.n = a->n, r.heads = a->heads, r.dim = a->dim;
  r.x_f32 = a->x_elem == OES_ELEM_F32, r.res_f32 = a->res_elem == OES_ELEM_F32;
  r.gate_act = a->gate_act, r.scale = a->scale;
  return launched(launch_norm(r, as_stream(stream)), "oes_norm");
}

// ============================================================================ bf16 product with an epilogue
extern "C" oes_status oes_linear_bf16(const void *w, int64_t w_row, const void *bias, int32_t N, int32_t K, const void *x,
                                      int64_t x_row, int32_t n, int32_t act, float scale, const void *res, int64_t res_row,
                                      void *y, int64_t y_row, int32_t y_elem, void *stream) {
  if (N < 1 || K < 8 || K % 8 || K > (1 << 20)) return fail(OES_ERR_ARG, "need N >= 1 and K a multiple of 8 up to 2^20");
  if (n < 0) return fail(OES_ERR_ARG, "n < 0");
  if (N > (1 << 22) || n > (1 << 19)) return fail(OES_ERR_UNSUPPORTED, "N = %d, n = %d: at most 2^22 rows and 2^19 tokens", N, n);
  if (act < OES_ACT_NONE || act > OES_ACT_SWIGLU) return fail(OES_ERR_ARG, "unknown act %d", act);
  if (y_elem != OES_ELEM_BF16 && y_elem != OES_ELEM_F32) return fail(OES_ERR_UNSUPPORTED, "y is bf16 or fp32");
  if (!isfinite(scale)) return fail(OES_ERR_ARG, "scale must be finite");
  if (n == 0) return OES_OK;
  if (!w || !x || !y) return fail(OES_ERR_ARG, "NULL input");
  if (n == 1) x_row = y_row = res_row = 0;   // the stride over a single row does not count
  if (N == 1 && act != OES_ACT_SWIGLU) w_row = 0;
  const int size = y_elem == OES_ELEM_F32 ? 4 : 2;
  if (!aligned(w, 16) || !aligned(x, 16) || w_row % 8 || x_row % 8) return fail(OES_ERR_ARG, "the rows of w and x must be 16-byte aligned");
  if (!aligned(bias, 2) || !aligned(y, size) || !aligned(res, size)) return fail(OES_ERR_ARG, "bias, y and res must be aligned to their elements");
  if (w_row < 0 || x_row < 0 || y_row < 0 || res_row < 0) return fail(OES_ERR_ARG, "strides must be >= 0");
  if (((N > 1 || act == OES_ACT_SWIGLU) && w_row < K) || (n > 1 && (x_row < K || y_row < N || (res && res_row < N))))
    return fail(OES_ERR_ARG, "w_row, x_row < K or y_row, res_row < N");
  if (y == res && y_row != res_row) return fail(OES_ERR_ARG, "in place, y has the stride of res");
  if (y == x || y == w || y == bias) return fail(OES_ERR_ARG, "y must not be an input other than res");
  DenseArgs a = {};
  a.w = static_cast<const uint16_t *>(w);
  a.bias = static_cast<const uint16_t *>(bias);
  a.x = static_cast<const uint16_t *>(x);
  a.res = res;
  a.y = y;
  a.w_row = w_row, a.x_row = x_row, a.res_row = res_row, a.y_row = y_row;
  a.N = N, a.K = K, a.n = n, a.act = act, a.y_f32 = y_elem == OES_ELEM_F32;
  a.scale = scale;
  if (!linear_bf16_fits(a)) return too_large();
  return launched(launch_linear_bf16(a, as_stream(stream)), "oes_linear_bf16");
}

// ============================================================================ sampling
namespace {
oes_status check_sample(int32_t n, int32_t vocab) {
  if (n < 0 || vocab < 1) return fail(OES_ERR_ARG, "need n >= 0 and vocab >= 1");
  if (n > (1 << 16) || vocab > (1 << 20)) return fail(OES_ERR_UNSUPPORTED, "n = %d, vocab = %d: at most 2^16 rows of 2^20", n, vocab);
  if (n > 0 && !sample_fits(n, vocab)) return too_large();
  return OES_OK;
}
}  // namespace

extern "C" oes_status oes_sample_workspace(int32_t n, int32_t vocab, int64_t *bytes) {
  if (!bytes) return fail(OES_ERR_ARG, "bytes is NULL");
  oes_status st = check_sample(n, vocab);
  if (st != OES_OK) return st;
  *bytes = sample_workspace_bytes(n, vocab);
  return OES_OK;
}

extern "C" oes_status oes_sample(const void *logits, int32_t elem, int64_t row, int32_t n, int32_t vocab,
                                 const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                                 const float *u, int32_t *ids, float *logprob, void *workspace, int64_t workspace_bytes,
                                 void *stream) {
  oes_status st = check_sample(n, vocab);
  if (st != OES_OK) return st;
  if (elem != OES_ELEM_BF16 && elem != OES_ELEM_F32) return fail(OES_ERR_UNSUPPORTED, "logits are bf16 or fp32");
  if (n == 0) return OES_OK;
  if (!logits || !u || !ids) return fail(OES_ERR_ARG, "logits / u / ids are NULL");
  if (!aligned(logits, elem == OES_ELEM_F32 ? 4 : 2) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
      !aligned(min_p, 4) || !aligned(u, 4) || !aligned(ids, 4) || !aligned(logprob, 4))
    return fail(OES_ERR_ARG, "pointers must be aligned to their elements");
  if (n > 1 && row < vocab) return fail(OES_ERR_ARG, "row < vocab");
  if (n == 1) row = 0;
  const int64_t need = sample_workspace_bytes(n, vocab);
  if (workspace_bytes < need) return fail(OES_ERR_ARG, "workspace %lld < %lld bytes", (long long)workspace_bytes, (long long)need);
  if (need > 0 && (!workspace || !aligned(workspace, 16))) return fail(OES_ERR_ARG, "workspace is NULL or not 16-byte aligned");
  SampleArgs a = {};
  a.logits = logits;
  a.row = row;
  a.f32 = elem == OES_ELEM_F32;
  a.n = n, a.vocab = vocab;
  a.temperature = temperature, a.top_p = top_p, a.min_p = min_p, a.u = u;
  a.top_k = top_k;
  a.ids = ids;
  a.logprob = logprob;
  a.ws = static_cast<uint8_t *>(workspace);
  return launched(launch_sample(a, as_stream(stream)), "oes_sample");
}
