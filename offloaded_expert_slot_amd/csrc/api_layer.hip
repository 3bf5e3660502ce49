// Host side of the operators around the expert step: argument checks and launches of
// the 4-bit linear product, the rotary positions, attention over the paged cache, the
// weights its entries receive, and the eviction by them.

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

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
