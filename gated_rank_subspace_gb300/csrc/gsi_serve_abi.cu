// C ABI of the serving operators: argument checks and dispatch.  The contract
// of every entry point is in include/gsi.h.

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "gsi_common.cuh"
#include "gsi_kernels.h"

namespace gsi {

static gsi_status refuse(gsi_status s, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return record_error(s, buf);
}
static gsi_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return record_error(GSI_OK, "");
  return refuse(GSI_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}
static bool on(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// A pointer that has to be there, aligned to n bytes.
static gsi_status need(const void* p, uintptr_t n, const char* name) {
  if (!p) return refuse(GSI_ERR_INVALID_ARG, "%s is NULL", name);
  if (!on(p, n)) return refuse(GSI_ERR_INVALID_ARG, "%s is not %d-byte aligned", name, int(n));
  return GSI_OK;
}
#define GSI_NEED(p, n)                        \
  do {                                        \
    const gsi_status st_ = need(p, n, #p);    \
    if (st_ != GSI_OK) return st_;            \
  } while (0)

static int elem(gsi_dtype dt) { return dt == GSI_BF16 ? 2 : 4; }
static bool known(gsi_dtype dt) { return dt == GSI_F32 || dt == GSI_BF16; }
static bool page_ok(int64_t p) { return p >= 16 && p <= 256 && (p & (p - 1)) == 0; }
static int log2_of(int64_t p) {
  int s = 0;
  while ((int64_t(1) << s) < p) ++s;
  return s;
}

static gsi_status check_cache(const gsi_cache_desc* c) {
  if (!c) return refuse(GSI_ERR_INVALID_ARG, "cache descriptor is NULL");
  if (!known(c->dtype)) return refuse(GSI_ERR_INVALID_ARG, "unknown dtype %d", int(c->dtype));
  if (c->n_pages < 0 || c->n_heads <= 0 || c->head_dim <= 0)
    return refuse(GSI_ERR_INVALID_ARG, "cache sizes must be positive (pages=%lld heads=%lld head_dim=%lld)",
                  (long long)c->n_pages, (long long)c->n_heads, (long long)c->head_dim);
  if (!page_ok(c->page_size))
    return refuse(GSI_ERR_UNSUPPORTED, "page_size=%lld is not a power of two from 16 to 256", (long long)c->page_size);
  const int es = elem(c->dtype);
  if (c->head_dim > 256 || (c->head_dim * es) % 16)
    return refuse(GSI_ERR_UNSUPPORTED, "head_dim=%lld is above 256 or not a multiple of 16 bytes", (long long)c->head_dim);
  if (c->n_heads > 4096 || c->n_pages > (int64_t(1) << 31) - 1)
    return refuse(GSI_ERR_UNSUPPORTED, "more than 4096 heads or 2^31 pages");
  const int64_t st[3] = {c->page_stride, c->head_stride, c->token_stride}, n[3] = {c->n_pages, c->n_heads, c->page_size};
  for (int i = 0; i < 3; ++i) {
    if (st[i] < 0 || (st[i] == 0 && n[i] > 1)) return refuse(GSI_ERR_INVALID_ARG, "a cache stride is not positive");
    if ((st[i] * es) % 16) return refuse(GSI_ERR_UNSUPPORTED, "a cache stride is not a multiple of 16 bytes");
    if (st[i] >= int64_t(1) << 38) return refuse(GSI_ERR_UNSUPPORTED, "a cache stride is above 2^38");
  }
  if (c->n_pages > 0) {
    GSI_NEED(c->K, 16);
    GSI_NEED(c->V, 16);
  }
  return GSI_OK;
}

static gsi_status check_heads(const gsi_cache_desc* c, int64_t n_q_heads) {
  if (n_q_heads <= 0 || n_q_heads % c->n_heads)
    return refuse(GSI_ERR_INVALID_ARG, "n_q_heads=%lld is not a multiple of the cache's %lld heads", (long long)n_q_heads,
                  (long long)c->n_heads);
  if (n_q_heads / c->n_heads > 128) return refuse(GSI_ERR_UNSUPPORTED, "more than 128 query heads share a key/value head");
  return GSI_OK;
}

static gsi_status check_norm(const gsi_norm* n, const char* name) {
  if (!n) return GSI_OK;
  if (n->kind != GSI_NORM_NONE && n->kind != GSI_NORM_RMS && n->kind != GSI_NORM_LAYER)
    return refuse(GSI_ERR_INVALID_ARG, "%s: unknown norm %d", name, int(n->kind));
  if (n->kind != GSI_NORM_NONE && !(n->eps >= 0.f && std::isfinite(n->eps)))
    return refuse(GSI_ERR_INVALID_ARG, "%s: eps must be >= 0 and finite", name);
  if (!on(n->weight, 16) || !on(n->bias, 16))
    return refuse(GSI_ERR_INVALID_ARG, "%s: weight or bias is not 16-byte aligned", name);
  return GSI_OK;
}

}  // namespace gsi

using namespace gsi;

extern "C" {

gsi_status gsi_paged_plan(const int32_t* cached, const int32_t* fresh, int64_t n_req, int32_t* table,
                          int64_t table_width, const int32_t* free_pages, int64_t capacity, const int32_t* n_free,
                          int64_t page_size, int64_t n_tokens, int32_t* q_start, int32_t* kv_len, int64_t* slots,
                          int32_t* token_req, int32_t* positions, int32_t* n_free_out, int32_t* status, void* stream) {
  if (n_req < 0 || n_tokens < 0 || table_width < 0 || capacity < 0)
    return refuse(GSI_ERR_INVALID_ARG, "a size is negative (n_req=%lld n_tokens=%lld table_width=%lld capacity=%lld)",
                  (long long)n_req, (long long)n_tokens, (long long)table_width, (long long)capacity);
  if (!page_ok(page_size))
    return refuse(GSI_ERR_UNSUPPORTED, "page_size=%lld is not a power of two from 16 to 256", (long long)page_size);
  if (n_req > (int64_t(1) << 20) || n_tokens > (int64_t(1) << 24) || table_width >= (int64_t(1) << 31) / page_size ||
      capacity > (int64_t(1) << 31) - 1)
    return refuse(GSI_ERR_UNSUPPORTED, "more than 2^20 requests, 2^24 tokens or 2^31 places of a request");
  GSI_NEED(q_start, 4);
  GSI_NEED(n_free, 4);
  GSI_NEED(n_free_out, 4);
  GSI_NEED(status, 4);
  if (n_req > 0) {
    GSI_NEED(cached, 4);
    GSI_NEED(fresh, 4);
    GSI_NEED(kv_len, 4);
    if (table_width > 0) GSI_NEED(table, 4);
  }
  if (capacity > 0) GSI_NEED(free_pages, 4);
  if (n_tokens > 0) {
    GSI_NEED(slots, 8);
    GSI_NEED(token_req, 4);
    GSI_NEED(positions, 4);
  }
  if (kv_len && kv_len == cached) return refuse(GSI_ERR_INVALID_ARG, "kv_len is cached: the lengths are read and written");
  if (n_free_out == n_free) return refuse(GSI_ERR_INVALID_ARG, "n_free_out is n_free: it is read and written");
  if (injected_failure()) return refuse(GSI_ERR_CUDA, "injected failure (gsi_debug_fail_after)");
  PlanArgs a{};
  a.cached = cached;
  a.fresh = fresh;
  a.n_req = int(n_req);
  a.table = table;
  a.width = table_width;
  a.free_pages = free_pages;
  a.capacity = capacity;
  a.n_free = n_free;
  a.page_shift = log2_of(page_size);
  a.n_tokens = int(n_tokens);
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.slots = slots;
  a.token_req = token_req;
  a.positions = positions;
  a.n_free_out = n_free_out;
  a.status = status;
  return launched(launch_paged_plan(a, static_cast<cudaStream_t>(stream)), "page plan launch");
}

gsi_status gsi_paged_trim(const int32_t* kv_len, const int32_t* kept, int64_t n_req, const int32_t* table,
                          int64_t table_width, int32_t* free_pages, int64_t capacity, const int32_t* n_free,
                          int64_t page_size, int32_t* n_free_out, int32_t* status, void* stream) {
  if (n_req < 0 || table_width < 0 || capacity < 0)
    return refuse(GSI_ERR_INVALID_ARG, "a size is negative (n_req=%lld table_width=%lld capacity=%lld)", (long long)n_req,
                  (long long)table_width, (long long)capacity);
  if (!page_ok(page_size))
    return refuse(GSI_ERR_UNSUPPORTED, "page_size=%lld is not a power of two from 16 to 256", (long long)page_size);
  if (n_req > (int64_t(1) << 20) || table_width >= (int64_t(1) << 31) / page_size || capacity > (int64_t(1) << 31) - 1)
    return refuse(GSI_ERR_UNSUPPORTED, "more than 2^20 requests or 2^31 places of a request");
  GSI_NEED(n_free, 4);
  GSI_NEED(n_free_out, 4);
  GSI_NEED(status, 4);
  if (n_req > 0) {
    GSI_NEED(kv_len, 4);
    GSI_NEED(kept, 4);
    if (table_width > 0) GSI_NEED(table, 4);
  }
  if (capacity > 0) GSI_NEED(free_pages, 4);
  if (n_free_out == n_free) return refuse(GSI_ERR_INVALID_ARG, "n_free_out is n_free: it is read and written");
  if (injected_failure()) return refuse(GSI_ERR_CUDA, "injected failure (gsi_debug_fail_after)");
  TrimArgs a{};
  a.kv_len = kv_len;
  a.kept = kept;
  a.n_req = int(n_req);
  a.table = table;
  a.width = table_width;
  a.free_pages = free_pages;
  a.capacity = capacity;
  a.n_free = n_free;
  a.page_shift = log2_of(page_size);
  a.n_free_out = n_free_out;
  a.status = status;
  return launched(launch_paged_trim(a, static_cast<cudaStream_t>(stream)), "page trim launch");
}

// The arguments that both appends share; *nothing: there is no token.
static gsi_status append_args(const gsi_cache_desc* cache, const void* X, gsi_dtype xdt, int64_t row_stride,
                              const int64_t* slots, int64_t T, int64_t n_q_heads, void* Q, AppendArgs& a, bool* nothing) {
  gsi_status s = check_cache(cache);
  if (s != GSI_OK) return s;
  if (!known(xdt)) return refuse(GSI_ERR_INVALID_ARG, "unknown dtype %d", int(xdt));
  if (T < 0 || n_q_heads < 0)
    return refuse(GSI_ERR_INVALID_ARG, "a size is negative (T=%lld n_q_heads=%lld)", (long long)T, (long long)n_q_heads);
  if (T > (int64_t(1) << 24) || n_q_heads > 4096)
    return refuse(GSI_ERR_UNSUPPORTED, "more than 2^24 tokens or 4096 heads");
  *nothing = T == 0;
  if (T == 0) return GSI_OK;
  const int64_t values = (n_q_heads + 2 * cache->n_heads) * cache->head_dim;
  if (T == 1) row_stride = 0;  // there is no next row
  if (row_stride < values && T > 1)
    return refuse(GSI_ERR_INVALID_ARG, "row_stride=%lld is below the row's %lld values", (long long)row_stride, (long long)values);
  if ((row_stride * elem(xdt)) % 16) return refuse(GSI_ERR_UNSUPPORTED, "row_stride is not a multiple of 16 bytes");
  if (row_stride >= int64_t(1) << 38) return refuse(GSI_ERR_UNSUPPORTED, "row_stride is above 2^38");
  GSI_NEED(X, 16);
  GSI_NEED(slots, 8);
  if (Q && n_q_heads > 0) GSI_NEED(Q, 16);
  a.X = X;
  a.row_stride = row_stride;
  a.slots = slots;
  a.T = int(T);
  a.hq = int(n_q_heads);
  a.hkv = int(cache->n_heads);
  a.dim = int(cache->head_dim);
  a.page_shift = log2_of(cache->page_size);
  a.n_slots = cache->n_pages * cache->page_size;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.K = cache->K;
  a.V = cache->V;
  a.Q = Q;
  return GSI_OK;
}

gsi_status gsi_cache_append(const gsi_cache_desc* cache, const void* X, gsi_dtype xdt, int64_t row_stride,
                            const int64_t* slots, int64_t T, int64_t n_q_heads, void* Q, void* stream) {
  AppendArgs a{};
  bool nothing = false;
  const gsi_status s = append_args(cache, X, xdt, row_stride, slots, T, n_q_heads, Q, a, &nothing);
  if (s != GSI_OK) return s;
  if (nothing) return record_error(GSI_OK, "");
  if (injected_failure()) return refuse(GSI_ERR_CUDA, "injected failure (gsi_debug_fail_after)");
  return launched(launch_cache_append(a, xdt, cache->dtype, static_cast<cudaStream_t>(stream)), "cache append launch");
}

gsi_status gsi_rotary_rates(int64_t dim, double base, gsi_rotary_scaling scaling, double factor, double context,
                            double fast, double slow, double* rates, float* scale) {
  if (dim <= 0 || dim % 2) return refuse(GSI_ERR_INVALID_ARG, "dim=%lld is not positive and even", (long long)dim);
  if (dim > 256) return refuse(GSI_ERR_UNSUPPORTED, "dim=%lld is above 256", (long long)dim);
  if (!(base > 1.0) || !std::isfinite(base)) return refuse(GSI_ERR_INVALID_ARG, "base must be above 1 and finite");
  if (scaling < GSI_ROTARY_NONE || scaling > GSI_ROTARY_BANDS) return refuse(GSI_ERR_INVALID_ARG, "unknown scaling %d", int(scaling));
  if (scaling != GSI_ROTARY_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return refuse(GSI_ERR_INVALID_ARG, "factor must be at least 1 and finite");
  if (scaling == GSI_ROTARY_NTK && dim <= 2) return refuse(GSI_ERR_INVALID_ARG, "a larger base needs dim above 2");
  if (scaling == GSI_ROTARY_YARN || scaling == GSI_ROTARY_BANDS) {
    if (!(context > 0.0) || !std::isfinite(context)) return refuse(GSI_ERR_INVALID_ARG, "context must be positive and finite");
    if (!(fast > slow) || !(slow > 0.0) || !std::isfinite(fast))
      return refuse(GSI_ERR_INVALID_ARG, "fast > slow > 0 is needed, both finite");
  }
  GSI_NEED(rates, 8);
  GSI_NEED(scale, 4);
  rotary_rates(int(dim), base, scaling, factor, context, fast, slow, rates, scale);
  return record_error(GSI_OK, "");
}

gsi_status gsi_rotary_phases(const double* rates, int64_t n, uint64_t* phases) {
  if (n < 0) return refuse(GSI_ERR_INVALID_ARG, "n=%lld is negative", (long long)n);
  if (n == 0) return record_error(GSI_OK, "");
  GSI_NEED(rates, 8);
  GSI_NEED(phases, 8);
  for (int64_t i = 0; i < n; ++i)
    if (!(std::fabs(rates[i]) <= 1099511627776.0))
      return refuse(GSI_ERR_INVALID_ARG, "rate %lld is not finite, or above 2^40 in magnitude", (long long)i);
  for (int64_t i = 0; i < n; ++i) phases[i] = rotary_phase(rates[i]);
  return record_error(GSI_OK, "");
}

gsi_status gsi_rotary_append(const gsi_cache_desc* cache, const void* X, gsi_dtype xdt, int64_t row_stride,
                             const int64_t* slots, const int32_t* positions, const int32_t* token_req,
                             const int32_t* offsets, int64_t n_req, int64_t T, int64_t n_q_heads,
                             const gsi_rotary* rotary, void* Q, void* stream) {
  RotaryArgs r{};
  bool nothing = false;
  const gsi_status s = append_args(cache, X, xdt, row_stride, slots, T, n_q_heads, Q, r.to, &nothing);
  if (s != GSI_OK) return s;
  if (!rotary) return refuse(GSI_ERR_INVALID_ARG, "rotary is NULL");
  if (rotary->layout != GSI_ROTARY_HALF && rotary->layout != GSI_ROTARY_PAIRS)
    return refuse(GSI_ERR_INVALID_ARG, "unknown layout %d", int(rotary->layout));
  if (rotary->dim <= 0 || rotary->dim % 2 || rotary->dim > cache->head_dim)
    return refuse(GSI_ERR_INVALID_ARG, "rotary dim=%lld is not even and within 2 .. %lld", (long long)rotary->dim,
                  (long long)cache->head_dim);
  if (!std::isfinite(rotary->scale)) return refuse(GSI_ERR_INVALID_ARG, "scale must be finite");
  if (n_req < 0) return refuse(GSI_ERR_INVALID_ARG, "a size is negative (n_req=%lld)", (long long)n_req);
  if (n_req > (int64_t(1) << 20)) return refuse(GSI_ERR_UNSUPPORTED, "more than 2^20 requests");
  if (nothing) return record_error(GSI_OK, "");
  const uint64_t* phases = rotary->phases;
  GSI_NEED(phases, 8);
  GSI_NEED(positions, 4);
  if (!on(token_req, 4) || !on(offsets, 4)) return refuse(GSI_ERR_INVALID_ARG, "token_req or offsets is not 4-byte aligned");
  if (injected_failure()) return refuse(GSI_ERR_CUDA, "injected failure (gsi_debug_fail_after)");
  r.positions = positions;
  r.token_req = token_req;
  r.offsets = offsets;
  r.n_req = int(n_req);
  r.turned = int(rotary->dim);
  r.pairs = rotary->layout == GSI_ROTARY_PAIRS;
  r.scale = rotary->scale;
  r.phases = phases;
  return launched(launch_rotary_append(r, xdt, cache->dtype, static_cast<cudaStream_t>(stream)), "rotary append launch");
}

size_t gsi_paged_attention_workspace_size(const gsi_cache_desc* cache, int64_t n_q_heads) {
  if (check_cache(cache) != GSI_OK || check_heads(cache, n_q_heads) != GSI_OK) return 0;
  record_error(GSI_OK, "");
  return attention_work_bytes(cache->dtype, int(cache->head_dim), int(n_q_heads / cache->n_heads));
}

gsi_status gsi_paged_attention_lse(const gsi_cache_desc* cache, const void* Q, int64_t q_stride, int64_t N,
                                   int64_t n_q_heads, const int32_t* q_start, const int32_t* kv_len,
                                   const int32_t* table, int64_t table_width, int64_t n_req, int64_t max_q, float scale,
                                   int causal, int64_t window, void* O, float* LSE, void* workspace, size_t ws_bytes,
                                   void* stream) {
  gsi_status s = check_cache(cache);
  if (s != GSI_OK) return s;
  if (N < 0 || n_req < 0 || table_width < 0 || max_q < 0)
    return refuse(GSI_ERR_INVALID_ARG, "a size is negative (N=%lld n_req=%lld table_width=%lld max_q=%lld)", (long long)N,
                  (long long)n_req, (long long)table_width, (long long)max_q);
  if ((s = check_heads(cache, n_q_heads)) != GSI_OK) return s;
  if (!std::isfinite(scale)) return refuse(GSI_ERR_INVALID_ARG, "scale must be finite");
  if (window < 0 || (window > 0 && !causal))
    return refuse(GSI_ERR_INVALID_ARG, "window must be >= 0, and 0 where the attention is not causal");
  if (N > (int64_t(1) << 24) || n_req > (int64_t(1) << 20) ||
      table_width > ((int64_t(1) << 31) - 512) / cache->page_size)  // a tile's end stays within 31 bits
    return refuse(GSI_ERR_UNSUPPORTED, "more than 2^24 tokens, 2^20 requests or 2^31 - 512 places of a request");
  if (N == 0 || n_req == 0) return record_error(GSI_OK, "");
  const int64_t values = n_q_heads * cache->head_dim;
  if (N == 1) q_stride = values;  // there is no next row
  if (q_stride < values)
    return refuse(GSI_ERR_INVALID_ARG, "q_stride=%lld is below the row's %lld values", (long long)q_stride, (long long)values);
  if ((q_stride * elem(cache->dtype)) % 16) return refuse(GSI_ERR_UNSUPPORTED, "q_stride is not a multiple of 16 bytes");
  if (q_stride >= int64_t(1) << 38) return refuse(GSI_ERR_UNSUPPORTED, "q_stride is above 2^38");
  GSI_NEED(Q, 16);
  GSI_NEED(O, 16);
  if (!on(LSE, 4)) return refuse(GSI_ERR_INVALID_ARG, "LSE is not 4-byte aligned");
  GSI_NEED(q_start, 4);
  GSI_NEED(kv_len, 4);
  if (table_width > 0) GSI_NEED(table, 4);
  const size_t want = attention_work_bytes(cache->dtype, int(cache->head_dim), int(n_q_heads / cache->n_heads));
  if (!workspace) return refuse(GSI_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", want);
  if (!on(workspace, 256)) return refuse(GSI_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < want) return refuse(GSI_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", ws_bytes, want);
  if (injected_failure()) return refuse(GSI_ERR_CUDA, "injected failure (gsi_debug_fail_after)");
  AttnArgs a{};
  a.K = cache->K;
  a.V = cache->V;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.n_pages = cache->n_pages;
  a.page_shift = log2_of(cache->page_size);
  a.hkv = int(cache->n_heads);
  a.group = int(n_q_heads / cache->n_heads);
  a.dim = int(cache->head_dim);
  a.Q = Q;
  a.q_stride = q_stride;
  a.O = O;
  a.N = int(N);
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.table = table;
  a.width = cache->n_pages ? table_width : 0;  // an empty cache holds no keys
  a.n_req = int(n_req);
  a.scale = scale;
  a.causal = causal != 0;
  // a window of 2^31 or more hides nothing
  a.window = window >= (int64_t(1) << 31) ? 0 : int(window);
  a.work = workspace;
  a.LSE = LSE;
  return launched(launch_paged_attention(a, cache->dtype, max_q, static_cast<cudaStream_t>(stream)), "paged attention launch");
}

gsi_status gsi_paged_attention(const gsi_cache_desc* cache, const void* Q, int64_t q_stride, int64_t N,
                               int64_t n_q_heads, const int32_t* q_start, const int32_t* kv_len,
                               const int32_t* table, int64_t table_width, int64_t n_req, int64_t max_q, float scale,
                               int causal, int64_t window, void* O, void* workspace, size_t ws_bytes, void* stream) {
  return gsi_paged_attention_lse(cache, Q, q_stride, N, n_q_heads, q_start, kv_len, table, table_width, n_req, max_q, scale,
                                 causal, window, O, nullptr, workspace, ws_bytes, stream);
}

static gsi_status check_marks(const gsi_cache_desc* c, const gsi_key_marks* m) {
  if (!m) return refuse(GSI_ERR_INVALID_ARG, "marks is NULL");
  if (c->n_pages == 0) return GSI_OK;
  const float* weight = m->weight;
  const int32_t* place = m->place;
  GSI_NEED(weight, 16);
  GSI_NEED(place, 16);
  return GSI_OK;
}

size_t gsi_key_weights_workspace_size(void) { return key_weights_work_bytes(); }

gsi_status gsi_key_weights(const gsi_cache_desc* cache, const void* Q, int64_t q_stride, int64_t N, int64_t n_q_heads,
                           const float* LSE, const int32_t* q_start, const int32_t* kv_len, const int32_t* held,
                           const int32_t* offsets, const int32_t* table, int64_t table_width, int64_t n_req,
                           int64_t max_q, float scale, int causal, const gsi_key_marks* marks, void* workspace,
                           size_t ws_bytes, void* stream) {
  gsi_status s = check_cache(cache);
  if (s != GSI_OK) return s;
  if (N < 0 || n_req < 0 || table_width < 0 || max_q < 0)
    return refuse(GSI_ERR_INVALID_ARG, "a size is negative (N=%lld n_req=%lld table_width=%lld max_q=%lld)", (long long)N,
                  (long long)n_req, (long long)table_width, (long long)max_q);
  if ((s = check_heads(cache, n_q_heads)) != GSI_OK) return s;
  if (!std::isfinite(scale)) return refuse(GSI_ERR_INVALID_ARG, "scale must be finite");
  if (N > (int64_t(1) << 24) || n_req > (int64_t(1) << 20) || table_width > ((int64_t(1) << 31) - 512) / cache->page_size)
    return refuse(GSI_ERR_UNSUPPORTED, "more than 2^24 tokens, 2^20 requests or 2^31 - 512 places of a request");
  if ((s = check_marks(cache, marks)) != GSI_OK) return s;
  if (n_req == 0 || table_width == 0 || cache->n_pages == 0) return record_error(GSI_OK, "");
  const int64_t values = n_q_heads * cache->head_dim;
  if (N <= 1) q_stride = values;  // there is no next row
  if (q_stride < values)
    return refuse(GSI_ERR_INVALID_ARG, "q_stride=%lld is below the row's %lld values", (long long)q_stride, (long long)values);
  if ((q_stride * elem(cache->dtype)) % 16) return refuse(GSI_ERR_UNSUPPORTED, "q_stride is not a multiple of 16 bytes");
  if (q_stride >= int64_t(1) << 38) return refuse(GSI_ERR_UNSUPPORTED, "q_stride is above 2^38");
  if (N > 0) {
    GSI_NEED(Q, 16);
    GSI_NEED(LSE, 4);
  }
  GSI_NEED(q_start, 4);
  GSI_NEED(kv_len, 4);
  GSI_NEED(table, 4);
  if (!on(held, 4) || !on(offsets, 4)) return refuse(GSI_ERR_INVALID_ARG, "held or offsets is not 4-byte aligned");
  const size_t want = key_weights_work_bytes();
  if (!workspace) return refuse(GSI_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", want);
  if (!on(workspace, 256)) return refuse(GSI_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < want) return refuse(GSI_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", ws_bytes, want);
  if (injected_failure()) return refuse(GSI_ERR_CUDA, "injected failure (gsi_debug_fail_after)");
  KeyWeightArgs a{};
  a.K = cache->K;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.n_pages = cache->n_pages;
  a.page_shift = log2_of(cache->page_size);
  a.hkv = int(cache->n_heads);
  a.group = int(n_q_heads / cache->n_heads);
  a.dim = int(cache->head_dim);
  a.Q = Q;
  a.q_stride = q_stride;
  a.LSE = LSE;
  a.N = int(N);
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.held = held;
  a.offsets = offsets;
  a.table = table;
  a.width = table_width;
  a.n_req = int(n_req);
  a.scale = scale;
  a.causal = causal != 0;
  a.weight = marks->weight;
  a.place = marks->place;
  a.work = workspace;
  return launched(launch_key_weights(a, cache->dtype, max_q, static_cast<cudaStream_t>(stream)), "key weights launch");
}

static gsi_status check_evict(const gsi_cache_desc* cache, int64_t n_req, int64_t budget) {
  const gsi_status s = check_cache(cache);
  if (s != GSI_OK) return s;
  if (n_req < 0) return refuse(GSI_ERR_INVALID_ARG, "a size is negative (n_req=%lld)", (long long)n_req);
  if (budget < 1) return refuse(GSI_ERR_INVALID_ARG, "budget=%lld is not positive", (long long)budget);
  if (n_req > (int64_t(1) << 20) || n_req * cache->n_heads > int64_t(1) << 27 || budget > (int64_t(1) << 31) - 1)
    return refuse(GSI_ERR_UNSUPPORTED, "more than 2^20 requests, 2^27 heads of them or 2^31 keys");
  return GSI_OK;
}

size_t gsi_cache_evict_workspace_size(const gsi_cache_desc* cache, int64_t n_req, int64_t budget) {
  if (check_evict(cache, n_req, budget) != GSI_OK) return 0;
  record_error(GSI_OK, "");
  return evict_work_bytes(n_req * cache->n_heads, budget);
}

gsi_status gsi_cache_evict(const gsi_cache_desc* cache, const int32_t* kv_len, const int32_t* table,
                           int64_t table_width, int64_t n_req, const gsi_key_marks* marks, int64_t budget,
                           int64_t recent, int64_t sinks, const int32_t* offsets, int32_t* kept, int32_t* offsets_out,
                           void* workspace, size_t ws_bytes, void* stream) {
  gsi_status s = check_evict(cache, n_req, budget);
  if (s != GSI_OK) return s;
  if (recent < 0 || sinks < 0 || recent > budget || sinks > budget - recent)
    return refuse(GSI_ERR_INVALID_ARG, "recent=%lld and sinks=%lld are not within the budget of %lld", (long long)recent,
                  (long long)sinks, (long long)budget);
  if (table_width < 0) return refuse(GSI_ERR_INVALID_ARG, "a size is negative (table_width=%lld)", (long long)table_width);
  if (table_width > ((int64_t(1) << 31) - 512) / cache->page_size)
    return refuse(GSI_ERR_UNSUPPORTED, "more than 2^31 - 512 places of a request");
  if ((s = check_marks(cache, marks)) != GSI_OK) return s;
  if (n_req == 0) return record_error(GSI_OK, "");
  GSI_NEED(kv_len, 4);
  if (table_width > 0) GSI_NEED(table, 4);
  GSI_NEED(kept, 4);
  if (!on(offsets, 4) || !on(offsets_out, 4)) return refuse(GSI_ERR_INVALID_ARG, "offsets or offsets_out is not 4-byte aligned");
  if (kept == kv_len || kept == offsets || (offsets_out && (offsets_out == offsets || offsets_out == kv_len || offsets_out == kept)))
    return refuse(GSI_ERR_INVALID_ARG, "kept or offsets_out is an array that is read, or both are one");
  const size_t want = evict_work_bytes(n_req * cache->n_heads, budget);
  if (!workspace) return refuse(GSI_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", want);
  if (!on(workspace, 256)) return refuse(GSI_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < want) return refuse(GSI_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", ws_bytes, want);
  if (injected_failure()) return refuse(GSI_ERR_CUDA, "injected failure (gsi_debug_fail_after)");
  EvictArgs a{};
  a.K = cache->K;
  a.V = cache->V;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.n_pages = cache->n_pages;
  a.page_shift = log2_of(cache->page_size);
  a.hkv = int(cache->n_heads);
  a.elem = elem(cache->dtype);
  a.row_bytes = int(cache->head_dim) * a.elem;
  a.kv_len = kv_len;
  a.table = table;
  a.width = table_width;
  a.n_req = int(n_req);
  a.weight = marks->weight;
  a.place = marks->place;
  a.budget = int(budget);
  a.recent = int(recent);
  a.sinks = int(sinks);
  a.offsets = offsets;
  a.kept = kept;
  a.offsets_out = offsets_out;
  a.moves = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + kEvictMovesAt);
  a.err = &static_cast<Ctrl*>(workspace)->err;
  return launched(launch_cache_evict(a, static_cast<cudaStream_t>(stream)), "cache eviction launch");
}

gsi_status gsi_verify_drafts(const void* target, gsi_dtype tdt, int64_t target_stride, const void* draft, gsi_dtype ddt,
                             int64_t draft_stride, int64_t N, int64_t vocab, const int32_t* tokens,
                             const float* uniforms, const float* samples, const int32_t* q_start,
                             const int32_t* kv_len, int64_t n_req, int32_t* out, int32_t* accepted, int32_t* kept,
                             void* stream) {
  if (!known(tdt) || (draft && !known(ddt))) return refuse(GSI_ERR_INVALID_ARG, "unknown dtype");
  if (N < 0 || n_req < 0 || vocab <= 0)
    return refuse(GSI_ERR_INVALID_ARG, "sizes must be positive (N=%lld n_req=%lld vocab=%lld)", (long long)N, (long long)n_req,
                  (long long)vocab);
  if (N > (int64_t(1) << 24) || n_req > (int64_t(1) << 20) || vocab > (int64_t(1) << 24))
    return refuse(GSI_ERR_UNSUPPORTED, "more than 2^24 rows, 2^20 requests or 2^24 tokens of a vocabulary");
  if (n_req == 0) return record_error(GSI_OK, "");
  if (N <= 1) target_stride = draft_stride = vocab;  // there is no next row
  if (target_stride < vocab || (draft && draft_stride < vocab))
    return refuse(GSI_ERR_INVALID_ARG, "a row's stride is below its %lld values", (long long)vocab);
  if (target_stride >= int64_t(1) << 38 || (draft && draft_stride >= int64_t(1) << 38))
    return refuse(GSI_ERR_UNSUPPORTED, "a row's stride is above 2^38");
  if (N > 0) {
    GSI_NEED(target, uintptr_t(elem(tdt)));
    if (draft) GSI_NEED(draft, uintptr_t(elem(ddt)));
    GSI_NEED(tokens, 4);
    GSI_NEED(uniforms, 4);
    GSI_NEED(samples, 4);
    GSI_NEED(out, 4);
    if (out == tokens) return refuse(GSI_ERR_INVALID_ARG, "out is tokens: they are read and written");
  }
  GSI_NEED(q_start, 4);
  GSI_NEED(accepted, 4);
  if ((kv_len == nullptr) != (kept == nullptr)) return refuse(GSI_ERR_INVALID_ARG, "kept and kv_len go together");
  if (!on(kv_len, 4) || !on(kept, 4)) return refuse(GSI_ERR_INVALID_ARG, "kv_len or kept is not 4-byte aligned");
  if (accepted == kept || accepted == kv_len) return refuse(GSI_ERR_INVALID_ARG, "accepted is kept or kv_len");
  if (injected_failure()) return refuse(GSI_ERR_CUDA, "injected failure (gsi_debug_fail_after)");
  VerifyArgs a{};
  a.target = target;
  a.target_stride = target_stride;
  a.draft = draft;
  a.draft_stride = draft_stride;
  a.N = int(N);
  a.vocab = int(vocab);
  a.tokens = tokens;
  a.uniforms = uniforms;
  a.samples = samples;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.n_req = int(n_req);
  a.out = out;
  a.accepted = accepted;
  a.kept = kept;
  return launched(launch_verify_drafts(a, tdt, draft ? ddt : tdt, static_cast<cudaStream_t>(stream)), "draft verification launch");
}

gsi_status gsi_norm_residual(const void* H, gsi_dtype hdt, const void* Y, gsi_dtype ydt, int64_t T, int64_t d,
                             float alpha, const gsi_norm* post, const float* gate, int64_t gate_rows,
                             const int32_t* gate_index, const gsi_norm* pre, void* H_out, void* X, gsi_dtype xdt,
                             void* stream) {
  if (!known(hdt) || !known(ydt) || !known(xdt)) return refuse(GSI_ERR_INVALID_ARG, "unknown dtype");
  if (T < 0 || d <= 0) return refuse(GSI_ERR_INVALID_ARG, "sizes must be positive (T=%lld d=%lld)", (long long)T, (long long)d);
  if (d % 8 || d > 16384) return refuse(GSI_ERR_UNSUPPORTED, "d=%lld is not a multiple of 8 or above 16384", (long long)d);
  if (T > (int64_t(1) << 24)) return refuse(GSI_ERR_UNSUPPORTED, "T=%lld above 2^24", (long long)T);
  if (!std::isfinite(alpha)) return refuse(GSI_ERR_INVALID_ARG, "alpha must be finite");
  gsi_status s = check_norm(post, "post");
  if (s != GSI_OK) return s;
  if ((s = check_norm(pre, "pre")) != GSI_OK) return s;
  if (gate && gate_rows < 1) return refuse(GSI_ERR_INVALID_ARG, "gate_rows=%lld is not positive", (long long)gate_rows);
  if (gate && gate_rows > (int64_t(1) << 31) - 1) return refuse(GSI_ERR_UNSUPPORTED, "gate_rows above 2^31");
  if (T == 0) return record_error(GSI_OK, "");
  GSI_NEED(H, 16);
  if (!on(Y, 16) || !on(gate, 16) || !on(H_out, 16) || !on(X, 16))
    return refuse(GSI_ERR_INVALID_ARG, "Y, gate, H_out or X is not 16-byte aligned");
  if (gate_index && !on(gate_index, 4)) return refuse(GSI_ERR_INVALID_ARG, "gate_index is not 4-byte aligned");
  if (!H_out && !X) return refuse(GSI_ERR_INVALID_ARG, "H_out and X are both NULL");
  if (injected_failure()) return refuse(GSI_ERR_CUDA, "injected failure (gsi_debug_fail_after)");
  NormArgs a{};
  a.H = H;
  a.Y = Y;
  a.T = int(T);
  a.d = int(d);
  a.alpha = alpha;
  if (post) {
    a.post = post->kind;
    a.post_eps = post->eps;
    a.post_w = post->weight;
    a.post_b = post->bias;
  }
  if (pre) {
    a.pre = pre->kind;
    a.pre_eps = pre->eps;
    a.pre_w = pre->weight;
    a.pre_b = pre->bias;
  }
  a.gate = gate;
  a.gate_rows = int(gate_rows);
  a.gate_index = gate_index;
  a.H_out = H_out;
  a.X = X;
  return launched(launch_norm_residual(a, hdt, ydt, xdt, static_cast<cudaStream_t>(stream)), "norm launch");
}

}  // extern "C"
