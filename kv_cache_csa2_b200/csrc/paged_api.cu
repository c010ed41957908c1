// The C ABI of the head and paged-cache calls (include/csa2.h, part p): argument
// validation, strides filled in, dispatch to the launchers.
#include <algorithm>

#include "common.cuh"
#include "paged.h"

using namespace csa2;

#define REQUIRE(cond, ...) \
  do {                     \
    if (!(cond)) return fail(CSA2_ERR_INVALID, __VA_ARGS__); \
  } while (0)

namespace {

bool known(csa2_dtype t) { return t == CSA2_BF16 || t == CSA2_F16; }

// csa2_heads -> HeadRows (checked; T rows of D channels).
csa2_status rows_of(const char* fn, const char* name, const csa2_heads* h, int64_t T, int D, HeadRows* out) {
  REQUIRE(h->heads > 0 && h->heads <= 65535, "%s: %s has %d heads", fn, name, h->heads);
  out->heads = h->heads;
  out->head_stride = h->head_stride ? h->head_stride : D;
  out->token_stride = h->token_stride ? h->token_stride : static_cast<int64_t>(h->heads) * out->head_stride;
  REQUIRE(out->head_stride % 8 == 0 && out->token_stride % 8 == 0 && out->head_stride >= 0 && out->token_stride >= 0,
          "%s: %s strides (%lld, %lld) must be non-negative multiples of 8", fn, name,
          (long long)out->token_stride, (long long)out->head_stride);
  out->data = h->data;
  if (T > 0) REQUIRE(h->data != nullptr && aligned16(h->data), "%s: %s is null or not 16-byte aligned", fn, name);
  return CSA2_OK;
}

// An output's rows must not overlap one another: token-major or head-major.
csa2_status distinct_rows(const char* fn, const char* name, const HeadRows& r, int64_t T, int D) {
  const int64_t h = r.head_stride, t = r.token_stride, H = r.heads;
  const bool token_major = (H <= 1 || h >= D) && (T <= 1 || t >= (H - 1) * h + D);
  const bool head_major = (T <= 1 || t >= D) && (H <= 1 || h >= (T - 1) * t + D);
  REQUIRE(token_major || head_major, "%s: %s rows overlap (strides %lld, %lld)", fn, name, (long long)t, (long long)h);
  return CSA2_OK;
}

// The rows of a cache that is written must not overlap one another: taken from the smallest
// stride up, each dimension steps over all that lies within.
csa2_status distinct_cache_rows(const char* fn, const csa2_paged_kv* c, const PagedView& v) {
  struct Dim {
    int64_t n, stride;
  } d[3] = {{c->heads, v.head_stride}, {c->page_size, v.token_stride}, {c->n_pages, v.page_stride}};
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t extent = c->dim;
  for (const Dim& x : d) {
    if (x.n <= 1) continue;
    REQUIRE(x.stride >= extent, "%s: cache rows overlap (strides %lld, %lld, %lld)", fn, (long long)v.page_stride,
            (long long)v.token_stride, (long long)v.head_stride);
    extent += (x.n - 1) * x.stride;
  }
  return CSA2_OK;
}

csa2_status rope_of(const char* fn, const csa2_rope* r, int D, rope::RopeArgs* out) {
  *out = rope::RopeArgs{nullptr, 0, 0, 0, 0};
  if (!r) return CSA2_OK;
  REQUIRE(r->half > 0 && r->half % 8 == 0 && r->half <= rope::kMaxHalf && r->offset >= 0 && r->offset % 8 == 0 &&
              r->offset <= D - 2 * r->half,
          "%s: rotation of channels [%d, %d + 2*%d) of %d: half and offset must be multiples of 8 inside the row", fn,
          r->offset, r->offset, r->half, D);
  REQUIRE(r->inv_freq != nullptr, "%s: rotation without inv_freq", fn);
  *out = rope::RopeArgs{r->inv_freq, r->half, r->offset, r->interleaved ? 1 : 0, r->inverse ? 1 : 0};
  return CSA2_OK;
}

csa2_status view_of(const char* fn, const csa2_paged_kv* c, PagedView* v, int64_t* max_len) {
  REQUIRE(c != nullptr, "%s: cache is null", fn);
  REQUIRE(c->fmt == CSA2_KV_BF16 || c->fmt == CSA2_KV_FP4 || c->fmt == CSA2_KV_F16, "%s: unknown cache format %d", fn,
          int(c->fmt));
  const bool fp4 = c->fmt == CSA2_KV_FP4;
  REQUIRE(c->dim > 0 && c->dim <= 512 && c->dim % (fp4 ? 32 : 8) == 0, "%s: cache width %d", fn, c->dim);
  REQUIRE(c->heads > 0 && c->heads <= 65535, "%s: cache has %d heads", fn, c->heads);
  REQUIRE(c->page_size >= 1 && c->page_size <= 65536 && (c->page_size & (c->page_size - 1)) == 0,
          "%s: page_size=%d must be a power of two up to 65536", fn, c->page_size);
  REQUIRE(c->n_pages >= 0 && c->n_pages <= 0x7fffffffLL && c->max_pages >= 0 && c->B >= 0 && c->max_len >= 0,
          "%s: negative size", fn);
  REQUIRE(c->table_stride == 0 || c->table_stride >= c->max_pages, "%s: table_stride %lld < max_pages %d", fn,
          (long long)c->table_stride, c->max_pages);
  v->head_stride = c->head_stride;
  v->token_stride = c->token_stride;
  v->page_stride = c->page_stride;
  if (!c->head_stride && !c->token_stride && !c->page_stride) {
    v->head_stride = c->dim;
    v->token_stride = static_cast<int64_t>(c->heads) * c->dim;
    v->page_stride = v->token_stride * c->page_size;
  }
  const int unit = fp4 ? 32 : 8;
  REQUIRE(v->head_stride % unit == 0 && v->token_stride % unit == 0 && v->page_stride % unit == 0 &&
              (v->head_stride >= c->dim || c->heads == 1) && (v->token_stride >= c->dim || c->page_size == 1) &&
              (v->page_stride >= c->dim || c->n_pages <= 1),
          "%s: cache strides (%lld, %lld, %lld) must be multiples of %d and at least the row", fn,
          (long long)v->page_stride, (long long)v->token_stride, (long long)v->head_stride, unit);
  if (c->n_pages > 0) {
    REQUIRE(c->k != nullptr && aligned16(c->k) && aligned16(c->v), "%s: cache rows null or not 16-byte aligned", fn);
    const bool own_v = c->v != nullptr && c->v != c->k;
    REQUIRE(!fp4 || (c->k_scales != nullptr && (!own_v || c->v_scales != nullptr)), "%s: FP4 cache without scales", fn);
    REQUIRE(!fp4 || (((reinterpret_cast<uintptr_t>(c->k_scales) | reinterpret_cast<uintptr_t>(c->v_scales)) & 1u) == 0),
            "%s: FP4 scales not 2-byte aligned", fn);
  }
  v->k = static_cast<const uint8_t*>(c->k);
  v->v = c->v ? static_cast<const uint8_t*>(c->v) : v->k;
  v->k_scales = c->k_scales;
  v->v_scales = v->v == v->k ? c->k_scales : c->v_scales;
  v->table = c->table;
  v->lens = c->lens;
  v->table_stride = c->table_stride ? c->table_stride : c->max_pages;
  v->n_pages = c->n_pages;
  v->page_shift = 0;
  while ((1 << v->page_shift) < c->page_size) ++v->page_shift;
  v->capacity = static_cast<int64_t>(c->max_pages) << v->page_shift;
  if (v->capacity > 0x7fffffffLL) v->capacity = 0x7fffffffLL;   // positions are int32
  v->heads = c->heads;
  v->B = c->B;
  if (max_len) *max_len = c->max_len > 0 && c->max_len < v->capacity ? c->max_len : v->capacity;
  return CSA2_OK;
}

// Checks shared by the two attention calls; fills everything but out / lse / error word.
csa2_status attn_of(const char* fn, const csa2_heads* q, int64_t T, const csa2_paged_kv* cache, float scale, int window,
                    int sinks, PagedAttn* a, int64_t* max_len) {
  CSA2_TRY(view_of(fn, cache, &a->kv, max_len));
  REQUIRE(cache->dim == 64 || cache->dim == 128 || cache->dim == 256 || cache->dim == 512,
          "%s: width %d must be 64, 128, 256 or 512", fn, cache->dim);
  REQUIRE(cache->fmt != CSA2_KV_FP4 || ((a->kv.head_stride | a->kv.token_stride | a->kv.page_stride) % 64 == 0 &&
                                        ((reinterpret_cast<uintptr_t>(a->kv.k_scales) |
                                          reinterpret_cast<uintptr_t>(a->kv.v_scales)) & 3u) == 0),
          "%s: an FP4 cache needs strides in multiples of 64 and 4-byte aligned scales", fn);
  REQUIRE(window >= 0 && sinks >= 0, "%s: negative window or sinks", fn);
  HeadRows rows;
  REQUIRE(q != nullptr, "%s: q is null", fn);
  CSA2_TRY(rows_of(fn, "q", q, T, cache->dim, &rows));
  REQUIRE(rows.heads % cache->heads == 0, "%s: %d query heads over %d cache heads", fn, rows.heads, cache->heads);
  a->fmt = cache->fmt;
  a->D = cache->dim;
  a->Hq = rows.heads;
  a->G = rows.heads / cache->heads;
  a->q = rows.data;
  a->q_token = rows.token_stride;
  a->q_head = rows.head_stride;
  a->scale = scale;
  a->window = window;
  a->sinks = sinks;
  if (T > 0 && cache->B > 0)
    REQUIRE(cache->lens != nullptr && (cache->table != nullptr || cache->max_pages == 0), "%s: lens or table is null", fn);
  return CSA2_OK;
}

}  // namespace

extern "C" {

csa2_status csa2_qk_norm_rope(csa2_dtype dtype, const csa2_heads* q, const float* q_weight,
                              const csa2_heads* q_out, const csa2_heads* k, const float* k_weight,
                              const csa2_heads* k_out, int64_t T, int D, float eps,
                              const int32_t* positions, const csa2_rope* rope, csa2_stream stream) {
  CSA2_TRY(fault_gate());
  const char* fn = "csa2_qk_norm_rope";
  REQUIRE(known(dtype), "%s: unknown dtype %d", fn, int(dtype));
  REQUIRE(T >= 0, "%s: T=%lld is negative", fn, (long long)T);
  REQUIRE(D >= 8 && D <= 512 && D % 8 == 0, "%s: D=%d must be a multiple of 8 in [8, 512]", fn, D);
  REQUIRE(q || k, "%s: neither q nor k given", fn);
  rope::RopeArgs r;
  CSA2_TRY(rope_of(fn, rope, D, &r));
  HeadRows in[2], out[2];
  const csa2_heads *ins[2] = {q, k}, *outs[2] = {q_out, k_out};
  const char *names[2] = {"q", "k"}, *onames[2] = {"q_out", "k_out"};
  for (int i = 0; i < 2; ++i) {
    if (!ins[i]) continue;
    CSA2_TRY(rows_of(fn, names[i], ins[i], T, D, &in[i]));
    REQUIRE(outs[i] != nullptr && outs[i]->heads == ins[i]->heads, "%s: %s is missing or has other heads than %s", fn,
            onames[i], names[i]);
    CSA2_TRY(rows_of(fn, onames[i], outs[i], T, D, &out[i]));
    CSA2_TRY(distinct_rows(fn, onames[i], out[i], T, D));
    REQUIRE(out[i].data != in[i].data || (out[i].token_stride == in[i].token_stride && out[i].head_stride == in[i].head_stride),
            "%s: %s starts at %s with other strides", fn, onames[i], names[i]);
  }
  REQUIRE(aligned16(q_weight) && aligned16(k_weight), "%s: weights not 16-byte aligned", fn);
  if (T == 0) return CSA2_OK;
  REQUIRE(!rope || positions, "%s: rotation without positions", fn);
  return launch_head_norm(dtype, in[0], q_weight, out[0], in[1], k_weight, out[1], T, D, eps, positions, r,
                          reinterpret_cast<cudaStream_t>(stream));
}

csa2_status csa2_paged_append(csa2_dtype dtype, const csa2_heads* k, const csa2_heads* v,
                              const int32_t* seq, const int32_t* pos, int64_t T,
                              const csa2_rope* rope, const csa2_paged_kv* cache,
                              csa2_stream stream) {
  CSA2_TRY(fault_gate());
  const char* fn = "csa2_paged_append";
  REQUIRE(known(dtype), "%s: unknown dtype %d", fn, int(dtype));
  REQUIRE(T >= 0, "%s: T=%lld is negative", fn, (long long)T);
  PagedView view;
  CSA2_TRY(view_of(fn, cache, &view, nullptr));
  CSA2_TRY(distinct_cache_rows(fn, cache, view));
  const bool fp4 = cache->fmt == CSA2_KV_FP4;
  REQUIRE((dtype == CSA2_F16) == (cache->fmt == CSA2_KV_F16), "%s: dtype %d does not match cache format %d", fn,
          int(dtype), int(cache->fmt));
  const bool shared = view.v == view.k;
  REQUIRE(k != nullptr && (v == nullptr) == shared, "%s: k is null, or v does not match a %s cache", fn,
          shared ? "shared" : "separate");
  rope::RopeArgs r;
  CSA2_TRY(rope_of(fn, rope, cache->dim, &r));
  REQUIRE(!fp4 || (r.half % 16 == 0 && r.offset % 16 == 0), "%s: FP4 needs rope half and offset in multiples of 16", fn);
  HeadRows kr, vr;
  CSA2_TRY(rows_of(fn, "k", k, T, cache->dim, &kr));
  if (v) CSA2_TRY(rows_of(fn, "v", v, T, cache->dim, &vr));
  REQUIRE(kr.heads == cache->heads && (!v || vr.heads == cache->heads), "%s: rows and cache differ in heads", fn);
  if (T == 0) return CSA2_OK;
  REQUIRE(seq && pos && (cache->B == 0 || cache->max_pages == 0 || cache->table), "%s: seq, pos or table is null", fn);
  view.err = device_error_word();
  return launch_paged_append(dtype, kr, vr, seq, pos, T, cache->dim, fp4, r, view,
                             reinterpret_cast<cudaStream_t>(stream));
}

size_t csa2_paged_decode_attn_workspace(const csa2_paged_kv* cache, int Hq, int window, int sinks, int chunk) {
  PagedAttn a = {};
  int64_t max_len = 0;
  if (view_of("csa2_paged_decode_attn_workspace", cache, &a.kv, &max_len) != CSA2_OK || Hq <= 0 ||
      Hq % cache->heads != 0 || window < 0 || sinks < 0 || chunk < 0 || chunk % 64 != 0)
    return 0;
  a.fmt = cache->fmt;
  a.D = cache->dim;
  a.Hq = Hq;
  a.G = Hq / cache->heads;
  a.window = window;
  a.sinks = sinks;
  return paged_decode_workspace(a, max_len, chunk);
}

csa2_status csa2_paged_decode_attn(const csa2_heads* q, const csa2_paged_kv* cache, float scale,
                                   int window, int sinks, int chunk, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, csa2_stream stream) {
  CSA2_TRY(fault_gate());
  const char* fn = "csa2_paged_decode_attn";
  PagedAttn a = {};
  int64_t max_len = 0;
  CSA2_TRY(attn_of(fn, q, cache ? cache->B : 0, cache, scale, window, sinks, &a, &max_len));
  REQUIRE(chunk >= 0 && chunk % 64 == 0, "%s: chunk=%d must be a multiple of 64", fn, chunk);
  if (cache->B == 0) return CSA2_OK;
  REQUIRE(cache->B <= 65535, "%s: B=%d above 65535", fn, cache->B);
  if (static_cast<int64_t>(a.kv.heads) * ((a.G + 15) / 16) > 65535)
    return fail(CSA2_ERR_UNSUPPORTED, "%s: %d query heads over %d cache heads", fn, a.Hq, a.kv.heads);
  REQUIRE(out != nullptr && aligned16(out), "%s: out is null or not 16-byte aligned", fn);
  const size_t need = paged_decode_workspace(a, max_len, chunk);
  if (workspace_bytes < need || (need > 0 && (!workspace || !aligned16(workspace))))
    return fail(CSA2_ERR_OOM, "%s: workspace %zu < %zu bytes, or not 16-byte aligned", fn, workspace_bytes, need);
  a.out = out;
  a.lse = lse;
  a.kv.err = device_error_word();
  return launch_paged_decode(a, max_len, chunk, workspace, reinterpret_cast<cudaStream_t>(stream));
}

csa2_status csa2_paged_window_attn(const csa2_heads* q, const int32_t* cu_q, int64_t T,
                                   const csa2_paged_kv* cache, float scale, int window, int sinks,
                                   void* out, float* lse, csa2_stream stream) {
  CSA2_TRY(fault_gate());
  const char* fn = "csa2_paged_window_attn";
  REQUIRE(T >= 0 && T <= 0x7fffffffLL, "%s: bad T=%lld", fn, (long long)T);
  PagedAttn a = {};
  CSA2_TRY(attn_of(fn, q, T, cache, scale, window, sinks, &a, nullptr));
  if (T == 0 || cache->B == 0) return CSA2_OK;
  REQUIRE(cu_q != nullptr, "%s: cu_q is null", fn);
  if (static_cast<int64_t>(a.kv.heads) * ((a.G + 15) / 16) > 65535)
    return fail(CSA2_ERR_UNSUPPORTED, "%s: %d query heads over %d cache heads", fn, a.Hq, a.kv.heads);
  REQUIRE(out != nullptr && aligned16(out), "%s: out is null or not 16-byte aligned", fn);
  a.out = out;
  a.lse = lse;
  a.kv.err = device_error_word();
  return launch_paged_window(a, cu_q, T, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
