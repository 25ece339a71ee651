// C-ABI entry points of the 8-bit key/value cache: argument validation and
// launches on the caller's stream.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "cache.cuh"

namespace vattn {
namespace {

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return record_error(code, buf);
}
int ok() { return record_error(VATTN_OK, ""); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define REQUIRE_PTR(p)                                                                \
  do {                                                                                \
    if (!(p)) return fail(VATTN_ERR_INVALID_ARG, "%s is NULL", #p);                   \
    if (!aligned16(p)) return fail(VATTN_ERR_ALIGN, "%s is not 16-byte aligned", #p); \
  } while (0)
// int32 arrays (lengths, tables, counts): natural alignment, so that rows and
// elements of larger arrays can be passed
#define REQUIRE_INTS(p)                                                                                        \
  do {                                                                                                         \
    if (!(p)) return fail(VATTN_ERR_INVALID_ARG, "%s is NULL", #p);                                            \
    if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(VATTN_ERR_ALIGN, "%s is not 4-byte aligned", #p);     \
  } while (0)

#define CHECK_LAUNCH(expr, what)                                                                        \
  do {                                                                                                  \
    cudaError_t e_ = (expr);                                                                            \
    if (e_ != cudaSuccess) return fail(VATTN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e_));         \
  } while (0)

int build_geom(const vattn_cache_geom* in, cache::Geom* g) {
  if (!in) return fail(VATTN_ERR_INVALID_ARG, "geom is NULL");
  if (in->streams < 0 || in->pages < 0) return fail(VATTN_ERR_INVALID_ARG, "streams/pages must be >= 0");
  if (in->q_heads <= 0 || in->kv_heads <= 0) return fail(VATTN_ERR_INVALID_ARG, "q_heads/kv_heads must be > 0");
  if (in->q_heads % in->kv_heads)
    return fail(VATTN_ERR_SHAPE, "q_heads %lld not a multiple of kv_heads %lld", (long long)in->q_heads,
                (long long)in->kv_heads);
  if (in->table_width <= 0) return fail(VATTN_ERR_INVALID_ARG, "table_width must be > 0");
  if (in->frame_tokens < 0 || in->window_frames < 0)
    return fail(VATTN_ERR_INVALID_ARG, "frame_tokens/window_frames must be >= 0");
  if (in->window_frames > 0 && in->frame_tokens == 0)
    return fail(VATTN_ERR_INVALID_ARG, "window_frames needs frame_tokens");
  if (in->head_dim != 64 && in->head_dim != 128)
    return fail(VATTN_ERR_UNSUPPORTED, "head_dim %lld not supported (64 or 128)", (long long)in->head_dim);
  const int pt = in->page_tokens;
  if (pt != 16 && pt != 32 && pt != 64 && pt != 128)
    return fail(VATTN_ERR_UNSUPPORTED, "page_tokens %d not supported (16, 32, 64 or 128)", pt);
  if (in->q_heads > 65535 || in->streams > 65535)
    return fail(VATTN_ERR_UNSUPPORTED, "q_heads and streams must be <= 65535");
  if (in->pages >= (1ll << 31) / pt) return fail(VATTN_ERR_UNSUPPORTED, "pages * page_tokens must be < 2^31");
  if (in->pages * in->kv_heads >= (1ll << 31))
    return fail(VATTN_ERR_UNSUPPORTED, "pages * kv_heads must be < 2^31");
  if (in->streams * in->kv_heads >= (1ll << 31))
    return fail(VATTN_ERR_UNSUPPORTED, "streams * kv_heads must be < 2^31");
  if ((long long)in->table_width * pt >= (1ll << 31) - 256)
    return fail(VATTN_ERR_UNSUPPORTED, "table_width * page_tokens must be < 2^31 - 256");
  g->streams = (int)in->streams;
  g->q_heads = (int)in->q_heads;
  g->kv_heads = (int)in->kv_heads;
  g->group = g->q_heads / g->kv_heads;
  g->d = (int)in->head_dim;
  g->pages = (int)in->pages;
  g->page_tokens = pt;
  g->page_shift = pt == 16 ? 4 : pt == 32 ? 5 : pt == 64 ? 6 : 7;
  g->width = in->table_width;
  g->frame = in->frame_tokens;
  g->window = in->window_frames;
  return VATTN_OK;
}

int check_tokens(int64_t n_tokens) {
  if (n_tokens < 0) return fail(VATTN_ERR_INVALID_ARG, "n_tokens must be >= 0");
  if (n_tokens >= (1ll << 31)) return fail(VATTN_ERR_UNSUPPORTED, "n_tokens must be < 2^31");
  return VATTN_OK;
}

// Query rows of a call: every stream may have max_new tokens.
int check_rows(const cache::Geom& g, int64_t max_new) {
  if (max_new * g.group >= (1ll << 31)) return fail(VATTN_ERR_UNSUPPORTED, "max_new * query heads per kv head >= 2^31");
  if (cache_many_items(g, max_new) >= (1ll << 31))
    return fail(VATTN_ERR_UNSUPPORTED, "streams * kv_heads * tiles of 256 query rows >= 2^31");
  return VATTN_OK;
}

int check_stride(const char* name, int64_t stride, int64_t heads, int64_t d) {
  if (stride < heads * d)
    return fail(VATTN_ERR_SHAPE, "%s %lld is less than heads * head_dim = %lld", name, (long long)stride,
                (long long)(heads * d));
  if (stride % 8) return fail(VATTN_ERR_ALIGN, "%s %lld is not a multiple of 8 elements", name, (long long)stride);
  return VATTN_OK;
}

size_t fwd_workspace(const cache::Geom& g, int64_t max_new) {
  if (g.streams == 0 || max_new == 0) return 0;
  return cache_few_fits(g, max_new) ? cache_few_workspace(g) : cache_many_workspace(g, max_new);
}
// What serves every max_new up to this one: fewer tokens can need more (one
// kernel always leaves partial results, the other only where items are few).
size_t fwd_workspace_most(const cache::Geom& g, int64_t max_new) {
  if (g.streams == 0 || max_new == 0) return 0;
  const size_t few = cache_few_fits(g, 1) ? cache_few_workspace(g) : 0;
  return cache_few_fits(g, max_new) ? few : std::max(few, cache_many_workspace_most(g, max_new));
}

}  // namespace
}  // namespace vattn

using namespace vattn;

extern "C" {

int vattn_cache_plan(const vattn_cache_geom* geom, const int32_t* new_tokens, const int32_t* kv_lens,
                     int32_t* block_table, int32_t* free_pages, const int32_t* n_free, int32_t* kv_lens_out,
                     int32_t* n_free_out, int32_t* q_starts, int32_t* slots, int64_t max_tokens, int32_t* result,
                     void* stream) {
  cache::Geom g;
  int r = build_geom(geom, &g);
  if (r) return r;
  if (max_tokens < 0) return fail(VATTN_ERR_INVALID_ARG, "max_tokens must be >= 0");
  if (max_tokens >= (1ll << 31)) return fail(VATTN_ERR_UNSUPPORTED, "max_tokens must be < 2^31");
  if (g.streams == 0) return ok();
  REQUIRE_INTS(new_tokens);
  REQUIRE_INTS(kv_lens);
  REQUIRE_INTS(block_table);
  REQUIRE_INTS(free_pages);
  REQUIRE_INTS(n_free);
  REQUIRE_INTS(kv_lens_out);
  REQUIRE_INTS(n_free_out);
  REQUIRE_INTS(q_starts);
  if (max_tokens > 0) REQUIRE_INTS(slots);
  REQUIRE_INTS(result);
  CachePlanArgs a;
  a.new_tokens = new_tokens;
  a.kv_lens = kv_lens;
  a.table = block_table;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.kv_lens_out = kv_lens_out;
  a.n_free_out = n_free_out;
  a.q_starts = q_starts;
  a.slots = slots;
  a.max_tokens = (int)max_tokens;
  a.result = result;
  CHECK_LAUNCH(launch_cache_plan(g, a, (cudaStream_t)stream), "cache_plan launch");
  return ok();
}

int vattn_cache_append(const vattn_cache_geom* geom, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, const int32_t* slots, int64_t n_tokens, void* kcache, void* vcache,
                       float* kscale, float* vscale, void* stream) {
  cache::Geom g;
  int r = build_geom(geom, &g);
  if (r) return r;
  if ((r = check_tokens(n_tokens))) return r;
  if (n_tokens * g.kv_heads >= (1ll << 34)) return fail(VATTN_ERR_UNSUPPORTED, "n_tokens * kv_heads must be < 2^34");
  if (n_tokens == 0) return ok();
  if ((r = check_stride("k_stride", k_stride, g.kv_heads, g.d))) return r;
  if ((r = check_stride("v_stride", v_stride, g.kv_heads, g.d))) return r;
  REQUIRE_PTR(k);
  REQUIRE_PTR(v);
  REQUIRE_INTS(slots);
  REQUIRE_PTR(kcache);
  REQUIRE_PTR(vcache);
  REQUIRE_PTR(kscale);
  REQUIRE_PTR(vscale);
  CacheAppendArgs a;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.n_tokens = (int)n_tokens;
  a.kc = kcache;
  a.vc = vcache;
  a.ks = kscale;
  a.vs = vscale;
  a.ctl = current_ctl();
  CHECK_LAUNCH(launch_cache_append(g, a, (cudaStream_t)stream), "cache_append launch");
  return ok();
}

int vattn_cache_workspace_size(const vattn_cache_geom* geom, int64_t n_tokens, int64_t max_new, size_t* bytes) {
  cache::Geom g;
  int r = build_geom(geom, &g);
  if (r) return r;
  if ((r = check_tokens(n_tokens))) return r;
  if (max_new < 0) return fail(VATTN_ERR_INVALID_ARG, "max_new must be >= 0");
  if (!bytes) return fail(VATTN_ERR_INVALID_ARG, "bytes is NULL");
  if (max_new > n_tokens) max_new = n_tokens;
  if ((r = check_rows(g, max_new))) return r;
  *bytes = fwd_workspace_most(g, max_new);
  return ok();
}

int vattn_cache_fwd(const vattn_cache_geom* geom, const void* q, int64_t q_stride, const int32_t* q_starts,
                    const int32_t* kv_lens, const int32_t* block_table, const void* kcache, const void* vcache,
                    const float* kscale, const float* vscale, float scale, int64_t n_tokens, int64_t max_new,
                    void* o, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  cache::Geom g;
  int r = build_geom(geom, &g);
  if (r) return r;
  if ((r = check_tokens(n_tokens))) return r;
  if (max_new < 0) return fail(VATTN_ERR_INVALID_ARG, "max_new must be >= 0");
  const float scale_log2 = scale * 1.4426950408889634f;  // the kernels' exponentials are of base 2
  if (!(scale > 0.f) || std::isinf(scale_log2))
    return fail(VATTN_ERR_INVALID_ARG, "scale must be positive, and scale * log2(e) finite");
  if (max_new > n_tokens) max_new = n_tokens;
  if ((r = check_rows(g, max_new))) return r;
  if (g.streams == 0 || n_tokens == 0 || max_new == 0) return ok();
  if (g.pages == 0) return fail(VATTN_ERR_INVALID_ARG, "pages must be > 0");
  if ((r = check_stride("q_stride", q_stride, g.q_heads, g.d))) return r;
  REQUIRE_PTR(q);
  REQUIRE_INTS(q_starts);
  REQUIRE_INTS(kv_lens);
  REQUIRE_INTS(block_table);
  REQUIRE_PTR(kcache);
  REQUIRE_PTR(vcache);
  REQUIRE_PTR(kscale);
  REQUIRE_PTR(vscale);
  REQUIRE_PTR(o);
  if (lse && !aligned16(lse)) return fail(VATTN_ERR_ALIGN, "lse is not 16-byte aligned");
  const size_t need = fwd_workspace(g, max_new);
  if (need > 0) {
    if (!workspace || ws_bytes < need)
      return fail(VATTN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? ws_bytes : 0);
    if (!aligned16(workspace)) return fail(VATTN_ERR_ALIGN, "workspace is not 16-byte aligned");
  }
  cache::FwdParams p;
  p.g = g;
  p.q = (const __nv_bfloat16*)q;
  p.q_stride = q_stride;
  p.q_starts = q_starts;
  p.kv_lens = kv_lens;
  p.table = block_table;
  p.kc = (const uint8_t*)kcache;
  p.vc = (const uint8_t*)vcache;
  p.ks = kscale;
  p.vs = vscale;
  p.scale_log2 = scale_log2;
  p.n_tokens = (int)n_tokens;
  p.max_new = (int)max_new;
  p.o = (__nv_bfloat16*)o;
  p.lse = lse;
  p.ctl = current_ctl();
  if (cache_few_fits(g, max_new))
    CHECK_LAUNCH(launch_cache_few(p, workspace, (cudaStream_t)stream), "cache_fwd launch");
  else
    CHECK_LAUNCH(launch_cache_many(p, workspace, (cudaStream_t)stream), "cache_fwd launch");
  return ok();
}

}  // extern "C"
