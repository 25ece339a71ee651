// The 8-bit paged key/value cache: parameters and device helpers shared by the
// plan, the append and the attention that reads it (include/vattn.h has the
// layouts).
#pragma once

#include "common.cuh"

namespace vattn {
namespace cache {

constexpr int SCALE_TOKENS = 16;  // tokens that share one scale per kv head
constexpr int E_MIN = -40;        // smallest scale exponent
constexpr uint8_t E4M3_NAN = 0x7f;

// Flattened, validated vattn_cache_geom.
struct Geom {
  int streams, q_heads, kv_heads, group, d;
  int pages, page_tokens, page_shift;  // page_tokens = 1 << page_shift
  int width;                           // block_table entries per stream
  int frame, window;
};

// Cache rows of one page and kv head start at row (page * kv_heads + h) *
// page_tokens; 64-bit, a pool may exceed 2^32 bytes.
__device__ __forceinline__ long long cache_row(const Geom& g, int page, int h, int off) {
  return ((long long)page * g.kv_heads + h) * g.page_tokens + off;
}

struct FwdParams {
  Geom g;
  const __nv_bfloat16* q;
  long long q_stride;  // elements between tokens
  const int* q_starts;
  const int* kv_lens;
  const int* table;
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  float scale_log2;  // scale * log2(e)
  int n_tokens, max_new;
  __nv_bfloat16* o;
  float* lse;
  DevCtl ctl;
};

// One stream's step, with every value brought into range (an out-of-range one
// is reported): its new tokens are q rows [row0, row0 + n), and it holds len
// tokens.
struct StreamStep {
  int row0, n, len;
};
__device__ __forceinline__ StreamStep stream_step(const FwdParams& p, int s) {
  const int a = p.q_starts[s], b = p.q_starts[s + 1], l = p.kv_lens[s];
  StreamStep r;
  r.row0 = min(max(a, 0), p.n_tokens);
  r.n = min(max(b, r.row0), p.n_tokens) - r.row0;
  const long long cap = (long long)p.g.width << p.g.page_shift;
  r.len = (int)min((long long)max(l, 0), cap);
  bool ok = a == r.row0 && b == r.row0 + r.n && l == r.len;
  if (r.n > p.max_new) {
    r.n = p.max_new;
    ok = false;
  }
  if (!ok) report_error(p.ctl.err_word, VATTN_ERR_DEVICE_BOUNDS);
  return r;
}

// Keys [lo, hi) that the stream's new token i sees.
__device__ __forceinline__ void key_range(const Geom& g, const StreamStep& st, int i, int* lo, int* hi) {
  *lo = 0;
  *hi = st.len;
  if (g.frame > 0) {
    const int pos = st.len - st.n + i;  // both below 2^31
    if (pos < 0) {
      *hi = 0;
      return;
    }
    const unsigned from = (unsigned)pos / (unsigned)g.frame * (unsigned)g.frame;  // first of its frame
    *hi = (int)min((unsigned)st.len, from + (unsigned)g.frame);
    if (g.window > 0) *lo = (int)max(0ll, (long long)from - (g.window - 1ll) * g.frame);
  }
}

// e4m3 pair (low byte first) -> f16 pair; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// The two pairs of four e4m3 bytes.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t v) {
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v));
  return r;
}

}  // namespace cache

// -- cache_store.cu --
struct CachePlanArgs {
  const int* new_tokens;
  const int* kv_lens;
  int* table;
  int* free_pages;
  const int* n_free;
  int* kv_lens_out;
  int* n_free_out;
  int* q_starts;
  int* slots;
  int max_tokens;
  int* result;
};
cudaError_t launch_cache_plan(const cache::Geom& g, const CachePlanArgs& a, cudaStream_t st);
struct CacheAppendArgs {
  const void* k;
  const void* v;
  long long k_stride, v_stride;
  const int* slots;
  int n_tokens;
  void* kc;
  void* vc;
  float* ks;
  float* vs;
  DevCtl ctl;
};
cudaError_t launch_cache_append(const cache::Geom& g, const CacheAppendArgs& a, cudaStream_t st);

// -- cache_attn_few.cu: max_new * group <= 16 query rows per stream and kv head --
bool cache_few_fits(const cache::Geom& g, long long max_new);
size_t cache_few_workspace(const cache::Geom& g);
cudaError_t launch_cache_few(const cache::FwdParams& p, void* workspace, cudaStream_t st);

// -- cache_attn_many.cu --
long long cache_many_items(const cache::Geom& g, long long max_new);  // thread blocks, before any is split
size_t cache_many_workspace(const cache::Geom& g, long long max_new);
size_t cache_many_workspace_most(const cache::Geom& g, long long max_new);  // of any max_new up to this one
cudaError_t launch_cache_many(const cache::FwdParams& p, void* workspace, cudaStream_t st);

// 3-D map over e4m3 cache pages [pages * kv_heads][page_tokens][d]: box = one
// page of one kv head, 128-byte swizzle (64-byte at d = 64).
bool make_tmap_pages(CUtensorMap* map, const void* base, int d, int page_tokens, long long heads, const char** err);

}  // namespace vattn
