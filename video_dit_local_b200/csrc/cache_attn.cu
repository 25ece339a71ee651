// Attention over the 8-bit key/value cache.
#include "cache.cuh"

namespace vattn {
namespace cache {

// One thread block per (token, query head): 128 keys at a time, a key per
// thread for the scores and a channel per thread for P V.
template <int D>
__global__ void __launch_bounds__(128) rows_kernel(const FwdParams p) {
  __shared__ float qs[D], w[128];
  __shared__ float red[4];
  __shared__ int pg[128];
  __shared__ int s_stream;
  const Geom& g = p.g;
  const int t = threadIdx.x;
  const int row = blockIdx.x, h = blockIdx.y, kvh = h / g.group;
  if (t == 0) {
    int s = -1;
    for (int i = 0; i < g.streams; ++i)
      if (p.q_starts[i] <= row && row < p.q_starts[i + 1]) s = i;
    s_stream = s;
  }
  if (t < D) qs[t] = __bfloat162float(p.q[(long long)row * p.q_stride + h * D + t]) * p.scale_log2;
  __syncthreads();
  const int s = s_stream;
  if (s < 0) return;
  const StreamStep st = stream_step(p, s);
  int lo, hi;
  key_range(g, st, row - st.row0, &lo, &hi);
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j0 = lo & ~127; j0 < hi; j0 += 128) {
    const int j = j0 + t;
    float x = -INFINITY;
    int page = -1;
    if (j >= lo && j < hi) {
      page = p.table[(long long)s * g.width + (j >> g.page_shift)];
      if ((unsigned)page >= (unsigned)g.pages) {
        report_error(p.ctl.err_word, VATTN_ERR_DEVICE_BOUNDS);
        page = -1;
      }
    }
    pg[t] = page;
    if (page >= 0) {
      const long long r = cache_row(g, page, kvh, j & (g.page_tokens - 1));
      const uint4* k = (const uint4*)(p.kc + r * D);
      float dot = 0.f;
      for (int c = 0; c < D / 16; ++c) {
        const uint4 v = k[c];
        const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
        for (int u = 0; u < 4; ++u) {
          const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(vv[u] & 0xffffu)));
          const float2 b = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(vv[u] >> 16)));
          const float* q = qs + c * 16 + u * 4;
          dot += a.x * q[0] + a.y * q[1] + b.x * q[2] + b.y * q[3];
        }
      }
      x = dot * p.ks[r >> 4];
    }
    float mx = x;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    if ((t & 31) == 0) red[t >> 5] = mx;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float e = exp2f(x - m_use);
    w[t] = e;
    float sum = e;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    __syncthreads();
    if ((t & 31) == 0) red[t >> 5] = sum;
    __syncthreads();
    const float alpha = exp2f(m - m_use);
    l = l * alpha + (red[0] + red[1]) + (red[2] + red[3]);
    acc *= alpha;
    m = m_new;
    if (t < D)
      for (int u = 0; u < 128; ++u) {
        if (pg[u] < 0) continue;
        const long long r = cache_row(g, pg[u], kvh, (j0 + u) & (g.page_tokens - 1));
        const float2 v = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)p.vc[r * D + t]));
        acc += w[u] * (v.x * p.vs[r >> 4]);
      }
    __syncthreads();
  }
  const size_t at = (size_t)row * g.q_heads + h;
  if (t < D) p.o[at * D + t] = __float2bfloat16(l == 0.f ? 0.f : acc / l);
  if (t == 0 && p.lse) p.lse[at] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace cache

size_t cache_fwd_workspace(const cache::Geom& g, long long, long long max_new) {
  return cache_few_fits(g, max_new) ? cache_few_workspace(g) : 0;
}

cudaError_t launch_cache_fwd(const cache::FwdParams& p, void* ws, cudaStream_t st) {
  using namespace cache;
  if (cache_few_fits(p.g, p.max_new)) return launch_cache_few(p, ws, st);
  const dim3 grid(p.n_tokens, p.g.q_heads);
  if (p.g.d == 128)
    rows_kernel<128><<<grid, 128, 0, st>>>(p);
  else
    rows_kernel<64><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace vattn
