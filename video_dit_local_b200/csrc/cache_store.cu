// Page bookkeeping and the quantising append of the 8-bit key/value cache.
#include "cache.cuh"

namespace vattn {
namespace cache {

// ---------------------------------------------------------------------------
// Plan.  have = ceil(len / P) pages are listed for a stream, ceil((len + n) / P)
// are needed; ending streams give theirs back first.  With exclusive running
// sums over the streams of the pages given (G_s) and taken (T_s) and of the new
// tokens (Q_s):
//   free[n_free + G_s + j] = table[s][j]                (s ends, j < have)
//   table[s][have + j] = free[n_free + G - 1 - T_s - j] (j < pages taken)
//   slot of token t of stream s: position len + t - Q_s in its pages.
// One thread block does the sums and the tables: it is a handful of dependent
// reads, and one block needs no hand-over between blocks.
// ---------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;

struct StreamPlan {
  int have, give, take, add;
};
__device__ __forceinline__ StreamPlan stream_plan(const Geom& g, int len, int n) {
  StreamPlan r;
  r.have = (len + g.page_tokens - 1) >> g.page_shift;
  r.give = n < 0 ? r.have : 0;
  r.add = max(n, 0);
  r.take = n < 0 ? 0 : ((len + r.add + g.page_tokens - 1) >> g.page_shift) - r.have;
  return r;
}

// Exclusive block-wide sums of three values; *total the sums themselves.
__device__ __forceinline__ int3 block_exclusive_sums(int3 v, int3* total, int3* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int3 x = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(~0u, x.x, o), b = __shfl_up_sync(~0u, x.y, o), c = __shfl_up_sync(~0u, x.z, o);
    if (lane >= o) {
      x.x += a;
      x.y += b;
      x.z += c;
    }
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int3 before = make_int3(0, 0, 0), all = make_int3(0, 0, 0);
  for (int w = 0; w < PLAN_THREADS / 32; ++w) {
    const int3 t = warp_sums[w];
    if (w < warp) before = make_int3(before.x + t.x, before.y + t.y, before.z + t.z);
    all = make_int3(all.x + t.x, all.y + t.y, all.z + t.z);
  }
  *total = all;
  return make_int3(before.x + x.x - v.x, before.y + x.y - v.y, before.z + x.z - v.z);
}

// Last s in [0, n) with first[s] <= i (first is non-decreasing, first[0] <= i).
__device__ __forceinline__ int last_at_most(const int* first, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const Geom g, const CachePlanArgs a) {
  __shared__ int3 warp_sums[PLAN_THREADS / 32];
  __shared__ int first[PLAN_THREADS], have_s[PLAN_THREADS];
  __shared__ unsigned long long tot_add;
  __shared__ long long tot_give, tot_take;
  __shared__ int worst, longest;
  const int t = threadIdx.x;
  const long long cap = (long long)g.width << g.page_shift;
  if (t == 0) {
    tot_add = 0;
    tot_give = tot_take = 0;
    worst = VATTN_PLAN_OK;
    longest = 0;
  }
  __syncthreads();
  const int n_free = *a.n_free;

  // totals and the verdict, before anything is written
  for (int s = t; s < g.streams; s += PLAN_THREADS) {
    const int len = a.kv_lens[s], n = a.new_tokens[s];
    if (len < 0 || len > cap) {
      atomicMax(&worst, VATTN_PLAN_BAD_STATE);
      continue;
    }
    if (n >= 0 && len + (long long)n > cap) {
      atomicMax(&worst, VATTN_PLAN_TABLE_FULL);
      continue;
    }
    const StreamPlan r = stream_plan(g, len, n);
    atomicAdd(&tot_add, (unsigned long long)r.add);
    atomicAdd((unsigned long long*)&tot_give, (unsigned long long)r.give);
    atomicAdd((unsigned long long*)&tot_take, (unsigned long long)r.take);
    atomicMax(&longest, n < 0 ? 0 : len + r.add);
    for (int j = 0; j < r.give; ++j)
      if ((unsigned)a.table[(long long)s * g.width + j] >= (unsigned)g.pages) atomicMax(&worst, VATTN_PLAN_BAD_STATE);
  }
  __syncthreads();
  int verdict = worst;
  if (verdict == VATTN_PLAN_OK) {
    if (n_free < 0 || n_free + tot_give > g.pages)
      verdict = VATTN_PLAN_BAD_STATE;
    else if ((long long)tot_add > a.max_tokens)
      verdict = VATTN_PLAN_NO_SLOTS;
    else if (tot_take > n_free + tot_give)
      verdict = VATTN_PLAN_NO_PAGES;
  }
  if (verdict != VATTN_PLAN_OK) {
    int top = 0;
    for (int s = t; s < g.streams; s += PLAN_THREADS) {
      const int len = a.kv_lens[s];
      a.kv_lens_out[s] = len;
      top = max(top, len);
    }
    for (int s = t; s <= g.streams; s += PLAN_THREADS) a.q_starts[s] = 0;
    __syncthreads();
    if (t == 0) longest = 0;
    __syncthreads();
    atomicMax(&longest, top);
    __syncthreads();
    if (t == 0) {
      *a.n_free_out = n_free;
      a.result[0] = verdict;
      a.result[1] = 0;
      a.result[2] = n_free;
      a.result[3] = longest;
    }
    return;
  }
  const int avail = n_free + (int)tot_give;

  // pages of ending streams onto the stack
  if (tot_give > 0) {
    int base = n_free;
    for (int s0 = 0; s0 < g.streams; s0 += PLAN_THREADS) {
      const int s = s0 + t;
      int give = 0;
      if (s < g.streams) give = stream_plan(g, a.kv_lens[s], a.new_tokens[s]).give;
      int3 all;
      const int3 ex = block_exclusive_sums(make_int3(give, 0, 0), &all, warp_sums);
      first[t] = ex.x;
      __syncthreads();
      for (int i = t; i < all.x; i += PLAN_THREADS) {
        const int u = last_at_most(first, PLAN_THREADS, i);
        a.free_pages[base + i] = a.table[(long long)(s0 + u) * g.width + (i - first[u])];
      }
      base += all.x;
      __syncthreads();
    }
  }
  // new pages off the stack, lengths and token ranges
  int taken = 0, token0 = 0;
  for (int s0 = 0; s0 < g.streams; s0 += PLAN_THREADS) {
    const int s = s0 + t;
    StreamPlan r = {0, 0, 0, 0};
    int len = 0, n = 0;
    if (s < g.streams) {
      len = a.kv_lens[s];
      n = a.new_tokens[s];
      r = stream_plan(g, len, n);
    }
    int3 all;
    const int3 ex = block_exclusive_sums(make_int3(r.take, r.add, 0), &all, warp_sums);
    first[t] = ex.x;
    have_s[t] = r.have;
    if (s < g.streams) {
      a.q_starts[s] = token0 + ex.y;
      a.kv_lens_out[s] = n < 0 ? 0 : len + r.add;
    }
    __syncthreads();
    for (int i = t; i < all.x; i += PLAN_THREADS) {
      const int u = last_at_most(first, PLAN_THREADS, i);
      a.table[(long long)(s0 + u) * g.width + have_s[u] + (i - first[u])] = a.free_pages[avail - 1 - taken - i];
    }
    taken += all.x;
    token0 += all.y;
    __syncthreads();
  }
  if (t == 0) {
    a.q_starts[g.streams] = token0;
    *a.n_free_out = avail - taken;
    a.result[0] = VATTN_PLAN_OK;
    a.result[1] = token0;
    a.result[2] = avail - taken;
    a.result[3] = longest;
  }
}

// Slots of the new tokens, from the tables that plan_kernel left.
__global__ void __launch_bounds__(256) slots_kernel(const Geom g, const CachePlanArgs a) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= a.max_tokens) return;
  int slot = -1;
  if (t < a.q_starts[g.streams]) {
    const int s = last_at_most(a.q_starts, g.streams, t);
    const int pos = a.kv_lens_out[s] - a.q_starts[s + 1] + t;
    const int page = a.table[(long long)s * g.width + (pos >> g.page_shift)];
    if ((unsigned)page < (unsigned)g.pages) slot = (page << g.page_shift) + (pos & (g.page_tokens - 1));
  }
  a.slots[t] = slot;
}

// ---------------------------------------------------------------------------
// Append.  A warp takes one 16-token block of one kv head (K and V): its new
// rows are read once into registers (all loads in flight together), the block's
// absmax gives the scale exponent, and the bytes leave in whole cache rows.
// Bound by HBM: 4 d bytes in, 2 d bytes out per token and kv head.
// ---------------------------------------------------------------------------

// Smallest e >= E_MIN with the bf16 magnitude `bits` (finite) <= 448 * 2^e:
// (1 + m/128) 2^(E-127) <= 1.75 * 2^(8+e).
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int e = (int)(bits >> 7) - 127 - 8 + ((bits & 0x7f) > 96 ? 1 : 0);
  return max(e, E_MIN);
}
__device__ __forceinline__ float pow2(int e) {  // e in [-126, 127]
  return __int_as_float((e + 127) << 23);
}

template <int D>
__global__ void __launch_bounds__(256) append_kernel(const Geom g, const CacheAppendArgs a, int span) {
  constexpr int LPR = D / 8;         // lanes per row (16 bytes of bf16 each)
  constexpr int RPL = 32 / LPR;      // rows per warp-wide load
  constexpr int NL = 16 / RPL;       // loads of a whole block
  const int warp = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int c = lane % LPR, r0 = lane / LPR;
  const int h = warp % g.kv_heads;
  const long long i0 = (long long)(warp / g.kv_heads) * span;
  if (i0 >= a.n_tokens) return;
  // lane j: slot of token i0 + j (a block that starts among the first `span` may go on past them)
  const int n_slots = g.pages << g.page_shift;
  auto slot_at = [&](long long i) {
    const int x = i >= 0 && i < a.n_tokens ? __ldg(a.slots + i) : -1;
    return x < n_slots ? x : -1;
  };
  const int my = slot_at(i0 + lane), before = slot_at(i0 - 1);
  const int up = __shfl_up_sync(~0u, my, 1), prev = lane == 0 ? before : up;
  // a block belongs to the first of its new tokens
  uint32_t leads = __ballot_sync(~0u, lane < span && my >= 0 && !(prev >= 0 && prev + 1 == my && (my & 15) != 0));
  for (; leads; leads &= leads - 1) {
    const int lead = __ffs(leads) - 1;
    const int slot = __shfl_sync(~0u, my, lead);
    const long long i = i0 + lead;
    const int held = slot & 15;
    // its new tokens: consecutive slots from there on
    const bool same = lane >= lead && lane - lead + held < 16 && my == slot + lane - lead;
    const int n = __ffs(~(__ballot_sync(~0u, same) >> lead)) - 1;
    const int page = slot >> g.page_shift, off = (slot & (g.page_tokens - 1)) - held;
    const long long row = cache_row(g, page, h, off);
    const long long sidx = row >> 4;
    // rows are counted from the block's first: row r is new token i + r - held
    uint4 kx[NL], vx[NL];
    const __nv_bfloat16* kp = (const __nv_bfloat16*)a.k + h * D + c * 8;
    const __nv_bfloat16* vp = (const __nv_bfloat16*)a.v + h * D + c * 8;
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const int r = l * RPL + r0 - held;
      const bool in = r >= 0 && r < n;
      kx[l] = in ? __ldg((const uint4*)(kp + (i + r) * a.k_stride)) : make_uint4(0, 0, 0, 0);
      vx[l] = in ? __ldg((const uint4*)(vp + (i + r) * a.v_stride)) : make_uint4(0, 0, 0, 0);
    }
    uint32_t km = 0, vm = 0, poison = 0;
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      auto row_max = [](const uint4& x) {
        uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                              __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
        return max(m & 0xffffu, m >> 16);
      };
      uint32_t a_k = row_max(kx[l]), a_v = row_max(vx[l]);
      uint32_t both = (a_k << 16) | a_v;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) both = __vmaxu2(both, __shfl_xor_sync(~0u, both, o));
      a_k = both >> 16;
      a_v = both & 0xffffu;
      if (a_k >= 0x7f80u || a_v >= 0x7f80u) {  // a NaN or an infinity: the token gives no magnitude
        poison |= 1u << l;
      } else {
        km = max(km, a_k);
        vm = max(vm, a_v);
      }
    }
#pragma unroll
    for (int o = 16; o >= LPR; o >>= 1) {
      km = max(km, __shfl_xor_sync(~0u, km, o));
      vm = max(vm, __shfl_xor_sync(~0u, vm, o));
    }
    int ke = scale_exponent(km), ve = scale_exponent(vm);
    int ke_old = ke, ve_old = ve;
    if (held > 0) {
      ke_old = (__float_as_int(a.ks[sidx]) >> 23) - 127;
      ve_old = (__float_as_int(a.vs[sidx]) >> 23) - 127;
      ke = max(ke, ke_old);
      ve = max(ve, ve_old);
    }
    __syncwarp();
    if (lane == 0) {
      a.ks[sidx] = pow2(ke);
      a.vs[sidx] = pow2(ve);
    }
    auto store = [&](const uint4& x, uint8_t* base, int r, int e, int e_old, bool nan, bool zero) {
      uint2* dst = (uint2*)(base + (row + r) * D + c * 8);
      if (r < held) {  // held before: bring to the new scale
        if (e == e_old) return;
        const float f = pow2(max(e_old - e, -126));
        const uint2 w = *dst;
        uint32_t out[2];
        const uint32_t in[2] = {w.x, w.y};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float2 lo = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(in[u] & 0xffffu)));
          const float2 hi = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(in[u] >> 16)));
          out[u] = pack_e4m3x2(lo.x * f, lo.y * f) | (pack_e4m3x2(hi.x * f, hi.y * f) << 16);
        }
        *dst = make_uint2(out[0], out[1]);
        return;
      }
      if (r >= held + n || zero) {
        *dst = make_uint2(0, 0);
      } else if (nan) {
        *dst = make_uint2(0x01010101u * E4M3_NAN, 0x01010101u * E4M3_NAN);
      } else {
        const float f = pow2(-e);
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        uint32_t out[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) out[u] = pack_e4m3x2(bf16lo(in[u]) * f, bf16hi(in[u]) * f);
        *dst = make_uint2(out[0] | (out[1] << 16), out[2] | (out[3] << 16));
      }
    };
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const int r = l * RPL + r0;
      const bool bad = (poison >> l) & 1;
      store(kx[l], (uint8_t*)a.kc, r, ke, ke_old, bad, false);
      store(vx[l], (uint8_t*)a.vc, r, ve, ve_old, false, bad);
    }
  }
}

}  // namespace cache

cudaError_t launch_cache_plan(const cache::Geom& g, const CachePlanArgs& a, cudaStream_t st) {
  using namespace cache;
  plan_kernel<<<1, PLAN_THREADS, 0, st>>>(g, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.max_tokens == 0) return e;
  slots_kernel<<<(a.max_tokens + 255) / 256, 256, 0, st>>>(g, a);
  return cudaGetLastError();
}

cudaError_t launch_cache_append(const cache::Geom& g, const CacheAppendArgs& a, cudaStream_t st) {
  using namespace cache;
  // Tokens a warp looks through for blocks to take.  16: one warp a block of a
  // long run of tokens, where 1 would start 15 idle warps for each that works
  // (two 1080p frames, 24 heads of 128: 85 us against 182); 1: blocks of single
  // tokens side by side instead of one after the other, as long as 16 would
  // leave the GPU short of warps.
  const int span = (long long)a.n_tokens / 16 * g.kv_heads >= 148 * 16 ? 16 : 1;
  const long long warps = (long long)((a.n_tokens + span - 1) / span) * g.kv_heads;
  const long long blocks = (warps + 7) / 8;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  if (g.d == 128)
    append_kernel<128><<<(int)blocks, 256, 0, st>>>(g, a, span);
  else
    append_kernel<64><<<(int)blocks, 256, 0, st>>>(g, a, span);
  return cudaGetLastError();
}

}  // namespace vattn
