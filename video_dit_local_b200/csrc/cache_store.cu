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
// Every page id that a stream gives, takes or goes on filling is checked before
// the state changes.
// Bound by the latency of its handful of dependent reads, so one thread block
// does it all with one scan: a thread sums a run of streams, the block scans the
// threads' sums, and pages (and the slots of few tokens) are dealt out to all
// threads by a search in those sums.  Slots of many tokens are a second, wide
// kernel.
// ---------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;
// Tokens whose slots the planning block lists itself: 1000 new tokens of 1000
// streams take 6.7 us so and 8.4 us with the second kernel, 4000 tokens of 100
// streams 8.7 and 7.2 us.
constexpr int PLAN_SLOTS = 2048;

struct StreamPlan {
  int len, have, give, take, add;
};
__device__ __forceinline__ StreamPlan stream_plan(const Geom& g, const CachePlanArgs& a, int s) {
  StreamPlan r;
  r.len = a.kv_lens[s];
  const int n = a.new_tokens[s];
  r.have = (r.len + g.page_tokens - 1) >> g.page_shift;
  r.give = n < 0 ? r.have : 0;
  r.add = max(n, 0);
  r.take = n < 0 ? 0 : ((r.len + r.add + g.page_tokens - 1) >> g.page_shift) - r.have;
  return r;
}

// Last i in [0, n) with first[i] <= x (first is non-decreasing, first[0] <= x).
template <class T>
__device__ __forceinline__ int last_at_most(const T* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int slot_of(const Geom& g, const int* table, int s, int pos) {
  return (table[(long long)s * g.width + (pos >> g.page_shift)] << g.page_shift) + (pos & (g.page_tokens - 1));
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const Geom g, const CachePlanArgs a, int list_slots) {
  __shared__ long long warp_give[32], warp_take[32], warp_add[32];
  __shared__ int warp_longest[32], warp_worst[32];
  __shared__ int give0[PLAN_THREADS], take0[PLAN_THREADS], add0[PLAN_THREADS];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const long long cap = (long long)g.width << g.page_shift;
  const int n_free = *a.n_free;
  const int per = (g.streams + PLAN_THREADS - 1) / PLAN_THREADS;
  const int s0 = min(t * per, g.streams), s1 = min(s0 + per, g.streams);
  auto in_pool = [&](int page) { return (unsigned)page < (unsigned)g.pages; };

  // sums and the verdict, before anything is written
  long long give = 0, take = 0, add = 0;
  int longest = 0, worst = VATTN_PLAN_OK, filled = 0;
  bool bad = false, fills = false;
  for (int s = s0; s < s1; ++s) {
    const int len = a.kv_lens[s], n = a.new_tokens[s];
    if (len < 0 || len > cap) {
      worst = max(worst, VATTN_PLAN_BAD_STATE);
    } else if (n >= 0 && len + (long long)n > cap) {
      worst = max(worst, VATTN_PLAN_TABLE_FULL);
    } else {
      const StreamPlan r = stream_plan(g, a, s);
      give += r.give;
      take += r.take;
      add += r.add;
      longest = max(longest, n < 0 ? 0 : len + r.add);
      // the page that the stream goes on filling (looked at later on: nothing waits for it here)
      bad |= fills && !in_pool(filled);
      fills = r.add > 0 && (len & (g.page_tokens - 1));
      if (fills) filled = a.table[(long long)s * g.width + (len >> g.page_shift)];
    }
  }
  const long long my_give = give, my_take = take, my_add = add;
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(~0u, give, o), y = __shfl_up_sync(~0u, take, o), z = __shfl_up_sync(~0u, add, o);
    if (lane >= o) {
      give += x;
      take += y;
      add += z;
    }
    longest = max(longest, __shfl_xor_sync(~0u, longest, o));
    worst = max(worst, __shfl_xor_sync(~0u, worst, o));
  }
  if (lane == 31) {
    warp_give[warp] = give;
    warp_take[warp] = take;
    warp_add[warp] = add;
    warp_longest[warp] = longest;
    warp_worst[warp] = worst;
  }
  __syncthreads();
  long long tot_give, tot_take, tot_add;
  {  // every warp scans the warps' sums
    const long long wg = warp_give[lane], wt = warp_take[lane], wa = warp_add[lane];
    long long sg = wg, st = wt, sa = wa;
    longest = warp_longest[lane];
    worst = warp_worst[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(~0u, sg, o), y = __shfl_up_sync(~0u, st, o), z = __shfl_up_sync(~0u, sa, o);
      if (lane >= o) {
        sg += x;
        st += y;
        sa += z;
      }
      longest = max(longest, __shfl_xor_sync(~0u, longest, o));
      worst = max(worst, __shfl_xor_sync(~0u, worst, o));
    }
    tot_give = __shfl_sync(~0u, sg, 31);
    tot_take = __shfl_sync(~0u, st, 31);
    tot_add = __shfl_sync(~0u, sa, 31);
    give += __shfl_sync(~0u, sg - wg, warp) - my_give;
    take += __shfl_sync(~0u, st - wt, warp) - my_take;
    add += __shfl_sync(~0u, sa - wa, warp) - my_add;
  }
  int verdict = worst;
  if (verdict == VATTN_PLAN_OK) {
    if (n_free < 0 || n_free + tot_give > g.pages)
      verdict = VATTN_PLAN_BAD_STATE;
    else if (tot_add > a.max_tokens)
      verdict = VATTN_PLAN_NO_SLOTS;
    else if (tot_take > n_free + tot_give)
      verdict = VATTN_PLAN_NO_PAGES;
  }
  // (sums that passed fit an int: at most pages, and max_tokens)
  give0[t] = (int)give;
  take0[t] = (int)take;
  add0[t] = (int)add;
  __syncthreads();

  if (verdict == VATTN_PLAN_OK) {
    bad |= fills && !in_pool(filled);
    // what is taken from below the pages that ending streams give
    for (int i = (int)tot_give + t; i < (int)tot_take; i += PLAN_THREADS)
      bad |= !in_pool(a.free_pages[n_free + (int)tot_give - 1 - i]);
    // pages of ending streams onto the stack: above its top, so nothing is lost if one turns out bad
    for (int i = t; i < (int)tot_give; i += PLAN_THREADS) {
      const int u = last_at_most(give0, PLAN_THREADS, i);
      int s = u * per, j = i - give0[u];
      for (int x; j >= (x = stream_plan(g, a, s).give); ++s) j -= x;
      const int page = a.table[(long long)s * g.width + j];
      bad |= !in_pool(page);
      a.free_pages[n_free + i] = page;
    }
    if (__syncthreads_or(bad)) verdict = VATTN_PLAN_BAD_STATE;
  }
  if (verdict != VATTN_PLAN_OK) {
    int top = 0;
    for (int s = s0; s < s1; ++s) {
      const int len = a.kv_lens[s];
      a.kv_lens_out[s] = len;
      a.q_starts[s] = 0;
      top = max(top, len);
    }
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) warp_longest[warp] = top;
    __syncthreads();
    if (list_slots)
      for (int i = t; i < a.max_tokens; i += PLAN_THREADS) a.slots[i] = -1;
    if (t == 0) {
      for (int w = 0; w < PLAN_THREADS / 32; ++w) top = max(top, warp_longest[w]);
      a.q_starts[g.streams] = 0;
      *a.n_free_out = n_free;
      a.result[0] = verdict;
      a.result[1] = 0;
      a.result[2] = n_free;
      a.result[3] = top;
    }
    return;
  }

  // new pages off the stack
  const int avail = n_free + (int)tot_give;
  for (int i = t; i < (int)tot_take; i += PLAN_THREADS) {
    const int u = last_at_most(take0, PLAN_THREADS, i);
    int s = u * per, j = i - take0[u];
    for (int x; j >= (x = stream_plan(g, a, s).take); ++s) j -= x;
    a.table[(long long)s * g.width + stream_plan(g, a, s).have + j] = a.free_pages[avail - 1 - i];
  }
  __syncthreads();
  // slots, from the lengths before the step
  if (list_slots) {
    for (int i = t; i < a.max_tokens; i += PLAN_THREADS) {
      int slot = -1;
      if (i < (int)tot_add) {
        const int u = last_at_most(add0, PLAN_THREADS, i);
        int s = u * per, j = i - add0[u];
        for (int x; j >= (x = stream_plan(g, a, s).add); ++s) j -= x;
        slot = slot_of(g, a.table, s, a.kv_lens[s] + j);
      }
      a.slots[i] = slot;
    }
    __syncthreads();
  }
  // the lengths may be updated in place: last
  int q = (int)add;
  for (int s = s0; s < s1; ++s) {
    const StreamPlan r = stream_plan(g, a, s);
    const int n = a.new_tokens[s];
    a.q_starts[s] = q;
    a.kv_lens_out[s] = n < 0 ? 0 : r.len + r.add;
    q += r.add;
  }
  if (t == 0) {
    a.q_starts[g.streams] = (int)tot_add;
    *a.n_free_out = avail - (int)tot_take;
    a.result[0] = VATTN_PLAN_OK;
    a.result[1] = (int)tot_add;
    a.result[2] = avail - (int)tot_take;
    a.result[3] = longest;
  }
}

// Slots of many new tokens, from the tables and lengths that plan_kernel left.
__global__ void __launch_bounds__(256) slots_kernel(const Geom g, const CachePlanArgs a) {
  const unsigned at = blockIdx.x * 256 + threadIdx.x;  // up to 255 past max_tokens, which may be 2^31 - 1
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (at >= (unsigned)a.max_tokens) return;
  const int t = (int)at;
  int slot = -1;
  if (t < a.q_starts[g.streams]) {
    const int s = last_at_most(a.q_starts, g.streams, t);
    slot = slot_of(g, a.table, s, a.kv_lens_out[s] - a.q_starts[s + 1] + t);
  }
  a.slots[t] = slot;
}

// ---------------------------------------------------------------------------
// Append.  A warp takes one 16-token block of one kv head (K and V): its new
// rows are read once into registers (all loads in flight together), the block's
// absmax gives the scale exponent, and the bytes leave in whole cache rows.
// Bound by HBM: 4 d bytes in, 2 d bytes out per token and kv head (two 1080p
// frames, 24 heads of 128, from a fused projection: 52-55 us, 6 TB/s).  That
// leaves about 600 instructions a block: a block of sixteen finite new tokens,
// which is what a frame is made of, takes a path without predicates.
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

// Warps of a thread block: small blocks fit the registers better (eight
// warps took 29% longer for two 1080p frames, one warp twice as long for ragged
// chunks).
constexpr int APPEND_WARPS = 4;

template <int D>
__global__ void __launch_bounds__(APPEND_WARPS * 32) append_kernel(const Geom g, const CacheAppendArgs a, int span) {
  constexpr int LPR = D / 8;         // lanes per row (16 bytes of bf16 each)
  constexpr int RPL = 32 / LPR;      // rows per warp-wide load
  constexpr int NL = 16 / RPL;       // loads of a whole block
  const int warp = blockIdx.x * APPEND_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int c = lane % LPR, r0 = lane / LPR;
  const int h = warp % g.kv_heads;
  const long long i0 = (long long)(warp / g.kv_heads) * span;
  if (i0 >= a.n_tokens) return;
  // lane j: slot of token i0 + j (a block that starts among the first `span` may go on past them)
  const int n_slots = g.pages << g.page_shift;
  auto slot_at = [&](long long i) {
    const int x = i >= 0 && i < a.n_tokens ? __ldg(a.slots + i) : -1;
    if (x < n_slots) return x;
    report_error(a.ctl.err_word, VATTN_ERR_DEVICE_BOUNDS);
    return -1;
  };
  const int my = slot_at(i0 + lane), earlier = slot_at(i0 - 32 + lane);
  const int before = __shfl_sync(~0u, earlier, 31), up = __shfl_up_sync(~0u, my, 1), prev = lane == 0 ? before : up;
  // a block belongs to the first of its new tokens
  uint32_t leads = __ballot_sync(~0u, lane < span && my >= 0 && !(prev >= 0 && prev + 1 == my && (my & 15) != 0));
  for (; leads; leads &= leads - 1) {
    const int lead = __ffs(leads) - 1;
    const int slot = __shfl_sync(~0u, my, lead);
    const long long i = i0 + lead;
    const int held = slot & 15;
    // a block that the list comes back to after a gap (or a slot listed twice): another warp writes it
    if (__any_sync(~0u, (earlier >> 4) == (slot >> 4) || (lane < lead && (my >> 4) == (slot >> 4)))) {
      report_error(a.ctl.err_word, VATTN_ERR_DEVICE_BOUNDS);
      continue;
    }
    // its new tokens: consecutive slots from there on
    const bool same = lane >= lead && lane - lead + held < 16 && my == slot + lane - lead;
    const int n = __ffs(~(__ballot_sync(~0u, same) >> lead)) - 1;
    const int page = slot >> g.page_shift, off = (slot & (g.page_tokens - 1)) - held;
    const long long row = cache_row(g, page, h, off);
    const long long sidx = row >> 4;
    // rows are counted from the block's first: row r is new token i + r - held
    uint4 kx[NL], vx[NL];
    const __nv_bfloat16* kp = (const __nv_bfloat16*)a.k + (i + r0 - held) * a.k_stride + h * D + c * 8;
    const __nv_bfloat16* vp = (const __nv_bfloat16*)a.v + (i + r0 - held) * a.v_stride + h * D + c * 8;
    const bool full = n == 16;  // then held = 0
    uint32_t km2 = 0, vm2 = 0;  // largest magnitudes, two packed
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const int r = l * RPL + r0 - held;
      const bool in = full || (r >= 0 && r < n);
      kx[l] = in ? __ldg((const uint4*)(kp + l * RPL * a.k_stride)) : make_uint4(0, 0, 0, 0);
      vx[l] = in ? __ldg((const uint4*)(vp + l * RPL * a.v_stride)) : make_uint4(0, 0, 0, 0);
    }
    auto magnitude = [](const uint4& x) {
      return __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    };
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      km2 = __vmaxu2(km2, magnitude(kx[l]));
      vm2 = __vmaxu2(vm2, magnitude(vx[l]));
    }
    uint32_t both = max(km2 & 0xffffu, km2 >> 16) << 16 | max(vm2 & 0xffffu, vm2 >> 16);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) both = __vmaxu2(both, __shfl_xor_sync(~0u, both, o));
    uint32_t km = both >> 16, vm = both & 0xffffu, poison = 0;
    if (km >= 0x7f80u || vm >= 0x7f80u) {  // a NaN or an infinity somewhere: its token gives no magnitude
      km = vm = 0;
#pragma unroll
      for (int l = 0; l < NL; ++l) {
        const uint32_t k2 = magnitude(kx[l]), v2 = magnitude(vx[l]);
        uint32_t row = max(k2 & 0xffffu, k2 >> 16) << 16 | max(v2 & 0xffffu, v2 >> 16);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) row = __vmaxu2(row, __shfl_xor_sync(~0u, row, o));
        if ((row >> 16) >= 0x7f80u || (row & 0xffffu) >= 0x7f80u) {
          poison |= 1u << l;
        } else {
          km = max(km, row >> 16);
          vm = max(vm, row & 0xffffu);
        }
      }
#pragma unroll
      for (int o = 16; o >= LPR; o >>= 1) {
        km = max(km, __shfl_xor_sync(~0u, km, o));
        vm = max(vm, __shfl_xor_sync(~0u, vm, o));
      }
    }
    const bool clean = full && __all_sync(~0u, poison == 0);
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
    auto quantise = [](const uint4& x, float f) {
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
      uint32_t out[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) out[u] = pack_e4m3x2(bf16lo(in[u]) * f, bf16hi(in[u]) * f);
      return make_uint2(out[0] | (out[1] << 16), out[2] | (out[3] << 16));
    };
    if (clean) {  // sixteen new tokens, nothing to keep or to mark
      uint2* kd = (uint2*)((uint8_t*)a.kc + (row + r0) * D + c * 8);
      uint2* vd = (uint2*)((uint8_t*)a.vc + (row + r0) * D + c * 8);
      const float kf = pow2(-ke), vf = pow2(-ve);
#pragma unroll
      for (int l = 0; l < NL; ++l) {
        kd[l * RPL * D / 8] = quantise(kx[l], kf);
        vd[l * RPL * D / 8] = quantise(vx[l], vf);
      }
      continue;
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
        *dst = quantise(x, pow2(-e));
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
  const bool few = a.max_tokens <= PLAN_SLOTS;
  plan_kernel<<<1, PLAN_THREADS, 0, st>>>(g, a, few ? 1 : 0);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || few) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(((unsigned)a.max_tokens + 255) / 256);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, slots_kernel, g, a);
}

cudaError_t launch_cache_append(const cache::Geom& g, const CacheAppendArgs& a, cudaStream_t st) {
  using namespace cache;
  // Tokens a warp looks through for blocks to take.  16: one warp a block of a
  // long run of tokens, where 1 starts 15 idle warps for each that works (24
  // heads of 128, 10,000 token-blocks: 23 us against 72 for one run of tokens,
  // 22 against 54 for chunks of 1 to 90); 1: blocks of short chunks side by side
  // instead of one after the other, as long as 16 leaves the GPU short of warps
  // (500 blocks: 5.0 us against 5.9 for such chunks).  At 1000 blocks the two
  // meet for such chunks; runs are faster with 16 at any size.
  const int span = (long long)a.n_tokens / 16 * g.kv_heads >= 148 * 16 ? 16 : 1;
  const long long warps = (long long)((a.n_tokens + span - 1) / span) * g.kv_heads;
  const long long blocks = (warps + APPEND_WARPS - 1) / APPEND_WARPS;
  if (g.d == 128)
    append_kernel<128><<<(int)blocks, APPEND_WARPS * 32, 0, st>>>(g, a, span);
  else
    append_kernel<64><<<(int)blocks, APPEND_WARPS * 32, 0, st>>>(g, a, span);
  return cudaGetLastError();
}

}  // namespace vattn
