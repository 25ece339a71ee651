// Attention over the 8-bit key/value cache for many query rows (whole latent
// frames): bound by the tensor pipe and the softmax, on tcgen05.
//
// A thread block takes the query rows (token, query head of the group) of one
// stream and kv head in tiles of 128 and streams the keys they see in blocks of
// 128.  20 warps:
//   warps 0-7 and 8-15 two softmax groups, each with an S and an O accumulator
//                      in TMEM; a row's 128 scores are shared by two threads,
//                      64 each (720p frame over ten: 1.89 ms; 1.93 with one
//                      thread a row and half as many warps).  TWO = true: a
//                      tile of rows each (256 rows a thread block), on the same
//                      key blocks, so that one conversion of V serves 256
//                      rows; false (no stream has more than 128 rows): one
//                      tile, alternate key blocks, joined at the end;
//   warps 16, 17       convert V, e4m3 -> f16, from one swizzled tile into the
//                      other that P V reads;
//   warp 18            K and V pages by TMA, and the blocks' scales;
//   warp 19            issues the MMAs and owns the TMEM allocation.
//
// Q K^T runs on the cached bytes as they are (kind::f8f6f4).  A bf16 query has
// 8 significant bits, an e4m3 value 4: each row is scaled by a power of two
// into [128, 256) and split into two e4m3 values, hi + lo, whose products with
// K add up in the same accumulator.  hi + lo is exact down to the e4m3 step
// 2^-9, that is to 2^-17 of the row's largest element, and the two fp8 passes
// cost what one bf16 pass would, without converting a key.  P V runs on f16: P
// keeps 11 bits and V, converted exactly, is the part whose rows past a
// stream's end must be zeroed anyway.
//
// Scales are powers of two per 16 keys: K's enters the factor of those 16
// scores; V's the exponent of P, x_j = s_j + log2(vs), with the row sum taking
// P 2^-log2(vs).  The reference m of a row moves only when its maximum grows by
// more than 2^8 (then O is rescaled); P = 2^(x - m + 7) <= 2^15 in f16.
#include <algorithm>

#include "cache.cuh"
#include "fwd_common.cuh"

namespace vattn {
namespace cache {
namespace many {

using fwd::idesc_e4m3_f32;
using fwd::mma_ss_e4m3;

constexpr int BM = 128, BN = 128;
constexpr int THREADS = 640, SOFTMAX = 512;
constexpr int WARP_V = 16, V_WARPS = 2, WARP_K = 18, WARP_MMA = 19;
constexpr int NV = 2;   // ring stages of V as f16
// Scale ring: block j + 8 is written after Q K^T of block j + 5 (or j + 6) is
// done, which is issued after P of block j + 2, whose group has long read block
// j's slot.
constexpr int NS = 8;
constexpr float RESCALE = 8.0f;
constexpr float P_SHIFT = 7.0f;
constexpr int SUBS = BN / SCALE_TOKENS;

// Of each 16 keys of a block: K's scale, log2 of V's, and 2^-log2 of V's.
struct alignas(16) Scales {
  float k[SUBS], e[SUBS], inv[SUBS];
};

template <int D, bool TWO>
struct Smem {
  static constexpr int TILES = TWO ? 2 : 1;     // tiles of query rows
  static constexpr int NK = TWO && D == 128 ? 2 : 3;  // ring stages of K and of V's bytes
  // S accumulators (TMEM columns 128 b ..) and O accumulators (from column 128 NB, d columns a group).  At d = 64 a
  // third S fits: Q K^T then runs ahead of the softmax (see the MMA warp).
  static constexpr int NB = D == 64 ? 3 : 2;
  // Barriers that say S is there: unit n's is n % NSB, which one group only waits for, and in each of its phases (at
  // three accumulators the groups take turns with each).
  static constexpr int NSB = NB % 2 ? 2 * NB : NB;
  static constexpr uint32_t O = 128 * NB;
  static constexpr int QK = 128 * D;            // 128 rows of bytes
  static constexpr int V = 128 * D * 2;         // 128 rows of f16
  static constexpr int OFF_Q = 0;               // hi and lo of each tile
  static constexpr int OFF_K = TILES * 2 * QK;
  static constexpr int OFF_V8 = OFF_K + NK * QK;  // V as cached, in step with K
  static constexpr int OFF_V = OFF_V8 + NK * QK;
  static constexpr int OFF_SC = OFF_V + NV * V;              // NS x Scales
  static constexpr int OFF_XCH = OFF_SC + NS * (int)sizeof(Scales);
  static constexpr int OFF_BAR = OFF_XCH + 4 * 128 * 8;      // [group][half][row] pairs of floats
  static constexpr int NBAR = 1 + 3 * NK + 2 * NV + NSB + NB + 2 + 1 + NS + 8;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int TOTAL = OFF_MISC + 16;
  static constexpr int ALLOC = TOTAL + 1024;
};

struct Params {
  FwdParams f;
  int q_tiles;   // tiles of rows (of all of a thread block's) that a stream can have
  int whole;     // items (a tile of rows, kv head and stream) with a thread block each
  int splits;    // thread blocks that share the keys of each of the other items
  float* part;   // partial results [item - whole][split][row][d], then (m, l) pairs
  float2* part_ml;
};

// Up to RANKED streams come longest first, so that the long ones do not start
// last (ragged prompts: 165 against 181 us): the stream whose length is the
// rank-th.  All threads of the block take part.
constexpr int RANKED = 128;
__device__ __forceinline__ int stream_of_rank(const FwdParams& p, int rank) {
  const int n = p.g.streams;
  if (n == 1 || n > RANKED) return rank;
  __shared__ int lens[RANKED];
  __shared__ int found;
  const int t = threadIdx.x;
  if (t < n) lens[t] = p.kv_lens[t];
  __syncthreads();
  if (t < n) {
    const int mine = lens[t];
    int before = 0;
    for (int i = 0; i < n; ++i) before += lens[i] > mine || (lens[i] == mine && i < t);
    if (before == rank) found = t;
  }
  __syncthreads();
  return found;
}

// Item -> tile, kv head, stream (by rank), tiles fastest: thread blocks that run
// at the same time read the same keys.  Later tiles see more keys under a causal
// mask: they come first.
struct Item {
  int tile, h, s;
};
__device__ __forceinline__ Item item_of(const Params& pp, int item) {
  const Geom& g = pp.f.g;
  const int rest = item / pp.q_tiles;
  Item r;
  r.tile = pp.q_tiles - 1 - (item - rest * pp.q_tiles);
  r.s = rest / g.kv_heads;
  r.h = rest - r.s * g.kv_heads;
  return r;
}

// Instruction descriptor, kind::f16, f16 x f16 -> f32, B MN-major (V rows are keys).
constexpr uint32_t idesc_f16_pv(int N) {
  return (1u << 4) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}
// K-major byte rows: 128-byte swizzle at d = 128, 64-byte at d = 64.
template <int D>
__device__ __forceinline__ uint64_t desc_bytes(uint32_t start) {
  if (D == 128) return smem_desc_sw128(start, 16, 1024);
  return (smem_desc_sw128(start, 16, 512) & ~(7ull << 61)) | (4ull << 61);
}
// 16-byte chunk c of byte row r in those layouts.
template <int D>
__device__ __forceinline__ uint32_t byte_chunk(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The keys of a tile of rows: blocks [first, first + count) of 128, those of
// the tokens [lo, hi).
struct TileKeys {
  int lo, hi, first, count;
};
__device__ __forceinline__ TileKeys tile_keys(const Geom& g, const StreamStep& st, int row0, int rows) {
  TileKeys t;
  int x;
  key_range(g, st, row0 / g.group, &t.lo, &x);
  key_range(g, st, (row0 + rows - 1) / g.group, &x, &t.hi);
  t.hi = max(t.hi, t.lo);
  t.first = t.lo / BN;
  t.count = t.hi > t.lo ? (t.hi + BN - 1) / BN - t.first : 0;
  return t;
}

template <int D, bool TWO>
__global__ void __launch_bounds__(THREADS, 1)
    many_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const Params pp) {
  using L = Smem<D, TWO>;
  constexpr int NK = L::NK, NB = L::NB, NSB = L::NSB;
  constexpr int ROWS = L::TILES * BM;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const FwdParams& p = pp.f;
  const Geom& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // what this block computes
  const int spare = (int)blockIdx.x - pp.whole;
  const bool whole = spare < 0;
  const int shared = whole ? 0 : spare / pp.splits;
  const int splits = whole ? 1 : pp.splits, split = whole ? 0 : spare - shared * pp.splits;
  const Item it = item_of(pp, whole ? (int)blockIdx.x : pp.whole + shared);
  const int tile = it.tile, h = it.h, s = stream_of_rank(p, it.s);
  const StreamStep st = stream_step(p, s);
  const int row0 = tile * ROWS;
  const int rows = min(ROWS, st.n * g.group - row0);
  if (rows <= 0) return;
  const TileKeys tk = tile_keys(g, st, row0, rows);
  const int b0 = tk.first + (int)((long long)tk.count * split / splits);
  const int nblk = tk.first + (int)((long long)tk.count * (split + 1) / splits) - b0;
  if (nblk == 0) {
    // no keys here: rows that see none at all are written by the first split, the join skips the rest
    if (tk.count == 0 && split == 0) {
      for (int i = threadIdx.x; i < rows * (D / 8); i += THREADS) {
        const int r = row0 + i / (D / 8), tok = r / g.group;
        const size_t at = (size_t)(st.row0 + tok) * g.q_heads + h * g.group + (r - tok * g.group);
        *(uint4*)(p.o + at * D + (i % (D / 8)) * 8) = make_uint4(0, 0, 0, 0);
        if (i % (D / 8) == 0 && p.lse) p.lse[at] = -INFINITY;
      }
    }
    return;
  }

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* kv_full = bars + 1;      // K and V bytes of a stage have landed
  uint64_t* k_empty = kv_full + NK;  // Q K^T with K of a stage is done
  uint64_t* v8_empty = k_empty + NK; // V's bytes of a stage are converted
  uint64_t* v_full = v8_empty + NK;
  uint64_t* v_empty = v_full + NV;
  uint64_t* s_full = v_empty + NV;   // S of a unit is in TMEM
  uint64_t* p_full = s_full + NSB;   // P of an accumulator is
  uint64_t* pv_done = p_full + NB;   // a group's last P V is done (three S accumulators)
  uint64_t* o_final = pv_done + 2;
  uint64_t* sc_full = o_final + 1;
  uint64_t* max_full = sc_full + NS;  // [group][quad]: both halves of the rows' maxima are there
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  float2* xch = reinterpret_cast<float2*>(smem + L::OFF_XCH);
  Scales* scales = reinterpret_cast<Scales*>(smem + L::OFF_SC);
  WaitCtx wc;
  wc.abort_flag = abort_flag;
  wc.timeout_ns = p.ctl.timeout_ns;
  wc.err_word = p.ctl.err_word;

  if (threadIdx.x == 0) {
    mbar_init(q_full, SOFTMAX);
    for (int i = 0; i < NK; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v8_empty[i], V_WARPS);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&v_full[i], V_WARPS);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < NSB; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < NB; ++i) mbar_init(&p_full[i], 8);
    for (int i = 0; i < 2; ++i) mbar_init(&pv_done[i], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&max_full[i], 2);
    mbar_init(o_final, 1);
    for (int i = 0; i < NS; ++i) mbar_init(&sc_full[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == WARP_K && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int* table = p.table + (long long)s * g.width;
  // Page of the 16 keys from `key` on; -1: none of them is to be read.
  auto page_at = [&](int key) {
    if (key >= tk.hi || key + SCALE_TOKENS <= tk.lo) return -1;
    const int pg = __ldg(table + (key >> g.page_shift));
    if ((unsigned)pg >= (unsigned)g.pages) {
      report_error(p.ctl.err_word, VATTN_ERR_DEVICE_BOUNDS);
      return -1;
    }
    return pg;
  };

  if (warp == WARP_K) {
    // Lanes 0-7 follow K's scales and pages, lanes 8-15 V's scales, one lane
    // for 16 keys; pages are fetched two blocks ahead and scales one, so that
    // the dependent loads do not stand in a row.
    const int sub = lane & 7;
    const float* sp = lane < 8 ? p.ks : p.vs;
    auto page_of = [&](int j) { return j < nblk && lane < 16 ? page_at((b0 + j) * BN + sub * SCALE_TOKENS) : -1; };
    auto scale_of = [&](int j, int pg) {
      return pg < 0 ? 0.f
                    : __ldg(sp + (cache_row(g, pg, h, ((b0 + j) * BN + sub * SCALE_TOKENS) & (g.page_tokens - 1)) >> 4));
    };
    int pg = page_of(0), pg_next = page_of(1);
    float sc = scale_of(0, pg);
    const int lanes_per_page = g.page_tokens >> 4;
    int issued = 0;
    bool ok = true;
    for (int j = 0; j < nblk; ++j) {
      const int pg_after = page_of(j + 2);
      const float sc_next = scale_of(j + 1, pg_next);
      const int sg = j % NK;
      const uint32_t free_phase = ((j / NK) & 1) ^ 1;
      ok = __all_sync(~0u, mbar_wait(&k_empty[sg], free_phase, wc) && mbar_wait(&v8_empty[sg], free_phase, wc));
      if (!ok || (p.ctl.debug_flags & VATTN_DEBUG_SKIP_ARRIVAL)) break;
      // one box of page_tokens rows for each page that holds a key to be read
      // (its first 16 keys may lie before the window: any of its groups of 16 names it)
      int page = pg;
      for (int i = 1; i < lanes_per_page; ++i) page = max(page, __shfl_down_sync(~0u, pg, i));
      const bool want = lane < 8 && lane % lanes_per_page == 0 && page >= 0;
      const uint32_t wanted = __ballot_sync(~0u, want);
      if (lane == 0) mbar_arrive_expect_tx(&kv_full[sg], 2 * __popc(wanted) * g.page_tokens * D);
      __syncwarp();
      if (want) {
        const int at = sg * L::QK + lane * SCALE_TOKENS * D;
        tma_load_3d(smem + L::OFF_K + at, &tm_k, &kv_full[sg], 0, 0, page * g.kv_heads + h);
        tma_load_3d(smem + L::OFF_V8 + at, &tm_v, &kv_full[sg], 0, 0, page * g.kv_heads + h);
      }
      ++issued;
      // 16 keys that are not read have scale 0: exponent -127, and P = 0
      if (lane < 8) {
        scales[j % NS].k[lane] = sc;
      } else if (lane < 16) {
        const int bits = __float_as_int(sc) & 0x7f800000;
        scales[j % NS].e[lane - 8] = (float)((bits >> 23) - 127);
        scales[j % NS].inv[lane - 8] = __int_as_float((254 << 23) - max(bits, 1 << 23));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc_full[j % NS]);
      pg = pg_next;
      pg_next = pg_after;
      sc = sc_next;
    }
    if (lane == 0)  // every issued copy has landed before the block can exit (a no-op unless aborted)
      for (int j = max(issued - NK, 0); j < issued; ++j) mbar_wait_drain(&kv_full[j % NK], (j / NK) & 1, wc);
  } else if (warp >= WARP_V && warp < WARP_V + V_WARPS) {
    constexpr int RP = 512 / D;            // rows of a warp-wide read, 16 bytes a lane
    constexpr int NL = BN / V_WARPS / RP;  // reads of a block
    const int half = (warp - WARP_V) * (BN / V_WARPS);
    // Eight lanes at a time read, and then store, four chunks of two rows.  d = 128: of rows r and r ^ 5, whose
    // swizzles differ in bit 2 (so the reads meet all banks) and in bit 0 (so the stores do); d = 64: of rows r, r + 1.
    const int c = D == 128 ? (lane & 3) | ((lane >> 1) & 4) : lane & 3;
    auto row_of = [&](int i) {
      return D == 128 ? half + 8 * (i >> 1) + ((2 * (i & 1) + (lane >> 4)) ^ (lane & 4 ? 5 : 0)) : half + i * RP + (lane >> 2);
    };
    for (int j = 0; j < nblk; ++j) {
      const int s8 = j % NK, sg = j % NV;
      if (!__all_sync(~0u, mbar_wait(&kv_full[s8], (j / NK) & 1, wc) &&
                               mbar_wait(&v_empty[sg], ((j / NV) & 1) ^ 1, wc)))
        break;
      const uint8_t* src = smem + L::OFF_V8 + s8 * L::QK;
      uint8_t* dst = smem + L::OFF_V + sg * L::V + (c >> 2) * (128 * 128);
      // rows outside the keys read become zeros: P is 0 there, and what a page holds past a stream's end may be NaN
      const int from = tk.lo - (b0 + j) * BN, to = tk.hi - (b0 + j) * BN;
      const bool all = from <= 0 && to >= BN;
#pragma unroll 8
      for (int i = 0; i < NL; ++i) {
        const int r = row_of(i);
        uint4 x = *(const uint4*)(src + byte_chunk<D>(r, c));
        if (!all && (r < from || r >= to)) x = make_uint4(0, 0, 0, 0);
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        uint32_t out[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) e4m3x4_to_f16x2(in[u], out[2 * u], out[2 * u + 1]);
        // 16 channels: two 16-byte chunks of the row's 128-byte box
        const int at = (2 * (c & 3)) ^ (r & 7);
        *(uint4*)(dst + r * 128 + (at << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
        *(uint4*)(dst + r * 128 + ((at ^ 1) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&v8_empty[s8]);
        mbar_arrive(&v_full[sg]);
      }
    }
  } else if (warp == WARP_MMA) {
    if (lane == 0) {
      const uint32_t q_base = smem_u32(smem + L::OFF_Q);
      const uint32_t k_base = smem_u32(smem + L::OFF_K);
      const uint32_t v_base = smem_u32(smem + L::OFF_V);
      bool ok = mbar_wait(q_full, 0, wc);
      // Unit n: S and then O of group n & 1, with key block n / 2 (TWO) or n, in S accumulator n % NB.  Two
      // accumulators: Q K^T of unit n + 2 follows P V of unit n, and the group waits for both.  Three: it follows P V
      // of unit n - 1, so that the next S is there when the group has stored its P.
      auto issue_qk = [&](int n) -> bool {
        const int j = TWO ? n >> 1 : n, w = n & 1, sg = j % NK, b = n % NB;
        if (!mbar_wait(&kv_full[sg], (j / NK) & 1, wc)) return false;
        tc_fence_after();
        const uint32_t kb = k_base + sg * L::QK, qb = q_base + (TWO ? w : 0) * 2 * L::QK;
#pragma unroll
        for (int part = 0; part < 2; ++part)  // hi, lo
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_ss_e4m3(tmem + (uint32_t)(b * 128), desc_bytes<D>(qb + part * L::QK + kk * 32),
                        desc_bytes<D>(kb + kk * 32), idesc_e4m3_f32(BM, BN), part + kk > 0);
        tc_commit(&s_full[n % NSB]);
        if (!TWO || w == 1) tc_commit(&k_empty[sg]);
        return true;
      };
      auto issue_pv = [&](int n) -> bool {
        const int j = TWO ? n >> 1 : n, w = n & 1, sg = j % NV, b = n % NB;
        if (!mbar_wait(&p_full[b], (n / NB) & 1, wc)) return false;
        if (!mbar_wait(&v_full[sg], (j / NV) & 1, wc)) return false;
        tc_fence_after();
        const uint32_t vb = v_base + sg * L::V;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_ts(tmem + L::O + (uint32_t)(w * D), tmem + (uint32_t)(b * 128) + kk * 8,
                 smem_desc_sw128(vb + kk * 2048, 128 * 128, 1024), idesc_f16_pv(D), (n >= 2 || kk > 0) ? 1u : 0u);
        if (NB > 2) tc_commit(&pv_done[w]);
        if (!TWO || w == 1) tc_commit(&v_empty[sg]);
        return true;
      };
      const int units = TWO ? 2 * nblk : nblk;
      for (int n = 0; ok && n < min(NB, units); ++n) ok = issue_qk(n);
      for (int n = 0; ok && n < units; ++n) {
        ok = issue_pv(n);
        if (ok && n + NB < units) ok = issue_qk(n + NB);
      }
      tc_commit(o_final);
      // every MMA this thread issued must be finished before TMEM is freed
      mbar_wait_drain(o_final, 0, wc);
    }
  } else {
    // ---------------- softmax groups ----------------
    const int w = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
    const int row = quad * 32 + lane;                    // in its tile
    const int brow = (TWO ? w * BM : 0) + row;           // in the thread block's rows
    const bool real = brow < rows;
    // none of the warp's rows exists: it leaves P as it finds it, in rows that nobody reads
    const bool idle = brow - lane >= rows;
    const int tok = real ? (row0 + brow) / g.group : 0;
    const size_t out_row =
        (size_t)(st.row0 + tok) * g.q_heads + h * g.group + (real ? row0 + brow - tok * g.group : 0);
    int lo = 0, hi = 0x7fffffff;  // rows that do not exist mask nothing, and are not written
    if (real) key_range(g, st, tok, &lo, &hi);
    // the query rows, scaled and split into hi + lo, in the MMA's layout: a warp takes ROWS / 16 of them, 16 bytes
    // of bf16 a lane; the rows' factors and non-finite marks go through shared memory to the lanes that need them
    float c_row, poison;
    {
      constexpr int LPR = D / 8, RPI = 32 / LPR, ITERS = ROWS / 16 / RPI;
      const int c = lane % LPR;
      uint4 x[ITERS];
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const int r = warp * (ROWS / 16) + i * RPI + lane / LPR;
        const int t = r < rows ? (row0 + r) / g.group : 0;
        x[i] = r < rows ? __ldg((const uint4*)(p.q + (long long)(st.row0 + t) * p.q_stride +
                                               (long long)(h * g.group + row0 + r - t * g.group) * D) + c)
                        : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const int r = warp * (ROWS / 16) + i * RPI + lane / LPR;
        uint32_t m = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                              __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
        m = max(m & 0xffffu, m >> 16);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
        const int sh = m == 0 ? 0 : min(7 - ((int)(m >> 7) - 127), 126);
        const float up = __int_as_float((sh + 127) << 23);
        uint32_t hv[2], lv[2];
        const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t hh[2], ll[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = bf16lo(in[2 * u + e]) * up, b = bf16hi(in[2 * u + e]) * up;
            hh[e] = pack_e4m3x2(a, b);
            const float2 back = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)hh[e]));
            ll[e] = pack_e4m3x2(a - back.x, b - back.y);
          }
          hv[u] = hh[0] | (hh[1] << 16);
          lv[u] = ll[0] | (ll[1] << 16);
        }
        uint8_t* at = smem + L::OFF_Q + (r >> 7) * 2 * L::QK + byte_chunk<D>(r & 127, c >> 1) + (c & 1) * 8;
        *(uint2*)at = make_uint2(hv[0], hv[1]);
        *(uint2*)(at + L::QK) = make_uint2(lv[0], lv[1]);
        if (c == 0)
          xch[r] = make_float2(p.scale_log2 * __int_as_float((127 - sh) << 23),
                               m >= 0x7f80u ? __int_as_float(0x7fc00000) : 0.f);
      }
      fence_async_smem();
      mbar_arrive(q_full);
      named_bar_sync(1, SOFTMAX);
      c_row = xch[brow].x;
      poison = xch[brow].y;
      named_bar_sync(1, SOFTMAX);
    }
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    const uint32_t tO = tmem + lane_addr + L::O + (uint32_t)(w * D);
    float* my_max = (float*)xch + (w * 2 + half) * 256 + row;          // two slots, 128 floats apart
    const float* other_max = (float*)xch + (w * 2 + 1 - half) * 256 + row;
    float m_ref = -INFINITY, l_sum = 0.f;
    bool ok = true;
    int sb = w;             // barrier of the S of the group's unit 2 i + w ...
    uint32_t s_phase = 0;   // ... and the parity of its phase
    auto next_unit = [&] {
      sb += 2;
      if (sb >= NSB) {
        sb -= NSB;
        s_phase ^= 1u;
      }
    };
    for (int i = 0;; ++i, next_unit()) {
      const int j = TWO ? i : 2 * i + w;
      if (j >= nblk) break;
      const int acc = sb < NB ? sb : sb - NB;  // S accumulator: the unit modulo NB
      const uint32_t tS = tmem + lane_addr + (uint32_t)(acc * 128);
      ok = __all_sync(~0u, mbar_wait(&sc_full[j % NS], (j / NS) & 1, wc) && mbar_wait(&s_full[sb], s_phase, wc));
      if (!ok) break;
      tc_fence_after();
      if (idle) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[acc]);
        continue;
      }
      // this thread's 64 scores: keys 64 half .. of the block
      uint32_t sr[2][32];
      tmem_ld32(tS + half * 64, sr[0]);
      tmem_ld32(tS + half * 64 + 32, sr[1]);
      // x = S f + e for each 16 keys; f > 0, so that a masked score stays -inf
      const float4 k4 = *(const float4*)&scales[j % NS].k[half * 4], e4 = *(const float4*)&scales[j % NS].e[half * 4];
      const float4 i4 = *(const float4*)&scales[j % NS].inv[half * 4];
      const float f[4] = {fmaxf(c_row * k4.x, 1.17549435e-38f), fmaxf(c_row * k4.y, 1.17549435e-38f),
                          fmaxf(c_row * k4.z, 1.17549435e-38f), fmaxf(c_row * k4.w, 1.17549435e-38f)};
      const float e[4] = {e4.x, e4.y, e4.z, e4.w}, inv[4] = {i4.x, i4.y, i4.z, i4.w};
      tmem_wait_ld();
      const int from = lo - (b0 + j) * BN - half * 64, to = hi - (b0 + j) * BN - half * 64;
      if (from > 0 || to < BN / 2) {
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2)
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (q2 * 32 + c < from || q2 * 32 + c >= to) sr[q2][c] = __float_as_uint(-INFINITY);
      }
      float mx = -INFINITY;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          const uint32_t* v = &sr[b >> 1][(b & 1) * 16 + c];
          m0 = fmax3(m0, __uint_as_float(v[0]), __uint_as_float(v[1]));
          m1 = fmax3(m1, __uint_as_float(v[2]), __uint_as_float(v[3]));
        }
        mx = fmaxf(mx, fmaf(fmaxf(m0, m1), f[b], e[b]));
      }
      // the other half of the row: both threads go on with the same maximum
      // (and P may now take the place of scores that the other thread has read)
      my_max[(i & 1) * 128] = mx;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&max_full[w * 4 + quad]);
      ok = __all_sync(~0u, mbar_wait(&max_full[w * 4 + quad], i & 1, wc));
      if (!ok) break;
      tc_fence_after();
      mx = fmaxf(mx, other_max[(i & 1) * 128]);
      bool need = false;
      float alpha = 1.f;
      if (i == 0) {
        m_ref = mx;
      } else if (mx > m_ref + RESCALE) {
        need = true;
        alpha = ex2(m_ref - mx);
        m_ref = mx;
        l_sum *= alpha;
      }
      const float ref = (m_ref == -INFINITY ? 0.f : m_ref) - P_SHIFT;
#pragma unroll
      for (int q2 = 0; q2 < 2; ++q2) {
        uint32_t pk[16];
#pragma unroll
        for (int b2 = 0; b2 < 2; ++b2) {
          const int b = q2 * 2 + b2;
          const float2 ff = make_float2(f[b], f[b]), ee = make_float2(e[b] - ref, e[b] - ref);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t* v = &sr[q2][b2 * 16 + 2 * c];
            const float2 x = ffma2(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), ff, ee);
            const float2 pr = make_float2(ex2(x.x), ex2(x.y));
            sum = fadd2(sum, pr);
            pk[b2 * 8 + c] = pack_f16(pr.x, pr.y);
          }
          l_sum = fmaf(sum.x + sum.y, inv[b], l_sum);
        }
        tmem_st16(tS + half * 32 + q2 * 16, pk);
      }
      // Three accumulators: the group's last P V, waited for here by every unit whether O is rescaled or not.  A wait
      // knows a phase by its parity, so it has to come while that phase is the one under way or the last one
      // complete: P V of this unit cannot complete before this warp's arrival on p_full below, and the unit before
      // has waited for the phase before this one.  (It is done by now: the softmax of a unit takes longer.)
      if (NB > 2 && i > 0) {
        ok = __all_sync(~0u, mbar_wait(&pv_done[w], (i - 1) & 1, wc));
        if (!ok) break;
        tc_fence_after();
      }
      if (__any_sync(~0u, need)) {
        // O of this group is quiescent: the commit that signalled this S also
        // covers the previous P V into it (two accumulators; with three it was
        // waited for), and the next one waits for p_full.
#pragma unroll 1
        for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c0, o);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
          tmem_st32(tO + c0, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[acc]);
    }
    // ---------------- epilogue ----------------
    if (ok && !*abort_flag) ok = mbar_wait(o_final, 0, wc);
    ok = __all_sync(~0u, ok);
    tc_fence_after();
    named_bar_sync(1, SOFTMAX);  // the maxima's slots are read
    xch[(w * 2 + half) * 128 + row] = make_float2(m_ref, l_sum);
    named_bar_sync(1, SOFTMAX);
    if (ok && !*abort_flag) {
      // the two threads of a row have one reference and half the sum each; without TWO the groups' halves of the
      // keys are joined too.  Each thread writes SPAN channels.
      float m = m_ref, l = l_sum + xch[(w * 2 + 1 - half) * 128 + row].y, a0 = 1.f, a1 = 0.f;
      bool both = false;
      if constexpr (!TWO) {
        const float2 x0 = xch[(2 - 2 * w) * 128 + row];
        const float other_l = x0.y + xch[(3 - 2 * w) * 128 + row].y;
        m = fmaxf(m_ref, x0.x);
        const float m0 = m == -INFINITY ? 0.f : m;
        const float a_self = ex2(m_ref - m0), a_other = ex2(x0.x - m0);
        l = l * a_self + other_l * a_other;  // a group without blocks has l = 0 and m = -inf
        a0 = w == 0 ? a_self : a_other;
        a1 = w == 0 ? a_other : a_self;
        both = nblk >= 2;
      }
      if (lo < hi) l += poison;  // (a row that sees nothing stays empty whatever its query)
      const float norm = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      a0 *= norm;
      a1 *= norm;
      constexpr int SPAN = TWO ? D / 2 : D / 4;
      const int col0 = (TWO ? half : w * 2 + half) * SPAN;
      const uint32_t t0 = (TWO ? tO : tmem + lane_addr + L::O) + col0, t1 = tmem + lane_addr + L::O + D + col0;
      float o[SPAN];
#pragma unroll
      for (int c = 0; c < SPAN; c += 16) {
        uint32_t x1[16];
        tmem_ld16(t0 + c, reinterpret_cast<uint32_t*>(o) + c);
        if (!TWO && both) tmem_ld16(t1 + c, x1);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[c + e] = o[c + e] * a0 + (!TWO && both ? __uint_as_float(x1[e]) * a1 : 0.f);
      }
      // through shared memory (every tile in it is done with), so that a warp stores whole runs of a row
      uint8_t* stage = smem + warp * 32 * SPAN * 4;
      const size_t pr = ((size_t)shared * splits + split) * ROWS + (TWO ? w * BM : 0) + quad * 32;
      if (whole) {
        constexpr int NCH = SPAN / 8, SH = NCH >= 8 ? 0 : NCH == 4 ? 1 : 2;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
          *(uint4*)(stage + lane * SPAN * 2 + ((c ^ ((lane >> SH) & (NCH - 1))) << 4)) =
              make_uint4(pack_bf16(o[8 * c], o[8 * c + 1]), pack_bf16(o[8 * c + 2], o[8 * c + 3]),
                         pack_bf16(o[8 * c + 4], o[8 * c + 5]), pack_bf16(o[8 * c + 6], o[8 * c + 7]));
        __syncwarp();
        const int c = lane % NCH;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int r = i * (32 / NCH) + lane / NCH;
          const size_t to = __shfl_sync(~0u, out_row, r);
          const uint4 v = *(const uint4*)(stage + r * SPAN * 2 + ((c ^ ((r >> SH) & (NCH - 1))) << 4));
          if ((TWO ? w * BM : 0) + quad * 32 + r < rows) *(uint4*)(p.o + to * D + col0 + c * 8) = v;
        }
      } else {
        constexpr int NCH = SPAN / 4, SH = NCH >= 8 ? 0 : 1, MASK = NCH >= 8 ? 7 : NCH - 1;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
          *(float4*)(stage + lane * SPAN * 4 + ((c ^ ((lane >> SH) & MASK)) << 4)) =
              make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        __syncwarp();
        const int c = lane % NCH;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int r = i * (32 / NCH) + lane / NCH;
          const float4 v = *(const float4*)(stage + r * SPAN * 4 + ((c ^ ((r >> SH) & MASK)) << 4));
          *(float4*)(pp.part + (pr + r) * D + col0 + c * 4) = v;
        }
      }
      if (half == 0 && (TWO || w == 0) && real) {
        if (!whole)
          pp.part_ml[pr + lane] = make_float2(m, l);
        else if (p.lse)
          p.lse[out_row] = (m - P_SHIFT + __log2f(l)) * 0.69314718055994531f;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the splits of each row of the shared items, in their order; one warp a row.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const Params pp, int tile_rows) {
  const FwdParams& p = pp.f;
  const Geom& g = p.g;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const Item it = item_of(pp, pp.whole + blockIdx.x);
  const StreamStep st = stream_step(p, stream_of_rank(p, it.s));
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rows = min(tile_rows, st.n * g.group - it.tile * tile_rows);
  if (row >= rows) return;
  const TileKeys tk = tile_keys(g, st, it.tile * tile_rows, rows);
  if (tk.count == 0) return;
  constexpr int PER = D / 32;
  float acc[PER] = {};
  float m = -INFINITY, l = 0.f;
#pragma unroll 2
  for (int i = 0; i < pp.splits; ++i) {
    if ((long long)tk.count * i / pp.splits == (long long)tk.count * (i + 1) / pp.splits) continue;
    const size_t pr = ((size_t)blockIdx.x * pp.splits + i) * tile_rows + row;
    const float2 ml = __ldcg(pp.part_ml + pr);
    float v[PER];
#pragma unroll
    for (int c = 0; c < PER; c += 2)
      *(float2*)(v + c) = __ldcg((const float2*)(pp.part + pr * D + lane * PER + c));
    const float m_new = fmaxf(m, ml.x), ref = m_new == -INFINITY ? 0.f : m_new;
    const float a = ex2(m - ref), e = ex2(ml.x - ref);
    l = l * a + ml.y * e;
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = acc[c] * a + v[c] * e;
    m = m_new;
  }
  const int r = it.tile * tile_rows + row;
  const int tok = r / g.group;
  const size_t at = (size_t)(st.row0 + tok) * g.q_heads + it.h * g.group + (r - tok * g.group);
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < PER; c += 2)
    *(uint32_t*)(p.o + at * D + lane * PER + c) = pack_bf16(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0 && p.lse) p.lse[at] = (m - P_SHIFT + __log2f(l)) * 0.69314718055994531f;
}

// Query rows a thread block takes (see TWO).
int rows_of(const Geom& g, long long max_new) { return max_new * g.group > BM ? 2 * BM : BM; }
int tiles_of(const Geom& g, long long max_new) {
  const int rows = rows_of(g, max_new);
  return (int)((max_new * g.group + rows - 1) / rows);
}

// How the items are dealt out.  In units of a key block, a thread block costs
// its keys and about 3 for its start and end, and 3 more where partial results
// are written and joined; the cache's capacity stands in for the streams'
// lengths, which the host does not know (half of it for several streams).
//  - One stream: as many items as fill whole waves of the 148 SMs get a thread
//    block each, the rest are split into shares that fill the last waves (3000
//    token-causal queries over 9000 keys, 24 heads: 355 us, 469 unsplit).
//  - Else all items get the same number of splits: enough that the last ones
//    to finish are short, counting half the tiles as there.
constexpr int SMS = 148, MOST = SMS * 8;  // MOST bounds the partial results
struct Deal {
  long long items, whole;
  int splits;
};
Deal deal(const Geom& g, long long tiles) {
  Deal d;
  d.items = (long long)g.streams * g.kv_heads * tiles;
  d.whole = d.items;
  d.splits = 1;
  const double blocks = std::max(1.0, (double)g.width * g.page_tokens / BN * (g.streams == 1 ? 1.0 : 0.5));
  double least = 1e300;
  auto take = [&](long long whole, int splits, double cost) {
    if (cost < least) {
      least = cost;
      d.whole = splits == 1 ? d.items : whole;
      d.splits = splits;
    }
  };
  if (g.streams == 1) {
    // (costs count from the first of these waves on, so that the choice is the same whatever number comes before)
    const long long waves = d.items / SMS, w0 = std::max(0ll, waves - 2);
    for (long long w = w0; w <= waves; ++w) {
      const long long rest = d.items - w * SMS;
      for (int sp = 1; sp == 1 || (sp <= 64 && rest * sp <= MOST); ++sp)
        take(w * SMS, sp, (double)(w - w0) * (blocks + 3) + (double)((rest * sp + SMS - 1) / SMS) * (blocks / sp + (sp == 1 ? 3 : 6)));
    }
  } else {
    for (int sp = 1; sp == 1 || (sp <= 64 && d.items * sp <= MOST); ++sp) {
      const double each = blocks / sp + (sp == 1 ? 3 : 6);
      take(0, sp, std::max(1.0, 0.5 * d.items * sp / SMS) * each + each);
    }
  }
  return d;
}
size_t part_rows(const Deal& d, int rows) {
  return (size_t)(d.items - d.whole) * (d.splits == 1 ? 0 : d.splits) * rows;
}
size_t bytes_of(const Geom& g, size_t part_rows) { return part_rows * (g.d + 2) * sizeof(float); }

template <int D, bool TWO>
cudaError_t launch(const FwdParams& f, void* ws, cudaStream_t stream) {
  const int rows = rows_of(f.g, f.max_new);
  const Deal d = deal(f.g, tiles_of(f.g, f.max_new));
  const long long grid = d.whole + (d.items - d.whole) * d.splits;  // the items, or few more than MOST
  Params p;
  p.f = f;
  p.q_tiles = tiles_of(f.g, f.max_new);
  p.whole = (int)d.whole;
  p.splits = d.splits;
  p.part = (float*)ws;
  p.part_ml = (float2*)(p.part + part_rows(d, rows) * D);
  CUtensorMap tk, tv;
  const char* err = nullptr;
  const long long heads = (long long)f.g.pages * f.g.kv_heads;
  if (!make_tmap_pages(&tk, f.kc, D, f.g.page_tokens, heads, &err) ||
      !make_tmap_pages(&tv, f.vc, D, f.g.page_tokens, heads, &err))
    return cudaErrorInvalidValue;
  auto kernel = many_kernel<D, TWO>;
  constexpr int smem = Smem<D, TWO>::ALLOC;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)grid, THREADS, smem, stream>>>(tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || d.whole == d.items) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(d.items - d.whole), (unsigned)(rows / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, rows);
}

}  // namespace many
}  // namespace cache

long long cache_many_items(const cache::Geom& g, long long max_new) {
  return (long long)g.streams * g.kv_heads * cache::many::tiles_of(g, max_new);
}
size_t cache_many_workspace(const cache::Geom& g, long long max_new) {
  using namespace cache::many;
  return bytes_of(g, part_rows(deal(g, tiles_of(g, max_new)), rows_of(g, max_new)));
}
size_t cache_many_workspace_most(const cache::Geom& g, long long max_new) {
  using namespace cache::many;
  size_t most = 0;
  const long long one = std::min<long long>(max_new, BM / g.group);  // the most tokens of one tile of BM rows
  if (one > 0 && !cache_few_fits(g, one)) most = part_rows(deal(g, 1), BM);
  if (max_new * g.group <= BM) return bytes_of(g, most);
  // Tiles of 2 BM rows.  Several streams: none is split once two splits of each item are too many.  One stream: the
  // choice depends on what is left after whole waves, and from three waves on 148 tiles show every remainder.
  const long long per_tile = (long long)g.streams * g.kv_heads;
  long long last = tiles_of(g, max_new);
  last = std::min(last, g.streams > 1 ? MOST / 2 / per_tile : (2 * SMS - 1) / per_tile + 1 + SMS);
  for (long long tiles = tiles_of(g, BM / g.group + 1); tiles <= last; ++tiles)
    most = std::max(most, part_rows(deal(g, tiles), 2 * BM));
  return bytes_of(g, most);
}
cudaError_t launch_cache_many(const cache::FwdParams& p, void* ws, cudaStream_t st) {
  using namespace cache::many;
  const bool two = rows_of(p.g, p.max_new) > BM;
  if (p.g.d == 128) return two ? launch<128, true>(p, ws, st) : launch<128, false>(p, ws, st);
  return two ? launch<64, true>(p, ws, st) : launch<64, false>(p, ws, st);
}

}  // namespace vattn
