// Attention over the 8-bit key/value cache for few query rows: the new tokens
// of a stream times the query heads of a kv head make at most 16 rows.
//
// Bound by HBM: 2 d bytes for every key and kv head, read once, against 4 d
// flop for each row.  So the design serves the loads:
//  - every warp streams its own 32-key steps through a private ring in shared
//    memory with 16-byte asynchronous copies: no barrier between warps, and
//    three thread blocks of four warps keep about 100 KB in flight on an SM,
//    twice what the memory latency needs at full rate;
//  - a fixed grid shares all streams' 128-key tiles evenly, whatever their
//    lengths: thread blocks take equal runs of the tiles, which are laid out
//    stream by stream and head by head.  A (stream, head) that
//    spans several thread blocks leaves partial results that a second kernel
//    joins in a fixed order; it is launched early (programmatic dependent
//    launch) so that only its joins are exposed.
//  - the products run on mma.sync m16n8k16: 16 rows are far too few for a
//    tcgen05 tile, and the operands come from registers as they are converted.
//    Both are transposed, S^T = K Q^T and O^T = V^T P^T, so that keys and
//    channels fill the 16 rows of an instruction and the query rows its 8
//    columns: half the instructions and accumulators of the other way round.
//
// Numbers: e4m3 bytes become f16 exactly.  A query row is scaled by a power of
// two into f16's upper range, so its 8 significant bits are exact down to
// 2^-29 of the row's largest element.  The reference m of a row moves when a
// score passes it by more than 2^8; P = 2^(x - m + 7) <= 2^15 is f16, 11
// significant bits down to 2^-21 of 2^m.  A V scale is a power of two: it
// enters the exponent of P, x_j = s_j + log2(vs), and the row sum takes
// P 2^-log2(vs), so that O needs no scale and no weight overflows.
#include "cache.cuh"

namespace vattn {
namespace cache {
namespace few {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int STEP = 32;             // keys of a warp's step
constexpr int TILE = WARPS * STEP;   // keys of a thread block's step
constexpr int ROWS = 16;
constexpr int CTAS_PER_SM = 3;
constexpr int GRID = 148 * CTAS_PER_SM;
constexpr float P_SHIFT = 7.0f;      // P = 2^(x - m + 7)
constexpr float RESCALE = 8.0f;

// Two partial results a thread block: of the (stream, head) that began before
// its tiles (slot 0) and of the one that goes on after them (slot 1).
constexpr int SLOTS = GRID * 2;
// What a thread block leaves to be joined with the partial results of those
// after it, in its second slot: `blocks` of them share it (0: nothing).
struct Shared {
  int row0, head, rows, blocks;  // first token, kv head, query rows
};
inline size_t workspace_bytes(int d) {
  return (size_t)SLOTS * ROWS * (d + 2) * sizeof(float) + GRID * sizeof(Shared);
}
__device__ __forceinline__ Shared* shared_of(void* ws, int d) {
  return (Shared*)((float*)ws + (size_t)SLOTS * ROWS * (d + 2));
}
__device__ __forceinline__ float* slot_o(void* ws, int d, int slot) { return (float*)ws + (size_t)slot * ROWS * d; }
__device__ __forceinline__ float2* slot_ml(void* ws, int d, int slot) {
  return (float2*)((float*)ws + (size_t)SLOTS * ROWS * d) + (size_t)slot * ROWS;
}

template <int D>
struct Ring {
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr int HALF = STEP * D;                     // K or V bytes of a step
  static constexpr int SCALES = 16;                         // 2 K and 2 V scales
  static constexpr int STAGE = 2 * HALF + SCALES;
  static constexpr int WARP = STAGES * STAGE;
  static constexpr int MERGE = ROWS * D * 4 + ROWS * 8;     // a warp's partial result, over its own ring
  static constexpr int PER_WARP = WARP > MERGE ? WARP : MERGE;
  static constexpr int TOTAL = WARPS * PER_WARP;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;  // 0: the 16 bytes become zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 x 8 f16 matrix, a row's pair of columns per lane -> its transpose.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Shared-memory layouts of a step.  Lane (g, t) = (lane / 4, lane % 4) of the
// MMA fragments reads, eight lanes (two g, four t) at a time:
//  K: 16 bytes at chunk t (+ 4) of row g (+ 8): at d = 128 odd rows keep their
//     chunks 4 further on, so that the eight lanes meet all 32 banks (at d = 64
//     two rows fill them anyway);
//  V: chunk g of rows 2 t + const: chunks are turned by 2 (row / 2).  d = 64:
//     8-byte reads by 16 lanes; rows with bit 1 set swap with their neighbours,
//     rows with bit 2 set turn by two chunks.
template <int D>
__device__ __forceinline__ uint32_t k_at(int row, int chunk) {
  return D == 128 ? row * 128 + ((chunk ^ ((row & 1) << 2)) << 4) : row * 64 + (chunk << 4);
}
template <int D>
__device__ __forceinline__ uint32_t v_at(int row, int chunk) {
  return D == 128 ? row * 128 + ((chunk ^ (((row >> 1) & 3) << 1)) << 4)
                  : (row ^ ((row >> 1) & 1)) * 64 + ((chunk ^ (((row >> 2) & 1) << 1)) << 4);
}

// `total` tiles shared evenly: the first `extra` thread blocks take per + 1 of
// them, the others `per` (and those past the last tile none).  With few tiles a
// block no more blocks than needed take part: 792 tiles (one token over 4101
// keys, 24 heads) go to 396 blocks of two, not to 348 of two and 96 of one,
// which end at the same time but leave more to join (13.6 against 14.1 us); with
// many, the blocks of an SM share its bandwidth, and all of them are wanted
// (54 against 59 us for a few tokens in 16 streams).
struct Shares {
  long long per, extra, total;
  __device__ __forceinline__ explicit Shares(long long t) : total(t) {
    if (t < 4 * GRID) {
      per = ((uint32_t)t + GRID - 1) / GRID;
      extra = 0;
    } else {
      per = t < (1ll << 31) ? (uint32_t)t / GRID : t / GRID;
      extra = t - per * GRID;
    }
  }
  __device__ __forceinline__ long long first(int block) const {
    return min(block * per + min((long long)block, extra), total);
  }
  __device__ __forceinline__ int owner(long long tile) const {
    const long long wide = extra * (per + 1);  // tiles of the blocks that take one more
    const bool small = total < (1ll << 31);
    if (tile < wide) return small ? (uint32_t)tile / (uint32_t)(per + 1) : (int)(tile / (per + 1));
    return (int)extra + (small ? (uint32_t)(tile - wide) / (uint32_t)per : (int)((tile - wide) / per));
  }
};

// The tiles of one stream, for each kv head: keys [base, end), `tiles` of TILE.
struct StreamTiles {
  StreamStep st;
  int lo, base, end, tiles;  // base: lo rounded down to a step
};
__device__ __forceinline__ StreamTiles stream_tiles(const FwdParams& p, int s) {
  StreamTiles r;
  r.st = stream_step(p, s);
  r.lo = r.base = r.end = r.tiles = 0;
  if (r.st.n > 0) {
    int hi, x;
    key_range(p.g, r.st, 0, &r.lo, &x);
    key_range(p.g, r.st, r.st.n - 1, &x, &hi);
    r.base = r.lo & ~(STEP - 1);
    r.end = max(hi, r.base);
    r.tiles = max(1, (r.end - r.base + TILE - 1) / TILE);  // one that is empty still writes its rows
  }
  return r;
}

// Finds the stream of tile `want` (of all heads' tiles, stream by stream): its
// index, its first tile, and the total.  All threads of the block take part.
struct Place {
  int stream;
  long long first, total;
};
template <int NT, class Wanted>
__device__ __forceinline__ Place find_stream(const FwdParams& p, Wanted wanted, long long* sums, Place* out) {
  const int t = threadIdx.x;
  const int per = (p.g.streams + NT - 1) / NT;
  const int s0 = min(t * per, p.g.streams), s1 = min(s0 + per, p.g.streams);
  long long mine = 0;
  for (int s = s0; s < s1; ++s) mine += stream_tiles(p, s).tiles;
  mine *= p.g.kv_heads;
  long long x = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, x, o);
    if ((t & 31) >= o) x += y;
  }
  if ((t & 31) == 31) sums[t >> 5] = x;
  __syncthreads();
  long long before = x - mine, total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < (t >> 5)) before += sums[w];
    total += sums[w];
  }
  const long long want = wanted(total);
  if (want >= before && want < before + mine) {
    int s = s0;
    for (;; ++s) {
      const long long n = (long long)stream_tiles(p, s).tiles * p.g.kv_heads;
      if (want < before + n) break;
      before += n;
    }
    out->stream = s;
    out->first = before;
  }
  __syncthreads();
  Place r = *out;
  r.total = total;
  return r;
}

// NT: blocks of 8 query rows.
template <int D, int NT>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) few_kernel(const FwdParams p, void* ws) {
  using R = Ring<D>;
  constexpr int KS = D / 16;  // k-steps of S^T; m-tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long sums[WARPS];
  __shared__ Place place;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Geom& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int fg = lane >> 2, ft = lane & 3;
  uint8_t* mine = smem + warp * R::PER_WARP;
  const uint32_t ring = smem_u32(mine);

  const Place pl = find_stream<THREADS>(
      p,
      [](long long total) {
        const long long t = Shares(total).first(blockIdx.x);
        return t < total ? t : -1;
      },
      sums, &place);
  const Shares shares(pl.total);
  long long at = shares.first(blockIdx.x);
  const long long stop = shares.first(blockIdx.x + 1);
  Shared left = {0, 0, 0, 0};
  if (at >= stop) {
    if (threadIdx.x == 0) shared_of(ws, D)[blockIdx.x] = left;
    return;
  }
  int s = pl.stream;
  long long first = pl.first;  // first tile of stream s
  StreamTiles sp = stream_tiles(p, s);

  while (at < stop) {
    while (at >= first + (long long)sp.tiles * g.kv_heads) {
      first += (long long)sp.tiles * g.kv_heads;
      sp = stream_tiles(p, ++s);
    }
    const long long in_stream = at - first;
    const int h = in_stream < (1ll << 31) ? (uint32_t)in_stream / (uint32_t)sp.tiles : (int)(in_stream / sp.tiles);
    const int k0 = (int)(in_stream - (long long)h * sp.tiles);
    const int k1 = (int)min((long long)sp.tiles, k0 + (stop - at));
    const int rows = sp.st.n * g.group;
    if (k0 == 0 && k1 < sp.tiles)
      left = {sp.st.row0, h, rows, shares.owner(at + sp.tiles - 1) - (int)blockIdx.x + 1};
    at += k1 - k0;
    const int min_lo = sp.lo, max_hi = sp.end;

    // steps of this warp: keys sp.base + (k * WARPS + warp) * STEP, k in [k0, k1)
    const int* table = p.table + (long long)s * g.width;
    auto step_key = [&](int k) { return sp.base + (k * WARPS + warp) * STEP; };
    // Pages of a step's two 16-key halves as read from the table (-1: none of its keys is to be read).  They are
    // looked at only when the step is loaded, later on, so that no warp waits here.
    auto pages_of = [&](int k) {
      int2 r = make_int2(-1, -1);
      if (k < k1) {
        const int a = step_key(k), b = a + SCALE_TOKENS;
        if (a < max_hi && b > min_lo) r.x = __ldg(table + (a >> g.page_shift));
        if (b < max_hi && b + SCALE_TOKENS > min_lo) r.y = __ldg(table + (b >> g.page_shift));
      }
      return r;
    };
    auto load = [&](int k, const int2& raw) {
      if (k < k1) {
        const int key0 = step_key(k);
        const uint32_t dst = ring + ((k - k0) % R::STAGES) * R::STAGE;
        const int pg0 = raw.x < g.pages ? raw.x : -1, pg1 = raw.y < g.pages ? raw.y : -1;
        if ((pg0 < 0 && key0 < max_hi && key0 + SCALE_TOKENS > min_lo) ||
            (pg1 < 0 && key0 + SCALE_TOKENS < max_hi && key0 + STEP > min_lo))
          report_error(p.ctl.err_word, VATTN_ERR_DEVICE_BOUNDS);
        const long long row0 = cache_row(g, max(pg0, 0), h, key0 & (g.page_tokens - 1));
        const long long row1 = cache_row(g, max(pg1, 0), h, (key0 + SCALE_TOKENS) & (g.page_tokens - 1));
        constexpr int CH = D / 16, RP = 32 / CH;
        const int c = lane % CH, r0 = lane / CH;
        const long long off0 = row0 * D + r0 * D + c * 16, off1 = row1 * D + r0 * D + c * 16;
        if (pg0 >= 0 && pg1 >= 0 && key0 >= min_lo && key0 + STEP <= max_hi) {
          const uint8_t *k_a = p.kc + off0, *k_b = p.kc + off1, *v_a = p.vc + off0, *v_b = p.vc + off1;
#pragma unroll
          for (int i = 0; i < STEP / RP; ++i) {
            const bool second = i * RP >= SCALE_TOKENS;
            const int at = (i * RP % SCALE_TOKENS) * D;
            cp16(dst + k_at<D>(i * RP + r0, c), (second ? k_b : k_a) + at);
            cp16(dst + R::HALF + v_at<D>(i * RP + r0, c), (second ? v_b : v_a) + at);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < STEP / RP; ++i) {
            const int r = i * RP + r0;
            const bool second = i * RP >= SCALE_TOKENS;
            const bool in = (second ? pg1 : pg0) >= 0 && key0 + r < max_hi && key0 + r >= min_lo;
            const long long off = in ? (second ? off1 : off0) + (i * RP % SCALE_TOKENS) * D : 0;
            cp16(dst + k_at<D>(r, c), p.kc + off, in);
            cp16(dst + R::HALF + v_at<D>(r, c), p.vc + off, in);
          }
        }
        if (lane < 4) {
          const bool in = (lane & 1 ? pg1 : pg0) >= 0;
          const long long idx = in ? (lane & 1 ? row1 : row0) >> 4 : 0;
          cp4(dst + 2 * R::HALF + lane * 4, (lane & 2 ? p.vs : p.ks) + idx, in);
        }
      }
      cp_commit();
    };
    // query rows fg (+ 8) as f16 MMA fragments, each row scaled by a power of two; then what belongs to
    // the rows 2 ft, 2 ft + 1 (+ 8) whose scores this lane holds
    uint32_t qf[NT][KS][2];
    float c_row[NT][2], poison[NT][2];
    int lo[NT][2], hi[NT][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int r = fg + 8 * u;
      const bool in = r < rows;
      const int tok = in ? r / g.group : 0;
      const __nv_bfloat16* src = p.q + (long long)(sp.st.row0 + tok) * p.q_stride +
                                 (long long)(h * g.group + (in ? r - tok * g.group : 0)) * D;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        const uint2 w = in ? __ldg((const uint2*)(src + (kk >> 2) * 64 + 16 * ft + 4 * (kk & 3))) : make_uint2(0, 0);
        qf[u][kk][0] = w.x;
        qf[u][kk][1] = w.y;
      }
    }
    // the first keys are on their way before the rows are needed
    int2 next;
    {
      int2 raw[R::STAGES];
#pragma unroll
      for (int i = 0; i < R::STAGES; ++i) raw[i] = pages_of(k0 + i);
#pragma unroll
      for (int i = 0; i < R::STAGES; ++i) load(k0 + i, raw[i]);
      next = pages_of(k0 + R::STAGES);
    }
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      uint32_t m = 0;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
        m = __vmaxu2(m, __vmaxu2(qf[u][kk][0] & 0x7fff7fffu, qf[u][kk][1] & 0x7fff7fffu));
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(~0u, m, 1));
      m = max(m, __shfl_xor_sync(~0u, m, 2));
      const float bad = m >= 0x7f80u ? __int_as_float(0x7fc00000) : 0.f;
      const int sh = m == 0 ? 0 : min(14 - ((int)(m >> 7) - 127), 126);
      const float up = __int_as_float((sh + 127) << 23);
      const float down = p.scale_log2 * __int_as_float((127 - sh) << 23);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        qf[u][kk][0] = pack_f16(bf16lo(qf[u][kk][0]) * up, bf16hi(qf[u][kk][0]) * up);
        qf[u][kk][1] = pack_f16(bf16lo(qf[u][kk][1]) * up, bf16hi(qf[u][kk][1]) * up);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        c_row[u][e] = __shfl_sync(~0u, down, (2 * ft + e) * 4);
        poison[u][e] = __shfl_sync(~0u, bad, (2 * ft + e) * 4);
        const int row = 2 * ft + e + 8 * u;
        key_range(g, sp.st, row < rows ? row / g.group : 0, &lo[u][e], &hi[u][e]);
      }
    }
    int all_lo, all_hi, x;  // keys that every row sees
    key_range(g, sp.st, 0, &x, &all_hi);
    key_range(g, sp.st, sp.st.n - 1, &all_lo, &x);

    float o[NT][KS][4];
    float m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
      for (int j = 0; j < KS; ++j) o[u][j][0] = o[u][j][1] = o[u][j][2] = o[u][j][3] = 0.f;
      m_run[u][0] = m_run[u][1] = -INFINITY;
      l_run[u][0] = l_run[u][1] = 0.f;
    }

    for (int k = k0; k < k1; ++k) {
      if (k > k0) {  // into the stage that the last step left
        load(k + R::STAGES - 1, next);
        next = pages_of(k + R::STAGES);
      }
      cp_wait<R::STAGES - 1>();
      __syncwarp();
      const uint32_t st = ring + ((k - k0) % R::STAGES) * R::STAGE;
      const int key0 = step_key(k);
      if (key0 < max_hi) {
        // S^T: 16-key tile b, rows fg and fg + 8
        float sc[NT][2][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
          for (int u = 0; u < NT; ++u) sc[u][b][0] = sc[u][b][1] = sc[u][b][2] = sc[u][b][3] = 0.f;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 w0 = lds128(st + k_at<D>(16 * b + fg, ft + 4 * c));
            const uint4 w1 = lds128(st + k_at<D>(16 * b + fg + 8, ft + 4 * c));
            const uint32_t a[4] = {w0.x, w0.y, w0.z, w0.w}, e[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t f[4];
              e4m3x4_to_f16x2(a[i], f[0], f[2]);
              e4m3x4_to_f16x2(e[i], f[1], f[3]);
#pragma unroll
              for (int u = 0; u < NT; ++u) mma16816(sc[u][b], f, qf[u][c * 4 + i][0], qf[u][c * 4 + i][1]);
            }
          }
        }
        const bool whole = key0 >= all_lo && key0 + STEP <= all_hi;
        float kf[2], ev[2], inv[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          kf[b] = lds32(st + 2 * R::HALF + b * 4);
          const int bits = __float_as_int(lds32(st + 2 * R::HALF + 8 + b * 4)) & 0x7f800000;
          ev[b] = (float)((bits >> 23) - 127);
          inv[b] = __int_as_float((254 << 23) - max(bits, 1 << 23));
        }
        uint32_t pf[NT][2][2];  // P^T as MMA fragments
        bool over = false;
        float mx[NT][2];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float f = fmaxf(c_row[u][e] * kf[b], 1.17549435e-38f), off = ev[b] + poison[u][e];
#pragma unroll
              for (int i = 0; i < 2; ++i) sc[u][b][2 * i + e] = fmaf(sc[u][b][2 * i + e], f, off);
            }
          }
        if (!whole) {
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = key0 + 8 * i + fg;
                if (key < lo[u][e] || key >= hi[u][e]) sc[u][i >> 1][2 * (i & 1) + e] = -INFINITY;
              }
        }
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[u][e] = fmaxf(fmaxf(sc[u][0][e], sc[u][0][2 + e]), fmaxf(sc[u][1][e], sc[u][1][2 + e]));
            over = over || mx[u][e] > m_run[u][e] + RESCALE;
          }
        if (__any_sync(~0u, over)) {
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float m = mx[u][e];
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, w));
              const float m_new = fmaxf(m_run[u][e], m);
              alpha[e] = m_new == -INFINITY ? 1.f : ex2(m_run[u][e] - m_new);
              m_run[u][e] = m_new;
              l_run[u][e] *= alpha[e];
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              o[u][j][0] *= alpha[0];
              o[u][j][1] *= alpha[1];
              o[u][j][2] *= alpha[0];
              o[u][j][3] *= alpha[1];
            }
          }
        }
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          const float ref0 = (m_run[u][0] == -INFINITY ? 0.f : m_run[u][0]) - P_SHIFT;
          const float ref1 = (m_run[u][1] == -INFINITY ? 0.f : m_run[u][1]) - P_SHIFT;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float a0 = ex2(sc[u][b][0] - ref0), a1 = ex2(sc[u][b][1] - ref1);
            const float b0 = ex2(sc[u][b][2] - ref0), b1 = ex2(sc[u][b][3] - ref1);
            l_run[u][0] = fmaf(a0 + b0, inv[b], l_run[u][0]);
            l_run[u][1] = fmaf(a1 + b1, inv[b], l_run[u][1]);
            pf[u][b][0] = transpose8x8(pack_f16(a0, a1));
            pf[u][b][1] = transpose8x8(pack_f16(b0, b1));
          }
        }
        // O^T += V^T P^T: rows fg, fg + 8 of channel tile j are the channels (D / 8) fg + 2 j, + 1
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t w[4][D / 32];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * b + 2 * ft + (r & 1) + 8 * (r >> 1);
            if constexpr (D == 128) {
              const uint4 v = lds128(st + R::HALF + v_at<D>(row, fg));
              w[r][0] = v.x;
              w[r][1] = v.y;
              w[r][2] = v.z;
              w[r][3] = v.w;
            } else {
              const uint2 v = lds64(st + R::HALF + v_at<D>(row, fg >> 1) + (fg & 1) * 8);
              w[r][0] = v.x;
              w[r][1] = v.y;
            }
          }
#pragma unroll
          for (int q4 = 0; q4 < D / 32; ++q4) {
            // four keys' bytes of four channels -> key pairs of each channel
            const uint32_t a0 = __byte_perm(w[0][q4], w[1][q4], 0x5140), a1 = __byte_perm(w[0][q4], w[1][q4], 0x7362);
            const uint32_t b0 = __byte_perm(w[2][q4], w[3][q4], 0x5140), b1 = __byte_perm(w[2][q4], w[3][q4], 0x7362);
            uint32_t f0[4], f1[4];
            e4m3x4_to_f16x2(a0, f0[0], f0[1]);
            e4m3x4_to_f16x2(b0, f0[2], f0[3]);
            e4m3x4_to_f16x2(a1, f1[0], f1[1]);
            e4m3x4_to_f16x2(b1, f1[2], f1[3]);
#pragma unroll
            for (int u = 0; u < NT; ++u) {
              mma16816(o[u][q4 * 2], f0, pf[u][b][0], pf[u][b][1]);
              mma16816(o[u][q4 * 2 + 1], f1, pf[u][b][0], pf[u][b][1]);
            }
          }
        }
      }
      __syncwarp();  // the stage is free
    }
    cp_wait<0>();
    __syncwarp();

    // the warps' results, over their rings
    {
      float* mo = (float*)mine;
      float2* ml = (float2*)(mine + ROWS * D * 4);
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = l_run[u][e];
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l += __shfl_xor_sync(~0u, l, w);
          const int row = 2 * ft + e + 8 * u;
          if (fg == 0) ml[row] = make_float2(m_run[u][e], l);
#pragma unroll
          for (int j = 0; j < KS; j += 2)
            *(float4*)(mo + row * D + (D / 8) * fg + 2 * j) =
                make_float4(o[u][j][e], o[u][j][2 + e], o[u][j + 1][e], o[u][j + 1][2 + e]);
        }
    }
    __syncthreads();
    const bool complete = k0 == 0 && k1 == sp.tiles;
    const int slot = blockIdx.x * 2 + (k0 == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < rows * (D / 4); i += THREADS) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4;
      float2 ml[WARPS];
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        ml[w] = ((const float2*)(smem + w * R::PER_WARP + ROWS * D * 4))[r];
        m = fmaxf(m, ml[w].x);
      }
      const float m0 = m == -INFINITY ? 0.f : m;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float a = ex2(ml[w].x - m0);
        const float4 v = *(const float4*)(smem + w * R::PER_WARP + (r * D + c) * 4);
        l += ml[w].y * a;
        acc.x += v.x * a;
        acc.y += v.y * a;
        acc.z += v.z * a;
        acc.w += v.w * a;
      }
      if (complete) {
        const int tok = r / g.group;
        const size_t at_o = (size_t)(sp.st.row0 + tok) * g.q_heads + h * g.group + (r - tok * g.group);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        *(uint2*)(p.o + at_o * D + c) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (c == 0 && p.lse) p.lse[at_o] = (m - P_SHIFT + log2f(l)) * 0.69314718055994531f;
      } else {
        *(float4*)(slot_o(ws, D, slot) + r * D + c) = acc;
        if (c == 0) slot_ml(ws, D, slot)[r] = make_float2(m, l);
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) shared_of(ws, D)[blockIdx.x] = left;
}

// Joins the partial results of a row of a (stream, head) that several thread
// blocks share, the first of them blockIdx.x: their weights first, then groups
// of d / 4 threads take every so-manieth one, with several loads in flight.
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const FwdParams p, void* ws) {
  constexpr int LANES = D / 4, GROUPS = 128 / LANES;
  __shared__ float weight[GRID];
  __shared__ float red[4];
  __shared__ float4 accs[128];
  const Geom& g = p.g;
  const int t = threadIdx.x, r = blockIdx.y, c0 = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 left = __ldcg((const int4*)(shared_of(ws, D) + c0));
  const int row0 = left.x, h = left.y, n = left.w;
  if (n == 0 || r >= left.z) return;
  // partial result i: block c0 keeps it in its second slot, the others in their first
  auto slot_of = [&](int i) { return (c0 + i) * 2 + (i == 0 ? 1 : 0); };
  auto block_reduce = [&](float v, bool sum) {
    for (int o = 16; o > 0; o >>= 1) {
      const float w = __shfl_xor_sync(~0u, v, o);
      v = sum ? v + w : fmaxf(v, w);
    }
    __syncthreads();
    if ((t & 31) == 0) red[t >> 5] = v;
    __syncthreads();
    return sum ? (red[0] + red[1]) + (red[2] + red[3]) : fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  };
  constexpr int PER = (GRID + 127) / 128;
  float2 ml[PER];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    ml[i] = t + 128 * i < n ? __ldcg(slot_ml(ws, D, slot_of(t + 128 * i)) + r) : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, ml[i].x);
  }
  m = block_reduce(m, false);
  const float m0 = m == -INFINITY ? 0.f : m;
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (t + 128 * i < n) {
      const float w = ex2(ml[i].x - m0);
      weight[t + 128 * i] = w;
      l += ml[i].y * w;
    }
  l = block_reduce(l, true);
  const int c = (t % LANES) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = t / LANES; i < n; i += GROUPS) {
    const float4 v = __ldcg((const float4*)(slot_o(ws, D, slot_of(i)) + r * D + c));
    const float w = weight[i];
    acc.x = fmaf(v.x, w, acc.x);
    acc.y = fmaf(v.y, w, acc.y);
    acc.z = fmaf(v.z, w, acc.z);
    acc.w = fmaf(v.w, w, acc.w);
  }
  accs[t] = acc;
  __syncthreads();
  if (t >= LANES) return;
  for (int i = 1; i < GROUPS; ++i) {
    const float4 v = accs[t + i * LANES];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const int tok = r / g.group;
  const size_t at_o = (size_t)(row0 + tok) * g.q_heads + h * g.group + (r - tok * g.group);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *(uint2*)(p.o + at_o * D + c) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (c == 0 && p.lse) p.lse[at_o] = (m - P_SHIFT + log2f(l)) * 0.69314718055994531f;
}

template <int D>
cudaError_t launch(const FwdParams& p, void* ws, cudaStream_t st) {
  constexpr int smem = Ring<D>::TOTAL;
  auto kernel = p.max_new * p.g.group > 8 ? few_kernel<D, 2> : few_kernel<D, 1>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<GRID, THREADS, smem, st>>>(p, ws);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(GRID, (unsigned)(p.max_new * p.g.group));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, ws);
}

}  // namespace few
}  // namespace cache

bool cache_few_fits(const cache::Geom& g, long long max_new) { return max_new * g.group <= cache::few::ROWS; }
size_t cache_few_workspace(const cache::Geom& g) { return cache::few::workspace_bytes(g.d); }
cudaError_t launch_cache_few(const cache::FwdParams& p, void* ws, cudaStream_t st) {
  return p.g.d == 128 ? cache::few::launch<128>(p, ws, st) : cache::few::launch<64>(p, ws, st);
}

}  // namespace vattn
