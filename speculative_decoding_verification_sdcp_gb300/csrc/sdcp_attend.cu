// sdcp_attend.cu - sdcp_attend_kv: attention of a round's rows over the paged 4-bit cache.
//
//   out[row][h] = sum_t p_t value_t / sum_t p_t,   p_t = 2^(c q.key_t - m),  c = scale log2(e),
//
// in one pass over the tokens with a running reference m of each (row, head).
//
// All query heads that share a cached head, over all rows of a session, are the columns of one
// product with that head's tokens, so the cache is read once for them (M_b + 1 rows of 8 heads are
// 72 columns at M_b = 8).  A tile is 128 tokens, and the tokens are the rows of both products on the
// tensor cores (tcgen05, M = 128):
//   S[t][j] = key_t . q_j        A = keys, from tensor memory; B = queries, from shared memory
//   O[d][j] += v_t[d] p_t[j]     A = values, B = weights, both from shared memory
// so the cost grows with the columns that are there (a multiple of 16), not with a padded 128.
//
// A thread owns one token of a tile: it reads the token's codes (16 bytes a group, coalesced over
// the tokens by the cache's layout) and turns them into numbers n s in its registers.  n and s have
// four significant bits each, so n s is exact in bfloat16 and, for scales up to 60, in binary16, and
// one fused multiply-add gives it: with the code as the low bits of a constant 128 + 8 + n (bfloat16)
// or 1024 + 8 + n (binary16), the subtrahends 136 s and 1032 s are exact too.  Keys are bfloat16 (as
// the queries are), values and weights binary16: a weight keeps 11 bits.
//
// The reference m only has to keep the weights in range: weights are 2^7 at m, and m moves only
// when a weight would pass 2^15 (binary16 ends below 2^16), which after a head's first tile is rare.
// The weights of a tile are therefore computed at once with the m at hand; a block-wide vote, taken
// at the barrier that the tile needs anyway, sends it through the slow path that finds the tile's
// column maxima, rescales O and repeats the weights.  The sum of weights is of the rounded ones, in
// binary32, a partial sum per thread and column.
//
// Work: the tiles of all (session, cached head, block of columns) items in one line, cut evenly
// over the CTAs (two an SM), whatever the lengths.  A CTA's first and last items may be parts; their
// O, m and sum go to the workspace, and a second kernel joins them in the order of the line.
#include <climits>
#include <math.h>
#include <mutex>

#include "sdcp_kv.cuh"

namespace sdcp {
namespace {

constexpr int kThreads2 = 256;    // two groups of 128: keys and values; half of the columns each
constexpr int kTile = 128;        // tokens of a tile
constexpr int kCols = 96;         // columns of an item
constexpr int kColsHalf = kCols / 2;
constexpr int kMaxCtas = 320;     // CTAs a launch has at most (sizes the workspace)
constexpr int kTmemCols = 256;    // tensor memory of a CTA: keys 0..63, S from 64, O from 160
constexpr uint32_t kTmemS = 64, kTmemO = 160;
constexpr float kLift = 7.0f;     // a weight is 2^kLift at its reference
constexpr float kTop = 15.0f;     // and 2^kTop at most

// How a session's work is cut: kv heads x `chunks` items of at most `w` columns, `tiles` units each:
// the most tiles any chunk needs (its own may be fewer), after kItemUnits for the item itself.
struct SessionPlan {
  int32_t w, chunks, tiles;
};
constexpr int32_t kItemUnits = 2;  // what an item's start and end cost, in tiles

struct AttendArgs {
  KvView kv;
  KvSessions s;
  const __nv_bfloat16* q;
  int64_t q_stride;
  int32_t q_heads;
  float c;
  __nv_bfloat16* out;
  int32_t* status;
  uint32_t* error;   // non-zero: a bounded wait gave up
  int64_t* units;    // [B] units of a session: kv heads x chunks x tiles; 0 for a refused one
  SessionPlan* plans;  // [B]
  int64_t* prefix;   // [B+1]
  float* parts;      // [kMaxCtas * 2] of Part<D>
  int32_t ctas;
};

template <int D> struct Part {
  float o[kCols][D];
  float m[kCols];
  float l[kCols];
};

__device__ __forceinline__ SessionPlan session_plan(int32_t len, int32_t rows, int32_t share, int32_t window) {
  SessionPlan p;
  const int64_t cols = (int64_t)rows * share;
  p.chunks = (int32_t)((cols + kCols - 1) / kCols);
  const int64_t even = (cols + p.chunks - 1) / p.chunks;
  p.w = (int32_t)((even + 15) / 16 * 16);
  p.chunks = (int32_t)((cols + p.w - 1) / p.w);
  int64_t span = (int64_t)len + rows;
  if (window > 0) span = min(span, (int64_t)window - 1 + (p.w + share - 2) / share + 1 + 31);
  p.tiles = (int32_t)((span + kTile - 1) / kTile) + kItemUnits;
  return p;
}
// a / b where both are rarely beyond 32 bits
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line of tiles over the CTAs: CTA k has [first(k), first(k + 1)).
struct Line {
  int64_t total, each, more;
  int32_t ctas;
  __device__ __forceinline__ Line(int64_t t, int32_t most) {
    total = t;
    ctas = (int32_t)min((int64_t)most, max(t, (int64_t)1));
    each = quotient(t, ctas);
    more = t - each * ctas;
  }
  __device__ __forceinline__ int64_t first(int32_t k) const { return k * each + min((int64_t)k, more); }
  __device__ __forceinline__ int32_t cta_of(int64_t t) const {
    const int64_t big = more * (each + 1);
    return t < big ? (int32_t)quotient(t, each + 1) : (int32_t)(more + quotient(t - big, each));
  }
};

// ---- tensor core and tensor memory primitives (PTX ISA, tcgen05) -------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* at, int cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(at)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
               "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const float (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "f"(r[0]), "f"(r[1]), "f"(r[2]),
               "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t at, float (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "r"(at)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
               "l"(b), "r"(idesc), "r"((uint32_t)add)
               : "memory");
}
__device__ __forceinline__ void mma_smem_a(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
               "l"(b), "r"(idesc), "r"((uint32_t)add)
               : "memory");
}
// A shared-memory matrix of 128-byte swizzled atoms (8 rows of 128 bytes).  lead: bytes between
// atoms along the contiguous dimension (used where that is not the product's inner one); step:
// bytes between atoms along the other.
__device__ __forceinline__ uint64_t smem_matrix(const void* p, uint32_t lead, uint32_t step) {
  return (uint64_t)((smem_u32(p) & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(step >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
constexpr uint32_t kIdescF32 = 1u << 4, kIdescBf16 = 1u << 7 | 1u << 10, kIdescTransposeBoth = 1u << 15 | 1u << 16, kIdescM128 = 8u << 24;

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// sum += the low and the high half of w (binary16), each in binary32
__device__ __forceinline__ void add_halves(uint32_t w, float& lo, float& hi) {
  asm("{ .reg .f16 a, b; mov.b32 {a, b}, %2; add.f32.f16 %0, a, %0; add.f32.f16 %1, b, %1; }" : "+f"(lo), "+f"(hi) : "r"(w));
}
// Largest of a warp's values, NaN left out.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sums of eight values over a warp: each exchange halves the values a lane carries, and lanes
// 0..7 end with the sum of value `lane`.
__device__ __forceinline__ float warp_sum8(const float* x, int lane) {
  float y[4], z[2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float keep = (lane & 4) ? x[k + 4] : x[k], give = (lane & 4) ? x[k] : x[k + 4];
    y[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 4);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float keep = (lane & 2) ? y[k + 2] : y[k], give = (lane & 2) ? y[k] : y[k + 2];
    z[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 2);
  }
  const float keep = (lane & 1) ? z[1] : z[0], give = (lane & 1) ? z[0] : z[1];
  float s = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 1);
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
  return s;
}

// Byte g of w in both halves of a word.
__device__ __forceinline__ uint32_t twice(uint32_t w, int g) { return __byte_perm(w, 0u, 0x4040u + 0x0101u * g); }

// A word of eight codes as pairs of numbers n s.  bfloat16: the four bits in the low end of
// 128 + 8 + n; the pairs of a word lie four bits apart.
__device__ __forceinline__ void word_bf16(uint32_t w, uint32_t s, uint32_t c, uint32_t* r) {
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = fma_bf16x2(((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u, s, c);
}
// binary16: 1024 + 8 + n in the low four bits, or 1024 + 16 (8 + n) in the next four, with s / 16.
__device__ __forceinline__ void word_f16(uint32_t w, uint32_t s, uint32_t c, uint32_t s16, uint32_t c16, uint32_t* r) {
  const uint32_t h = w >> 8;
  r[0] = fma_f16x2((w & 0x000F000Fu) | 0x64006400u, s, c);
  r[1] = fma_f16x2((w & 0x00F000F0u) | 0x64006400u, s16, c16);
  r[2] = fma_f16x2((h & 0x000F000Fu) | 0x64006400u, s, c);
  r[3] = fma_f16x2((h & 0x00F000F0u) | 0x64006400u, s16, c16);
}

template <int D> struct AttendSmem {
  static constexpr int kAtoms = D / 64;                 // 128-byte atoms along the channels
  static constexpr int kQ = kAtoms * kCols * 128;       // queries: [atom][column][128 bytes]
  static constexpr int kV = kAtoms * kTile * 128;       // values: [atom][token][128 bytes]
  static constexpr int kP = 2 * kTile * 128;            // weights: [atom of 64 columns][token][128 bytes]
  static constexpr size_t kBytes = (size_t)kQ + kV + kP + 1024;  // and the alignment to 1024
};

// ---- plan: statuses and tiles of the sessions ---------------------------------------------
__global__ void __launch_bounds__(kCheckThreads) attend_plan_kernel(const AttendArgs a) {
  let_next_start();
  const int32_t b = (int32_t)blockIdx.x;
  const int32_t st = kv_session_status(a.kv, a.s, b);
  if (threadIdx.x == 0) {
    a.status[b] = st;
    int64_t units = 0;
    if (st == SDCP_S_OK) {
      const SessionPlan p = session_plan(a.s.start[b], a.s.offsets[b + 1] - a.s.offsets[b] + 1, a.q_heads / a.kv.heads, a.s.window);
      units = (int64_t)p.chunks * p.tiles * a.kv.heads;
      a.plans[b] = p;
    }
    a.units[b] = units;
    if (b == 0) *a.error = 0u;
  }
}

// ---- the products -------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads2, 2) attend_kernel(const AttendArgs a) {
  using Sm = AttendSmem<D>;
  constexpr int kGroups = D / kKvGroup;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* const s_q = sm;
  unsigned char* const s_v = sm + Sm::kQ;
  unsigned char* const s_p = s_v + Sm::kV;
  __shared__ __align__(16) float s_nm[kCols];    // kLift - m: what a scaled score is shifted by
  __shared__ __align__(16) float s_f[kCols];     // factors of a rescale
  __shared__ __align__(16) int32_t s_last[kCols];  // last position of a column
  __shared__ int32_t s_row[kCols], s_at[kCols];    // a column's row, and its place among the output's heads
  __shared__ float s_red[4][kCols];
  __shared__ uint64_t s_bar_s, s_bar_o;
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead;
  __shared__ long long s_scan[kThreads2 / 32];
  __shared__ long long s_total, s_base;
  __shared__ int32_t s_session;

  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wg = tid >> 7, tok = tid & 127;
  const int32_t cta = (int32_t)blockIdx.x;
  wait_for_previous();

  // this CTA's part of the line: a prefix sum over the sessions, a stretch of them per thread
  {
    const int32_t per = (a.s.B + kThreads2 - 1) / kThreads2;
    const int32_t b0 = min(tid * per, a.s.B), b1 = min(b0 + per, a.s.B);
    long long mine = 0;
    for (int32_t b = b0; b < b1; ++b) mine += a.units[b];
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_scan[warp] = incl;
    if (tid == 0) s_dead = 0;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads2 / 32; ++w) {
      if (w < warp) before += s_scan[w];
      all += s_scan[w];
    }
    const long long start = before + incl - mine;
    const Line line(all, a.ctas);
    if (cta == 0) {
      long long at = start;
      for (int32_t b = b0; b < b1; ++b) {
        a.prefix[b] = at;
        at += a.units[b];
      }
      if (tid == 0) a.prefix[a.s.B] = all;
    }
    if (tid == 0) s_total = all;
    if (cta >= line.ctas || all == 0) return;
    const int64_t mine0 = line.first(cta);
    if (mine0 >= start && mine0 < start + mine) {
      long long at = start;
      int32_t b = b0;
      while (mine0 >= at + a.units[b]) at += a.units[b++];
      s_session = b;
      s_base = at;
    }
  }
  if (warp == 0) tmem_alloc(&s_tmem, kTmemCols);
  if (tid == 0) {
    mbar_init(&s_bar_s, 1);
    mbar_init(&s_bar_o, 1);
    fence_barrier_init();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t my_lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes of tensor memory, in bits 16 up
  const Line line(s_total, a.ctas);
  int64_t t = line.first(cta);
  const int64_t t_end = line.first(cta + 1);
  int32_t b = s_session;
  int64_t base = s_base;
  const int32_t share = a.q_heads / a.kv.heads;
  const uint32_t win = a.s.window > 0 ? (uint32_t)a.s.window : 0x80000000u;
  uint32_t ph_s = 0, ph_o = 0;  // phases of the two barriers
  bool dead = false;

  // where the line enters its first item; from there on it walks
  SessionPlan pl = a.plans[b];
  int64_t item = quotient(t - base, pl.tiles);
  int32_t unit0 = (int32_t)(t - base - item * pl.tiles);
  int32_t kvh = (int32_t)quotient(item, pl.chunks), chunk = (int32_t)(item - (int64_t)kvh * pl.chunks);
  int32_t off = a.s.offsets[b], rows = a.s.offsets[b + 1] - off + 1, len = a.s.start[b];

  while (t < t_end && !dead) {
    if (kvh == a.kv.heads) {  // the next session that has work
      do ++b;
      while (a.units[b] == 0);
      pl = a.plans[b];
      off = a.s.offsets[b], rows = a.s.offsets[b + 1] - off + 1, len = a.s.start[b];
      kvh = 0;
    }
    const int32_t units = (int32_t)min((int64_t)(pl.tiles - unit0), t_end - t);  // of this item, here
    const bool whole = units == pl.tiles;
    const int32_t slot = cta * 2 + (t == line.first(cta) ? 0 : 1);
    const int64_t c0 = (int64_t)chunk * pl.w;
    const int32_t n = (int32_t)min((int64_t)pl.w, (int64_t)rows * share - c0);
    const int32_t n16 = (n + 15) / 16;      // blocks of 16 columns; a group of threads has eight of each
    const int32_t i0 = (int32_t)quotient(c0, share), g0 = (int32_t)(c0 - (int64_t)i0 * share);
    const int32_t i1 = i0 + (g0 + n - 1) / share;
    const uint32_t end = (uint32_t)(len + i1) + 1u;  // one past the last position any column sees
    const uint32_t lowest = a.s.window > 0 ? (uint32_t)max((int64_t)0, (int64_t)len + i0 + 1 - a.s.window) : 0u;
    const uint32_t begin = lowest & ~31u;            // the first tile's start; tokens below `lowest` are not read
    const int32_t real = (int32_t)((end - begin + kTile - 1) / kTile);  // tiles that hold something
    const int32_t k0 = max(unit0 - kItemUnits, 0), k1 = min(max(unit0 + units - kItemUnits, 0), real);
    const int64_t row0 = (int64_t)off + b;
    const int32_t head_now = kvh;
    t += units;
    unit0 = 0;
    if (++chunk == pl.chunks) {
      chunk = 0;
      ++kvh;
    }

    // queries of the columns, zero past them, and the columns' state
    __syncthreads();
    if (tid < kCols) {
      const int32_t r = (g0 + tid) / share;
      s_row[tid] = r;
      s_at[tid] = r * a.q_heads + g0 + tid - r * share;
      s_nm[tid] = tid < n ? INFINITY : kLift;
      s_last[tid] = tid < n ? len + i0 + r : INT_MAX;
    }
    __syncthreads();
    const __nv_bfloat16* const q0 = a.q + (row0 + i0) * a.q_stride + (int64_t)head_now * share * D;
    for (int k = tid; k < n16 * 16 * (D / 8); k += kThreads2) {
      const int j = k / (D / 8), ch = k % (D / 8);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (j < n) v = *reinterpret_cast<const uint4*>(q0 + s_row[j] * a.q_stride + (s_at[j] - s_row[j] * a.q_heads) * D + ch * 8);
      *reinterpret_cast<uint4*>(s_q + (ch / 8) * (kCols * 128) + j * 128 + (((ch & 7) ^ (j & 7)) << 4)) = v;
    }
    fence_async_smem();
    float l[kColsHalf];
#pragma unroll
    for (int j = 0; j < kColsHalf; ++j) l[j] = 0.0f;
    const uint32_t idesc_n = (uint32_t)(n16 * 16 / 8) << 17;
    const uint8_t* const head = a.kv.pages + ((int64_t)head_now * 2 + wg) * a.kv.block;
    const int32_t* const table = a.kv.page_table + (int64_t)b * a.kv.max_pages;

    // a tile ahead: the page of the next token, and its codes
    uint4 code[kGroups];
    uint32_t scales = 0;
    int32_t next_page = 0;
    const uint32_t group_bytes = 16u << a.kv.log_page, slot_mask = (1u << a.kv.log_page) - 1u;
    auto find_page = [&](int32_t k) {
      const uint32_t pos = begin + (uint32_t)k * kTile + (uint32_t)tok;
      if (k < k1 && pos >= lowest && pos < end) next_page = table[pos >> a.kv.log_page];
    };
    auto fetch = [&](int32_t k) {
      const uint32_t pos = begin + (uint32_t)k * kTile + (uint32_t)tok;
      scales = 0u;  // a token that is not read becomes finite numbers, whose weight is zero
      if (k < k1 && pos >= lowest && pos < end) {
        const uint32_t slot_in = pos & slot_mask;
        const uint8_t* blk = head + (int64_t)next_page * a.kv.page;
        const uint8_t* at = blk + slot_in * 16u;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          code[g] = *reinterpret_cast<const uint4*>(at);
          at += group_bytes;
        }
        blk += (D / 2 << a.kv.log_page) + slot_in * (D / kKvGroup);
        if (D == 128) scales = *reinterpret_cast<const uint32_t*>(blk);
        else scales = *reinterpret_cast<const uint16_t*>(blk);
      }
    };
#pragma unroll
    for (int g = 0; g < kGroups; ++g) code[g] = make_uint4(0u, 0u, 0u, 0u);
    find_page(k0);
    fetch(k0);
    find_page(k0 + 1);
    __syncthreads();

    for (int32_t k = k0; k < k1; ++k) {
      const bool first = k == k0;
      const uint32_t lo = begin + (uint32_t)k * kTile, pos = lo + (uint32_t)tok;
      // keys to tensor memory, then S; values to shared memory (once the previous O product has read it)
      if (wg == 0) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const uint32_t s = twice(scales, g) * 16u + (kScaleBias << 4) * 0x10001u;
          const uint32_t c = fma_bf16x2(s, 0xC308C308u, 0u);  // -136 s
          uint32_t r[16];
          word_bf16(code[g].x, s, c, r);
          word_bf16(code[g].y, s, c, r + 4);
          word_bf16(code[g].z, s, c, r + 8);
          word_bf16(code[g].w, s, c, r + 12);
          tmem_st16(tmem + my_lanes + g * 16, r);
        }
        tmem_wait_st();
        fence_before();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (tid == 0) {
          fence_after();
          const uint64_t bq = smem_matrix(s_q, 0, 1024);
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            mma_tmem_a(tmem + kTmemS, tmem + x * 8, bq + (uint64_t)(((x / 4) * (kCols * 128) + (x % 4) * 32) >> 4),
                       kIdescF32 | kIdescBf16 | kIdescM128 | idesc_n, x > 0);
          mma_commit(&s_bar_s);
        }
      }
      if (!first) {
        dead |= !mbar_wait_for(&s_bar_o, ph_o, nullptr);
        ph_o ^= 1u;
      }
      if (wg == 1) {
        unsigned char* const dst = s_v + tok * 128;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const uint32_t s = twice(scales, g) << 7;
          const uint32_t s16 = fma_f16x2(s, 0x2C002C00u, 0u);                                   // s / 16
          const uint32_t c = fma_f16x2(s, 0xE408E408u, 0u), c16 = fma_f16x2(s, 0xD480D480u, 0u);  // -1032 s, -72 s
          const uint32_t w[4] = {code[g].x, code[g].y, code[g].z, code[g].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t r[4];
            word_f16(w[x], s, c, s16, c16, r);
            const int ch = (g & 1) * 4 + x;
            *reinterpret_cast<uint4*>(dst + (g >> 1) * (kTile * 128) + ((ch ^ (tok & 7)) << 4)) = make_uint4(r[0], r[1], r[2], r[3]);
          }
        }
      }
      fetch(k + 1);
      find_page(k + 2);

      // weights of this group's columns with the references at hand
      dead |= !mbar_wait_for(&s_bar_s, ph_s, nullptr);
      ph_s ^= 1u;
      fence_after();
      const bool masked = lo + kTile - 1 > (uint32_t)(len + i0) || (uint32_t)(len + i1) - lo >= win;
      uint32_t w16[kColsHalf / 2];
      float top = -INFINITY;
      unsigned char* const dst_p = s_p + tok * 128;
      const int place = (wg ^ (tok & 7)) << 4;  // of a block of eight columns in its 128 bytes: block 2 cb + wg
      auto weights = [&](int cb, bool judge) {
        const int j0 = cb * 16 + wg * 8;
        float x[8];
        tmem_ld8(tmem + my_lanes + kTmemS + j0, x);
        const float4 n0 = *reinterpret_cast<const float4*>(&s_nm[j0]), n1 = *reinterpret_cast<const float4*>(&s_nm[j0 + 4]);
        const float nm[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], a.c, nm[j]);
        if (masked) {
          const int4 e0 = *reinterpret_cast<const int4*>(&s_last[j0]), e1 = *reinterpret_cast<const int4*>(&s_last[j0 + 4]);
          const int32_t last[8] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if ((uint32_t)last[j] - pos >= win) x[j] = -INFINITY;
        }
        if (judge) {
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, x[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) w16[cb * 4 + j] = pack_f16x2(ex2(x[2 * j]), ex2(x[2 * j + 1]));
        *reinterpret_cast<uint4*>(dst_p + (cb >> 2) * (kTile * 128) + (place ^ ((2 * cb & 7) << 4))) =
            make_uint4(w16[cb * 4], w16[cb * 4 + 1], w16[cb * 4 + 2], w16[cb * 4 + 3]);
      };
      if (!first) {  // no reference yet on the first one
#pragma unroll
        for (int cb = 0; cb < kColsHalf / 8; ++cb)
          if (cb < n16) weights(cb, true);
      }
      if (dead) s_dead = 1;
      fence_async_smem();
      fence_before();
      if (__syncthreads_or(top > kTop || first)) {
        // slow path: the columns' maxima over the tile, new references, O and the sums rescaled
        fence_after();
        for (int cb = 0; cb < n16; ++cb) {
          const int j0 = cb * 16 + wg * 8;
          float x[8];
          tmem_ld8(tmem + my_lanes + kTmemS + j0, x);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = masked && (uint32_t)s_last[j0 + j] - pos >= win ? -INFINITY : x[j] * a.c;
            const float m = warp_max(y);
            if (lane == 0) s_red[warp & 3][j0 + j] = m;
          }
        }
        __syncthreads();
        if (tid < n) {
          const float m = fmaxf(fmaxf(s_red[0][tid], s_red[1][tid]), fmaxf(s_red[2][tid], s_red[3][tid]));
          const float nm0 = s_nm[tid], nm1 = fminf(nm0, kLift - m);
          s_nm[tid] = nm1;
          s_f[tid] = nm0 == nm1 ? 1.0f : ex2(nm1 - nm0);
        } else if (tid < kCols) {
          s_f[tid] = 1.0f;
        }
        __syncthreads();
#pragma unroll
        for (int cb = 0; cb < kColsHalf / 8; ++cb)
          if (cb < n16) {
            const int j0 = cb * 16 + wg * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) l[cb * 8 + j] *= s_f[j0 + j];
            if (!first) {
              float o[8];
              tmem_ld8(tmem + my_lanes + kTmemO + j0, o);
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] *= s_f[j0 + j];
              tmem_st8(tmem + my_lanes + kTmemO + j0, o);
            }
            weights(cb, false);
          }
        tmem_wait_st();
        fence_async_smem();
        fence_before();
        __syncthreads();
      }
      dead = s_dead != 0;
      if (dead) break;
      if (tid == 128) {
        fence_after();
        const uint64_t av = smem_matrix(s_v, D == 128 ? kTile * 128 : 0, 1024), bp = smem_matrix(s_p, kTile * 128, 1024);
#pragma unroll
        for (int x = 0; x < kTile / 16; ++x)
          mma_smem_a(tmem + kTmemO, av + (uint64_t)(x * 2048 >> 4), bp + (uint64_t)(x * 2048 >> 4),
                     kIdescF32 | kIdescTransposeBoth | kIdescM128 | idesc_n, !first || x > 0);
        mma_commit(&s_bar_o);
      }
#pragma unroll
      for (int cb = 0; cb < kColsHalf / 8; ++cb)
        if (cb < n16) {
#pragma unroll
          for (int j = cb * 4; j < cb * 4 + 4; ++j) add_halves(w16[j], l[2 * j], l[2 * j + 1]);
        }
    }
    if (dead) break;

    // O, references and sums of the item's columns
    if (k1 > k0) {
      dead |= !mbar_wait_for(&s_bar_o, ph_o, nullptr);
      ph_o ^= 1u;
      fence_after();
    }
#pragma unroll
    for (int cb = 0; cb < kColsHalf / 8; ++cb)
      if (cb < n16) {
        const float x = warp_sum8(&l[cb * 8], lane);
        if (lane < 8) s_red[warp & 3][cb * 16 + wg * 8 + lane] = x;
      }
    if (dead) s_dead = 1;
    __syncthreads();
    dead = s_dead != 0;
    if (dead) break;
    Part<D>* const part = reinterpret_cast<Part<D>*>(a.parts) + slot;
    if (tid < kCols) {
      const float sum = (s_red[0][tid] + s_red[1][tid]) + (s_red[2][tid] + s_red[3][tid]);
      s_f[tid] = __fdividef(1.0f, sum);
      if (!whole) {
        part->m[tid] = -s_nm[tid];
        part->l[tid] = sum;
      }
    }
    __syncthreads();
    __nv_bfloat16* const out0 = a.out + ((row0 + i0) * a.q_heads + (int64_t)head_now * share) * D + tok;
    for (int cb = 0; cb < n16; ++cb) {
      const int j0 = cb * 16 + wg * 8;
      float o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (k1 > k0) tmem_ld8(tmem + my_lanes + kTmemO + j0, o);
      if (tok < D) {
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 8; ++j) part->o[j0 + j][tok] = o[j];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j0 + j < n) out0[(int64_t)s_at[j0 + j] * D] = __float2bfloat16_rn(o[j] * s_f[j0 + j]);
        }
      }
    }
    fence_before();
  }
  __syncthreads();
  if (s_dead != 0) {
    // a product that never completed: give it the time of one more bounded wait, then report
    (void)mbar_wait_for(&s_bar_s, ph_s, nullptr);
    (void)mbar_wait_for(&s_bar_o, ph_o, nullptr);
    if (tid == 0) atomicOr(a.error, 1u);
    __syncthreads();
  }
  if (warp == 0) tmem_free(tmem, kTmemCols);
}

// ---- the joining of parts -----------------------------------------------------------------
constexpr int kJoinThreads = 256;

// One warp per row and query head: a row of a refused session becomes zero, a row whose item was cut
// is the parts' sum, a row that one CTA wrote is left.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendArgs a, int64_t rows) {
  constexpr int kPer = D / 32;
  const int lane = (int)(threadIdx.x & 31u);
  wait_for_previous();
  const bool failed = *a.error != 0u;
  if (failed)
    for (int64_t b = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; b < a.s.B; b += (int64_t)gridDim.x * kJoinThreads)
      a.status[b] = SDCP_S_INTERNAL;
  const Line line(a.prefix[a.s.B], a.ctas);
  const int32_t share = a.q_heads / a.kv.heads;
  const Part<D>* const parts = reinterpret_cast<const Part<D>*>(a.parts);
  for (int64_t at = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5); at < rows * a.q_heads;
       at += (int64_t)gridDim.x * (kJoinThreads / 32)) {
    const int64_t row = quotient(at, a.q_heads);
    const int32_t h = (int32_t)(at - row * a.q_heads);
    const int32_t b = find_session(a.s.offsets, a.s.B, row, true);
    const int32_t off = a.s.offsets[b], last = a.s.offsets[b + 1] - off;
    const int64_t i = row - off - b;
    __nv_bfloat16* out = a.out + at * D + lane * kPer;
    float o[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[k] = 0.0f;
    if (!failed && a.units[b] > 0 && i >= 0 && i <= last) {
      const SessionPlan pl = a.plans[b];
      const int32_t kvh = h / share;
      const int64_t col = i * share + (h - kvh * share);
      const int64_t part = quotient(col, pl.w);
      const int64_t first = a.prefix[b] + ((int64_t)kvh * pl.chunks + part) * pl.tiles;
      const int32_t j = (int32_t)(col - part * pl.w);
      const int32_t c_lo = line.cta_of(first), c_hi = line.cta_of(first + pl.tiles - 1);
      if (c_lo == c_hi) continue;
      float m = -INFINITY;
      for (int32_t c = c_lo + lane; c <= c_hi; c += 32)
        m = fmaxf(m, parts[c * 2 + (c == c_lo && line.first(c) < first ? 1 : 0)].m[j]);
      m = warp_max(m);
      float sum = 0.0f;
      for (int32_t c = c_lo; c <= c_hi; ++c) {
        const Part<D>& p = parts[c * 2 + (c == c_lo && line.first(c) < first ? 1 : 0)];
        const float pm = p.m[j];
        if (pm == -INFINITY && p.l[j] == 0.0f) continue;  // nothing of the column in this part
        const float f = pm == m ? 1.0f : ex2(pm - m);
        sum += p.l[j] * f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) o[k] += p.o[j][lane * kPer + k] * f;
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) o[k] = __fdividef(o[k], sum);
    }
    const __nv_bfloat162 v0 = __floats2bfloat162_rn(o[0], o[1]);
    *reinterpret_cast<__nv_bfloat162*>(out) = v0;
    if (kPer == 4) *reinterpret_cast<__nv_bfloat162*>(out + 2) = __floats2bfloat162_rn(o[kPer - 2], o[kPer - 1]);
  }
}

constexpr size_t kHeader = 256;
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Once per device: the kernels' dynamic shared memory.
constexpr int kMaxDevices = 64;
struct AttendDevice {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
AttendDevice g_attend_device[kMaxDevices];
bool attend_ready() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  AttendDevice& d = g_attend_device[dev];
  std::call_once(d.once, [&] {
    d.err = cudaFuncSetAttribute(attend_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)AttendSmem<128>::kBytes);
    if (d.err == cudaSuccess)
      d.err = cudaFuncSetAttribute(attend_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)AttendSmem<64>::kBytes);
    if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(attend_kernel<128>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(attend_kernel<64>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  });
  return d.err == cudaSuccess;
}

template <int D>
cudaError_t launch_attend(const AttendArgs& a, int sms, cudaStream_t st) {
  attend_plan_kernel<<<(unsigned)a.s.B, kCheckThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_after(attend_kernel<D>, (unsigned)a.ctas, kThreads2, AttendSmem<D>::kBytes, st, a);
  if (e != cudaSuccess) return e;
  const int64_t rows = a.s.total + a.s.B, warps = rows * a.q_heads;
  const int64_t blocks = min((warps + kJoinThreads / 32 - 1) / (kJoinThreads / 32), (int64_t)sms * 16);
  return launch_after(attend_join_kernel<D>, (unsigned)blocks, kJoinThreads, 0, st, a, rows);
}

}  // namespace
}  // namespace sdcp

using namespace sdcp;

extern "C" size_t sdcp_attend_workspace_bytes(int32_t B, int64_t total_drafts, int32_t q_heads,
                                              int32_t kv_heads, int32_t head_dim) {
  if (B < 0 || total_drafts < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  return kHeader + round256((size_t)B * sizeof(SessionPlan)) + round256(((size_t)B * 2 + 1) * sizeof(int64_t)) +
         (size_t)kMaxCtas * 2 * (head_dim == 128 ? sizeof(Part<128>) : sizeof(Part<64>));
}

extern "C" int sdcp_attend_kv(const sdcp_kv_cache* cache, int32_t B, const int32_t* m_offsets,
                              int64_t total_drafts, const int32_t* kv_len, const void* q,
                              int64_t q_stride, int32_t q_heads, float scale, int32_t window,
                              void* out, int32_t* status, void* workspace, size_t workspace_bytes,
                              void* stream) {
  KvView kv;
  const int rc = kv_view(cache, &kv);
  if (rc != SDCP_OK) return rc;
  const size_t need = sdcp_attend_workspace_bytes(B, total_drafts, q_heads, cache->kv_heads, cache->head_dim);
  if (need == 0 || window < 0 || !isfinite(scale)) return SDCP_E_INVALID;
  if (total_drafts + B > (int64_t)INT32_MAX / 2 || q_heads > (1 << 20)) return SDCP_E_TOO_LARGE;
  if (B == 0) return SDCP_OK;
  const int32_t D = cache->head_dim;
  if (!m_offsets || !kv_len || !q || !out || !status) return SDCP_E_INVALID;
  if (q_stride < (int64_t)q_heads * D) return SDCP_E_INVALID;
  if (((uintptr_t)q & 15u) != 0 || ((uintptr_t)out & 15u) != 0 || q_stride % 8 != 0) return SDCP_E_ALIGN;
  if (!workspace || ((uintptr_t)workspace & 255u) != 0 || workspace_bytes < need) return SDCP_E_WORKSPACE;
  DeviceInfo di;
  if (!device_info(&di) || !attend_ready()) return SDCP_E_DEVICE;
  char* w = static_cast<char*>(workspace);
  char* const plans = w + kHeader;
  char* const lines = plans + round256((size_t)B * sizeof(SessionPlan));
  int64_t* const units = reinterpret_cast<int64_t*>(lines);
  const KvSessions s{B, m_offsets, total_drafts, 1, kv_len, window, INT32_MAX};
  const AttendArgs a{kv, s, static_cast<const __nv_bfloat16*>(q), q_stride, q_heads, scale * 1.4426950408889634f,
                     static_cast<__nv_bfloat16*>(out), status, reinterpret_cast<uint32_t*>(w), units,
                     reinterpret_cast<SessionPlan*>(plans), units + B,
                     reinterpret_cast<float*>(lines + round256(((size_t)B * 2 + 1) * sizeof(int64_t))),
                     min(2 * di.sms, kMaxCtas)};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 128 ? launch_attend<128>(a, di.sms, st) : launch_attend<64>(a, di.sms, st);
  return e == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}
