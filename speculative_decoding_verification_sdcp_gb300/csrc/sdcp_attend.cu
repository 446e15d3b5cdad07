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
// the queries are), values and weights binary16: a weight keeps 11 bits (bfloat16 would keep 8, the matrix
// instruction's 32-bit type 11 as well at half the rate), which is little beside the output's own rounding
// to bfloat16 (relative error against 64 bits 0.0017, 0.0017 with weights of 32 bits).
// Exponentials are the hardware's (2 units in the last place of binary32), and so is the last division.
//
// The reference m only has to keep the weights in range: weights are 2^7 at m, and m moves only
// when a weight would pass 2^15 (binary16 ends below 2^16), which after an item's first tile is rare.
// The weights of a tile are therefore computed at once with the m at hand; a vote of the threads that
// compute them sends the tile through the slow path that finds its column maxima, rescales O and
// repeats the weights.  The sum of weights is of the rounded ones, in binary32, a partial sum per
// thread and column.
//
// What bounds it is the instructions of the turning and of the weights and their latencies, so
// several CTAs share an SM, and within one the products run beside the other work: eight warps all
// follow the same steps of a tile (turn half of the keys' channels each, then half of the values',
// then weigh half of the columns each), and a ninth issues S as soon as the keys are there, behind
// which the values are turned, and O behind the next tile's keys.  Loads are one tile ahead.  Roles
// in warps of their own (keys, values, weights; one CTA an SM, two tiles deep) were slower (203 us
// for the 20 columns below against 182 when the same eight warps did everything): several kinds of
// instruction streams on a scheduler starve one another.
//
// Measured (128 channels, 8 cached heads): 4 contexts of about 105000 tokens, 5 rows, 32 heads: 161 us,
// 454 MB of cache at 2.8 TB/s; 64 contexts of 500 .. 8200, 9 rows, 64 heads: 181 us, 60 % of the issue
// slots and a quarter of the tensor cores' cycles used.  The time of a
// tile hardly depends on its columns up to 32 (16 contexts of 30000: 166 us at 4 and at 16 columns,
// 182 at 32), so what a tile costs is its turning, its waits and its votes.
//
// Work: the tiles of all (session, cached head, block of columns) items in one line, a tile as
// long as its columns make it, cut evenly over the CTAs.  All blocks of columns of a session count as many
// tiles as its longest: that is even where they see about as many tokens, but of a long round into a
// short context (a prompt) the first blocks see few, and about half of the line is then no work.  A CTA's
// first and last items may be parts; their O, m and sum go to the workspace, and a second kernel joins
// them in the order of the line.
#include <climits>
#include <math.h>
#include <mutex>
#include <type_traits>

#include "sdcp_kv.cuh"

namespace sdcp {
namespace {

constexpr int kComputeThreads = 256;                  // two groups of 128, a token of the tile each
constexpr int kAttendThreads = kComputeThreads + 32;  // and the warp that issues the products
constexpr int kTile = 128;                            // tokens of a tile
constexpr int kMaxSms = 160;                          // sizes the workspace
// Two shapes: at most 32 columns an item and three CTAs an SM, or at most 96 and two.
template <int kColumns> struct Shape {
  static constexpr int kCols = kColumns;
  static constexpr int kHalf = kCols / 2;                   // columns of a thread
  static constexpr int kCtas = kCols == 32 ? 3 : 2;         // of an SM
  static constexpr uint32_t kTmemS = 64, kTmemO = 64 + kCols;  // tensor memory: keys, S, O
  static constexpr int kTmemCols = kCols == 32 ? 128 : 256;
};
constexpr float kLift = 7.0f;     // a weight is 2^kLift at its reference
constexpr float kTop = 15.0f;     // and 2^kTop at most

// How a session's work is cut: kv heads x `chunks` items of at most `w` columns, `tiles` units each:
// the most tiles any chunk needs (its own may be fewer), after kItemUnits for the item itself.
struct SessionPlan {
  int32_t w, chunks, tiles, cost;  // cost: of a unit, on the line
};
// What an item's start and end cost, in tiles (512 items of 72 columns, 4 .. 64 tiles: 189 us with 2,
// 183 with 3, 185 with 4, 189 with 8; with 32 long items any does).
constexpr int32_t kItemUnits = 3;
// What a tile of w columns costs on the line: kTileCost + w / 16 (16 contexts of 30000 tokens, 16 to 96
// columns: 200 to 281 us with 128 channels, 160 to 250 with 64).  Sessions of 14 .. 119 columns over a
// window of 1000: 93 us, 101 with one cost for all.
constexpr int32_t kTileCost = 8;

// The item that a CTA begins and another one goes on with: its parts are the CTA's second (or, where
// it began with it, first) and the first of the CTAs after it, up to `last`.  n = 0: none.
struct Cut {
  int32_t n, first_slot, last;
  int32_t row_head;  // place of column 0 among the heads of the output row of column 0
  int64_t row;       // and that row
  int32_t g0, pad;
};

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
  int64_t* units;    // [B] length of a session on the line: kv heads x chunks x tiles x cost; 0 for a refused one
  SessionPlan* plans;  // [B]
  float* parts;      // [ctas * 2] of Part
  Cut* cuts;         // [ctas]
  int32_t ctas;
  int32_t cols;      // columns an item has at most
  int32_t dim;       // channels of a head
};

template <int D, int kCols> struct Part {
  float o[kCols][D];
  float m[kCols];
  float l[kCols];
};

__device__ __forceinline__ SessionPlan session_plan(int32_t len, int32_t rows, int32_t share, int32_t window, int32_t most) {
  SessionPlan p;
  const int64_t cols = (int64_t)rows * share;
  p.chunks = (int32_t)((cols + most - 1) / most);
  const int64_t even = (cols + p.chunks - 1) / p.chunks;
  p.w = (int32_t)((even + 15) / 16 * 16);
  p.chunks = (int32_t)((cols + p.w - 1) / p.w);
  int64_t span = (int64_t)len + rows;
  if (window > 0) span = min(span, (int64_t)window - 1 + (p.w + share - 2) / share + 1 + 31);
  p.tiles = (int32_t)((span + kTile - 1) / kTile) + kItemUnits;
  p.cost = kTileCost + p.w / 16;
  return p;
}
// a / b where both are rarely beyond 32 bits
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line over the CTAs: CTA k has the units that begin in [first(k), first(k + 1)).
struct Line {
  int64_t total, each, more;
  int32_t ctas;
  __device__ __forceinline__ Line(int64_t t, int32_t most) {
    total = t;
    ctas = (int32_t)min((int64_t)most, max(quotient(t, kTileCost + 1), (int64_t)1));
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
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
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
// Bounded wait for a phase.  Waits here are a few hundred cycles, a tile's step, so it polls a while
// without reading a clock; false after kWaitNs, or when another warp has given up.
__device__ __forceinline__ bool poll_phase(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p, q; .reg .u32 n;\n"
      "mov.u32 n, 0;\n"
      "POLL:\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "@p bra DONE;\n"
      "add.u32 n, n, 1;\n"
      "setp.lt.u32 q, n, 4096;\n"
      "@q bra POLL;\n"
      "DONE:\n"
      "selp.u32 %0, 1, 0, p; }"
      : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, const volatile int* dead) {
  if (mbar_try_wait(bar, parity) || poll_phase(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!poll_phase(bar, parity))
    if ((dead != nullptr && *dead) || global_ns() - t0 > kWaitNs) return false;
  return true;
}
// A shared-memory matrix of swizzled atoms (8 rows of 128 or 64 bytes).  lead: bytes between atoms
// along the contiguous dimension (used where that is not the product's inner one); step: bytes
// between atoms along the other.
constexpr uint64_t kSwizzle128 = (uint64_t)2 << 61, kSwizzle64 = (uint64_t)4 << 61;
__device__ __forceinline__ uint64_t smem_matrix(const void* p, uint32_t lead, uint32_t step, uint64_t swizzle) {
  return (uint64_t)((smem_u32(p) & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(step >> 4) << 32 | (uint64_t)1 << 46 |
         swizzle;
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
// (beyond the range: its end, so that what the slow path takes back is finite)
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
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

// Eight values folded over a warp: each exchange halves the values a lane carries, and lanes 0..7 end
// with value `lane` of all lanes.
template <typename F>
__device__ __forceinline__ float warp_fold8(const float* x, int lane, F op) {
  float y[4], z[2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float keep = (lane & 4) ? x[k + 4] : x[k], give = (lane & 4) ? x[k] : x[k + 4];
    y[k] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 4));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float keep = (lane & 2) ? y[k + 2] : y[k], give = (lane & 2) ? y[k] : y[k + 2];
    z[k] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 2));
  }
  const float keep = (lane & 1) ? z[1] : z[0], give = (lane & 1) ? z[0] : z[1];
  float s = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 1));
  s = op(s, __shfl_xor_sync(0xFFFFFFFFu, s, 8));
  return op(s, __shfl_xor_sync(0xFFFFFFFFu, s, 16));
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared4(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async16_or_zero(uint32_t dst, const void* src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Byte g of w in both halves of a word.
__device__ __forceinline__ uint32_t twice(uint32_t w, int g) { return __byte_perm(w, 0u, 0x4040u + 0x0101u * g); }

// (a & kMask) | c in one instruction; c is a constant that the compiler is kept from loading anew at
// each use (kept(), once).
template <uint32_t kMask> __device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "n"(kMask), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t kept(uint32_t x) {
  uint32_t y;
  asm volatile("mov.b32 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A word of eight codes as pairs of numbers n s.  bfloat16: the four bits in the low end of
// 128 + 8 + n (one: 128 twice); the pairs of a word lie four bits apart.
__device__ __forceinline__ void word_bf16(uint32_t w, uint32_t one, uint32_t s, uint32_t c, uint32_t* r) {
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = fma_bf16x2(and_or<0x000F000Fu>(w >> (4 * j), one), s, c);
}
// binary16: 1024 + 8 + n in the low four bits, or 1024 + 16 (8 + n) in the next four, with s / 16
// (one: 1024 twice).
__device__ __forceinline__ void word_f16(uint32_t w, uint32_t one, uint32_t s, uint32_t c, uint32_t s16, uint32_t c16, uint32_t* r) {
  const uint32_t h = w >> 8;
  r[0] = fma_f16x2(and_or<0x000F000Fu>(w, one), s, c);
  r[1] = fma_f16x2(and_or<0x00F000F0u>(w, one), s16, c16);
  r[2] = fma_f16x2(and_or<0x000F000Fu>(h, one), s, c);
  r[3] = fma_f16x2(and_or<0x00F000F0u>(h, one), s16, c16);
}

template <int D, int kCols> struct AttendSmem {
  static constexpr int kAtoms = D / 64;                        // 128-byte atoms along the channels
  static constexpr int kQ = kAtoms * kCols * 128;              // queries: [atom][column][128 bytes]
  static constexpr int kV = kAtoms * kTile * 128;              // values: [atom][token][128 bytes]
  static constexpr bool kNarrow = kCols == 32;                 // weights: [token][64 bytes], swizzled in 64 bytes,
  static constexpr int kP = kNarrow ? kTile * 64 : (kCols + 63) / 64 * kTile * 128;  // or [atom of 64 columns][token][128 bytes]
  static constexpr int kC = 2 * kTile * (D / 2 + 8);           // codes and scales of the next keys and values
  static constexpr size_t kBytes = (size_t)kQ + kV + kP + kC + 1024;  // and the alignment to 1024
};

// One step of a CTA's way along the line: an item, or the part of it that is the CTA's.
struct Item {
  int32_t b, off, len, kvh;
  int32_t n, i0, g0;            // columns, and the row and head of the first
  uint32_t lowest, begin, end;  // positions: first read, first of tile 0, one past the last
  int32_t k0, k1;               // tiles
  int32_t slot;                 // of the parts
  int32_t whole;                // all of the item's tiles are here
};
// The way itself, walked by the ninth warp, an item ahead: the divisions stay out of the other
// warps' registers and off their way.
struct Walk {
  int64_t t, t_end, t_first;
  SessionPlan pl;
  int32_t b, off, rows, len, kvh, chunk, unit0;
  __device__ __forceinline__ void load(const AttendArgs& a) {
    pl = a.plans[b];
    off = a.s.offsets[b];
    rows = a.s.offsets[b + 1] - off + 1;
    len = a.s.start[b];
  }
  __device__ __forceinline__ void begin(const AttendArgs& a, const Line& line, int32_t session, int64_t base) {
    t_end = line.first((int32_t)blockIdx.x + 1);
    b = session;
    load(a);
    int64_t unit = quotient(line.first((int32_t)blockIdx.x) - base + pl.cost - 1, pl.cost);
    if (unit * pl.cost >= a.units[b]) {  // the CTA begins with the next session, if there is one
      base += a.units[b];
      unit = 0;
      if (base < t_end) {
        do ++b;
        while (a.units[b] == 0);
        load(a);
      }
    }
    t = t_first = base + unit * pl.cost;
    const int64_t item = quotient(unit, pl.tiles);
    unit0 = (int32_t)(unit - item * pl.tiles);
    kvh = (int32_t)quotient(item, pl.chunks);
    chunk = (int32_t)(item - (int64_t)kvh * pl.chunks);
  }
  // the next item; false at the end of the CTA's part
  __device__ __forceinline__ bool next(const AttendArgs& a, const Line& line, Item& it) {
    if (t >= t_end) return false;
    if (kvh == a.kv.heads) {  // the next session that has work
      do ++b;
      while (a.units[b] == 0);
      load(a);
      kvh = 0;
    }
    const int32_t share = a.q_heads / a.kv.heads;
    const int32_t units = (int32_t)min((int64_t)(pl.tiles - unit0), quotient(t_end - t + pl.cost - 1, pl.cost));
    const int64_t c0 = (int64_t)chunk * pl.w;
    it.b = b, it.off = off, it.len = len, it.kvh = kvh;
    it.n = (int32_t)min((int64_t)pl.w, (int64_t)rows * share - c0);
    it.i0 = (int32_t)quotient(c0, share);
    it.g0 = (int32_t)(c0 - (int64_t)it.i0 * share);
    const int32_t i1 = it.i0 + (it.g0 + it.n - 1) / share;
    it.end = (uint32_t)(len + i1) + 1u;
    it.lowest = a.s.window > 0 ? (uint32_t)max((int64_t)0, (int64_t)len + it.i0 + 1 - a.s.window) : 0u;
    it.begin = it.lowest & ~31u;
    const int32_t real = (int32_t)((it.end - it.begin + kTile - 1) / kTile);
    it.k0 = max(unit0 - kItemUnits, 0);
    it.k1 = min(max(unit0 + units - kItemUnits, 0), real);
    it.slot = (int32_t)blockIdx.x * 2 + (t == t_first ? 0 : 1);
    it.whole = units == pl.tiles;
    if (!it.whole && unit0 == 0)  // the CTA's last item, and others go on with it
      a.cuts[blockIdx.x] = Cut{it.n, it.slot, line.cta_of(t + (int64_t)(pl.tiles - 1) * pl.cost), kvh * share + it.g0, (int64_t)off + b + it.i0, it.g0, 0};
    t += (int64_t)units * pl.cost;
    unit0 = 0;
    if (++chunk == pl.chunks) {
      chunk = 0;
      ++kvh;
    }
    return true;
  }
};
// The barriers and small arrays of a CTA.
template <int kCols> struct AttendShared {
  __align__(16) float nm[kCols];      // kLift - m: what a scaled score is shifted by
  __align__(16) int32_t last[kCols];  // last position of a column
  int32_t at[kCols];                  // a column's place among the output's heads
  __align__(16) float f[kCols];       // factors of a rescale; reciprocal sums
  float red[4][kCols];
  uint64_t k_full, s_full, p_full, pv_done, drained;
  long long scan[kAttendThreads / 32];
  long long base;
  int32_t session;
  uint32_t tmem;
  int dead;
  Walk walk;
  Item item[2];  // item j in item[j & 1]; one without tiles ends them
};

// ---- plan: statuses and tiles of the sessions ---------------------------------------------
__global__ void __launch_bounds__(kCheckThreads) attend_plan_kernel(const AttendArgs a) {
  let_next_start();
  const int32_t b = (int32_t)blockIdx.x;
  const int32_t st = kv_session_status(a.kv, a.s, b, a.status);
  if (st != SDCP_S_OK) {  // its rows become zero (what another session has of them is written later)
    const int64_t lo = min(max((int64_t)a.s.offsets[b], (int64_t)0), a.s.total), hi = min(max((int64_t)a.s.offsets[b + 1], lo), a.s.total);
    const int64_t row = (int64_t)a.q_heads * a.dim / 8;
    uint4* const out = reinterpret_cast<uint4*>(a.out);
    for (int64_t x = (lo + b) * row + threadIdx.x; x < (hi + b + 1) * row; x += kCheckThreads) out[x] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (threadIdx.x == 0) {
    a.status[b] = st;
    int64_t units = 0;
    if (st == SDCP_S_OK) {
      const SessionPlan p = session_plan(a.s.start[b], a.s.offsets[b + 1] - a.s.offsets[b] + 1, a.q_heads / a.kv.heads, a.s.window, a.cols);
      units = (int64_t)p.chunks * p.tiles * a.kv.heads * p.cost;
      a.plans[b] = p;
    }
    a.units[b] = units;
    if (b == 0) *a.error = 0u;
  }
}

// ---- the products -------------------------------------------------------------------------
// The next item that has tiles; a part that holds no tile of its item is marked at once.  One thread.
template <int D, int kCols>
__device__ __forceinline__ void plan_item(const AttendArgs& a, AttendShared<kCols>& sh, const Line& line, uint32_t j) {
  Item it;
  bool more;
  Walk walk = sh.walk;
  auto nothing_in = [&](int32_t slot) {
    Part<D, kCols>* const part = reinterpret_cast<Part<D, kCols>*>(a.parts) + slot;
    for (int x = 0; x < kCols; ++x) {
      part->m[x] = -INFINITY;
      part->l[x] = 0.0f;
    }
  };
  if (j == 0 && walk.t >= walk.t_end) nothing_in((int32_t)blockIdx.x * 2);  // no unit begins here
  while ((more = walk.next(a, line, it)) && it.k0 >= it.k1) nothing_in(it.slot);
  if (!more) it.k0 = it.k1 = 0;
  sh.walk = walk;
  sh.item[j & 1u] = it;
}

// The ninth warp: S of a tile when its keys are in tensor memory, O when its weights are in shared
// memory (the values are there before the weights).  One thread.
template <int D, int kCols>
__device__ __forceinline__ void multiply(const AttendArgs& a, AttendShared<kCols>& sh, const Line& line, const unsigned char* s_q, const unsigned char* s_v,
                                         const unsigned char* s_p, uint32_t tmem) {
  using Sm = AttendSmem<D, kCols>;
  using Sh = Shape<kCols>;
  constexpr uint32_t kPRow = Sm::kNarrow ? 64 : 128;
  const uint64_t q_mat = smem_matrix(s_q, 0, 1024, kSwizzle128),
                 v_mat = smem_matrix(s_v, D == 128 ? kTile * 128 : 0, 1024, kSwizzle128),
                 p_mat = smem_matrix(s_p, kTile * kPRow, 8 * kPRow, Sm::kNarrow ? kSwizzle64 : kSwizzle128);
  uint32_t i = 0;
  for (uint32_t j = 0;; ++j) {
    __syncthreads();  // item j is planned, and the previous one is done with
    if (sh.dead) {    // products under way end before the tensor memory is given back
      if ((threadIdx.x & 31u) == 0) {
        mma_commit(&sh.drained);
        (void)wait_phase(&sh.drained, 0u, nullptr);
        atomicOr(a.error, 1u);
      }
      return;
    }
    const int32_t tiles = sh.item[j & 1u].k1 - sh.item[j & 1u].k0;
    if (tiles <= 0) return;
    const uint32_t idesc = kIdescF32 | kIdescM128 | (uint32_t)((sh.item[j & 1u].n + 15) / 16 * 2) << 17;
    if ((threadIdx.x & 31u) == 0) {
      for (int32_t k = 0; k < tiles; ++k, ++i) {
        const uint32_t par = i & 1u;
        if (!wait_phase(&sh.k_full, par, &sh.dead)) { sh.dead = 1; break; }
        fence_after();
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          mma_tmem_a(tmem + Sh::kTmemS, tmem + (uint32_t)x * 8u, q_mat + (uint64_t)(((x / 4) * (kCols * 128) + (x % 4) * 32) >> 4),
                     idesc | kIdescBf16, x > 0);
        mma_commit(&sh.s_full);
        if (k == 0) plan_item<D, kCols>(a, sh, line, j + 1);
        if (!wait_phase(&sh.p_full, par, &sh.dead)) { sh.dead = 1; break; }
        fence_after();
#pragma unroll
        for (int x = 0; x < kTile / 16; ++x)
          mma_smem_a(tmem + Sh::kTmemO, v_mat + (uint64_t)(x * 2048 >> 4), p_mat + (uint64_t)(x * 16 * kPRow >> 4), idesc | kIdescTransposeBoth,
                     k > 0 || x > 0);
        mma_commit(&sh.pv_done);
      }
    }
    __syncwarp();
  }
}

// The eight warps' steps.
template <int D, int kCols>
__device__ __forceinline__ void attend_tiles(const AttendArgs& a, AttendShared<kCols>& sh, unsigned char* s_q, unsigned char* s_v,
                                             unsigned char* s_p, unsigned char* s_c, uint32_t tmem) {
  using Sm = AttendSmem<D, kCols>;
  using Sh = Shape<kCols>;
  constexpr int kOwn = D / kKvGroup / 2;  // channel groups of a thread
  constexpr int kBlocks = Sh::kHalf / 8;
  const int tid = (int)kept(threadIdx.x), lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int wg = warp >> 2, tok = tid & 127;
  const uint32_t my_lanes = __shfl_sync(0xFFFFFFFFu, tmem + ((uint32_t)(warp & 3) << 21), 0);  // 32 lanes of tensor memory, in bits 16 up
  const uint32_t one_k = kept(0x43004300u), one_v = kept(0x64006400u);
  const uint32_t win = a.s.window > 0 ? (uint32_t)a.s.window : 0x80000000u;
  const int32_t share = a.q_heads / a.kv.heads;
  const uint32_t swizzled = (uint32_t)(tok * 128) + ((uint32_t)(tok & 7) << 4);
  // values: channels (wg * kOwn + g) * 32 of the token; weights: block 2 cb + wg of eight columns
  const uint32_t v_at = smem_u32(s_v) + (D == 128 ? (uint32_t)(wg * kTile * 128) + swizzled : swizzled ^ ((uint32_t)wg << 6));
  const uint32_t p_at =
      smem_u32(s_p) + (Sm::kNarrow ? (uint32_t)(tok * 64) + ((uint32_t)(wg ^ ((tok >> 1) & 3)) << 4) : swizzled ^ ((uint32_t)wg << 4));
  const uint32_t s_at = my_lanes + Sh::kTmemS + (uint32_t)(wg * 8);
  auto meet = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
  auto any = [](bool p) {
    uint32_t r;
    asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.or.pred q, 1, 256, p; selp.u32 %0, 1, 0, q; }" : "=r"(r) : "r"((uint32_t)p) : "memory");
    return r != 0;
  };
  // the thread's codes of the next keys, [group][thread][16 bytes], then [thread][4 bytes] of scales; the values' after them
  constexpr uint32_t kCodes = kComputeThreads * (kOwn * 16 + 4);
  static_assert(2 * kCodes == Sm::kC, "codes");
  const uint32_t c_at = smem_u32(s_c) + (uint32_t)tid * 16u, sb_at = smem_u32(s_c) + kComputeThreads * kOwn * 16 + (uint32_t)tid * 4u;
  const int sb_shift = D == 128 ? wg * 16 : (tok & 1) * 16 + wg * 8;  // of the thread's own scales (tiles start at even tokens)
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(sb_at), "r"(0u) : "memory");
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(sb_at + kCodes), "r"(0u) : "memory");
  uint32_t i = 0;  // tiles so far
  bool dead = false;  // a wait gave up: the eight warps agree on it at a vote, all nine at an item's start
  for (uint32_t j = 0;; ++j) {
    __syncthreads();
    if (sh.dead) {  // copies under way end before the shared memory is given back
      asm volatile("cp.async.wait_all;" ::: "memory");
      return;
    }
    const Item& it = sh.item[j & 1u];
    const int32_t tiles = it.k1 - it.k0;
    if (tiles <= 0) return;
    const int32_t n16 = (it.n + 15) / 16;  // blocks of 16 columns; a group of threads has eight of each

    // queries of the columns, zero past them (the oldest group of copies: they are there with the first
    // keys), and the columns' state
    {
      const __nv_bfloat16* const q0 = a.q + ((int64_t)it.off + it.b + it.i0) * a.q_stride + (int64_t)it.kvh * share * D;
      const int ch = tid % (D / 8);
      const uint32_t dst = smem_u32(s_q) + (uint32_t)(ch / 8) * (kCols * 128);
#pragma unroll 2
      for (int col = tid / (D / 8); col < n16 * 16; col += kComputeThreads / (D / 8)) {
        const int32_t c = min(col, it.n - 1) + it.g0, r = c / share;
        copy_async16_or_zero(dst + (uint32_t)col * 128u + (uint32_t)(((ch & 7) ^ (col & 7)) << 4), q0 + r * a.q_stride + (c - r * share) * D + ch * 8,
                             col < it.n);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    if (tid < kCols) {
      const int32_t r = (it.g0 + tid) / share;
      sh.at[tid] = r * a.q_heads + it.g0 + tid - r * share;
      sh.nm[tid] = tid < it.n ? INFINITY : kLift;
      sh.last[tid] = tid < it.n ? it.len + it.i0 + r : INT_MAX;
    }

    // a tile ahead: the page of the next token, and the copy of the thread's share of its codes to
    // the thread's own places in shared memory (a token that is not read keeps old codes: finite
    // numbers, whose weight is zero)
    const uint32_t lowest = it.lowest, end = it.end;
    uint32_t pos = it.begin + (uint32_t)it.k0 * kTile + (uint32_t)tok;
    const uint32_t in_page = (uint32_t)it.kvh * 2u * (uint32_t)a.kv.block;  // the head's keys
    const int32_t* const table = a.kv.page_table + (int64_t)it.b * a.kv.max_pages;
    auto page_of = [&](uint32_t p, bool some) { return some && p >= lowest && p < end ? table[p >> a.kv.log_page] : -1; };
    auto fetch = [&](int which, uint32_t p, int32_t page) {  // of the token at p, whose page is known (-1: nothing to read)
      if (page >= 0) {
        const uint32_t slot = p & ((1u << a.kv.log_page) - 1u);
        const uint8_t* const blk = a.kv.pages + (uint64_t)(uint32_t)page * (uint32_t)a.kv.page + (in_page + (which ? (uint32_t)a.kv.block : 0u));
        const uint32_t o = (((uint32_t)(wg * kOwn) << a.kv.log_page) + slot) * 16u;
        copy_async16(c_at + (uint32_t)which * kCodes, blk + o);
        if (kOwn == 2) copy_async16(c_at + (uint32_t)which * kCodes + kComputeThreads * 16, blk + (o + (16u << a.kv.log_page)));
        // four scale bytes of a token, or two each of a pair of tokens
        copy_async4(sb_at + (uint32_t)which * kCodes, blk + ((D / 2u << a.kv.log_page) + (D == 128 ? slot * 4u : (slot & ~1u) * 2u)));
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int32_t page = page_of(pos, true);
    fetch(0, pos, page);
    fetch(1, pos, page);
    page = page_of(pos + kTile, tiles > 1);

    const uint32_t low_last = (uint32_t)(it.len + it.i0), high_last = end - 1u;  // of the columns
    float l[Sh::kHalf];
#pragma unroll
    for (int x = 0; x < Sh::kHalf; ++x) l[x] = 0.0f;

    bool first = true;
    for (int32_t k = 0; k < tiles; ++k, ++i, pos += kTile, first = false) {
      // keys to tensor memory (the previous S has read the ones before)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      uint32_t sb = ld_shared4(sb_at) >> sb_shift;
#pragma unroll
      for (int g = 0; g < kOwn; ++g) {
        const uint4 c = ld_shared16(c_at + (uint32_t)g * (kComputeThreads * 16));
        const uint32_t s = twice(sb, g) * 16u + (kScaleBias << 4) * 0x10001u;
        const uint32_t m = fma_bf16x2(s, 0xC308C308u, 0u);  // -136 s
        uint32_t r[16];
        word_bf16(c.x, one_k, s, m, r);
        word_bf16(c.y, one_k, s, m, r + 4);
        word_bf16(c.z, one_k, s, m, r + 8);
        word_bf16(c.w, one_k, s, m, r + 12);
        tmem_st16(my_lanes + (uint32_t)((wg * kOwn + g) * 16), r);
      }
      tmem_wait_st();
      if (first) fence_async_smem();  // the queries
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.k_full);
      fetch(0, pos + kTile, page);
      // values to shared memory, once the O product has read the ones before
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      sb = ld_shared4(sb_at + kCodes) >> sb_shift;
#pragma unroll
      for (int g = 0; g < kOwn; ++g) {
        const uint4 c = ld_shared16(c_at + kCodes + (uint32_t)g * (kComputeThreads * 16));
        const uint32_t s = twice(sb, g) << 7;
        const uint32_t s16 = fma_f16x2(s, 0x2C002C00u, 0u);                                   // s / 16
        const uint32_t m = fma_f16x2(s, 0xE408E408u, 0u), m16 = fma_f16x2(s, 0xD480D480u, 0u);  // -1032 s, -72 s
        uint32_t r[16];
        word_f16(c.x, one_v, s, m, s16, m16, r);
        word_f16(c.y, one_v, s, m, s16, m16, r + 4);
        word_f16(c.z, one_v, s, m, s16, m16, r + 8);
        word_f16(c.w, one_v, s, m, s16, m16, r + 12);
        if (g == 0 && i > 0) dead |= !wait_phase(&sh.pv_done, (i - 1u) & 1u, &sh.dead);
#pragma unroll
        for (int x = 0; x < 4; ++x) st_shared16(v_at ^ (uint32_t)((g * 4 + x) << 4), r[4 * x], r[4 * x + 1], r[4 * x + 2], r[4 * x + 3]);
      }
      fetch(1, pos + kTile, page);
      page = page_of(pos + 2 * kTile, k + 2 < tiles);

      // weights of this group's columns with the references at hand; into the sums
      const uint32_t lo = pos - (uint32_t)tok;
      const bool masked = lo + kTile - 1 > low_last || high_last - lo >= win;
      dead |= !wait_phase(&sh.s_full, i & 1u, &sh.dead);
      fence_after();
      float top = -INFINITY;
      auto block = [&](int cb, float(&x)[8], auto with_mask) {
        const int j0 = cb * 16 + wg * 8;
        const float4 n0 = *reinterpret_cast<const float4*>(&sh.nm[j0]), n1 = *reinterpret_cast<const float4*>(&sh.nm[j0 + 4]);
        const float nm[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
        for (int y = 0; y < 8; ++y) x[y] = fmaf(x[y], a.c, nm[y]);
        if (with_mask) {
          const int4 e0 = *reinterpret_cast<const int4*>(&sh.last[j0]), e1 = *reinterpret_cast<const int4*>(&sh.last[j0 + 4]);
          const int32_t last[8] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
#pragma unroll
          for (int y = 0; y < 8; ++y)
            if ((uint32_t)last[y] - pos >= win) x[y] = -INFINITY;
        }
#pragma unroll
        for (int y = 0; y < 8; ++y) top = fmaxf(top, x[y]);
        uint32_t w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) w[y] = pack_f16x2(ex2(x[2 * y]), ex2(x[2 * y + 1]));
        st_shared16((p_at ^ (uint32_t)((2 * cb & 7) << 4)) + (uint32_t)(cb >> 2) * (kTile * 128), w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int y = 0; y < 4; ++y) add_halves(w[y], l[cb * 8 + 2 * y], l[cb * 8 + 2 * y + 1]);
      };
      auto weights = [&](auto with_mask) {
#pragma unroll
        for (int cb = 0; cb < kBlocks; ++cb)
          if (cb < n16) {
            float x[8];
            tmem_ld8(s_at + (uint32_t)cb * 16u, x);
            tmem_wait_ld();
            block(cb, x, with_mask);
          }
      };
      bool again = false, gone = false;
      while (true) {
        if (!first || again) {  // no reference yet on the first one
          if (masked) weights(std::true_type{});
          else weights(std::false_type{});
        }
        fence_async_smem();
        fence_before();
        if (!any(!again && (top > kTop || first || dead))) break;
        // slow path: the tile's weights out of the sums, its columns' maxima, new references, O and
        // the sums rescaled, and the weights again
        if ((gone = any(dead))) break;
        again = true;
        fence_after();
        if (first) {  // (rolled: run once an item, its instructions are fetched anew each time)
#pragma unroll 1
          for (int cb = 0; cb < n16; ++cb) {
            const int j0 = cb * 16 + wg * 8;
            float x[8];
            tmem_ld8(s_at + (uint32_t)cb * 16u, x);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 8; ++y) x[y] = (uint32_t)sh.last[j0 + y] - pos >= win ? -INFINITY : x[y] * a.c;
            const float m = warp_fold8(x, lane, [](float p, float q) { return fmaxf(p, q); });  // NaN left out
            if (lane < 8) sh.red[warp & 3][j0 + lane] = m;
          }
        } else {
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb)
            if (cb < n16) {
              const int j0 = cb * 16 + wg * 8;
              float x[8];
              tmem_ld8(s_at + (uint32_t)cb * 16u, x);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                const bool hidden = masked && (uint32_t)sh.last[j0 + y] - pos >= win;
                const uint32_t w = pack_f16x2(hidden ? 0.0f : ex2(fmaf(x[y], a.c, sh.nm[j0 + y])), 0.0f);
                l[cb * 8 + y] -= __half2float(__ushort_as_half((unsigned short)w));
                x[y] = hidden ? -INFINITY : x[y] * a.c;
              }
              const float m = warp_fold8(x, lane, [](float p, float q) { return fmaxf(p, q); });
              if (lane < 8) sh.red[warp & 3][j0 + lane] = m;
            }
        }
        meet();
        if (tid < kCols) {
          float f = 1.0f;
          if (tid < it.n) {
            const float m = fmaxf(fmaxf(sh.red[0][tid], sh.red[1][tid]), fmaxf(sh.red[2][tid], sh.red[3][tid]));
            const float nm0 = sh.nm[tid], nm1 = fminf(nm0, kLift - m);
            sh.nm[tid] = nm1;
            f = nm0 == nm1 ? 1.0f : ex2(nm1 - nm0);
          }
          sh.f[tid] = f;
        }
        meet();
        if (!first) {
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb)
            if (cb < n16) {
              const int j0 = cb * 16 + wg * 8;
              float o[8];
              const uint32_t o_at = my_lanes + Sh::kTmemO + (uint32_t)j0;
              tmem_ld8(o_at, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                l[cb * 8 + y] *= sh.f[j0 + y];
                o[y] *= sh.f[j0 + y];
              }
              tmem_st8(o_at, o);
            }
          tmem_wait_st();
        }
      }
      if (gone) break;
#ifdef SDCP_TEST_WAIT_EXPIRY
      // Test build only (the flag is never set in the library): every fourth CTA keeps the weights of its
      // first tile to itself, so that the waits of its nine warps run out on purpose.
      if (tid == 0 && (blockIdx.x % 4 != 0 || i != 0)) mbar_arrive(&sh.p_full);
#else
      if (tid == 0) mbar_arrive(&sh.p_full);
#endif
    }

    // O, references and sums of the item's columns
    if (!dead) dead = !wait_phase(&sh.pv_done, (i - 1u) & 1u, &sh.dead);
    fence_after();
#pragma unroll
    for (int cb = 0; cb < kBlocks; ++cb)
      if (cb < n16) {
        const float x = warp_fold8(&l[cb * 8], lane, [](float p, float q) { return p + q; });
        if (lane < 8) sh.red[warp & 3][cb * 16 + wg * 8 + lane] = x;
      }
    if (any(dead)) {
      sh.dead = 1;
      continue;
    }
    Part<D, kCols>* const part = reinterpret_cast<Part<D, kCols>*>(a.parts) + it.slot;
    if (tid < kCols) {
      const float sum = (sh.red[0][tid] + sh.red[1][tid]) + (sh.red[2][tid] + sh.red[3][tid]);
      sh.f[tid] = __fdividef(1.0f, sum);
      if (!it.whole) {
        part->m[tid] = -sh.nm[tid];
        part->l[tid] = sum;
      }
    }
    meet();
    __nv_bfloat16* const out0 = a.out + (((int64_t)it.off + it.b + it.i0) * a.q_heads + (int64_t)it.kvh * share) * D + tok;
#pragma unroll 1
    for (int cb = 0; cb < n16; ++cb) {
      const int j0 = cb * 16 + wg * 8;
      float o[8];
      tmem_ld8(my_lanes + Sh::kTmemO + (uint32_t)j0, o);
      tmem_wait_ld();
      if (tok < D) {
        if (!it.whole) {
#pragma unroll
          for (int y = 0; y < 8; ++y) part->o[j0 + y][tok] = o[y];
        } else {
#pragma unroll
          for (int y = 0; y < 8; ++y)
            if (j0 + y < it.n) out0[(int64_t)sh.at[j0 + y] * D] = __float2bfloat16_rn(o[y] * sh.f[j0 + y]);
        }
      }
    }
    fence_before();
  }
}

template <int D, int kCols>
__global__ void __launch_bounds__(kAttendThreads, Shape<kCols>::kCtas) attend_kernel(const AttendArgs a) {
  using Sm = AttendSmem<D, kCols>;
  using Sh = Shape<kCols>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const s_q = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* const s_v = s_q + Sm::kQ;
  unsigned char* const s_p = s_v + Sm::kV;
  __shared__ AttendShared<kCols> sh;

  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t cta = (int32_t)blockIdx.x;
  wait_for_previous();

  // this CTA's part of the line: a prefix sum over the sessions, a stretch of them per thread
  const int32_t per = (a.s.B + kAttendThreads - 1) / kAttendThreads;
  const int32_t b0 = min(tid * per, a.s.B), b1 = min(b0 + per, a.s.B);
  long long mine = 0;
  for (int32_t b = b0; b < b1; ++b) mine += a.units[b];
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh.scan[warp] = incl;
  if (tid == 0) sh.dead = 0;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kAttendThreads / 32; ++w) {
    if (w < warp) before += sh.scan[w];
    all += sh.scan[w];
  }
  const long long start = before + incl - mine;
  const Line line(all, a.ctas);
  if (tid == 0) a.cuts[cta].n = 0;
  if (cta >= line.ctas || all == 0) return;
  const int64_t here = line.first(cta);
  if (here >= start && here < start + mine) {
    long long at = start;
    int32_t b = b0;
    while (here >= at + a.units[b]) at += a.units[b++];
    sh.session = b;
    sh.base = at;
  }
  if (warp == 8) tmem_alloc(&sh.tmem, Sh::kTmemCols);
  if (tid == 0) {
    mbar_init(&sh.k_full, kComputeThreads / 32);
    mbar_init(&sh.s_full, 1);
    mbar_init(&sh.p_full, 1);
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.drained, 1);
    fence_barrier_init();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;
  if (warp == 8) {
    if (lane == 0) {
      sh.walk.begin(a, line, sh.session, sh.base);
      plan_item<D, kCols>(a, sh, line, 0);
    }
    __syncwarp();
    multiply<D, kCols>(a, sh, line, s_q, s_v, s_p, tmem);
  } else {
    attend_tiles<D, kCols>(a, sh, s_q, s_v, s_p, s_p + Sm::kP, tmem);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 8) tmem_free(tmem, Sh::kTmemCols);
}

// ---- the joining of parts -----------------------------------------------------------------
constexpr int kJoinThreads = 128;
constexpr int kJoinCtas = 9;   // of an SM: as many as need no spills
constexpr int kJoinAhead = 4;  // parts whose O a warp has in flight

// One warp per CTA and column: where the CTA's last item goes on in others, the column is the sum of
// its parts, in the line's order.  Bound by latency (3 to 12 us of a call: one row of 2000 tokens, 72
// columns of 304 cuts), so a warp asks for all it needs at once: 21 to 16 us for the one row's call.
template <int D, int kCols>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtas) attend_join_kernel(const AttendArgs a, int32_t cols) {
  constexpr int kPer = D / 32;
  const int lane = (int)(threadIdx.x & 31u);
  const int32_t id = (int32_t)(blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5)), cta = id / cols, j = id - cta * cols;
  wait_for_previous();
  const uint32_t error = *a.error;
  const Cut cut = a.cuts[min(cta, a.ctas - 1)];
  if (error != 0u) {
    for (int64_t b = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; b < a.s.B; b += (int64_t)gridDim.x * kJoinThreads)
      a.status[b] = SDCP_S_INTERNAL;
    return;
  }
  if (cta >= a.ctas || j >= cut.n) return;
  const Part<D, kCols>* const parts = reinterpret_cast<const Part<D, kCols>*>(a.parts);
  const int32_t n = cut.last - cta + 1;
  auto part = [&](int32_t x) -> const Part<D, kCols>& { return parts[x == 0 ? cut.first_slot : 2 * (cta + x)]; };
  // references, sums and the first O are asked for together (an O that was not written has no weight)
  using Chunk = typename std::conditional<D == 128, float4, float2>::type;  // a lane's channels
  float pm = -INFINITY, pl = 0.0f, o[kPer], sum = 0.0f;
  __align__(16) float v[kJoinAhead][kPer];
  auto state = [&](int32_t x) {
    pm = x < n ? part(x).m[j] : -INFINITY;
    pl = x < n ? part(x).l[j] : 0.0f;
  };
  auto load = [&](int32_t x0) {
#pragma unroll
    for (int u = 0; u < kJoinAhead; ++u)
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[u][k] = 0.0f;
#pragma unroll
    for (int u = 0; u < kJoinAhead; ++u)
      if (x0 + u < n) *reinterpret_cast<Chunk*>(v[u]) = *reinterpret_cast<const Chunk*>(&part(x0 + u).o[j][lane * kPer]);
  };
  state(lane);
  load(0);
#pragma unroll
  for (int k = 0; k < kPer; ++k) o[k] = 0.0f;
  float m = pm;
  for (int32_t x = lane + 32; x < n; x += 32) m = fmaxf(m, part(x).m[j]);
  m = warp_max(m);
  for (int32_t x0 = 0; x0 < n; x0 += 32) {
    if (x0 > 0) state(x0 + lane);
    // a lane's part: its factor, 0 where it holds nothing of the column
    const float f = pm != -INFINITY || pl != 0.0f ? (pm == m ? 1.0f : ex2(pm - m)) : 0.0f;
    if (f != 0.0f) sum += pl * f;
    const int32_t here = min(32, n - x0);
    for (int32_t x = 0; x < here; x += kJoinAhead) {
      if (x0 + x > 0) load(x0 + x);
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) {
        const float fx = __shfl_sync(0xFFFFFFFFu, f, (x + u) & 31);
        if (x + u < here && fx != 0.0f) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) o[k] += v[u][k] * fx;
        }
      }
    }
  }
  sum = warp_reduce(sum, [](float x, float y) { return x + y; });
  const int32_t share = a.q_heads / a.kv.heads, r = (cut.g0 + j) / share;
  __nv_bfloat16* const out = a.out + ((cut.row + r) * a.q_heads + cut.row_head - cut.g0 + (cut.g0 + j - r * share)) * D;
#pragma unroll
  for (int k = 0; k < kPer; k += 2)
    *reinterpret_cast<__nv_bfloat162*>(out + lane * kPer + k) = __floats2bfloat162_rn(__fdividef(o[k], sum), __fdividef(o[k + 1], sum));
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
template <int D, int kCols> void set_shared(cudaError_t* e) {
  if (*e == cudaSuccess)
    *e = cudaFuncSetAttribute(attend_kernel<D, kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)AttendSmem<D, kCols>::kBytes);
  if (*e == cudaSuccess) *e = cudaFuncSetAttribute(attend_kernel<D, kCols>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
}
bool attend_ready() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  AttendDevice& d = g_attend_device[dev];
  std::call_once(d.once, [&] {
    set_shared<64, 32>(&d.err);
    set_shared<64, 96>(&d.err);
    set_shared<128, 32>(&d.err);
    set_shared<128, 96>(&d.err);
  });
  return d.err == cudaSuccess;
}

// Columns of an item: the small shape where a session has at most 32 on average (so one long round among
// many single rows is cut into small items).  Sessions with more
// are cut into several items by either shape.  16 contexts of 30000 tokens, 8 cached heads of 128
// channels, small shape against large: 166 and 199 us at 4 columns, 182 and 215 at 32, but 336 and 230
// at 36 (two small items read the cache twice) and 494 and 281 at 96.  64 channels: 157 and 178 at 32,
// 288 and 193 at 36.
int32_t columns_of(int32_t B, int64_t total, int32_t share) { return (total + B) * share <= (int64_t)32 * B ? 32 : 96; }

template <int D, int kCols>
cudaError_t launch_attend(AttendArgs a, int sms, cudaStream_t st) {
  a.ctas = min(sms, kMaxSms) * Shape<kCols>::kCtas;
  cudaError_t e = launch_offsets_check(a.s.offsets, a.s.B, a.status, st);
  if (e != cudaSuccess) return e;
  e = launch_after_if(a.s.B > kScanSessions, attend_plan_kernel, (unsigned)a.s.B, kCheckThreads, 0, st, a);
  if (e != cudaSuccess) return e;
  e = launch_after(attend_kernel<D, kCols>, (unsigned)a.ctas, kAttendThreads, AttendSmem<D, kCols>::kBytes, st, a);
  if (e != cudaSuccess) return e;
  const int32_t cols = (int32_t)min((int64_t)kCols, (a.s.total + a.s.B) * (a.q_heads / a.kv.heads));  // no item has more
  const int32_t warps = a.ctas * cols, per = kJoinThreads / 32;
  return launch_after(attend_join_kernel<D, kCols>, (unsigned)((warps + per - 1) / per), kJoinThreads, 0, st, a, cols);
}

// For either shape: a batch with fewer sessions may take the wider one, in the workspace of a larger batch.
template <int D> constexpr size_t parts_bytes() {
  constexpr size_t narrow = sizeof(Part<D, 32>) * Shape<32>::kCtas, wide = sizeof(Part<D, 96>) * Shape<96>::kCtas;
  return (narrow > wide ? narrow : wide) * kMaxSms * 2;
}

}  // namespace
}  // namespace sdcp

using namespace sdcp;

extern "C" size_t sdcp_attend_workspace_bytes(int32_t B, int64_t total_drafts, int32_t q_heads,
                                              int32_t kv_heads, int32_t head_dim) {
  if (B < 0 || total_drafts < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  return kHeader + round256((size_t)B * sizeof(SessionPlan)) + round256((size_t)B * sizeof(int64_t)) +
         round256(kMaxSms * 3 * sizeof(Cut)) + (head_dim == 128 ? parts_bytes<128>() : parts_bytes<64>());
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
  if (total_drafts > (int64_t)INT32_MAX / 2 - B || q_heads > (1 << 20)) return SDCP_E_TOO_LARGE;
  if (B == 0) return SDCP_OK;
  const int32_t D = cache->head_dim;
  if (!m_offsets || !kv_len || !q || !out || !status) return SDCP_E_INVALID;
  if (q_stride < (int64_t)q_heads * D) return SDCP_E_INVALID;
  if (((uintptr_t)q & 15u) != 0 || ((uintptr_t)out & 15u) != 0 || q_stride % 8 != 0) return SDCP_E_ALIGN;
  if (!on_words(m_offsets, kv_len, status)) return SDCP_E_ALIGN;
  if (!workspace || ((uintptr_t)workspace & 255u) != 0 || workspace_bytes < need) return SDCP_E_WORKSPACE;
  DeviceInfo di;
  if (!device_info(&di) || !attend_ready()) return SDCP_E_DEVICE;
  char* w = static_cast<char*>(workspace);
  char* const plans = w + kHeader;
  char* const lines = plans + round256((size_t)B * sizeof(SessionPlan));
  char* const cuts = lines + round256((size_t)B * sizeof(int64_t));
  char* const parts = cuts + round256(kMaxSms * 3 * sizeof(Cut));
  const KvSessions s{B, m_offsets, total_drafts, 1, kv_len, window, INT32_MAX};
  const AttendArgs a{kv, s, static_cast<const __nv_bfloat16*>(q), q_stride, q_heads, scale * 1.4426950408889634f,
                     static_cast<__nv_bfloat16*>(out), status, reinterpret_cast<uint32_t*>(w), reinterpret_cast<int64_t*>(lines),
                     reinterpret_cast<SessionPlan*>(plans), reinterpret_cast<float*>(parts), reinterpret_cast<Cut*>(cuts),
                     0, columns_of(B, total_drafts, q_heads / cache->kv_heads), D};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (D == 128) e = a.cols == 32 ? launch_attend<128, 32>(a, di.sms, st) : launch_attend<128, 96>(a, di.sms, st);
  else e = a.cols == 32 ? launch_attend<64, 32>(a, di.sms, st) : launch_attend<64, 96>(a, di.sms, st);
  return e == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}
