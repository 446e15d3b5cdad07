// sdcp_attend_shared.cu - sdcp_attend_shared_kv: attention of a round's rows over the paged 4-bit cache in
// groups of sessions whose first pages are the same.
//
//   out[row][h] = sum_t p_t value_t / sum_t p_t,   p_t = 2^(c q.key_t - m),  c = scale log2(e)
//
// The tokens of a group's shared pages are attended once, by the rows of all its sessions, and what lies
// behind them by each session's rows; the two sums are joined by their references m:
//   m = max(m1, m2),  out = (2^(m1 - m) O1 + 2^(m2 - m) O2) / (2^(m1 - m) l1 + 2^(m2 - m) l2).
//
// An item is a cached head and up to 256 pairs of a row and a query head of it, over a stretch of tokens
// in tiles of 128.  The pairs are the rows of both products on the tensor cores (tcgen05, M = 128):
//   S[j][t] = q_j . key_t        A = queries, B = keys, both from shared memory
//   O[j][d] += p_j[t] v_t[d]     A = weights, from tensor memory; B = values, from shared memory
// so a thread of the softmax owns a pair: its reference and sum are the thread's own, and a tile that is
// read and turned once serves two blocks of 128 pairs.  (The attention of sessions by themselves has few
// pairs for its tokens; its kernel makes the tokens the rows.)
//
// One CTA an SM: two groups of four warps for the softmax of a block each, four warps that read keys' codes and
// turn them into 16-bit numbers in shared memory, four for the values', and one that issues the products and
// plans the items.  With more than 128 pairs each tile goes through both blocks; an item with fewer has its
// tiles go through the blocks in turn, as two sums over every other tile that are joined at its end, so the
// products of one run beside the softmax of the other either way.
//
// A weight is 2^8 at the reference, and the reference moves (O, the sums and the tile's weights so far are
// rescaled, by the pair's thread alone) when the weights of 32 tokens sum to more than 2^15: no weight can
// pass binary16's range before the sum tells, and 32 tokens at the reference sum to 2^13.  So an ordinary step
// looks for no maximum.  Weights are binary16 for the product (11 bits, as in the attention of sessions); sums,
// scores and O are binary32.
//
// What bounds it is a block's chain of hand-overs: by time stamps a step of 128 channels takes some 4250 cycles
// (S 470 to issue and 350 until it is seen, the softmax 2000, 280 until its weights are seen, O 390, and 600
// until its end is seen and S may be written again, the weights being in its place); the two blocks run beside
// each other, so a step takes half of that, against 1024 cycles of the tensor cores (39 % of the time).
// Measured (graph replays): 64 sessions of 9 rows and 64 / 8 heads of 128 channels, one prompt of 6000 tokens:
// 173 us, 119 GFLOP at 0.69 PFLOP/s; prompts of 4000 .. 8200 for groups of eight: 194 us, 0.66; 16 sessions of 5
// rows and 32 / 8 heads, 100001 tokens: 178 us, 0.74; by the attention of sessions by themselves 230, 249 and 541 us.
// Tried and slower (the first of these, 168 us then): each tile's tokens halved between two groups of softmax
// warps, 187 us; a second warp for the second product, 172; registers split between the groups, 204 (of 195).
#include <cfloat>
#include <climits>
#include <mutex>
#include <type_traits>

#include "sdcp_tensor.cuh"

namespace sdcp {
namespace {

constexpr int kPairs = 128;           // of a block
constexpr int kMostPairs = 2 * kPairs;  // of an item
constexpr int kTile = 128;            // tokens
// Warps: one that issues products, four of each block's softmax, four that turn keys and four values.
constexpr int kProductWarp = 0, kSoftWarp = 4, kKeyWarp = 12, kValueWarp = 16;  // (warps 1..3 only take part in the barriers)
constexpr int kThreads = 20 * 32;
constexpr int kMaxSms = 160;          // sizes the workspace
constexpr int kItems = 4;             // planned ahead
constexpr int64_t kMostEntries = 1 << 30;  // groups and sessions together: places in their list stay in 32 bits
constexpr float kLift = 8.0f;         // a weight is 2^kLift at its reference
constexpr float kTopSum = 32768.0f;   // and 32 tokens' weights sum to this at most
// kLift - m before there is a reference.  Finite, so that a score of minus infinity (a product beyond binary32)
// has no weight then either; any other score's weight is infinite and sets the reference.
constexpr float kNoScore = FLT_MAX;
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;  // tensor memory: S (and the weights) of two blocks, O of two

// What a tile costs on the line (through one block, through two), and an item's start and end, in tiles.  Graph
// replays of the measured calls above and of ragged groups, us with 5, 8, 3 / 5, 10, 3 / 5, 8, 5 / 8, 13, 2: groups of
// eight 193 / 213 / 201 / 215, ragged 132 / 136 / 143 / 138, one document 177 / 180 / 179 / 191, one prompt 172 / 192 / 177 / 192.
constexpr int32_t kOneBlock = 5, kTwoBlocks = 8, kItemUnits = 3;
// What a pair's second part costs, in the same measure: 1 / kPairsAUnit.  A group's pages are attended together
// where that saves more than the parts cost: 64 sessions of 9 rows in groups of eight, 64 heads, with 512 / 2048
// shared tokens take 105 / 126 us together, 92 / 135 by themselves; of a row in pairs, 74 / 98 and 74 / 116.
constexpr int32_t kPairsAUnit = 3;

// Rows over a stretch of tokens: of a group over its shared pages, or of a session over what is behind them.
struct Entry {
  int32_t row0, rows;      // output rows
  int32_t begin;           // first token
  int32_t last;            // last token of the first row; later rows see `step` more each
  int32_t step;
  int32_t table_row;
  int32_t tiles;           // of any item
  int32_t full, rest;      // items of 256 pairs a cached head, and the pairs of the last one (0: none)
  int32_t joined;          // its pairs have another part
};
__device__ __forceinline__ int32_t cost_of(int32_t pairs) { return pairs > kPairs ? kTwoBlocks : kOneBlock; }
// of a tile with all items of a cached head
__device__ __forceinline__ int64_t cost_of_all(int64_t pairs) {
  return pairs / kMostPairs * kTwoBlocks + (pairs % kMostPairs > 0 ? cost_of((int32_t)(pairs % kMostPairs)) : 0);
}
struct Lengths {  // on the line
  int64_t item, rest, head;
  __device__ __forceinline__ explicit Lengths(const Entry& e) {
    const int64_t u = e.tiles + kItemUnits;
    item = u * kTwoBlocks;
    rest = e.rest > 0 ? u * cost_of(e.rest) : 0;
    head = e.full * item + rest;
  }
};

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// The line over the CTAs: CTA k has the units that begin in [first(k), first(k + 1)).
struct Line {
  int64_t total, each, more;
  int32_t ctas;
  __device__ __forceinline__ Line(int64_t t, int32_t most) {
    total = t;
    ctas = (int32_t)min((int64_t)most, max(quotient(t, kOneBlock), (int64_t)1));
    each = quotient(t, ctas);
    more = t - each * ctas;
  }
  __device__ __forceinline__ int64_t first(int32_t k) const { return k * each + min((int64_t)k, more); }
  __device__ __forceinline__ int32_t cta_of(int64_t t) const {
    const int64_t big = more * (each + 1);
    return t < big ? (int32_t)quotient(t, each + 1) : (int32_t)(more + quotient(t - big, each));
  }
};

struct Header {
  uint32_t error;   // non-zero: a bounded wait gave up
};

// The item that a CTA begins and others go on with: its parts are the CTA's `first_slot` and the first of the
// CTAs after it, up to `last`.  n = 0: none.
struct Cut {
  int32_t n, first_slot, last;  // n: pairs
  int32_t row, head, g0;        // output row of the first pair, first head of its cached head, and the pair's place among these
  int32_t joined, pad;          // as an item's
};

struct SharedArgs {
  KvView kv;
  KvSessions s;
  const int32_t* group_offsets;  // null: one group
  int32_t groups;
  const __nv_bfloat16* q;
  int64_t q_stride;
  int32_t q_heads;
  float c;
  __nv_bfloat16* out;
  int32_t* status;
  int32_t dim;
  int32_t ctas;
  Header* header;
  int32_t* group_status;  // [groups] where there are many: whether the group offsets are in order
  int32_t* lead;          // [B] the session of its group that a session's pages were compared with
  int32_t* common;        // [B] leading pages it has in common with that one
  Entry* entries;         // [groups + B]: groups, then sessions
  int64_t* units;         // [groups + B] length on the line
  Cut* cuts;              // [ctas]
  float* parts;           // [ctas * 2] of Part
  float* acc;             // [2][rows * q_heads] of O, where a pair has two parts
  float2* acc_ml;         // [2][rows * q_heads] references and sums (or kDone in place of a session's sum)
};
constexpr float kDone = -1.0f;  // not joined: the output is there, or the row is no session's
constexpr int64_t kFewPairs = 8192;

template <int D> struct Part {
  float o[kMostPairs][D];
  float m[kMostPairs];
  float l[kMostPairs];
};

// ---- plan ---------------------------------------------------------------------------------
// A block a session: its status, its group, and the pages that it has in common with `lead`, the group's first
// session whose numbers do not refuse it (an ended one's length is -1).
__global__ void __launch_bounds__(kCheckThreads) shared_check_kernel(const SharedArgs a) {
  __shared__ int32_t common, lead;
  let_next_start();
  const int32_t b = (int32_t)blockIdx.x;
  const int64_t pairs = (a.s.total + a.s.B) * a.q_heads;
  for (int64_t x = (int64_t)b * kCheckThreads + threadIdx.x; x < pairs; x += (int64_t)gridDim.x * kCheckThreads) a.acc_ml[pairs + x] = make_float2(0.0f, kDone);
  if (b >= a.s.B) return;
  const bool kernel_before = a.s.B > kScanSessions || a.groups > kScanSessions;
  if (kernel_before) wait_for_previous();
  int32_t st = kv_session_status(a.kv, a.s, b, a.status);
  int32_t first = 0;
  if (a.group_offsets != nullptr) {
    bool bad = a.group_offsets[0] != 0 || a.group_offsets[a.groups] != a.s.B;
    bad |= a.groups <= kScanSessions ? !offsets_in_order(a.group_offsets, a.groups) : a.group_status[0] != SDCP_S_OK;
    if (__syncthreads_or(bad)) {
      st = SDCP_S_BAD_PARAMS;
    } else {
      first = a.group_offsets[find_session(a.group_offsets, a.groups, b, false)];
    }
  }
  if (st != SDCP_S_OK) {  // its rows become zero (what another session has of them is written later)
    const int64_t lo = min(max((int64_t)a.s.offsets[b], (int64_t)0), a.s.total), hi = min(max((int64_t)a.s.offsets[b + 1], lo), a.s.total);
    const int64_t row = (int64_t)a.q_heads * a.dim / 8;
    uint4* const out = reinterpret_cast<uint4*>(a.out);
    for (int64_t x = (lo + b) * row + threadIdx.x; x < (hi + b + 1) * row; x += kCheckThreads) out[x] = make_uint4(0u, 0u, 0u, 0u);
  } else {
    // (pages that all rows of the round see whole)
    const int32_t n = a.s.start[b] >> a.kv.log_page;
    const int32_t* const mine = a.kv.page_table + (int64_t)b * a.kv.max_pages;
    auto compare = [&](int32_t f) {
      const int32_t* const other = a.kv.page_table + (int64_t)f * a.kv.max_pages;
      if (f != b)
        for (int32_t p = (int32_t)threadIdx.x; p < n; p += kCheckThreads)
          if (mine[p] != other[p]) {
            atomicMin(&common, p);
            break;
          }
    };
    auto refused = [&](int32_t lo, int32_t hi, int32_t start) {
      int64_t end;
      return kv_session_end(a.kv, a.s, lo, hi, start, &end) != SDCP_S_OK;
    };
    if (threadIdx.x == 0) {
      common = n;
      lead = first;
    }
    __syncthreads();
    const int32_t lo = a.s.offsets[first], hi = a.s.offsets[first + 1], start = a.s.start[first];  // (on their way during the comparison)
    compare(first);
    if (refused(lo, hi, start)) {
      __syncthreads();
      if (threadIdx.x == 0) {
        common = n;
        lead = b;
      }
      __syncthreads();
      for (int32_t f = first + 1 + (int32_t)threadIdx.x; f < b; f += kCheckThreads)
        if (!refused(a.s.offsets[f], a.s.offsets[f + 1], a.s.start[f])) {
          atomicMin(&lead, f);
          break;
        }
      __syncthreads();
      compare(lead);
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    a.status[b] = st;
    a.lead[b] = st == SDCP_S_OK ? lead : b;
    a.common[b] = st == SDCP_S_OK ? common : 0;
    if (st != SDCP_S_OK) a.units[a.groups + b] = 0;
    if (b == 0) a.header->error = 0u;
  }
}

__device__ __forceinline__ void plan_entry(const SharedArgs& a, int32_t id, Entry e) {
  const int64_t pairs = (int64_t)e.rows * (a.q_heads / a.kv.heads);
  const int64_t tokens = (int64_t)e.last + (int64_t)e.step * (e.rows - 1) + 1 - e.begin;
  e.tiles = (int32_t)((tokens + kTile - 1) / kTile);
  e.full = (int32_t)(pairs / kMostPairs);
  e.rest = (int32_t)(pairs % kMostPairs);
  a.entries[id] = e;
  a.units[id] = Lengths(e).head * a.kv.heads;
}

// A block a group: the pages that its sessions share, its entry and theirs.
__global__ void __launch_bounds__(kCheckThreads) shared_plan_kernel(const SharedArgs a) {
  __shared__ int32_t pages, low, high;  // of the members that are not refused
  __shared__ unsigned long long apart;  // what a tile costs that each of them attends for itself
  let_next_start();
  wait_for_previous();
  const int32_t g = (int32_t)blockIdx.x;
  const int32_t b0 = a.group_offsets ? min(max(a.group_offsets[g], 0), a.s.B) : 0, b1 = a.group_offsets ? min(max(a.group_offsets[g + 1], 0), a.s.B) : a.s.B;
  if (threadIdx.x == 0) {
    pages = INT_MAX;
    low = INT_MAX;
    high = -1;
    apart = 0;
  }
  __syncthreads();
  const int32_t share = a.q_heads / a.kv.heads;
  unsigned long long cost = 0;
  int32_t least = INT_MAX, lowest = INT_MAX, highest = -1, lead = -1;
  bool leads_differ = false;
  for (int32_t b = b0 + (int32_t)threadIdx.x; b < b1; b += kCheckThreads)
    if (a.status[b] == SDCP_S_OK) {
      least = min(least, a.common[b]);
      lowest = min(lowest, b);
      leads_differ |= highest >= 0 && a.lead[b] != lead;
      lead = a.lead[b];
      highest = b;
      cost += (unsigned long long)cost_of_all((int64_t)(a.s.offsets[b + 1] - a.s.offsets[b] + 1) * share);
    }
  if (highest >= 0) {
    atomicMin(&pages, least);
    atomicMin(&low, lowest);
    atomicMax(&high, highest);
    atomicAdd(&apart, cost);
  }
  __syncthreads();
  // A lead that an entry of its row refused (rare: no call leaves such a row): the pages compared anew, with the first
  // that is not refused.
  if (__syncthreads_or(highest >= 0 && (lead != low || leads_differ))) {
    const int32_t* const first = a.kv.page_table + (int64_t)low * a.kv.max_pages;
    if (threadIdx.x == 0) pages = a.s.start[low] >> a.kv.log_page;
    for (int32_t b = low + 1; b < b1; ++b) {
      __syncthreads();
      if (a.status[b] != SDCP_S_OK) continue;
      const int32_t n = min(pages, a.s.start[b] >> a.kv.log_page);
      const int32_t* const row = a.kv.page_table + (int64_t)b * a.kv.max_pages;
      int32_t same = n;
#pragma unroll 4
      for (int32_t p = (int32_t)threadIdx.x; p < n; p += kCheckThreads)
        if (row[p] != first[p]) same = min(same, p);
      __syncthreads();
      atomicMin(&pages, same);
    }
    __syncthreads();
  }
  int32_t shared = 0;
  if (high > low && pages > 0) {
    const int64_t tokens = (int64_t)pages << a.kv.log_page, tiles = (tokens + kTile - 1) / kTile;
    const int64_t pairs = (int64_t)(a.s.offsets[high + 1] + high + 1 - a.s.offsets[low] - low) * share, together = cost_of_all(pairs);
    if (tiles * ((int64_t)apart - together) > kItemUnits * together + pairs / kPairsAUnit) shared = (int32_t)tokens;
  }
  if (threadIdx.x == 0) {
    if (shared > 0) {
      const int32_t row0 = a.s.offsets[low] + low;  // (a refused one's offsets may be outside the batch)
      plan_entry(a, g, Entry{row0, a.s.offsets[high + 1] + high + 1 - row0, 0, shared - 1, 0, low, 0, 0, 0, 1});
    } else {
      a.units[g] = 0;
    }
  }
  for (int32_t b = b0 + (int32_t)threadIdx.x; b < b1; b += kCheckThreads)
    if (a.status[b] == SDCP_S_OK) {
      const int32_t off = a.s.offsets[b];
      plan_entry(a, a.groups + b, Entry{off + b, a.s.offsets[b + 1] - off + 1, shared, a.s.start[b], 1, b, 0, 0, 0, shared > 0});
    }
}

// ---- items --------------------------------------------------------------------------------
struct Item {
  int32_t n;                    // pairs; 0: no more items
  int32_t i0, g0;               // row (of the entry) and head of the first
  int32_t row0;                 // output row of the entry
  int32_t kvh, table_row;
  int32_t begin, end;           // first token of tile 0, one past the last token read
  int32_t last, step;           // of the entry
  int32_t k0, k1;               // tiles
  int32_t slot;                 // of the parts
  int32_t whole;                // all of the item's tiles are here
  int32_t joined;               // 0: alone; 1: a group's part; 2: a session's
};
// A CTA's way along the line, walked by the warp that issues the products, items ahead of it.
struct Walk {
  int64_t t, t_end, t_first;
  Entry en;
  int32_t e, kvh, chunk, unit0;
  __device__ __forceinline__ int32_t chunks() const { return en.full + (en.rest > 0); }
  __device__ __forceinline__ int32_t pairs() const { return chunk < en.full ? kMostPairs : en.rest; }
  __device__ __forceinline__ void begin(const SharedArgs& a, const Line& line, int32_t entry, int64_t base) {
    const int64_t from = line.first((int32_t)blockIdx.x);
    t_end = line.first((int32_t)blockIdx.x + 1);
    e = entry;
    en = a.entries[e];
    const Lengths len(en);
    int64_t r = from - base;
    kvh = (int32_t)quotient(r, len.head);
    r -= kvh * len.head;
    chunk = (int32_t)min(quotient(r, len.item), (int64_t)en.full);
    r -= chunk * len.item;
    const int32_t cost = cost_of(pairs());
    unit0 = (int32_t)quotient(r + cost - 1, cost);
    t = t_first = base + kvh * len.head + chunk * len.item + (int64_t)unit0 * cost;
    if (unit0 == en.tiles + kItemUnits) advance();
  }
  __device__ __forceinline__ void advance() {
    unit0 = 0;
    if (++chunk == chunks()) {
      chunk = 0;
      ++kvh;
    }
  }
  // the next item; false at the end of the CTA's part
  __device__ __forceinline__ bool next(const SharedArgs& a, const Line& line, Item& it) {
    if (t >= t_end) return false;
    if (kvh == a.kv.heads) {  // the next entry that has work
      do ++e;
      while (a.units[e] == 0);
      en = a.entries[e];
      kvh = 0;
    }
    const int32_t share = a.q_heads / a.kv.heads, all = en.tiles + kItemUnits, cost = cost_of(pairs());
    const int32_t units = (int32_t)min((int64_t)(all - unit0), quotient(t_end - t + cost - 1, cost));
    const int32_t c0 = chunk * kMostPairs;
    it.n = pairs();
    it.i0 = c0 / share;
    it.g0 = c0 - it.i0 * share;
    it.row0 = en.row0;
    it.kvh = kvh;
    it.table_row = en.table_row;
    it.begin = en.begin;
    it.last = en.last;
    it.step = en.step;
    it.end = en.last + en.step * (it.i0 + (it.g0 + it.n - 1) / share) + 1;
    const int32_t real = (it.end - it.begin - 1) / kTile + 1;  // (ends may be next to 2^31)
    it.k0 = max(unit0 - kItemUnits, 0);
    it.k1 = min(max(unit0 + units - kItemUnits, 0), real);
    it.slot = (int32_t)blockIdx.x * 2 + (t == t_first ? 0 : 1);
    it.whole = units == all;
    it.joined = en.joined ? (e < a.groups ? 1 : 2) : 0;
    if (!it.whole && unit0 == 0)  // the CTA's last item, and others go on with it
      a.cuts[blockIdx.x] = Cut{it.n, it.slot, line.cta_of(t + (int64_t)(all - 1) * cost), en.row0 + it.i0, kvh * share, it.g0, it.joined, 0};
    t += (int64_t)units * cost;
    advance();
    return true;
  }
};

template <int D> struct SharedSmem {
  static constexpr int kAtoms = D / 64;                   // 128-byte atoms along the channels
  static constexpr int kBlock = kAtoms * kTile * 128;     // [atom][pair or token][128 bytes]
  static constexpr size_t kBytes = (size_t)6 * kBlock + 1024;  // two of queries, keys and values; and the alignment to 1024
};
struct SharedState {
  Item item[kItems];
  float2 ml[2][2][kPairs];  // references and sums of the blocks, at an item's end; the next such item's beside them
  uint64_t item_full[kItems], item_free[kItems];
  uint64_t q_free[2], k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], pv_done[2], o_free, ml_full, drained;
  long long scan[kThreads / 32];
  long long base;
  int32_t entry;
  uint32_t tmem;
  int dead;
};

template <int D> __device__ __forceinline__ void nothing_in(const SharedArgs& a, int32_t slot) {
  Part<D>* const part = reinterpret_cast<Part<D>*>(a.parts) + slot;
  for (int x = (int)(threadIdx.x & 31u); x < kMostPairs; x += 32) {
    part->m[x] = -INFINITY;
    part->l[x] = 0.0f;
  }
}
// The next item that has tiles, into the ring; a part that holds no tile of its item is marked at once.
template <int D> __device__ __forceinline__ void plan_item(const SharedArgs& a, SharedState& sh, const Line& line, Walk& walk, bool& more, uint32_t j) {
  Item it;
  it.n = 0;
  if (j == 0 && walk.t >= walk.t_end) nothing_in<D>(a, (int32_t)blockIdx.x * 2);  // no unit begins here
  while (more && (more = walk.next(a, line, it)) && it.k0 >= it.k1) nothing_in<D>(a, it.slot);
  if (!more) it.n = it.k0 = it.k1 = 0;
  if ((threadIdx.x & 31u) == 0) {
    sh.item[j % kItems] = it;
    mbar_arrive(&sh.item_full[j % kItems]);
  }
  __syncwarp();
}

// ---- the products: a warp, whose registers of a product are uniform; one lane issues ----------
// (Issued from a branch that one thread takes, each product has its operands moved to uniform registers anew:
// the calls above took 20 to 30 % longer.)
__device__ __forceinline__ void issue_smem_a(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{ .reg .pred p, e; elect.sync _|e, 0xFFFFFFFF; setp.ne.u32 p, %4, 0; @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
      "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void issue_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{ .reg .pred p, e; elect.sync _|e, 0xFFFFFFFF; setp.ne.u32 p, %4, 0; @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
      "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void issue_commit(uint64_t* bar) {
  asm volatile(
      "{ .reg .pred e; elect.sync _|e, 0xFFFFFFFF; @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(smem_u32(bar))
      : "memory");
}

// Bounded wait for the phases of two barriers (if wanted), looked at together: a look takes some 150 cycles
// beside the stores of the warps that turn.
__device__ __forceinline__ bool wait_both(bool want_a, uint64_t* a, uint32_t parity_a, bool want_b, uint64_t* b, uint32_t parity_b, const volatile int* dead) {
  const bool odd = (threadIdx.x & 1u) != 0;
  uint64_t* const bar = odd ? b : a;
  const uint32_t parity = odd ? parity_b : parity_a;
  bool done = odd ? !want_b : !want_a;
  unsigned long long t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (!done) done = mbar_try_wait(bar, parity);
    if (__all_sync(0xFFFFFFFFu, done)) {
      __syncwarp();  // a lane has looked at one of the two; a vote alone does not order what it saw before the others' work
      return true;
    }
    if (n % 1024u == 0u) {
      if (t0 == 0) t0 = global_ns();
      if (__any_sync(0xFFFFFFFFu, *dead != 0 || global_ns() - t0 > kWaitNs)) return false;
    }
  }
}

template <int D>
__device__ __forceinline__ void multiply(const SharedArgs& a, SharedState& sh, const Line& line, Walk& walk, const unsigned char* s_q, const unsigned char* s_k,
                                         const unsigned char* s_v, uint32_t tmem) {
  using Sm = SharedSmem<D>;
  const uint64_t q_mat = smem_matrix(s_q, 0, 1024, kSwizzle128), k_mat = smem_matrix(s_k, 0, 1024, kSwizzle128),
                 v_mat = smem_matrix(s_v, D == 128 ? kTile * 128 : 0, 1024, kSwizzle128);
  constexpr uint32_t kIdescS = kIdescF32 | kIdescBf16 | kIdescM128 | (uint32_t)(kTile / 8) << 17;
  constexpr uint32_t kIdescO = kIdescF32 | kIdescM128 | (uint32_t)(D / 8) << 17 | 1u << 16;  // values: tokens along the rows
  bool more = true;
  plan_item<D>(a, sh, line, walk, more, 0);
  plan_item<D>(a, sh, line, walk, more, 1);
  uint32_t tiles = 0, q_used = 0, used0 = 0, used1 = 0;  // tiles, blocks of queries and steps of the blocks so far
  bool ok = true;
  for (uint32_t j = 0; ok; ++j) {
    const int32_t n = __shfl_sync(0xFFFFFFFFu, sh.item[j % kItems].n, 0);
    const bool two = n > kPairs;
    const int32_t n_tiles = __shfl_sync(0xFFFFFFFFu, sh.item[j % kItems].k1 - sh.item[j % kItems].k0, 0), steps = two ? 2 * n_tiles : n_tiles;
    if (n_tiles <= 0) break;
    auto score = [&](int32_t h) {  // S of step h
      const int x = h & 1;
      const uint32_t tile = tiles + (uint32_t)(two ? h >> 1 : h), buf = tile & 1u;
      const uint32_t used = x ? used1 : used0;
      // the keys, and the end of the product of the weights of the step before, in the same place
      ok = wait_both(!two || x == 0, &sh.k_full[buf], (tile >> 1) & 1u, used > 0, &sh.pv_done[x], (used - 1u) & 1u, &sh.dead);
      if (!ok) return;
      fence_after();
      const uint32_t qb = (q_used + (two ? (uint32_t)x : 0u)) & 1u;
      const uint64_t qm = q_mat + (uint64_t)(qb * Sm::kBlock >> 4), km = k_mat + (uint64_t)(buf * Sm::kBlock >> 4);
#pragma unroll
      for (int y = 0; y < D / 16; ++y) {
        const uint64_t at = (uint64_t)(((y / 4) * (kTile * 128) + (y % 4) * 32) >> 4);
        issue_smem_a(tmem + kTmemS + (uint32_t)x * 128u, qm + at, km + at, kIdescS, y > 0);
      }
      issue_commit(&sh.s_full[x]);
      if (!two || x == 1) issue_commit(&sh.k_free[buf]);
      if (h == steps - 1) {
        issue_commit(&sh.q_free[q_used & 1u]);
        if (two) issue_commit(&sh.q_free[(q_used + 1u) & 1u]);
      }
      used0 += x ? 0u : 1u;
      used1 += x ? 1u : 0u;
    };
    score(0);
    for (int32_t h = 0; h < steps && ok; ++h) {
      if (h + 1 < steps) score(h + 1);
      if (!ok) break;
      if (h == 0 && ok) {
        if (j >= 2) ok = wait_both(true, &sh.item_free[(j + 2) % kItems], ((j - 2) / kItems) & 1u, false, nullptr, 0u, &sh.dead);
        if (ok) plan_item<D>(a, sh, line, walk, more, j + 2);
      }
      const int x = h & 1;
      const uint32_t tile = tiles + (uint32_t)(two ? h >> 1 : h), buf = tile & 1u;
      // (of its own step: the one after may have been asked for, but needs this product first)
      if (ok) ok = wait_both(!two || x == 0, &sh.v_full[buf], (tile >> 1) & 1u, true, &sh.p_full[x], ((x ? used1 : used0) - 1u) & 1u, &sh.dead);
      if (ok && h == 0 && j > 0) ok = wait_both(true, &sh.o_free, (j - 1u) & 1u, false, nullptr, 0u, &sh.dead);
      if (!ok) break;
      fence_after();
#pragma unroll
      for (int y = 0; y < kTile / 16; ++y)
        issue_tmem_a(tmem + kTmemO + (uint32_t)(x * D), tmem + kTmemS + (uint32_t)(x * 128 + y / 2 * 32 + y % 2 * 8), v_mat + (uint64_t)((buf * Sm::kBlock + y * 2048) >> 4),
                   kIdescO, h > 1 || y > 0);
      if (!two || x == 1) issue_commit(&sh.v_free[buf]);
      issue_commit(&sh.pv_done[x]);  // the last of a step: when it is seen, none is under way
    }
    tiles += (uint32_t)n_tiles;
    q_used += two ? 2u : 1u;
  }
  if (!ok) {  // products under way end before the tensor memory is given back
    sh.dead = 1;
    issue_commit(&sh.drained);
    (void)wait_phase(&sh.drained, 0u, nullptr);
  }
}

// ---- the turning: four warps for the keys and four for the values, a token of the tile a thread ----
template <int D, bool kValues>
__device__ __forceinline__ void turn(const SharedArgs& a, SharedState& sh, unsigned char* s_q, unsigned char* s_to) {
  using Sm = SharedSmem<D>;
  constexpr int kGroups = D / kKvGroup;
  const int tok = (int)threadIdx.x & 127, lane = tok & 31;
  const uint32_t one = kept(kValues ? 0x64006400u : 0x43004300u);
  const uint32_t to = smem_u32(s_to) + (uint32_t)(tok * 128) + ((uint32_t)(tok & 7) << 4);  // a token's line in an atom, swizzled
  const int sb_shift = D == 128 ? 0 : (tok & 1) * 16;  // of the thread's own scales (tiles start at even tokens)
  const int32_t share = a.q_heads / a.kv.heads;
  uint64_t* const full = kValues ? sh.v_full : sh.k_full;
  uint64_t* const freed = kValues ? sh.v_free : sh.k_free;
  uint32_t tiles = 0, q_used = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {  // a warp agrees on it
    if (ok) ok = __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, &sh.dead));
  };
  for (uint32_t j = 0;; ++j) {
    wait(&sh.item_full[j % kItems], (j / kItems) & 1u);
    if (!ok) break;
    const Item it = sh.item[j % kItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.item_free[j % kItems]);
    const int32_t n_tiles = it.k1 - it.k0;
    if (n_tiles <= 0) break;
    // a tile ahead: the next token's codes and scales, and a tile before that its page
    uint32_t pos = (uint32_t)it.begin + (uint32_t)it.k0 * kTile + (uint32_t)tok;
    const uint32_t end = (uint32_t)it.end, in_page = ((uint32_t)it.kvh * 2u + (kValues ? 1u : 0u)) * (uint32_t)a.kv.block;
    const int32_t* const table = a.kv.page_table + (int64_t)it.table_row * a.kv.max_pages;
    auto page_of = [&](uint32_t p, bool some) { return some && p < end ? table[p >> a.kv.log_page] : -1; };
    uint4 c[kGroups], next[kGroups];
    uint32_t sb, next_sb;
    auto load = [&](uint32_t p, int32_t page) {  // of the token at p, whose page is known (-1: nothing to read, zeros)
#pragma unroll
      for (int g = 0; g < kGroups; ++g) next[g] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
      next_sb = 0u;
      if (page >= 0) {
        const uint32_t slot = p & ((1u << a.kv.log_page) - 1u);
        const uint8_t* const blk = a.kv.pages + (uint64_t)(uint32_t)page * (uint32_t)a.kv.page + in_page;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) next[g] = *reinterpret_cast<const uint4*>(blk + ((((uint32_t)g << a.kv.log_page) + slot) * 16u));
        // four scale bytes of a token, or two each of a pair of tokens
        next_sb = *reinterpret_cast<const uint32_t*>(blk + ((D / 2u << a.kv.log_page) + (D == 128 ? slot * 4u : (slot & ~1u) * 2u)));
      }
    };
    int32_t page = page_of(pos, true);
    if (!kValues) {  // queries of the pairs, zero past them: they are there with the first keys
      for (int x = 0; x < (it.n > kPairs ? 2 : 1); ++x, ++q_used) {
        if (q_used >= 2) wait(&sh.q_free[q_used & 1u], ((q_used >> 1) - 1u) & 1u);
        if (!ok) break;
        const __nv_bfloat16* const q0 = a.q + ((int64_t)it.row0 + it.i0) * a.q_stride + (int64_t)it.kvh * share * D;
        const int ch = tok % (D / 8);
        const uint32_t dst = smem_u32(s_q) + (q_used & 1u) * Sm::kBlock + (uint32_t)(ch / 8) * (kTile * 128);
#pragma unroll 4
        for (int col = tok / (D / 8); col < kPairs; col += 128 / (D / 8)) {
          const int32_t at = x * kPairs + col, c = min(at, it.n - 1) + it.g0, r = c / share;
          copy_async16_or_zero(dst + (uint32_t)col * 128u + (uint32_t)(((ch & 7) ^ (col & 7)) << 4), q0 + r * a.q_stride + (c - r * share) * D + ch * 8,
                               at < it.n);
        }
      }
    }
    load(pos, page);
    page = page_of(pos + kTile, n_tiles > 1);
    if (!kValues) asm volatile("cp.async.wait_all;" ::: "memory");
    for (int32_t k = 0; k < n_tiles && ok; ++k, ++tiles, pos += kTile) {
      const uint32_t buf = tiles & 1u;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) c[g] = next[g];
      sb = next_sb >> sb_shift;
      load(pos + kTile, page);
      page = page_of(pos + 2 * kTile, k + 2 < n_tiles);
      if (tiles >= 2) wait(&freed[buf], ((tiles >> 1) - 1u) & 1u);  // the products that read the ones before are done
      if (!ok) break;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        uint32_t r[16];
        if (kValues) {
          const uint32_t s = twice(sb, g) << 7;
          const uint32_t s16 = fma_f16x2(s, 0x2C002C00u, 0u);                                   // s / 16
          const uint32_t m = fma_f16x2(s, 0xE408E408u, 0u), m16 = fma_f16x2(s, 0xD480D480u, 0u);  // -1032 s, -72 s
          word_f16(c[g].x, one, s, m, s16, m16, r);
          word_f16(c[g].y, one, s, m, s16, m16, r + 4);
          word_f16(c[g].z, one, s, m, s16, m16, r + 8);
          word_f16(c[g].w, one, s, m, s16, m16, r + 12);
        } else {
          const uint32_t s = twice(sb, g) * 16u + (kScaleBias << 4) * 0x10001u;
          const uint32_t m = fma_bf16x2(s, 0xC308C308u, 0u);  // -136 s
          word_bf16(c[g].x, one, s, m, r);
          word_bf16(c[g].y, one, s, m, r + 4);
          word_bf16(c[g].z, one, s, m, r + 8);
          word_bf16(c[g].w, one, s, m, r + 12);
        }
        const uint32_t line = to + buf * Sm::kBlock + (uint32_t)(g / 2) * (kTile * 128);
#pragma unroll
        for (int y = 0; y < 4; ++y) st_shared16(line ^ (uint32_t)(((g & 1) * 4 + y) << 4), r[4 * y], r[4 * y + 1], r[4 * y + 2], r[4 * y + 3]);
      }
      fence_async_smem();  // (the item's queries too)
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[buf]);
    }
    if (!ok) break;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // before the shared memory is given back
  if (!ok) sh.dead = 1;
}

// ---- the softmax: four warps a block of pairs, a pair a thread --------------------------------
// Two numbers of binary32 in an instruction.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void halves_of(uint64_t x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Where the weights of tokens c .. c + 31 are too large (or there is no reference yet): the largest of the
// pair's scores from here to the tile's end, the reference that it sets, and what has been summed so far
// rescaled.  References are whole numbers apart, so that rescaling is exact (but for weights below binary16's
// normal ones).
struct Moved {
  float nm, f;  // kLift - m, and the factor of what has been summed
  bool ok;
};
template <int D>
__device__ __noinline__ Moved move_reference(SharedState& sh, int c, int32_t lim, float scale, uint32_t s_at, uint32_t o_at, bool some_before, int x,
                                             uint32_t used, float nm) {
  float m = -INFINITY;
#pragma unroll 1
  for (int d = c; d < kTile; d += 32) {
    float r[32];
    tmem_ld32(s_at + (uint32_t)d, r);
    tmem_loaded(r);
#pragma unroll
    for (int y = 0; y < 32; ++y) m = fmaxf(m, d + y > lim ? -INFINITY : r[y] * scale);  // NaN left out
  }
  const float old = nm;
  nm = fminf(nm, kLift - ceilf(m));
  const float by = nm - old;  // a whole number, or far below -126
  const float f = nm == old ? 1.0f : by > -126.0f ? __int_as_float((127 + (int)by) << 23) : 0.0f;
  bool ok = true;
#pragma unroll 1
  for (int d = 0; d < c; d += 32) {  // the tile's weights so far
#pragma unroll 1
    for (int e = 0; e < 16; e += 8) {
      float r[8];
      tmem_ld8(s_at + (uint32_t)(d + e), r);
      tmem_loaded(r);
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const float lo = __half2float(__ushort_as_half((unsigned short)(__float_as_uint(r[y]) & 0xFFFFu)));
        const float hi = __half2float(__ushort_as_half((unsigned short)(__float_as_uint(r[y]) >> 16)));
        r[y] = __uint_as_float(pack_f16x2(lo * f, hi * f));
      }
      tmem_st8(s_at + (uint32_t)(d + e), r);
    }
  }
  if (some_before) {
    ok = __all_sync(0xFFFFFFFFu, wait_phase(&sh.pv_done[x], (used - 1u) & 1u, &sh.dead));
    fence_after();
#pragma unroll 1
    for (int d = 0; d < D; d += 8) {
      float o[8];
      tmem_ld8(o_at + (uint32_t)d, o);
      tmem_loaded(o);
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] *= f;
      tmem_st8(o_at + (uint32_t)d, o);
    }
  }
  tmem_wait_st();
  return Moved{nm, f, ok};
}

template <int D>
__device__ __forceinline__ void soften(const SharedArgs& a, SharedState& sh, int x, uint32_t tmem) {
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = (int)threadIdx.x & 31, pair = (int)threadIdx.x & 127;
  const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // 32 lanes of tensor memory, in bits 16 up
  const uint32_t s_at = lanes + kTmemS + (uint32_t)x * 128u, o_at = lanes + kTmemO + (uint32_t)(x * D);
  const int32_t share = a.q_heads / a.kv.heads;
  uint32_t used = 0, used_other = 0, halves = 0;  // steps of the block and of the other one, and items of halves, so far
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {  // a warp agrees on it
    if (ok) ok = __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, &sh.dead));
    return ok;
  };
  for (uint32_t j = 0;; ++j) {
    if (!wait(&sh.item_full[j % kItems], (j / kItems) & 1u)) break;
    const Item it = sh.item[j % kItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.item_free[j % kItems]);
    const int32_t n_tiles = it.k1 - it.k0;
    if (n_tiles <= 0) break;
    const bool two = it.n > kPairs;
    const int32_t at = two ? x * kPairs + pair : pair;                   // of the item's pairs
    const int32_t row = it.i0 + (it.g0 + min(at, it.n - 1)) / share;     // of the entry's rows
    const bool live = at < it.n, some = __any_sync(0xFFFFFFFFu, live);
    int32_t limit = it.last + it.step * row - it.begin - it.k0 * kTile;  // last token that it sees, from the tile's start
    float nm = kNoScore, l = 0.0f;  // kLift - m: what a scaled score is shifted by, and the sum
    bool first = true;
    for (int32_t k = two ? 0 : x; k < n_tiles; k += two ? 1 : 2, ++used) {
      if (!wait(&sh.s_full[x], used & 1u)) break;
      fence_after();
      if (some) {
        const int32_t lim = limit - k * kTile;
        float sum = 0.0f;  // of the tile's weights
        // (rolled: five kinds of warps share a scheduler's instruction cache)
        auto tile = [&](auto with_mask) {
          const uint64_t c2 = pair_of(a.c, a.c), zero2 = pair_of(0.0f, 0.0f);
#pragma unroll 1
          for (int c = 0; c < kTile; c += 32) {
            float part;
            uint32_t w[16];
#pragma unroll 1
            for (bool moved = false;; moved = true) {
              float s[32];
              tmem_ld32(s_at + (uint32_t)c, s);
              tmem_loaded(s);
              const uint64_t nm2 = pair_of(nm, nm);
              uint64_t sums[2] = {0, 0};
#pragma unroll
              for (int y = 0; y < 32; y += 2) {
                float u, v;
                // The scaled score is rounded before the reference is taken off, as it was for the reference: with
                // one rounding the largest of huge scores would be off by a rounding of itself, out of any
                // range.  (As a sum with zero: a product and a sum of two numbers become one instruction.  2 %.)
                halves_of(add_pair(fma_pair(pair_of(s[y], s[y + 1]), c2, zero2), nm2), u, v);
                if (with_mask) {
                  if (c + y > lim) u = -INFINITY;
                  if (c + y + 1 > lim) v = -INFINITY;
                }
                u = ex2(u);
                v = ex2(v);
                sums[y / 2 % 2] = add_pair(sums[y / 2 % 2], pair_of(u, v));
                w[y / 2] = pack_f16x2(u, v);
              }
              float u, v;
              halves_of(add_pair(sums[0], sums[1]), u, v);
              part = u + v;
              if (moved || !__any_sync(0xFFFFFFFFu, part > kTopSum)) break;
              const Moved m = move_reference<D>(sh, c, lim, a.c, s_at, o_at, !first, x, used, nm);
              nm = m.nm;
              ok &= m.ok;
              l *= m.f;
              sum *= m.f;
            }
            sum += part;
            tmem_st16(s_at + (uint32_t)c, w);  // over the scores they come from
          }
        };
        if (__any_sync(0xFFFFFFFFu, lim < kTile - 1)) tile(std::true_type{});
        else tile(std::false_type{});
        if (!ok) break;
        l += sum;
        tmem_wait_st();
        first = false;
      }
      fence_before();
      __syncwarp();
#ifdef SDCP_TEST_WAIT_EXPIRY
      // Test build only (the flag is never set in the library): every fourth CTA keeps the weights of its
      // first step to itself, so that the waits of its warps run out on purpose.
      if (lane == 0 && (blockIdx.x % 4 != 0 || used != 0)) mbar_arrive(&sh.p_full[x]);
#else
      if (lane == 0) mbar_arrive(&sh.p_full[x]);
#endif
    }
    // O of the pairs: by the block's own threads, all channels, or half of the channels by each group's
    used_other += (uint32_t)(two ? n_tiles : x == 0 ? n_tiles / 2 : (n_tiles + 1) / 2);
    if (ok && (two || x == 0 || n_tiles > 1)) wait(&sh.pv_done[x], (used - 1u) & 1u);
    if (ok && !two && (x == 1 || n_tiles > 1)) wait(&sh.pv_done[x ^ 1], (used_other - 1u) & 1u);
    if (!ok) break;
    fence_after();
    if (nm == kNoScore && l == 0.0f) nm = INFINITY;  // a sum of nothing
    float f0 = nm == INFINITY && l == 0.0f ? 0.0f : 1.0f, f1 = 0.0f, top = nm, all = l;
    if (!two) {
      sh.ml[halves & 1u][x][pair] = make_float2(nm, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.ml_full);
      if (!wait(&sh.ml_full, halves & 1u)) break;
      const float2 u = sh.ml[halves & 1u][0][pair], v = sh.ml[halves & 1u][1][pair];
      ++halves;
      top = fminf(u.x, v.x);
      auto factor = [&](const float2& w) { return w.x == INFINITY && w.y == 0.0f ? 0.0f : w.x == top ? 1.0f : ex2(top - w.x); };
      f0 = factor(u);
      f1 = factor(v);
      all = (f0 != 0.0f ? u.y * f0 : 0.0f) + (f1 != 0.0f ? v.y * f1 : 0.0f);
    }
    const int32_t g = it.g0 + at - (row - it.i0) * share;  // head of the cached head's
    const int64_t place = ((int64_t)it.row0 + row) * a.q_heads + (int64_t)it.kvh * share + g;
    const bool direct = it.whole && it.joined == 0;
    const float scale = direct ? __fdividef(1.0f, all) : 1.0f;
    const int64_t pairs_all = (a.s.total + a.s.B) * a.q_heads;
    Part<D>* const part = reinterpret_cast<Part<D>*>(a.parts) + it.slot;
    float* const to = it.whole ? a.acc + ((it.joined == 1 ? 0 : pairs_all) + place) * D : part->o[at];
    if (live && !direct && (two || x == 0)) {
      if (it.whole) {
        a.acc_ml[(it.joined == 1 ? 0 : pairs_all) + place] = make_float2(-top, all);
      } else {
        part->m[at] = -top;
        part->l[at] = all;
      }
    }
    const uint32_t o0 = two ? o_at : lanes + kTmemO, o1 = lanes + kTmemO + (uint32_t)D;
    const int c0 = two ? 0 : x * (D / 2), c1 = two ? D : c0 + D / 2;
#pragma unroll 1
    for (int c = c0; c < c1; c += 16) {
      float o[16], w[16];
      tmem_ld16(o0 + (uint32_t)c, o);
      if (!two) tmem_ld16(o1 + (uint32_t)c, w);
      tmem_loaded(o);
      if (!two) tmem_loaded(w);
      if (live) {
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          o[y] = f0 != 0.0f ? o[y] * f0 : 0.0f;
          if (!two && f1 != 0.0f) o[y] += w[y] * f1;
          o[y] *= scale;
        }
        if (direct) {
          uint32_t b[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * y], o[2 * y + 1]);
            b[y] = *reinterpret_cast<const uint32_t*>(&h);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) reinterpret_cast<uint4*>(a.out + place * D + c)[y] = make_uint4(b[4 * y], b[4 * y + 1], b[4 * y + 2], b[4 * y + 3]);
        } else {
#pragma unroll
          for (int y = 0; y < 4; ++y) reinterpret_cast<float4*>(to + c)[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
        }
      }
      __syncwarp();
    }
    fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.o_free);
  }
  if (!ok) sh.dead = 1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attend_shared_kernel(const SharedArgs a) {
  using Sm = SharedSmem<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const s_q = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* const s_k = s_q + 2 * Sm::kBlock;
  unsigned char* const s_v = s_k + 2 * Sm::kBlock;
  __shared__ SharedState sh;

  const int tid = (int)threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int32_t cta = (int32_t)blockIdx.x, entries = a.groups + a.s.B;
  wait_for_previous();

  // this CTA's part of the line: a prefix sum over the entries, a stretch of them per thread
  const int32_t per = (entries + kThreads - 1) / kThreads;
  const int32_t e0 = min(tid * per, entries), e1 = min(e0 + per, entries);
  long long mine = 0;
  for (int32_t e = e0; e < e1; ++e) mine += a.units[e];
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
  for (int w = 0; w < kThreads / 32; ++w) {
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
    int32_t e = e0;
    while (here >= at + a.units[e]) at += a.units[e++];
    sh.entry = e;
    sh.base = at;
  }
  if (warp == kProductWarp) tmem_alloc(&sh.tmem, kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_free[i], 16);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_free[i], 1);
      mbar_init(&sh.k_full[i], 4);
      mbar_init(&sh.k_free[i], 1);
      mbar_init(&sh.v_full[i], 4);
      mbar_init(&sh.v_free[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.pv_done[i], 1);
    }
    mbar_init(&sh.o_free, 8);
    mbar_init(&sh.ml_full, 8);
    mbar_init(&sh.drained, 1);
    fence_barrier_init();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem, 0);
  if (warp >= kValueWarp) {
    turn<D, true>(a, sh, s_q, s_v);
  } else if (warp >= kKeyWarp) {
    turn<D, false>(a, sh, s_q, s_k);
  } else if (warp >= kSoftWarp) {
    soften<D>(a, sh, (warp - kSoftWarp) >> 2, tmem);
  } else {
    if (warp == kProductWarp) {
      Walk walk;
      walk.begin(a, line, sh.entry, sh.base);
      multiply<D>(a, sh, line, walk, s_q, s_k, s_v, tmem);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == kProductWarp) tmem_free(tmem, kTmemCols);
  if (tid == 0 && sh.dead) atomicOr(&a.header->error, 1u);
}

// ---- the joining of parts -----------------------------------------------------------------
// First the parts of items that were cut, then the two parts of pairs that have a group's and a session's.
// Four channels a lane, so a pair is a warp's, or half of one's.
constexpr int kJoinThreads = 128;
constexpr int kJoinAhead = 4;  // parts, or pairs, that a warp has in flight

// How much of a pair's sum a part with this reference and sum holds: 0 where it holds nothing of the pair.
__device__ __forceinline__ float factor_of(const float2& w, float m) { return w.x != -INFINITY || w.y != 0.0f ? (w.x == m ? 1.0f : ex2(w.x - m)) : 0.0f; }
__device__ __forceinline__ void store_bf16(__nv_bfloat16* to, float x, float y, float z, float w) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x, y), hi = __floats2bfloat162_rn(z, w);
  *reinterpret_cast<uint2*>(to) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// A CTA's last item and a pair of it: the sum of the parts, in the line's order, to where a whole item's would be.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) shared_cuts_kernel(const SharedArgs a) {
  constexpr int kLanes = D / 4, kOnce = 32 / kLanes;
  const int lane = (int)(threadIdx.x & 31u), own = lane / kLanes, sub = lane % kLanes;
  const int32_t id = (int32_t)(blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5)) * kOnce + own, cta = id / kMostPairs, j = id % kMostPairs;
  let_next_start();
  wait_for_previous();
  if (cta >= a.ctas || a.header->error != 0u) return;
  const Cut cut = a.cuts[cta];
  if (j - own >= cut.n) return;  // (a warp's pairs are of one item)
  const bool live = j < cut.n;
  const Part<D>* const parts = reinterpret_cast<const Part<D>*>(a.parts);
  const int32_t n = cut.last - cta + 1;
  auto part = [&](int32_t x) -> const Part<D>& { return parts[x == 0 ? cut.first_slot : 2 * (cta + x)]; };
  auto state = [&](int32_t x) { return x < n && live ? make_float2(part(x).m[j], part(x).l[j]) : make_float2(-INFINITY, 0.0f); };
  auto over_pair = [&](float v, auto op) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  };
  float2 w = state(sub);
  float m = w.x;
  for (int32_t x = sub + kLanes; x < n; x += kLanes) m = fmaxf(m, state(x).x);
  m = over_pair(m, [](float x, float y) { return fmaxf(x, y); });
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float sum = 0.0f;
  for (int32_t x0 = 0; x0 < n; x0 += kLanes) {
    if (x0 > 0) w = state(x0 + sub);
    const float f = factor_of(w, m);
    if (f != 0.0f) sum += w.y * f;
    const int32_t here = min(kLanes, n - x0);
    for (int32_t x = 0; x < here; x += kJoinAhead) {
      float4 v[kJoinAhead];
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u)
        if (x + u < here && live) v[u] = *reinterpret_cast<const float4*>(&part(x0 + x + u).o[j][sub * 4]);
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u) {
        const float fx = __shfl_sync(0xFFFFFFFFu, f, own * kLanes + ((x + u) & (kLanes - 1)));
        if (x + u < here && fx != 0.0f) {  // (an O that was not written has no weight)
          o.x += v[u].x * fx;
          o.y += v[u].y * fx;
          o.z += v[u].z * fx;
          o.w += v[u].w * fx;
        }
      }
    }
  }
  sum = over_pair(sum, [](float x, float y) { return x + y; });
  if (!live) return;
  const int32_t share = a.q_heads / a.kv.heads, r = (cut.g0 + j) / share;
  const int64_t place = ((int64_t)cut.row + r) * a.q_heads + cut.head + (cut.g0 + j - r * share);
  if (cut.joined == 0) {
    store_bf16(a.out + place * D + sub * 4, __fdividef(o.x, sum), __fdividef(o.y, sum), __fdividef(o.z, sum), __fdividef(o.w, sum));
  } else {
    const int64_t to = (cut.joined == 1 ? 0 : (a.s.total + a.s.B) * a.q_heads) + place;
    *reinterpret_cast<float4*>(a.acc + to * D + sub * 4) = o;
    if (sub == 0) a.acc_ml[to] = make_float2(m, sum);
  }
}

// The pairs that have two parts; a warp asks for those of a few pairs at once.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const SharedArgs a, int32_t steps) {
  constexpr int kLanes = D / 4, kOnce = 32 / kLanes;
  const int lane = (int)(threadIdx.x & 31u), own = lane / kLanes, c = lane % kLanes * 4;
  const int64_t warp = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5), pairs_all = (a.s.total + a.s.B) * a.q_heads;
  wait_for_previous();
  if (a.header->error != 0u) {
    for (int64_t b = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; b < a.s.B; b += (int64_t)gridDim.x * kJoinThreads)
      a.status[b] = SDCP_S_INTERNAL;
    return;
  }
  const int64_t first = warp * steps * kOnce + own;
  float2 w[kJoinAhead][2];
  float4 v[kJoinAhead][2];
#pragma unroll
  for (int u = 0; u < kJoinAhead; ++u) {
    const int64_t pair = first + u * kOnce;
    const bool some = u < steps && pair < pairs_all;
    w[u][1] = some ? a.acc_ml[pairs_all + pair] : make_float2(0.0f, kDone);
    w[u][0] = some ? a.acc_ml[pair] : make_float2(0.0f, 0.0f);
    if (some) {  // (asked for before it is known whether they are there)
      v[u][1] = *reinterpret_cast<const float4*>(a.acc + (pairs_all + pair) * D + c);
      v[u][0] = *reinterpret_cast<const float4*>(a.acc + pair * D + c);
    }
  }
#pragma unroll
  for (int u = 0; u < kJoinAhead; ++u) {
    if (w[u][1].y == kDone) continue;
    const float m = fmaxf(w[u][0].x, w[u][1].x), f0 = factor_of(w[u][0], m), f1 = factor_of(w[u][1], m);
    const float sum = (f0 != 0.0f ? w[u][0].y * f0 : 0.0f) + (f1 != 0.0f ? w[u][1].y * f1 : 0.0f);
    auto both = [&](float x, float y) { return __fdividef((f0 != 0.0f ? x * f0 : 0.0f) + (f1 != 0.0f ? y * f1 : 0.0f), sum); };
    store_bf16(a.out + (first + u * kOnce) * D + c, both(v[u][0].x, v[u][1].x), both(v[u][0].y, v[u][1].y), both(v[u][0].z, v[u][1].z),
               both(v[u][0].w, v[u][1].w));
  }
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// The workspace, piece by piece.
struct Layout {
  size_t group_status, lead, common, entries, units, cuts, parts, acc, acc_ml, bytes;
  Layout(int64_t B, int64_t total, int64_t groups, int64_t q_heads, int64_t dim) {
    size_t at = 256;  // the header
    auto take = [&](size_t n) {
      const size_t here = at;
      at += round256(n);
      return here;
    };
    const size_t pairs = (size_t)(total + B) * (size_t)q_heads;
    group_status = take((size_t)groups * 4);
    lead = take((size_t)B * 4);
    common = take((size_t)B * 4);
    entries = take((size_t)(groups + B) * sizeof(Entry));
    units = take((size_t)(groups + B) * 8);
    cuts = take(kMaxSms * sizeof(Cut));
    parts = take((size_t)kMaxSms * 2 * (dim == 128 ? sizeof(Part<128>) : sizeof(Part<64>)));
    acc = take(pairs * 2 * (size_t)dim * 4);
    acc_ml = take(pairs * 2 * 8);
    bytes = at;
  }
};

// Once per device: the kernels' dynamic shared memory.
constexpr int kMaxDevices = 64;
struct SharedDevice {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
SharedDevice g_shared_device[kMaxDevices];
template <int D> void set_shared(cudaError_t* e) {
  if (*e == cudaSuccess)
    *e = cudaFuncSetAttribute(attend_shared_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SharedSmem<D>::kBytes);
}
bool shared_ready() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  SharedDevice& d = g_shared_device[dev];
  std::call_once(d.once, [&] {
    set_shared<64>(&d.err);
    set_shared<128>(&d.err);
  });
  return d.err == cudaSuccess;
}

template <int D> cudaError_t launch_shared(const SharedArgs& a, cudaStream_t st) {
  cudaError_t e = launch_offsets_check(a.s.offsets, a.s.B, a.status, st);
  if (e != cudaSuccess) return e;
  if (a.group_offsets != nullptr) e = launch_offsets_check(a.group_offsets, a.groups, a.group_status, st);
  if (e != cudaSuccess) return e;
  const bool kernel_before = a.s.B > kScanSessions || a.groups > kScanSessions;
  // (blocks beyond the sessions help to mark the pairs)
  const int64_t marks = ((a.s.total + a.s.B) * a.q_heads + 8 * kCheckThreads - 1) / (8 * kCheckThreads);
  const unsigned blocks = (unsigned)max((int64_t)a.s.B, min(marks, (int64_t)2 * kMaxSms));
  e = launch_after_if(kernel_before, shared_check_kernel, blocks, kCheckThreads, 0, st, a);
  if (e != cudaSuccess) return e;
  e = launch_after(shared_plan_kernel, (unsigned)a.groups, kCheckThreads, 0, st, a);
  if (e != cudaSuccess) return e;
  e = launch_after(attend_shared_kernel<D>, (unsigned)a.ctas, kThreads, SharedSmem<D>::kBytes, st, a);
  if (e != cudaSuccess) return e;
  e = launch_after(shared_cuts_kernel<D>, (unsigned)(a.ctas * kMostPairs / (32 / (D / 4)) / (kJoinThreads / 32)), kJoinThreads, 0, st, a);
  if (e != cudaSuccess) return e;
  // Many pairs: a few a warp; few are spread over the warps that there are.
  const int64_t pairs = (a.s.total + a.s.B) * a.q_heads, once = 32 / (D / 4), per = kJoinThreads / 32;
  const int32_t steps = pairs > kFewPairs ? kJoinAhead : 1;
  const int64_t warps = (pairs + once * steps - 1) / (once * steps);
  return launch_after(shared_join_kernel<D>, (unsigned)((warps + per - 1) / per), kJoinThreads, 0, st, a, steps);
}

}  // namespace
}  // namespace sdcp

using namespace sdcp;

extern "C" size_t sdcp_attend_shared_workspace_bytes(int32_t B, int64_t total_drafts, int32_t n_groups, int32_t q_heads, int32_t kv_heads,
                                                     int32_t head_dim) {
  if (B < 0 || total_drafts < 0 || n_groups < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  if (total_drafts > (int64_t)INT32_MAX / 2 - B || q_heads > (1 << 20) || (total_drafts + B) * q_heads > (int64_t)INT32_MAX) return 0;
  if ((int64_t)n_groups + B > kMostEntries) return 0;
  return Layout(B, total_drafts, n_groups > 0 ? n_groups : 1, q_heads, head_dim).bytes;
}

extern "C" int sdcp_attend_shared_kv(const sdcp_kv_cache* cache, int32_t B, const int32_t* m_offsets, int64_t total_drafts, const int32_t* kv_len,
                                     int32_t n_groups, const int32_t* group_offsets, const void* q, int64_t q_stride, int32_t q_heads, float scale,
                                     void* out, int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  KvView kv;
  const int rc = kv_view(cache, &kv);
  if (rc != SDCP_OK) return rc;
  const int32_t D = cache->head_dim;
  if (B < 0 || total_drafts < 0 || n_groups < 0 || q_heads < 1 || q_heads % cache->kv_heads != 0 || !isfinite(scale)) return SDCP_E_INVALID;
  const size_t need = sdcp_attend_shared_workspace_bytes(B, total_drafts, n_groups, q_heads, cache->kv_heads, D);
  if (need == 0) return SDCP_E_TOO_LARGE;
  if (B == 0) return SDCP_OK;
  if (!m_offsets || !kv_len || !q || !out || !status || (n_groups > 0) != (group_offsets != nullptr)) return SDCP_E_INVALID;
  if (q_stride < (int64_t)q_heads * D) return SDCP_E_INVALID;
  if (((uintptr_t)q & 15u) != 0 || ((uintptr_t)out & 15u) != 0 || q_stride % 8 != 0) return SDCP_E_ALIGN;
  if (!on_words(m_offsets, kv_len, group_offsets, status)) return SDCP_E_ALIGN;
  if (!workspace || ((uintptr_t)workspace & 255u) != 0 || workspace_bytes < need) return SDCP_E_WORKSPACE;
  DeviceInfo di;
  if (!device_info(&di) || !shared_ready()) return SDCP_E_DEVICE;
  const int32_t groups = n_groups > 0 ? n_groups : 1;
  char* const w = static_cast<char*>(workspace);
  const Layout at(B, total_drafts, groups, q_heads, D);
  const KvSessions s{B, m_offsets, total_drafts, 1, kv_len, 0, INT32_MAX};
  const SharedArgs a{kv, s, group_offsets, groups, static_cast<const __nv_bfloat16*>(q), q_stride, q_heads, scale * 1.4426950408889634f,
                     static_cast<__nv_bfloat16*>(out), status, D, min(di.sms, kMaxSms), reinterpret_cast<Header*>(w),
                     reinterpret_cast<int32_t*>(w + at.group_status), reinterpret_cast<int32_t*>(w + at.lead), reinterpret_cast<int32_t*>(w + at.common),
                     reinterpret_cast<Entry*>(w + at.entries), reinterpret_cast<int64_t*>(w + at.units), reinterpret_cast<Cut*>(w + at.cuts),
                     reinterpret_cast<float*>(w + at.parts), reinterpret_cast<float*>(w + at.acc),
                     reinterpret_cast<float2*>(w + at.acc_ml)};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 128 ? launch_shared<128>(a, st) : launch_shared<64>(a, st);
  return e == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}
