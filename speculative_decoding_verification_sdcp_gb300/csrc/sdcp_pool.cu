// sdcp_pool.cu - the pages of the 4-bit cache between rounds: sdcp_fork_kv, sdcp_reserve_kv,
// sdcp_release_kv, sdcp_compact_kv (page tables and counts, once for all layers) and sdcp_copy_pages
// (the bytes, for each layer's cache).
//
// A pool is three arrays: a slot's row of the page table, the pages it holds, and for each page the
// number of rows that hold it (0: free).  There is no list of free pages to keep in step with the
// counts: a call that takes pages looks the counts over (4 bytes a page, 0.5 MB for 128 Ki pages), which
// is a small part of a launch's time, and always takes the lowest ones, so results depend on the state
// alone.  Counts change by integer atomics, whose order does not matter.
#include <climits>

#include "sdcp_kv.cuh"

namespace sdcp {
namespace {

// The pool as the kernels see it (checked on the host by pool_view).
struct PoolView {
  int32_t* table;  // [slots][max_pages]
  int32_t* held;   // [slots]
  int32_t* refs;   // [n_pages]
  int32_t n_pages, slots, max_pages, log_page;

  __device__ __forceinline__ int64_t pages_of(int64_t tokens) const { return (tokens + (1 << log_page) - 1) >> log_page; }
  __device__ __forceinline__ int32_t* row(int32_t b) const { return table + (int64_t)b * max_pages; }
  __device__ __forceinline__ bool inside(int32_t page) const { return page >= 0 && page < n_pages; }
  __device__ __forceinline__ bool holds(int32_t h) const { return h >= 0 && h <= max_pages; }
};

constexpr int32_t kMostEntries = 1 << 30;  // pages, slots and copies: indices stay in 32 bits beyond a loop's last step

int pool_view(const sdcp_kv_pool* p, PoolView* out) {
  if (!p || p->struct_size < sizeof(sdcp_kv_pool)) return SDCP_E_INVALID;
  if (p->page_tokens < 16 || p->page_tokens > 1024 || (p->page_tokens & (p->page_tokens - 1)) != 0) return SDCP_E_INVALID;
  if (p->n_pages < 1 || p->n_slots < 0 || p->max_pages < 1) return SDCP_E_INVALID;
  if (p->n_slots > 0 && (!p->page_table || !p->held)) return SDCP_E_INVALID;
  if (!p->refs) return SDCP_E_INVALID;
  if ((int64_t)p->max_pages * p->page_tokens > (int64_t)INT32_MAX || p->n_pages > kMostEntries || p->n_slots > kMostEntries) return SDCP_E_TOO_LARGE;
  if (!on_words(p->page_table, p->held, p->refs)) return SDCP_E_ALIGN;
  int log_page = 0;
  while ((1 << log_page) < p->page_tokens) ++log_page;
  *out = PoolView{p->page_table, p->held, p->refs, p->n_pages, p->n_slots, p->max_pages, log_page};
  return SDCP_OK;
}

// ---- rows: fork, release, the new places after a compaction -----------------------------
// A block a slot, bound by latency: a chain of four loads, then the row's entries, kEntries of them a thread
// in flight.  The block is as large as the longest row that the pool allows can use.  (192 rows of 8 .. 129
// entries forked: 4.8 us; 63 rows of 7000 entries given back: 8.5 us, 7 MB; both with cold caches.)
constexpr int kEntries = 8;
int row_threads(int32_t max_pages) {
  int t = 128;
  while (t < 1024 && t * kEntries < max_pages) t *= 2;
  return t;
}

__global__ void __launch_bounds__(1024) fork_kernel(const PoolView p, const int32_t* __restrict__ parent, const int32_t* __restrict__ length,
                                                    int32_t* status) {
  const int32_t b = (int32_t)blockIdx.x, a = parent[b];
  auto say = [&](int32_t st) {
    if (threadIdx.x == 0) status[b] = st;
  };
  if (a == -1) return say(SDCP_S_OK);
  // a parent that is itself forked in this call has no pages yet
  if (a < -1 || a >= p.slots || parent[a] != -1 || p.held[b] != 0) return say(SDCP_S_BAD_PARAMS);
  const int32_t h = p.held[a], len = length[b];
  if (!p.holds(h) || len < 0) return say(SDCP_S_BAD_PARAMS);
  const int32_t n = (int32_t)p.pages_of(len);
  if (n > h) return say(SDCP_S_LIMIT);
  const int32_t* const from = p.row(a);
  int32_t* const to = p.row(b);
  bool bad = false;
  int32_t e[kEntries];
  auto load = [&](int32_t i0) {
#pragma unroll
    for (int k = 0; k < kEntries; ++k) {
      const int32_t i = i0 + k * (int32_t)blockDim.x;
      e[k] = i < n ? from[i] : 0;
    }
#pragma unroll
    for (int k = 0; k < kEntries; ++k) bad |= !p.inside(e[k]);
  };
  const int32_t step = (int32_t)blockDim.x * kEntries, last = n > 0 ? (n - 1) / step * step : 0;
  for (int32_t i0 = (int32_t)threadIdx.x; i0 < n; i0 += step) load(i0);
  if (__syncthreads_or(bad)) return say(SDCP_S_BAD_PARAMS);
  for (int32_t i0 = (int32_t)threadIdx.x; i0 < n; i0 += step) {
    if (last > 0) load(i0);  // (a row of one step is still at hand)
#pragma unroll
    for (int k = 0; k < kEntries; ++k) {
      const int32_t i = i0 + k * (int32_t)blockDim.x;
      if (i < n) {
        to[i] = e[k];
        atomicAdd(&p.refs[e[k]], 1);
      }
    }
  }
  if (threadIdx.x == 0) p.held[b] = n;
  say(SDCP_S_OK);
}

__global__ void __launch_bounds__(1024) release_kernel(const PoolView p, const int32_t* __restrict__ keep, int32_t* status) {
  const int32_t b = (int32_t)blockIdx.x, tokens = keep[b], h = p.held[b];
  auto say = [&](int32_t st) {
    if (threadIdx.x == 0) status[b] = st;
  };
  if (tokens < 0) return say(SDCP_S_OK);
  if (!p.holds(h)) return say(SDCP_S_BAD_PARAMS);
  const int32_t n = (int32_t)min(p.pages_of(tokens), (int64_t)h);
  int32_t* const row = p.row(b);
  bool bad = false;
  int32_t e[kEntries];
  auto load = [&](int32_t i0) {
#pragma unroll
    for (int k = 0; k < kEntries; ++k) {
      const int32_t i = i0 + k * (int32_t)blockDim.x;
      e[k] = i < h ? row[i] : 0;
    }
#pragma unroll
    for (int k = 0; k < kEntries; ++k) bad |= !p.inside(e[k]);
  };
  const int32_t step = (int32_t)blockDim.x * kEntries;
  for (int32_t i0 = n + (int32_t)threadIdx.x; i0 < h; i0 += step) load(i0);
  if (__syncthreads_or(bad)) return say(SDCP_S_BAD_PARAMS);
  for (int32_t i0 = n + (int32_t)threadIdx.x; i0 < h; i0 += step) {
    if (h - n > step) load(i0);
#pragma unroll
    for (int k = 0; k < kEntries; ++k) {
      const int32_t i = i0 + k * (int32_t)blockDim.x;
      if (i < h) {
        row[i] = -1;
        atomicSub(&p.refs[e[k]], 1);
      }
    }
  }
  if (threadIdx.x == 0) p.held[b] = n;
  say(SDCP_S_OK);
}

__global__ void __launch_bounds__(1024) renumber_kernel(const PoolView p, const int32_t* n_live, const int32_t* to) {
  wait_for_previous();
  const int32_t b = (int32_t)blockIdx.x, h = min(p.held[b], p.max_pages), live = *n_live;
  int32_t* const row = p.row(b);
#pragma unroll kEntries
  for (int32_t i = (int32_t)threadIdx.x; i < h; i += (int32_t)blockDim.x) {
    const int32_t e = row[i];
    if (e >= live && e < p.n_pages) row[i] = to[e];
  }
}

// ---- a cluster over the slots and the pages: reserve, compact ----------------------------
// What a call takes depends on all slots before and all pages below, so one cluster does it: each of its
// blocks has a stretch of the slots and one of the pages, and a few sums are exchanged between its
// barriers.  (Kernels of their own for the steps would cost a launch each.)
constexpr int kMostBlocks = 8;
// One block where it has a thread for each slot and few pages to look over (no barrier beyond its own): pages
// reserved for 10 slots and for 258 of a pool of 5400 pages, 9.5 and 11.5 us with one block, 13 and 15 with
// eight; a pool of 12000 pages compacted, 10 us with one, 7 with eight.
constexpr int32_t kFewPages = 1 << 13;
constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;

template <int kBlocks> __device__ __forceinline__ void cluster_meet() {
  if (kBlocks == 1) {
    __syncthreads();
    return;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// x of block `rank` of the cluster
__device__ __forceinline__ long long of_block(const long long* x, int rank) {
  uint32_t at;
  long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(x)), "r"(rank));
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}
// The sums of x over the blocks before this one, and over all.
template <int kBlocks> __device__ __forceinline__ void over_blocks(const long long* x, int rank, long long* before, long long* all) {
  *before = *all = 0;
#pragma unroll
  for (int r = 0; r < kBlocks; ++r) {
    const long long v = kBlocks == 1 ? *x : of_block(x, r);
    if (r < rank) *before += v;
    *all += v;
  }
}
// Exclusive scan over the block; *total: the sum.  scratch: kPoolWarps entries.
__device__ __forceinline__ long long block_scan(long long v, long long* scratch, long long* total) {
  return group_excl_scan_ll(Group{kPoolThreads, 1}, v, scratch, total);
}

// A block's stretch of n things, and a warp's of those (a multiple of 32, so that its loads are whole lines).
struct Stretch {
  int32_t begin, end;
};
__device__ __forceinline__ Stretch part_of(int64_t n, int32_t part, int32_t parts, int32_t unit) {
  const int64_t each = ((n + parts - 1) / parts + unit - 1) / unit * unit;
  return Stretch{(int32_t)min(n, part * each), (int32_t)min(n, (part + 1) * each)};
}
template <int kBlocks> __device__ __forceinline__ Stretch warp_pages(const PoolView& p, int rank, int warp) {
  return part_of(p.n_pages, rank * kPoolWarps + warp, kBlocks * kPoolWarps, 32);
}
constexpr int kPagesAhead = 8;  // loads of a lane in flight
// The number of a warp's pages that `which` holds for.
template <typename F> __device__ __forceinline__ int32_t count_pages(const PoolView& p, const Stretch& s, F which) {
  const int lane = (int)(threadIdx.x & 31u);
  int32_t n = 0;
  for (int32_t i0 = s.begin; i0 < s.end; i0 += 32 * kPagesAhead) {
    int32_t r[kPagesAhead];
#pragma unroll
    for (int k = 0; k < kPagesAhead; ++k) r[k] = i0 + k * 32 + lane < s.end ? p.refs[i0 + k * 32 + lane] : INT_MIN;
#pragma unroll
    for (int k = 0; k < kPagesAhead; ++k) n += which(r[k]);
  }
  return (int32_t)__reduce_add_sync(0xFFFFFFFFu, (unsigned)n);
}

struct ReserveArgs {
  PoolView p;
  const int32_t *kv_len, *upto;
  int4* copies;
  int32_t* n_copies;
  int32_t* status;
  long long* start;     // [slots] place of a slot's first new page among all taken; < 0: none for it
  int32_t* replaced;    // [slots] how many of its held pages are replaced
  int32_t* free_pages;  // [n_pages] the lowest free pages, as many as are taken
  int32_t* dropped;     // [n_pages] for each page taken: the shared one that it replaces, or -1
};

// What a slot needs: of the entries [first, end), those in [first, mid) are held, and shared ones of them
// are replaced; those in [fresh, end) are new.
struct Need {
  int32_t first, mid, fresh, end;
  __device__ __forceinline__ int32_t n_fresh() const { return end - fresh; }
};
__device__ __forceinline__ int32_t slot_need(const PoolView& p, int32_t kv_len, int32_t upto, int32_t held, Need* n) {
  *n = Need{0, 0, 0, 0};
  if (upto <= kv_len) return SDCP_S_OK;
  if (kv_len < 0 || !p.holds(held) || p.pages_of(kv_len) > held) return SDCP_S_BAD_PARAMS;
  const int64_t end = p.pages_of(upto);
  if (end > p.max_pages) return SDCP_S_LIMIT;
  n->first = kv_len >> p.log_page;
  n->end = (int32_t)end;
  n->mid = max(n->first, min(held, n->end));
  n->fresh = max(n->first, min(max(held, n->first), n->end));
  return SDCP_S_OK;
}
constexpr int32_t kAlone = 8;  // entries that a thread does by itself; rows with more are the block's

// What a thread knows of its slot, from one barrier of the cluster to the next.
struct SlotState {
  Need n;
  int32_t kv_len, held;
  int32_t shared;    // how many of [first, mid) are shared, and which, where the thread does them by itself
  uint32_t which;
  int32_t status;
  long long place;   // of its first new page; < 0: none for it
  __device__ __forceinline__ bool alone() const { return n.mid - n.first <= kAlone && n.n_fresh() <= kAlone; }
};

// Bound by latency: three chains of loads (a slot's numbers, its entries, their counts; then the free pages)
// between barriers of the cluster.  What a slot needs is kept in registers from one to the next where a
// block has a thread for each of its slots (258 slots: 18.5 to 15 us, cold, with eight blocks).
template <int kCluster> __global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPoolThreads) reserve_kernel(const ReserveArgs a) {
  const PoolView& p = a.p;
  __shared__ long long scratch[kPoolWarps];
  __shared__ long long sum_need, sum_free, sum_taken, sum_copies, sum_long;
  __shared__ int32_t long_slots[kPoolThreads], found[kPoolThreads];
  __shared__ int32_t n_long, any_long, warp_free[kPoolWarps];
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)blockIdx.x;
  const Stretch mine = part_of(p.slots, rank, kCluster, 1), pages = warp_pages<kCluster>(p, rank, warp);
  const bool once = p.slots <= kCluster * kPoolThreads;  // a thread a slot
  const int32_t in_page = (1 << p.log_page) - 1;
  SlotState s;
  // the slot's numbers; the entries that it has to look at are counted apart
  auto look = [&](int32_t b) {
    s = SlotState{Need{0, 0, 0, 0}, 0, 0, 0, 0u, SDCP_S_OK, -1};
    if (b >= mine.end) return;
    s.kv_len = a.kv_len[b];
    s.held = p.held[b];
    s.status = slot_need(p, s.kv_len, a.upto[b], s.held, &s.n);
  };
  if (tid == 0) any_long = 0;

  // free pages, and the pages that each slot needs
  const int32_t n_free = count_pages(p, pages, [](int32_t r) { return r == 0 ? 1 : 0; });
  if (lane == 0) warp_free[warp] = n_free;
  long long carry = 0;
  for (int32_t b0 = mine.begin; b0 < mine.end; b0 += kPoolThreads) {
    const int32_t b = b0 + tid;
    look(b);
    if (tid == 0) n_long = 0;
    __syncthreads();
    if (s.n.mid - s.n.first <= kAlone) {
      for (int32_t i = s.n.first; i < s.n.mid; ++i) {
        const int32_t e = p.row(b)[i];
        if (!p.inside(e)) s.status = SDCP_S_BAD_PARAMS;
        else if (p.refs[e] > 1) s.which |= 1u << (i - s.n.first);
      }
      s.shared = __popc(s.which);
    } else {
      long_slots[atomicAdd(&n_long, 1)] = tid;
    }
    if (!s.alone()) any_long = 1;
    __syncthreads();
    for (int32_t k = 0; k < n_long; ++k) {  // one at a time by the block: the order does not matter
      const int32_t owner = long_slots[k], ob = b0 + owner;
      Need o;
      (void)slot_need(p, a.kv_len[ob], a.upto[ob], p.held[ob], &o);
      long long here = 0, all = 0;
      bool bad = false;
      for (int32_t i = o.first + tid; i < o.mid; i += kPoolThreads) {
        const int32_t e = p.row(ob)[i];
        if (!p.inside(e)) bad = true;
        else if (p.refs[e] > 1) ++here;
      }
      (void)block_scan(here, scratch, &all);
      bad = __syncthreads_or(bad) != 0;
      if (tid == 0) found[owner] = bad ? -1 : (int32_t)all;
      __syncthreads();
    }
    if (s.n.mid - s.n.first > kAlone) {
      s.shared = found[tid];
      if (s.shared < 0) s.status = SDCP_S_BAD_PARAMS;
    }
    const long long need = s.status == SDCP_S_OK ? (long long)s.shared + s.n.n_fresh() : 0;
    long long all = 0;
    const long long at = carry + block_scan(need, scratch, &all);
    carry += all;
    s.place = need > 0 ? at : -1;
    if (b < mine.end) {
      a.status[b] = s.status;
      if (!once) {
        a.start[b] = s.place;
        a.replaced[b] = s.shared;
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    sum_need = carry;
    sum_long = any_long;
    long long f = 0;
    for (int w = 0; w < kPoolWarps; ++w) f += warp_free[w];
    sum_free = f;
  }
  cluster_meet<kCluster>();

  // who gets them, how many copies there are before a slot's, and the free pages in order
  long long need_before, need_all, free_before, free_all, unused, long_all;
  over_blocks<kCluster>(&sum_need, rank, &need_before, &need_all);
  over_blocks<kCluster>(&sum_free, rank, &free_before, &free_all);
  over_blocks<kCluster>(&sum_long, rank, &unused, &long_all);
  constexpr int kCopyBits = 20;  // of a sum of both: the new pages above, the copies (at most one a thread) below
  long long taken_here = 0, copies_here = 0, copy_place = 0;
  for (int32_t b0 = mine.begin; b0 < mine.end; b0 += kPoolThreads) {
    const int32_t b = b0 + tid;
    if (!once) {
      look(b);
      if (b < mine.end) {
        s.place = a.start[b];
        s.shared = a.replaced[b];
      }
    }
    int copy = 0;
    long long taken = 0;
    if (b < mine.end && s.place >= 0) {
      taken = (long long)s.shared + s.n.n_fresh();
      s.place += need_before;
      if (s.place + taken > free_all) {
        a.status[b] = SDCP_S_LIMIT;
        s.place = -1;
        taken = 0;
      } else if (s.n.first < s.n.mid && (s.kv_len & in_page) != 0) {
        // the round's first page, if it holds tokens already and is shared
        copy = once && s.n.mid - s.n.first <= kAlone ? (int)(s.which & 1u) : p.refs[p.row(b)[s.n.first]] > 1;
      }
      a.start[b] = s.place;
    }
    long long all = 0;
    copy_place = block_scan(taken << kCopyBits | copy, scratch, &all) & ((1 << kCopyBits) - 1);
    taken_here += all >> kCopyBits;
    copies_here += all & ((1 << kCopyBits) - 1);
  }
  if (tid == 0) {
    sum_taken = taken_here;
    sum_copies = copies_here;
  }
  {
    long long at = free_before;
    for (int w = 0; w < warp; ++w) at += warp_free[w];
    const long long want = min(need_all, free_all);
    for (int32_t i0 = pages.begin; i0 < pages.end && at < want; i0 += 32) {
      const bool is = i0 + lane < pages.end && p.refs[i0 + lane] == 0;
      const unsigned who = __ballot_sync(0xFFFFFFFFu, is);
      const long long place = at + __popc(who & ((1u << lane) - 1u));
      if (is && place < want) a.free_pages[place] = i0 + lane;
      at += __popc(who);
    }
  }
  cluster_meet<kCluster>();

  // the pages into the rows
  long long copies_before, copies_all, taken_all;
  over_blocks<kCluster>(&sum_copies, rank, &copies_before, &copies_all);
  over_blocks<kCluster>(&sum_taken, rank, &unused, &taken_all);
  if (rank == 0 && tid == 0) *a.n_copies = (int32_t)copies_all;
  // Where each slot is a thread's alone, no count is looked at any more and a replaced page's goes down at once.
  // Else shared pages are still told by their counts, which change after the last barrier.
  const bool at_once = long_all == 0 && once;
  for (int32_t b0 = mine.begin; b0 < mine.end; b0 += kPoolThreads) {
    const int32_t b = b0 + tid;
    if (!once) {
      look(b);
      s.place = b < mine.end && s.status == SDCP_S_OK && s.n.first < s.n.end ? a.start[b] : -1;
    }
    if (tid == 0) n_long = 0;
    __syncthreads();
    auto replace = [&](int32_t ob, int32_t i, long long place) {  // entry i of slot ob by the page taken at `place`
      int32_t* const entry = p.row(ob) + i;
      const int32_t page = __ldcg(&a.free_pages[place]), old = *entry;
      *entry = page;
      p.refs[page] = 1;
      if (at_once) atomicSub(&p.refs[old], 1);
      else a.dropped[place] = old;
      return make_int2(old, page);
    };
    auto take = [&](int32_t ob, int32_t i, long long place) {
      const int32_t page = __ldcg(&a.free_pages[place]);
      p.row(ob)[i] = page;
      p.refs[page] = 1;
      if (!at_once) a.dropped[place] = -1;
    };
    auto is_shared = [&](int32_t i) { return once && s.n.mid - s.n.first <= kAlone ? (s.which >> (i - s.n.first) & 1u) != 0u : p.refs[p.row(b)[i]] > 1; };
    // the first page by the slot's own thread, whoever does the rest
    int4 record = make_int4(-1, -1, s.kv_len & in_page, 0);
    const bool first_done = s.place >= 0 && s.n.first < s.n.mid && record.z != 0 && is_shared(s.n.first);
    if (first_done) {
      const int2 r = replace(b, s.n.first, s.place);
      record.x = r.x;
      record.y = r.y;
    }
    if (s.place >= 0 && s.alone()) {
      long long place = s.place + (first_done ? 1 : 0);
      for (int32_t i = s.n.first + (first_done ? 1 : 0); i < s.n.mid; ++i)
        if (is_shared(i)) replace(b, i, place++);
      for (int32_t i = s.n.fresh; i < s.n.end; ++i) take(b, i, place++);
    } else if (s.place >= 0) {
      long_slots[atomicAdd(&n_long, 1)] = tid;
      found[tid] = first_done ? 1 : 0;
    }
    __syncthreads();
    for (int32_t k = 0; k < n_long; ++k) {
      const int32_t owner = long_slots[k], ob = b0 + owner, skip = found[owner];
      Need o;
      (void)slot_need(p, a.kv_len[ob], a.upto[ob], p.held[ob], &o);
      long long place = a.start[ob] + skip;
      for (int32_t i0 = o.first + skip; i0 < o.mid; i0 += kPoolThreads) {
        const int32_t i = i0 + tid;
        const bool is = i < o.mid && p.refs[p.row(ob)[i]] > 1;
        long long all = 0;
        const long long before = block_scan(is ? 1 : 0, scratch, &all);
        if (is) replace(ob, i, place + before);
        place += all;
      }
#pragma unroll 4
      for (int32_t i = o.fresh + tid; i < o.end; i += kPoolThreads) take(ob, i, place + (i - o.fresh));
    }
    if (!once) {
      long long all = 0;
      copy_place = block_scan(first_done ? 1 : 0, scratch, &all);
      if (first_done) a.copies[copies_before + copy_place] = record;
      copies_before += all;
    } else if (first_done) {
      a.copies[copies_before + copy_place] = record;
    }
    __syncthreads();  // rows are read by their held[] until here
    if (s.place >= 0) p.held[b] = max(s.held, s.n.end);
  }
  cluster_meet<kCluster>();

  // the replaced pages lose a holder
  if (at_once) return;
  for (long long i = (long long)rank * kPoolThreads + tid; i < taken_all; i += kCluster * kPoolThreads) {
    const int32_t old = __ldcg(&a.dropped[i]);
    if (old >= 0) atomicSub(&p.refs[old], 1);
  }
}

struct CompactArgs {
  PoolView p;
  int32_t* copies;  // [max_copies][4]
  int32_t max_copies;
  int32_t *n_copies, *n_live;
  int32_t* to;  // [n_pages] the new place of a page at or past n_live (its own, unless it is moved)
};

// With L pages live, a free page below L is hole number (page - live pages below it), and a live page at or
// past L is move number (live pages above it): move k goes to hole k.
template <int kCluster> __global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPoolThreads) compact_kernel(const CompactArgs a) {
  const PoolView& p = a.p;
  __shared__ long long sum_live;
  __shared__ int32_t warp_live[kPoolWarps];
  __shared__ int32_t n_moves;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)blockIdx.x;
  const Stretch pages = warp_pages<kCluster>(p, rank, warp);
  let_next_start();
  const int32_t n = count_pages(p, pages, [](int32_t r) { return r > 0 ? 1 : 0; });
  if (lane == 0) warp_live[warp] = n;
  __syncthreads();
  if (tid == 0) {
    long long s = 0;
    for (int w = 0; w < kPoolWarps; ++w) s += warp_live[w];
    sum_live = s;
  }
  cluster_meet<kCluster>();
  long long before, all;
  over_blocks<kCluster>(&sum_live, rank, &before, &all);
  const int32_t live = (int32_t)all;
  int32_t at = (int32_t)before;
  for (int w = 0; w < warp; ++w) at += warp_live[w];
  for (int32_t i0 = pages.begin; i0 < pages.end; i0 += 32 * kPagesAhead) {
    int32_t r[kPagesAhead];
#pragma unroll
    for (int k = 0; k < kPagesAhead; ++k) r[k] = i0 + k * 32 + lane < pages.end ? p.refs[i0 + k * 32 + lane] : INT_MIN;
#pragma unroll
    for (int k = 0; k < kPagesAhead; ++k) {
      const int32_t i = i0 + k * 32 + lane;
      const unsigned who = __ballot_sync(0xFFFFFFFFu, r[k] > 0);
      const int32_t below = at + __popc(who & ((1u << lane) - 1u));  // live pages before page i
      at += __popc(who);
      if (r[k] == INT_MIN && i >= pages.end) continue;
      if (i == live) *a.n_copies = min(live - below, a.max_copies);
      if (i >= live) a.to[i] = i;  // (free ones too: a row filled by hand may name one)
      if (i >= live && r[k] > 0) {
        const int32_t k_move = live - below - 1;
        if (k_move < a.max_copies) {
          a.copies[(int64_t)k_move * 4] = i;
          a.copies[(int64_t)k_move * 4 + 2] = 1 << p.log_page;
          a.copies[(int64_t)k_move * 4 + 3] = 0;
        }
      } else if (i < live && r[k] <= 0) {
        const int32_t hole = i - below;
        if (hole < a.max_copies) a.copies[(int64_t)hole * 4 + 1] = i;
      }
    }
  }
  if (rank == 0 && tid == 0) {
    *a.n_live = live;
    if (live == p.n_pages) *a.n_copies = 0;
  }
  cluster_meet<kCluster>();
  if (tid == 0) n_moves = __ldcg(a.n_copies);
  __syncthreads();
  for (int32_t k = rank * kPoolThreads + tid; k < n_moves; k += kCluster * kPoolThreads) {
    const int32_t from = __ldcg(&a.copies[(int64_t)k * 4]), hole = __ldcg(&a.copies[(int64_t)k * 4 + 1]);
    p.refs[hole] = __ldcg(&p.refs[from]);
    p.refs[from] = 0;
    a.to[from] = hole;
  }
}

// ---- copies -----------------------------------------------------------------------------
// A warp a block (one head's keys or values of a page), its 16-byte pieces in flight together.  Bound by memory:
// 2970 whole pages of 70 KB, 207 MB read and written, 60 us, 6.9 TB/s; 1300 parts of pages of 139 KB, 88 MB, 28 us.
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 8;

struct CopyArgs {
  uint8_t* pages;
  int64_t page;
  int32_t block, blocks;  // bytes of a block, blocks of a page
  int32_t n_pages, page_tokens, groups;
  const int4* copies;
  int32_t max_copies;
  const int32_t* n_copies;
  int32_t* status;
};

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs a) {
  const int lane = (int)(threadIdx.x & 31u);
  const int32_t n = *a.n_copies;
  auto good = [&](const int4& c) {
    return c.x >= 0 && c.x < a.n_pages && c.y >= 0 && c.y < a.n_pages && c.x != c.y && c.z >= 0 && c.z <= a.page_tokens;
  };
  const bool listed = n >= 0 && n <= a.max_copies;
  if (blockIdx.x == 0) {
    bool bad = !listed;
    for (int32_t i = (int32_t)threadIdx.x; listed && i < n; i += kCopyThreads) bad |= !good(a.copies[i]);
    bad = __syncthreads_or(bad) != 0;
    if (threadIdx.x == 0) *a.status = bad ? SDCP_S_BAD_PARAMS : SDCP_S_OK;
  }
  if (!listed) return;
  const int64_t units = (int64_t)n * a.blocks, warps = (int64_t)gridDim.x * (kCopyThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const int32_t i = (int32_t)(u / a.blocks);
    const int4 c = a.copies[i];
    if (!good(c)) continue;
    const int64_t in_page = (u - (int64_t)i * a.blocks) * a.block;
    const uint8_t* const from = a.pages + c.x * a.page + in_page;
    uint8_t* const to = a.pages + c.y * a.page + in_page;
    // a group's codes of c.z tokens, then the next group's; of a whole page the scales follow on
    const bool whole = c.z == a.page_tokens;
    const int32_t pieces = whole ? a.block / 16 : a.groups * c.z, skip = whole ? 0 : (a.page_tokens - c.z) * 16;
    for (int32_t j0 = lane; j0 < pieces; j0 += 32 * kCopyAhead) {
      uint4 v[kCopyAhead];
      int32_t at[kCopyAhead];
#pragma unroll
      for (int k = 0; k < kCopyAhead; ++k) {
        const int32_t j = j0 + k * 32;
        at[k] = j * 16 + (skip == 0 ? 0 : skip * ((j >= c.z) + (j >= 2 * c.z) + (j >= 3 * c.z)));
        if (j < pieces) v[k] = __ldcs(reinterpret_cast<const uint4*>(from + at[k]));
      }
#pragma unroll
      for (int k = 0; k < kCopyAhead; ++k)
        if (j0 + k * 32 < pieces) *reinterpret_cast<uint4*>(to + at[k]) = v[k];
    }
    if (!whole) {
      const int32_t scales = a.groups * a.page_tokens * 16, bytes = c.z * a.groups;  // groups is even
      for (int32_t j = lane * 2; j < bytes; j += 64)
        *reinterpret_cast<uint16_t*>(to + scales + j) = *reinterpret_cast<const uint16_t*>(from + scales + j);
    }
  }
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace
}  // namespace sdcp

using namespace sdcp;

extern "C" int sdcp_fork_kv(const sdcp_kv_pool* pool, const int32_t* parent, const int32_t* length, int32_t* status, void* stream) {
  PoolView p;
  const int rc = pool_view(pool, &p);
  if (rc != SDCP_OK) return rc;
  if (p.slots == 0) return SDCP_OK;
  if (!parent || !length || !status) return SDCP_E_INVALID;
  if (!on_words(parent, length, status)) return SDCP_E_ALIGN;
  DeviceInfo di;
  if (!device_info(&di)) return SDCP_E_DEVICE;
  fork_kernel<<<(unsigned)p.slots, row_threads(p.max_pages), 0, reinterpret_cast<cudaStream_t>(stream)>>>(p, parent, length, status);
  return cudaGetLastError() == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}

extern "C" int sdcp_release_kv(const sdcp_kv_pool* pool, const int32_t* keep, int32_t* status, void* stream) {
  PoolView p;
  const int rc = pool_view(pool, &p);
  if (rc != SDCP_OK) return rc;
  if (p.slots == 0) return SDCP_OK;
  if (!keep || !status) return SDCP_E_INVALID;
  if (!on_words(keep, status)) return SDCP_E_ALIGN;
  DeviceInfo di;
  if (!device_info(&di)) return SDCP_E_DEVICE;
  release_kernel<<<(unsigned)p.slots, row_threads(p.max_pages), 0, reinterpret_cast<cudaStream_t>(stream)>>>(p, keep, status);
  return cudaGetLastError() == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}

extern "C" size_t sdcp_pool_workspace_bytes(int32_t n_pages, int32_t n_slots) {
  if (n_pages < 1 || n_slots < 0 || n_pages > kMostEntries || n_slots > kMostEntries) return 0;
  return 2 * round256((size_t)n_pages * 4) + round256((size_t)n_slots * 8) + round256((size_t)n_slots * 4);
}

namespace {
int check_list(const PoolView& p, const sdcp_page_copy* copies, int32_t max_copies, const int32_t* n_copies, const void* workspace,
               size_t workspace_bytes) {
  if (max_copies < 0 || (max_copies > 0 && !copies) || !n_copies) return SDCP_E_INVALID;
  if (max_copies > kMostEntries) return SDCP_E_TOO_LARGE;
  if (((uintptr_t)copies & 15u) != 0 || !on_words(n_copies)) return SDCP_E_ALIGN;
  if (!workspace || ((uintptr_t)workspace & 255u) != 0 || workspace_bytes < sdcp_pool_workspace_bytes(p.n_pages, p.slots)) return SDCP_E_WORKSPACE;
  return SDCP_OK;
}
}  // namespace

extern "C" int sdcp_reserve_kv(const sdcp_kv_pool* pool, const int32_t* kv_len, const int32_t* upto, sdcp_page_copy* copies, int32_t max_copies,
                               int32_t* n_copies, int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  PoolView p;
  int rc = pool_view(pool, &p);
  if (rc == SDCP_OK) rc = check_list(p, copies, max_copies, n_copies, workspace, workspace_bytes);
  if (rc != SDCP_OK) return rc;
  if (max_copies < p.slots || (p.slots > 0 && (!kv_len || !upto || !status))) return SDCP_E_INVALID;
  if (!on_words(kv_len, upto, status)) return SDCP_E_ALIGN;
  DeviceInfo di;
  if (!device_info(&di)) return SDCP_E_DEVICE;
  char* w = static_cast<char*>(workspace);
  int32_t* const free_pages = reinterpret_cast<int32_t*>(w);
  w += round256((size_t)p.n_pages * 4);
  int32_t* const dropped = reinterpret_cast<int32_t*>(w);
  w += round256((size_t)p.n_pages * 4);
  long long* const start = reinterpret_cast<long long*>(w);
  w += round256((size_t)p.slots * 8);
  const ReserveArgs a{p, kv_len, upto, reinterpret_cast<int4*>(copies), n_copies, status, start, reinterpret_cast<int32_t*>(w), free_pages, dropped};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p.slots <= kPoolThreads && p.n_pages <= kFewPages) reserve_kernel<1><<<1, kPoolThreads, 0, st>>>(a);
  else reserve_kernel<kMostBlocks><<<kMostBlocks, kPoolThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}

extern "C" int sdcp_compact_kv(const sdcp_kv_pool* pool, sdcp_page_copy* copies, int32_t max_copies, int32_t* n_copies, int32_t* n_live,
                               void* workspace, size_t workspace_bytes, void* stream) {
  PoolView p;
  int rc = pool_view(pool, &p);
  if (rc == SDCP_OK) rc = check_list(p, copies, max_copies, n_copies, workspace, workspace_bytes);
  if (rc != SDCP_OK) return rc;
  if (!n_live) return SDCP_E_INVALID;
  if (!on_words(n_live)) return SDCP_E_ALIGN;
  DeviceInfo di;
  if (!device_info(&di)) return SDCP_E_DEVICE;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int32_t* const to = static_cast<int32_t*>(workspace);
  const CompactArgs a{p, reinterpret_cast<int32_t*>(copies), max_copies, n_copies, n_live, to};
  if (p.n_pages <= kFewPages) compact_kernel<1><<<1, kPoolThreads, 0, st>>>(a);
  else compact_kernel<kMostBlocks><<<kMostBlocks, kPoolThreads, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SDCP_E_LAUNCH;
  if (p.slots == 0) return SDCP_OK;
  return launch_after(renumber_kernel, (unsigned)p.slots, (unsigned)row_threads(p.max_pages), 0, st, p, (const int32_t*)n_live, (const int32_t*)to) == cudaSuccess
             ? SDCP_OK
             : SDCP_E_LAUNCH;
}

extern "C" int sdcp_copy_pages(const sdcp_kv_cache* cache, const sdcp_page_copy* copies, int32_t max_copies, const int32_t* n_copies,
                               int32_t* status, void* stream) {
  if (!cache || cache->struct_size < sizeof(sdcp_kv_cache)) return SDCP_E_INVALID;
  const size_t page = sdcp_kv_page_bytes(cache->page_tokens, cache->kv_heads, cache->head_dim);
  if (page == 0 || cache->n_pages < 1 || !cache->pages || max_copies < 0 || (max_copies > 0 && !copies) || !n_copies || !status) return SDCP_E_INVALID;
  if (max_copies > kMostEntries) return SDCP_E_TOO_LARGE;
  if (((uintptr_t)cache->pages & 15u) != 0 || ((uintptr_t)copies & 15u) != 0 || !on_words(n_copies, status)) return SDCP_E_ALIGN;
  DeviceInfo di;
  if (!device_info(&di)) return SDCP_E_DEVICE;
  const int32_t blocks = 2 * cache->kv_heads;
  const CopyArgs a{cache->pages, (int64_t)page, (int32_t)(page / (size_t)blocks), blocks, cache->n_pages, cache->page_tokens,
                   cache->head_dim / kKvGroup, reinterpret_cast<const int4*>(copies), max_copies, n_copies, status};
  const int64_t units = (int64_t)max_copies * blocks, per = kCopyThreads / 32;
  const int64_t grid = max((int64_t)1, min((units + per - 1) / per, (int64_t)di.sms * 8));
  copy_kernel<<<(unsigned)grid, kCopyThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}
