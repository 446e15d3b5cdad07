// sdcp_kv.cuh - the paged 4-bit cache of keys and values: geometry, the checks of its sessions,
// the lookup of a row's session, and the code that the cache kernels share.
#pragma once

#include "sdcp_device.cuh"

namespace sdcp {

constexpr int kKvGroup = 32;  // channels that share a scale

// The cache as the kernels see it (checked on the host by kv_view).
struct KvView {
  uint8_t* pages;
  const int32_t* page_table;
  int32_t n_pages;
  int32_t max_pages;
  int32_t heads;
  int32_t log_page;   // page_tokens = 1 << log_page
  int32_t block;      // bytes of one head's keys or values in a page
  int64_t page;       // bytes of a page

  __device__ __forceinline__ int32_t page_tokens() const { return 1 << log_page; }
};

// SDCP_OK and the view, or the error of an unusable description.
int kv_view(const sdcp_kv_cache* cache, KvView* out);

// How a call's sessions lie on the cache.
struct KvSessions {
  int32_t B;
  const int32_t* offsets;  // [B+1]
  int64_t total;           // offsets[B]
  int32_t extra;           // rows of a session beyond its offsets' difference (1: target rows)
  const int32_t* start;    // [B] position of a session's first row
  int32_t window;          // positions a row sees (0: from the start); -1: rows see themselves alone
  int32_t limit;           // positions below this only (the rotary table); INT32_MAX: none
};

// The status of session b, found by a whole block of kCheckThreads: the batch's offsets in order, its own
// in range, a start that is not negative, the last position inside the page table's row and the limit,
// every page that the rows touch inside the pool.  A kernel of one block a session writes status[] before
// the call's main kernel, which reads it.
constexpr int kCheckThreads = 128;
__device__ __forceinline__ int32_t kv_session_status(const KvView& kv, const KvSessions& s, int32_t b, const int32_t* status) {
  const int32_t lo = s.offsets[b], hi = s.offsets[b + 1], start = s.start[b];
  if (s.B > kScanSessions) wait_for_previous();  // (it writes status[] too)
  bool bad = s.B <= kScanSessions ? !offsets_in_order(s.offsets, s.B) : status[b] != SDCP_S_OK;
  if (lo < 0 || hi < lo || (int64_t)hi > s.total || start < 0) return SDCP_S_BAD_PARAMS;
  const int64_t end = (int64_t)start + (hi - lo) + s.extra;  // one past the last position
  if (end == start) return __syncthreads_or(bad) ? SDCP_S_BAD_PARAMS : SDCP_S_OK;  // no rows
  if (end > min((int64_t)kv.max_pages << kv.log_page, (int64_t)s.limit)) return SDCP_S_LIMIT;
  const int64_t first = s.window < 0 ? start : s.window == 0 ? 0 : max((int64_t)0, (int64_t)start + 1 - s.window);
  for (int64_t p = (first >> kv.log_page) + threadIdx.x; p <= (end - 1) >> kv.log_page; p += kCheckThreads) {
    const int32_t page = kv.page_table[(int64_t)b * kv.max_pages + p];
    bad |= page < 0 || page >= kv.n_pages;
  }
  return __syncthreads_or(bad) ? SDCP_S_BAD_PARAMS : SDCP_S_OK;
}

// Scale bytes 8 e + m stand for (1 + m / 8) 2^(e - 15): the three mantissa bits and the exponent
// of a binary32 whose exponent is re-biased by 112.
constexpr uint32_t kScaleLow = 8u, kScaleHigh = 167u, kScaleBias = 112u << 3;
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float((byte + kScaleBias) << 20); }
// The smallest scale >= most / 7 (most >= 0, may be infinite), as its byte.
__device__ __forceinline__ uint32_t scale_byte(float most) {
  const uint32_t u = __float_as_uint(__fdiv_rn(most, 7.0f)) + 0xFFFFFu;
  const int32_t v = (int32_t)(u >> 20) - (int32_t)kScaleBias;
  return (uint32_t)min(max(v, (int32_t)kScaleLow), (int32_t)kScaleHigh);
}

// Bytes in a block: a group's 16 bytes of codes of token slot t, and its scale byte.
__device__ __forceinline__ int32_t code_at(int32_t group, int32_t slot, int32_t log_page) {
  return ((group << log_page) + slot) << 4;
}
template <int D>
__device__ __forceinline__ int32_t scale_at(int32_t group, int32_t slot, int32_t log_page) {
  return (D / 2 << log_page) + slot * (D / kKvGroup) + group;
}

}  // namespace sdcp
