// sdcp_logits.cu - sdcp_adjust_logits: penalties for repeated tokens, biases and grammar masks
// on the rows of a ragged batch.
//
//   z = l;  seen: z = z > 0 ? z / r : z * r;  z -= f c;  c > 0: z -= p;  z += bias;  masked: -inf
//
// A CTA owns a slice of the vocabulary of one session, for all its rows: the history is the same
// for every row, so the slice's occurrence counts are built once, in shared memory.  Row i also
// counts the drafts x[0 .. i-1]; the few that fall into the slice are kept as a list.
//
// It is bound by memory: every logit is read and written once (in place: only what changes).  So the
// rows are first streamed with their masks alone, in 16-byte blocks, and the few tokens that a
// penalty or a bias applies to are written again, from a list of them in rising order, after a
// barrier: the second write meets lines that are still in L2.  With the arithmetic inside the
// streaming loop (unrolled over a block's elements) the kernel starved for instructions (3058 us for
// the large call below).
//
// Measured: 1024 sessions, 5 rows of 152064 bfloat16, histories of up to 1024 tokens: 620 us, 3.1 GB
// at 5.1 TB/s; in place, where a quarter of the rows is masked and the others are not streamed: 508 us.
// 96 sessions, 1 .. 16 draft rows of 50257, histories of up to 16384: 80 us, 170 MB; there the listed
// tokens are as much work as the rows, and the slices of frequent ones take longest.
#include <climits>

#include "sdcp_device.cuh"

namespace sdcp {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjUnroll = 4;             // blocks a thread has in flight
constexpr int kAdjCtas = 5;               // CTAs of an SM
constexpr int kAhead = 2;                 // rows of a listed token in flight (8.5 rows: 82 us with 2 or 4, 86 with 8, 88 one by one)
static_assert(kAdjThreads >= kScanSessions, "an offset a thread");
constexpr uint32_t kNowhere = 0xFFFFFFFFu;
constexpr uint32_t kInPrompt = 1u << 31;  // of a slice's word: the token is in the prompt
constexpr uint32_t kCountMask = ~kInPrompt;

struct AdjustArgs {
  const void* logits;
  void* out;
  int64_t V;
  int32_t B;
  int32_t extra;  // rows of a session beyond its drafts: 1 (target rows) or 0
  const int32_t* m_offsets;
  int64_t total;
  const int32_t* tokens;
  const sdcp_logit_controls* controls;
  const int32_t* history;
  int64_t history_stride;
  const int32_t* bias_tokens;
  const float* bias_values;
  int64_t n_bias;
  const uint32_t* masks;
  int64_t mask_stride;
  int64_t n_masks;
  const int32_t* mask_rows;
  int32_t* status;
  int32_t slice;    // tokens of a CTA, a power of two
  int32_t n_slices; // of a session
  int32_t by_part;  // CTAs in the order of the slices, not of the sessions
};

// One listed draft of the slice: its token (relative to the slice) and its position.
struct SliceDraft {
  int32_t at;
  int32_t pos;
};

// A vote of the block (rare: out of the way of the rest).
__device__ __noinline__ bool all_in_order(const int32_t* offsets, int32_t B) { return __syncthreads_and(offsets_in_order(offsets, B)) != 0; }

template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// E mask bits from token t on (t + E - 1 < V), 1 = may be chosen.
template <int E>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* mask, int64_t t) {
  const uint32_t sh = (uint32_t)t & 31u;
  uint32_t w = mask[t >> 5] >> sh;
  if (sh + E > 32u) w |= mask[(t >> 5) + 1] << (32u - sh);
  return w & ((1u << E) - 1u);
}

// A block of E logits with -inf where its mask bit is clear.
__device__ __forceinline__ uint4 masked_block(uint4 q, uint32_t keep, const float*) {
  const uint32_t ninf = 0xFF800000u;
  return make_uint4(keep & 1u ? q.x : ninf, keep & 2u ? q.y : ninf, keep & 4u ? q.z : ninf, keep & 8u ? q.w : ninf);
}
__device__ __forceinline__ uint32_t masked_pair(uint32_t w, uint32_t keep) {
  const uint32_t lo = keep & 1u ? w & 0xFFFFu : 0xFF80u, hi = keep & 2u ? w & 0xFFFF0000u : 0xFF800000u;
  return lo | hi;
}
__device__ __forceinline__ uint4 masked_block(uint4 q, uint32_t keep, const __nv_bfloat16*) {
  return make_uint4(masked_pair(q.x, keep), masked_pair(q.y, keep >> 2), masked_pair(q.z, keep >> 4), masked_pair(q.w, keep >> 6));
}

// Shared memory of a CTA, for a slice of n tokens: words [n] (kInPrompt | outputs), marks [n / 32] (a
// bit a token that something applies to), listed [n] (those tokens, rising), bias [n] where there are any.
__host__ __device__ constexpr size_t adjust_smem(int32_t slice, bool biased) {
  return (size_t)slice * 4 + (size_t)slice / 8 + (size_t)slice * 2 + (biased ? (size_t)slice * 4 : 0);
}

template <typename T>
__global__ void __launch_bounds__(kAdjThreads, kAdjCtas) adjust_kernel(const AdjustArgs a) {
  constexpr int E = Elem<T>::kPerVec;
  constexpr uint32_t kAll = (1u << E) - 1u;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ SliceDraft s_drafts[SDCP_MAX_M];
  __shared__ int32_t s_ndrafts;
  __shared__ const uint32_t* s_mask[SDCP_MAX_M + 1];  // the rows' masks, null: none
  __shared__ int32_t s_sum[kAdjThreads / 32];
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t per = (uint32_t)(a.by_part ? a.B : a.n_slices), major = blockIdx.x / per, minor = blockIdx.x % per;
  const int32_t b = (int32_t)(a.by_part ? minor : major), part = (int32_t)(a.by_part ? major : minor);
  const int64_t v0 = (int64_t)part * a.slice;
  const int32_t n = (int32_t)min((int64_t)a.slice, a.V - v0);

  // the session: offsets, controls, masks and biases, checked by every CTA of it
  const int32_t lo = a.m_offsets[b], hi = a.m_offsets[b + 1];
  const sdcp_logit_controls ctl = a.controls[b];
  auto refuse = [&] {  // no row is known to be the session's own: none is written
    if (part == 0 && tid == 0) a.status[b] = SDCP_S_BAD_PARAMS;
  };
  const bool scan = a.B <= kScanSessions;
  if (!scan) wait_for_previous();  // (it writes status[] too)
  if (lo < 0 || hi < lo || (int64_t)hi > a.total) return refuse();
  const bool fine = scan ? tid >= a.B || a.m_offsets[tid] <= a.m_offsets[tid + 1] : a.status[b] == SDCP_S_OK;
  auto out_of_order = [&] {  // a vote, and so a barrier too
    if (__syncthreads_and(fine)) return false;
    return scan || !all_in_order(a.m_offsets, a.B);  // (status[b] may be of the session's first CTA, for something else)
  };
  const int32_t M = hi - lo;
  const int32_t rows = M + a.extra;
  const int64_t row0 = (int64_t)lo + (int64_t)b * a.extra;
  const T* const in = static_cast<const T*>(a.logits) + row0 * a.V + v0;
  T* const out = static_cast<T*>(a.out) + row0 * a.V + v0;
  bool bad = M > SDCP_MAX_M || !(ctl.repetition > 0.0f && ctl.repetition < INFINITY) || !isfinite(ctl.frequency) ||
             !isfinite(ctl.presence) || (int64_t)ctl.history_len > a.history_stride || ctl.prompt_len > ctl.history_len ||
             (int64_t)ctl.bias_offset + ctl.bias_count > a.n_bias;

  if (bad) {
    if (out_of_order()) return refuse();
  } else {
    uint32_t* const words = reinterpret_cast<uint32_t*>(smem);
    uint32_t* const marks = words + a.slice;
    uint16_t* const listed = reinterpret_cast<uint16_t*>(marks + a.slice / 32);
    float* const bias = reinterpret_cast<float*>(listed + a.slice);
    const bool has_bias = ctl.bias_count != 0u;
    for (int k = tid; k < a.slice / 4; k += kAdjThreads) reinterpret_cast<uint4*>(words)[k] = make_uint4(0u, 0u, 0u, 0u);
    for (int k = tid; k < a.slice / 32; k += kAdjThreads) marks[k] = 0u;
    if (has_bias)
      for (int k = tid; k < a.slice / 4; k += kAdjThreads) reinterpret_cast<uint4*>(bias)[k] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) s_ndrafts = 0;
    // what the slice is told apart by: all asked for at once, before the barrier
    const int32_t* const hist = a.history + (int64_t)b * a.history_stride;
    constexpr int kBatch = 8;  // tokens of the history that a thread has in flight
    int32_t token[kBatch];
    auto load_history = [&](uint32_t k0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) token[u] = k0 + u * kAdjThreads < ctl.history_len ? hist[k0 + u * kAdjThreads] : -1;
    };
    load_history((uint32_t)tid);
    const int32_t draft = tid < M ? a.tokens[lo + tid] : -1;
    if (tid < rows) {
      int32_t r = a.mask_rows ? a.mask_rows[row0 + tid] : -1;
      if (r < -1 || (int64_t)r >= a.n_masks) {
        bad = true;
        r = -1;
      }
      s_mask[tid] = r < 0 ? nullptr : a.masks + (int64_t)r * a.mask_stride;
    }
    if (out_of_order()) return refuse();

    // the slice's counts, biases and drafts
    for (uint32_t k0 = (uint32_t)tid; k0 < ctl.history_len; k0 += kBatch * kAdjThreads) {
      if (k0 != (uint32_t)tid) load_history(k0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t at = (uint32_t)token[u] - (uint32_t)v0;  // beyond the slice: >= n
        if (at < (uint32_t)n) {
          if (k0 + u * kAdjThreads < ctl.prompt_len) atomicOr(&words[at], kInPrompt);
          else atomicAdd(&words[at], 1u);
          atomicOr(&marks[at >> 5], 1u << (at & 31u));
        }
      }
    }
    for (uint32_t k = tid; k < ctl.bias_count; k += kAdjThreads) {
      const int32_t t = a.bias_tokens[ctl.bias_offset + k];
      const int32_t before = k ? a.bias_tokens[ctl.bias_offset + k - 1] : -1;
      bad |= t <= before || (int64_t)t >= a.V;
      const uint32_t at = (uint32_t)t - (uint32_t)v0;
      if (at < (uint32_t)n) {
        bias[at] = a.bias_values[ctl.bias_offset + k];
        atomicOr(&marks[at >> 5], 1u << (at & 31u));
      }
    }
    if (tid < M) {
      const uint32_t at = (uint32_t)draft - (uint32_t)v0;
      if (at < (uint32_t)n) {
        s_drafts[atomicAdd(&s_ndrafts, 1)] = SliceDraft{(int32_t)at, tid};
        atomicOr(&marks[at >> 5], 1u << (at & 31u));
      }
    }

    // The rows and their masks.  The slice of a row is cut at 16-byte boundaries of memory: block k
    // covers the tokens k E - lead .. k E - lead + E - 1 of the row, the first and the last may be
    // partial.  A thread goes down the rows with a block, then with its next one.
    const bool in_place = a.logits == a.out;
    const bool alike = (((uintptr_t)in ^ (uintptr_t)out) & 15u) == 0;
    const int32_t lead0 = (int32_t)(((uintptr_t)in & 15u) / sizeof(T)), step = (int32_t)(a.V & (E - 1));
    const int32_t blocks = alike ? (n + E - 1) / E + 1 : 0;
    {
      int32_t k = tid, i = 0, lead = lead0;
      uint32_t at = (uint32_t)k * E;  // of the block's first logit from `in`, plus lead (at most 65 rows of 2^24)
      while (rows > 0 && k < blocks) {  // (a session without drafts has no draft rows)
        uint4 q[kAdjUnroll];
        uint32_t to[kAdjUnroll], keep[kAdjUnroll];
#pragma unroll
        for (int u = 0; u < kAdjUnroll; ++u) {
          const int32_t t = k * E - lead;
          to[u] = kNowhere;
          if (k < blocks) {
            if (t >= 0 && t + E <= n) {
              const uint32_t* const mask = s_mask[i];
              keep[u] = mask == nullptr ? kAll : mask_bits<E>(mask, v0 + t);
              if (!in_place || keep[u] != kAll) {
                to[u] = at - (uint32_t)lead;
                q[u] = *reinterpret_cast<const uint4*>(in + to[u]);
              }
            }
            at += (uint32_t)a.V;
            lead = (lead + step) & (E - 1);
            if (++i == rows) {
              i = 0;
              k += kAdjThreads;
              at = (uint32_t)k * E;
              lead = lead0;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kAdjUnroll; ++u)
          if (to[u] != kNowhere)
            *reinterpret_cast<uint4*>(out + to[u]) = keep[u] == kAll ? q[u] : masked_block(q[u], keep[u], static_cast<const T*>(nullptr));
      }
    }
    // what the blocks left: the ends of the rows, or all of them where the two addresses differ modulo 16
    const int32_t ends = alike ? 2 * E : n;
    for (int32_t x = tid; x < rows * ends; x += kAdjThreads) {
      const int32_t i = x / ends, e = x - i * ends;
      int32_t t = e;
      if (alike) {
        const int32_t lead = (int32_t)((lead0 + (int64_t)i * step) & (E - 1));
        const int32_t head = (E - lead) & (E - 1), tail = head + (max(n - head, 0) / E) * E;  // [head, tail) is in blocks
        t = e < E ? e : tail + e - E;
        if ((e < E ? t >= head : t < head) || t >= n) continue;
      }
      const uint32_t* const mask = s_mask[i];
      const bool keep = mask == nullptr || mask_bits<1>(mask, v0 + t) != 0u;
      if (!in_place || !keep) out[(int64_t)i * a.V + t] = keep ? in[(int64_t)i * a.V + t] : from_float<T>(__uint_as_float(0xFF800000u));
    }
    bad = __syncthreads_or(bad) != 0;

    if (!bad) {
      // the marked tokens, rising: a stretch of the marks per thread, and their number before it
      const int per = (a.slice / 32 + kAdjThreads - 1) / kAdjThreads, w0 = min(tid * per, a.slice / 32), w1 = min(w0 + per, a.slice / 32);
      int32_t mine = 0;
      for (int w = w0; w < w1; ++w) mine += __popc(marks[w]);
      int32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_sum[warp] = incl;
      __syncthreads();
      int32_t at = incl - mine, total = 0;
#pragma unroll
      for (int w = 0; w < kAdjThreads / 32; ++w) {
        if (w < warp) at += s_sum[w];
        total += s_sum[w];
      }
      for (int w = w0; w < w1; ++w)
        for (uint32_t m = marks[w]; m != 0u; m &= m - 1u) listed[at++] = (uint16_t)(w * 32 + __ffs((int)m) - 1);
      __syncthreads();

      // their logits, in every row
      const int32_t nd = s_ndrafts;
      const float rep = ctl.repetition, freq = ctl.frequency, pres = ctl.presence;
      int32_t side = 1;  // threads of a token, a row each
      while (side < 32 && side < rows && total * side < kAdjThreads) side *= 2;
      const int32_t first = tid & (side - 1);
#pragma unroll 1
      for (int32_t x = tid / side; x < total; x += kAdjThreads / side) {
        const int32_t t = listed[x];
        const uint32_t w = words[t];
        const float bt = has_bias ? bias[t] : 0.0f;
        uint64_t drafted = 0;  // the places where the token is a draft
        for (int d = 0; d < nd; ++d)
          if (s_drafts[d].at == t) drafted |= 1ull << s_drafts[d].pos;
        const T* pr = in + (int64_t)first * a.V + t;
        T* po = out + (int64_t)first * a.V + t;
        // kAhead rows at a time: their mask words together, then their logits together
#pragma unroll 1
        for (int32_t r0 = first; r0 < rows; r0 += kAhead * side, pr += kAhead * side * a.V, po += kAhead * side * a.V) {
          uint32_t bits[kAhead], c[kAhead];
          float z[kAhead];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const int32_t r = r0 + u * side;
            const uint32_t* const mask = r < rows ? s_mask[r] : nullptr;
            bits[u] = r < rows ? ~0u : 0u;
            if (mask != nullptr) bits[u] = mask[(v0 + t) >> 5];
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const int32_t r = r0 + u * side;
            c[u] = (w & kCountMask) + (uint32_t)__popcll(r < 64 ? drafted & ((1ull << r) - 1ull) : drafted);
            bits[u] = (bits[u] >> ((uint32_t)(v0 + t) & 31u)) & 1u;
            if ((w & kInPrompt) == 0u && c[u] == 0u && bt == 0.0f) bits[u] = 0u;
            if (bits[u] != 0u) z[u] = to_float(pr[(int64_t)u * side * a.V]);
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u)
            if (bits[u] != 0u) {
              float y = z[u];
              if ((w & kInPrompt) != 0u || c[u] != 0u) y = y > 0.0f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
              if (c[u] != 0u) y = __fsub_rn(__fsub_rn(y, __fmul_rn(freq, (float)c[u])), pres);
              po[(int64_t)u * side * a.V] = from_float<T>(__fadd_rn(y, bt));
            }
        }
      }
    }
  }
  if (part == 0 && tid == 0) a.status[b] = M > SDCP_MAX_M ? SDCP_S_LIMIT : bad ? SDCP_S_BAD_PARAMS : SDCP_S_OK;
  if (bad) {
    const T nan = from_float<T>(__uint_as_float(0x7FC00000u));
    for (int r = 0; r < rows; ++r)
      for (int k = tid; k < n; k += kAdjThreads) out[(int64_t)r * a.V + k] = nan;
  }
}

template <typename T>
cudaError_t launch_adjust(const AdjustArgs& a, cudaStream_t stream) {
  const size_t smem = adjust_smem(a.slice, a.n_bias > 0);
  return launch_after_if(a.B > kScanSessions, adjust_kernel<T>, (unsigned)a.B * (unsigned)a.n_slices, kAdjThreads, smem, stream, a);
}

// Tokens of a slice: 4096 while a session has fewer than eight rows on average (what a CTA does
// besides streaming is then spread over more tokens: 5 rows of 152064, 623 us against 814 with
// 2048), else 2048 (unevenly repeated tokens are spread over more CTAs: 8.5 rows of 50257, 82 us
// against 110 with 4096, 112 with 1024), and down to 512 where that leaves SMs without a CTA.
int32_t adjust_slice(int64_t V, int32_t B, int64_t rows, int sms) {
  int32_t slice = rows < (int64_t)8 * B ? 4096 : 2048;
  while (slice > 512 && (V + slice - 1) / slice * B < (int64_t)2 * sms) slice /= 2;
  return slice;
}

}  // namespace
}  // namespace sdcp

extern "C" int sdcp_adjust_logits(const void* logits, void* out, int dtype, int64_t V, int32_t B,
                                  int rows, const int32_t* m_offsets, int64_t total_drafts,
                                  const int32_t* draft_tokens, const sdcp_logit_controls* controls,
                                  const int32_t* history, int64_t history_stride,
                                  const int32_t* bias_tokens, const float* bias_values,
                                  int64_t n_bias, const uint32_t* masks, int64_t mask_stride,
                                  int64_t n_masks, const int32_t* mask_rows, int32_t* status,
                                  void* stream) {
  using namespace sdcp;
  if (B < 0 || total_drafts < 0 || V < 1 || history_stride < 0 || n_bias < 0 || n_masks < 0) return SDCP_E_INVALID;
  if (dtype != SDCP_F32 && dtype != SDCP_BF16) return SDCP_E_INVALID;
  if (rows != SDCP_ROWS_TARGET && rows != SDCP_ROWS_DRAFT) return SDCP_E_INVALID;
  if (V > SDCP_MAX_VOCAB) return SDCP_E_TOO_LARGE;
  if (total_drafts > INT32_MAX || total_drafts + B + total_drafts > (int64_t)INT32_MAX / 2) return SDCP_E_TOO_LARGE;
  if (B == 0) return SDCP_OK;
  if (!m_offsets || !controls || !status || (total_drafts > 0 && !draft_tokens)) return SDCP_E_INVALID;
  if (rows == SDCP_ROWS_TARGET || total_drafts > 0)
    if (!logits || !out) return SDCP_E_INVALID;
  if ((history_stride > 0 && !history) || (n_bias > 0 && (!bias_tokens || !bias_values))) return SDCP_E_INVALID;
  if (mask_rows && n_masks > 0 && (!masks || mask_stride < (V + 31) / 32)) return SDCP_E_INVALID;
  const size_t esz = dtype == SDCP_BF16 ? 2 : 4;
  if (((uintptr_t)logits % esz) != 0 || ((uintptr_t)out % esz) != 0) return SDCP_E_ALIGN;
  if (!on_words(m_offsets, draft_tokens, controls, history, bias_tokens, bias_values, masks, mask_rows, status)) return SDCP_E_ALIGN;
  DeviceInfo di;
  if (!device_info(&di)) return SDCP_E_DEVICE;
  const int32_t slice = adjust_slice(V, B, total_drafts + (rows == SDCP_ROWS_TARGET ? B : 0), di.sms);
  const int64_t n_slices = (V + slice - 1) / slice;
  if (n_slices * B > (int64_t)INT32_MAX) return SDCP_E_TOO_LARGE;
  const AdjustArgs a{logits, out, V, B, rows == SDCP_ROWS_TARGET ? 1 : 0, m_offsets, total_drafts, draft_tokens,
                     controls, history, history_stride, bias_tokens, bias_values, n_bias, masks, mask_stride,
                     n_masks, mask_rows, status, slice, (int32_t)n_slices,
                     // the slices of frequent tokens (low ids) take longest: first, where the grid is a few waves
                     // (3 waves: 82 us against 97; 51 waves, whose rows are better read one after another: 659 against 623)
                     n_slices * B < (int64_t)8 * kAdjCtas * di.sms ? 1 : 0};
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch_offsets_check(m_offsets, B, status, s) != cudaSuccess) return SDCP_E_LAUNCH;
  const cudaError_t e = dtype == SDCP_BF16 ? launch_adjust<__nv_bfloat16>(a, s) : launch_adjust<float>(a, s);
  return e == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}
