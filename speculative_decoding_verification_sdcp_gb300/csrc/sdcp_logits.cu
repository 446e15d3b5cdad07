// sdcp_logits.cu - sdcp_adjust_logits: penalties for repeated tokens, biases and grammar masks
// on the rows of a ragged batch.
//
// A CTA owns a slice of the vocabulary of one session and handles that slice of all the session's
// rows: the history is the same for every row, so the slice's occurrence counts are built once, in
// shared memory, and used M + 1 times.  Row i also counts the drafts x[0 .. i-1]; the few of them
// that fall into the slice are kept as a list, which only tokens that are listed look at.
//
//   z = l;  seen: z = z > 0 ? z / r : z * r;  z -= f c;  c > 0: z -= p;  z += bias;  masked: -inf
//
// Everything else is a copy, in 16-byte blocks of memory.
#include <climits>

#include "sdcp_device.cuh"

namespace sdcp {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjUnroll = 4;             // blocks a thread has in flight
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
};

// One listed draft of the slice: its token (relative to the slice) and its position.
struct SliceDraft {
  int32_t at;
  int32_t pos;
};

// What the slow path needs about one row.
struct RowView {
  const uint32_t* mask;  // the row's mask words, or null
  int32_t i;             // drafts before this row
};

template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

struct Slice {
  const uint32_t* words;   // [slice] kInPrompt | outputs
  const float* bias;       // [slice], or null
  const uint32_t* touched; // a bit per 8 tokens: something may apply to one of them
  const SliceDraft* drafts;
  int32_t n_drafts;
  float rep, freq, pres;
};

// The logit of token `at` (relative to the slice) of a row, `keep` = its mask bit.
template <typename T>
__device__ __forceinline__ T adjust_one(const Slice& s, int32_t at, int32_t i, bool keep, T l) {
  if (!keep) return from_float<T>(__uint_as_float(0xFF800000u));
  const uint32_t w = s.words[at];
  uint32_t c = w & kCountMask;
  for (int k = 0; k < s.n_drafts; ++k) c += (s.drafts[k].at == at && s.drafts[k].pos < i) ? 1u : 0u;
  const bool seen = (w & kInPrompt) != 0u || c != 0u;
  const float b = s.bias ? s.bias[at] : 0.0f;
  if (!seen && b == 0.0f) return l;
  float z = to_float(l);
  if (seen) z = z > 0.0f ? __fdiv_rn(z, s.rep) : __fmul_rn(z, s.rep);
  if (c != 0u) {
    z = __fsub_rn(z, __fmul_rn(s.freq, (float)c));
    z = __fsub_rn(z, s.pres);
  }
  z = __fadd_rn(z, b);
  return from_float<T>(z);
}

// E mask bits from token t on (t + E - 1 < V), 1 = may be chosen.
template <int E>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* mask, int64_t t) {
  const uint32_t sh = (uint32_t)t & 31u;
  uint32_t w = mask[t >> 5] >> sh;
  if (sh + E > 32u) w |= mask[(t >> 5) + 1] << (32u - sh);
  return w & ((1u << E) - 1u);
}

template <typename T>
__global__ void __launch_bounds__(kAdjThreads) adjust_kernel(const AdjustArgs a) {
  constexpr int E = Elem<T>::kPerVec;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ SliceDraft s_drafts[SDCP_MAX_M];
  __shared__ int32_t s_ndrafts;
  const int tid = (int)threadIdx.x;
  const int32_t b = (int32_t)(blockIdx.x / (uint32_t)a.n_slices);
  const int32_t part = (int32_t)(blockIdx.x % (uint32_t)a.n_slices);
  const int64_t v0 = (int64_t)part * a.slice;
  const int32_t n = (int32_t)min((int64_t)a.slice, a.V - v0);

  // the session: offsets, controls, masks and biases, checked by every CTA of it
  const int32_t lo = a.m_offsets[b], hi = a.m_offsets[b + 1];
  if (lo < 0 || hi < lo || (int64_t)hi > a.total) {
    if (part == 0 && tid == 0) a.status[b] = SDCP_S_BAD_PARAMS;
    return;
  }
  const int32_t M = hi - lo;
  const int32_t rows = M + a.extra;
  const int64_t row0 = (int64_t)lo + (int64_t)b * a.extra;
  const sdcp_logit_controls ctl = a.controls[b];
  bool bad = !(ctl.repetition > 0.0f && ctl.repetition < INFINITY) || !isfinite(ctl.frequency) ||
             !isfinite(ctl.presence) || (int64_t)ctl.history_len > a.history_stride ||
             ctl.prompt_len > ctl.history_len || (int64_t)ctl.bias_offset + ctl.bias_count > a.n_bias;
  if (M <= SDCP_MAX_M && !bad) {
    if (a.mask_rows != nullptr)
      for (int i = tid; i < rows; i += kAdjThreads) {
        const int32_t r = a.mask_rows[row0 + i];
        bad |= r < -1 || (int64_t)r >= a.n_masks;
      }
    for (uint32_t k = tid; k < ctl.bias_count; k += kAdjThreads) {
      const int32_t t = a.bias_tokens[ctl.bias_offset + k];
      const int32_t before = k ? a.bias_tokens[ctl.bias_offset + k - 1] : -1;
      bad |= t <= before || (int64_t)t >= a.V;
    }
  }

  uint32_t* words = reinterpret_cast<uint32_t*>(smem);
  uint32_t* touched = words + a.slice;
  float* bias = reinterpret_cast<float*>(touched + a.slice / 256);
  const bool has_bias = ctl.bias_count != 0u;
  for (int k = tid; k < a.slice; k += kAdjThreads) {
    words[k] = 0u;
    if (has_bias) bias[k] = 0.0f;
  }
  for (int k = tid; k < a.slice / 256; k += kAdjThreads) touched[k] = 0u;
  if (tid == 0) s_ndrafts = 0;
  const int32_t st = M > SDCP_MAX_M ? SDCP_S_LIMIT : __syncthreads_or(bad) ? SDCP_S_BAD_PARAMS : SDCP_S_OK;
  if (part == 0 && tid == 0) a.status[b] = st;

  const T* in = static_cast<const T*>(a.logits) + row0 * a.V + v0;
  T* out = static_cast<T*>(a.out) + row0 * a.V + v0;
  if (st != SDCP_S_OK) {
    const T nan = from_float<T>(__uint_as_float(0x7FC00000u));
    for (int i = 0; i < rows; ++i)
      for (int k = tid; k < n; k += kAdjThreads) out[(int64_t)i * a.V + k] = nan;
    return;
  }

  // the slice's counts, biases and drafts
  const int32_t* hist = a.history + (int64_t)b * a.history_stride;
  for (uint32_t k = tid; k < ctl.history_len; k += kAdjThreads) {
    const uint32_t at = (uint32_t)((int64_t)hist[k] - v0);
    if (at < (uint32_t)n) {
      if (k < ctl.prompt_len) atomicOr(&words[at], kInPrompt);
      else atomicAdd(&words[at], 1u);
      atomicOr(&touched[at >> 8], 1u << ((at >> 3) & 31u));
    }
  }
  for (uint32_t k = tid; k < ctl.bias_count; k += kAdjThreads) {
    const uint32_t at = (uint32_t)((int64_t)a.bias_tokens[ctl.bias_offset + k] - v0);
    if (at < (uint32_t)n) {
      bias[at] = a.bias_values[ctl.bias_offset + k];
      atomicOr(&touched[at >> 8], 1u << ((at >> 3) & 31u));
    }
  }
  for (int k = tid; k < M; k += kAdjThreads) {
    const uint32_t at = (uint32_t)((int64_t)a.tokens[lo + k] - v0);
    if (at < (uint32_t)n) {
      s_drafts[atomicAdd(&s_ndrafts, 1)] = SliceDraft{(int32_t)at, k};
      atomicOr(&touched[at >> 8], 1u << ((at >> 3) & 31u));
    }
  }
  __syncthreads();

  const Slice s{words, has_bias ? bias : nullptr, touched, s_drafts, s_ndrafts, ctl.repetition, ctl.frequency, ctl.presence};
  const bool in_place = a.logits == a.out;

  // The slice of a row is cut at 16-byte boundaries of memory: block k covers the tokens from
  // k E - lead on, the first and the last may be partial.  Rows whose two addresses differ modulo
  // 16 go element by element.
  const int32_t slots = (n + E - 1) / E + 1;
  int32_t i = 0, k = tid;
  while (k >= slots) { k -= slots; ++i; }
  while (i < rows) {
    uint4 q[kAdjUnroll];
    int32_t ui[kAdjUnroll], ut[kAdjUnroll];  // row, first token (relative to the slice)
    uint32_t keep[kAdjUnroll];               // mask bits of a whole block
    int kind[kAdjUnroll];                    // 0: nothing to do, 1: a whole block, 2: element by element
#pragma unroll
    for (int u = 0; u < kAdjUnroll; ++u) {
      kind[u] = 0;
      ui[u] = i;
      if (i < rows) {
        const T* pr = in + (int64_t)i * a.V;
        const T* po = out + (int64_t)i * a.V;
        const int32_t lead = (int32_t)(((uintptr_t)pr & 15u) / sizeof(T));
        const int32_t t = k * E - lead;
        ut[u] = t;
        if (t < n) {
          const bool whole = t >= 0 && t + E <= n && (((uintptr_t)pr ^ (uintptr_t)po) & 15u) == 0;
          kind[u] = whole ? 1 : 2;
          if (whole) {
            const int32_t mr = a.mask_rows ? a.mask_rows[row0 + i] : -1;
            keep[u] = mr < 0 ? (1u << E) - 1u : mask_bits<E>(a.masks + (int64_t)mr * a.mask_stride, v0 + t);
            const uint32_t t1 = touched[t >> 8] >> ((t >> 3) & 31);
            const int32_t e = t + E - 1;
            const uint32_t any = (t1 | (touched[e >> 8] >> ((e >> 3) & 31))) & 1u;
            keep[u] |= any << 31;
            if (in_place && any == 0u && keep[u] == (1u << E) - 1u) kind[u] = 0;
            else q[u] = *reinterpret_cast<const uint4*>(pr + t);
          }
        }
        k += kAdjThreads;
        while (k >= slots) { k -= slots; ++i; }
      }
    }
#pragma unroll
    for (int u = 0; u < kAdjUnroll; ++u) {
      const T* pr = in + (int64_t)ui[u] * a.V;
      T* po = out + (int64_t)ui[u] * a.V;
      if (kind[u] == 1) {
        T* e = reinterpret_cast<T*>(&q[u]);
        if (keep[u] != (1u << E) - 1u) {
          if (keep[u] >> 31) {
#pragma unroll
            for (int j = 0; j < E; ++j) e[j] = adjust_one<T>(s, ut[u] + j, ui[u], (keep[u] >> j) & 1u, e[j]);
          } else {
#pragma unroll
            for (int j = 0; j < E; ++j)
              if (!((keep[u] >> j) & 1u)) e[j] = from_float<T>(__uint_as_float(0xFF800000u));
          }
        }
        *reinterpret_cast<uint4*>(po + ut[u]) = q[u];
      } else if (kind[u] == 2) {
        const int32_t mr = a.mask_rows ? a.mask_rows[row0 + ui[u]] : -1;
        const uint32_t* mask = mr < 0 ? nullptr : a.masks + (int64_t)mr * a.mask_stride;
        for (int32_t t = max(ut[u], 0); t < min(ut[u] + E, n); ++t) {
          const bool keep1 = mask == nullptr || mask_bits<1>(mask, v0 + t) != 0u;
          po[t] = adjust_one<T>(s, t, ui[u], keep1, pr[t]);
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_adjust(const AdjustArgs& a, cudaStream_t stream) {
  const size_t smem = (size_t)a.slice * 4 + (size_t)a.slice / 256 * 4 + (a.n_bias > 0 ? (size_t)a.slice * 4 : 0);
  adjust_kernel<T><<<(unsigned)a.B * (unsigned)a.n_slices, kAdjThreads, smem, stream>>>(a);
  return cudaGetLastError();
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
  if (total_drafts + B + total_drafts > (int64_t)INT32_MAX / 2) return SDCP_E_TOO_LARGE;
  if (B == 0) return SDCP_OK;
  if (!m_offsets || !controls || !status || (total_drafts > 0 && !draft_tokens)) return SDCP_E_INVALID;
  if (rows == SDCP_ROWS_TARGET || total_drafts > 0)
    if (!logits || !out) return SDCP_E_INVALID;
  if ((history_stride > 0 && !history) || (n_bias > 0 && (!bias_tokens || !bias_values))) return SDCP_E_INVALID;
  if (mask_rows && n_masks > 0 && (!masks || mask_stride < (V + 31) / 32)) return SDCP_E_INVALID;
  const size_t esz = dtype == SDCP_BF16 ? 2 : 4;
  if (((uintptr_t)logits % esz) != 0 || ((uintptr_t)out % esz) != 0) return SDCP_E_ALIGN;
  const int32_t slice = 4096;
  const int64_t n_slices = (V + slice - 1) / slice;
  if (n_slices * B > (int64_t)INT32_MAX) return SDCP_E_TOO_LARGE;
  const AdjustArgs a{logits, out, V, B, rows == SDCP_ROWS_TARGET ? 1 : 0, m_offsets, total_drafts, draft_tokens,
                     controls, history, history_stride, bias_tokens, bias_values, n_bias, masks, mask_stride,
                     n_masks, mask_rows, status, slice, (int32_t)n_slices};
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SDCP_BF16 ? launch_adjust<__nv_bfloat16>(a, s) : launch_adjust<float>(a, s);
  return e == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}
