// sdcp_kv.cu - the paged 4-bit cache: sdcp_append_kv (rotation, quantisation, the write) and
// sdcp_read_kv (cached tokens as values), and the check of a call's sessions.
#include <climits>

#include "sdcp_kv.cuh"

namespace sdcp {

int kv_view(const sdcp_kv_cache* c, KvView* out) {
  if (!c || c->struct_size < sizeof(sdcp_kv_cache)) return SDCP_E_INVALID;
  const size_t page = sdcp_kv_page_bytes(c->page_tokens, c->kv_heads, c->head_dim);
  if (page == 0 || c->n_pages < 1 || c->max_pages < 1 || !c->pages || !c->page_table) return SDCP_E_INVALID;
  if ((int64_t)c->max_pages * c->page_tokens > (int64_t)INT32_MAX) return SDCP_E_TOO_LARGE;
  if (((uintptr_t)c->pages & 15u) != 0) return SDCP_E_ALIGN;
  int log_page = 0;
  while ((1 << log_page) < c->page_tokens) ++log_page;
  *out = KvView{c->pages, c->page_table, c->n_pages, c->max_pages, c->kv_heads, log_page,
                (int32_t)(page / 2 / (size_t)c->kv_heads), (int64_t)page};
  return SDCP_OK;
}

namespace {

__global__ void __launch_bounds__(kCheckThreads) kv_check_kernel(const KvView kv, const KvSessions s, int32_t* status) {
  let_next_start();
  const int32_t st = kv_session_status(kv, s, (int32_t)blockIdx.x);
  if (threadIdx.x == 0) status[blockIdx.x] = st;
}

cudaError_t launch_kv_check(const KvView& kv, const KvSessions& s, int32_t* status, cudaStream_t stream) {
  kv_check_kernel<<<(unsigned)s.B, kCheckThreads, 0, stream>>>(kv, s, status);
  return cudaGetLastError();
}

// ---- append ---------------------------------------------------------------------------

constexpr int kAppendThreads = 256;
constexpr int kChan = 4;  // channels of a lane

struct AppendArgs {
  KvView kv;
  KvSessions s;
  const void *k, *v, *q;
  int64_t k_stride, v_stride, q_stride;
  int32_t q_heads;
  void* q_out;
  const float* table;  // null: no rotation
  int32_t rot;
  int32_t interleaved;
  const int32_t* status;
};

__device__ __forceinline__ void load4(const float* p, float (&x)[kChan]) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[kChan]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[kChan]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[kChan]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ float elem(const float* p) { return *p; }
__device__ __forceinline__ float elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// One warp handles 32 / (D / 4) heads at a time, four channels a lane.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / kChan;           // lanes of a head
  constexpr int kHeads = 32 / kLanes;         // heads of a warp
  const int lane = (int)(threadIdx.x & 31u), warp = (int)(threadIdx.x >> 5);
  const int64_t row = blockIdx.x;
  wait_for_previous();
  const int32_t b = find_session(a.s.offsets, a.s.B, row, true);
  const int64_t i = row - a.s.offsets[b] - b;
  if (a.status[b] != SDCP_S_OK || i < 0 || i > (int64_t)a.s.offsets[b + 1] - a.s.offsets[b]) return;
  const int32_t pos = a.s.start[b] + (int32_t)i;

  // this lane's channels, and the cosines and signed sines they turn by
  const int c0 = (lane % kLanes) * kChan;
  float cs[kChan], sn[kChan];
  bool turns[kChan];
  int other[kChan];  // the channel each turns with
#pragma unroll
  for (int j = 0; j < kChan; ++j) {
    const int c = c0 + j, half = a.rot / 2;
    turns[j] = a.table != nullptr && c < a.rot;
    cs[j] = 1.0f;
    sn[j] = 0.0f;
    other[j] = c;
    if (turns[j]) {
      const bool second = a.interleaved ? (c & 1) != 0 : c >= half;
      const int pair = a.interleaved ? c >> 1 : second ? c - half : c;
      other[j] = a.interleaved ? c ^ 1 : second ? c - half : c + half;
      const float* t = a.table + (int64_t)pos * a.rot;
      cs[j] = t[pair];
      sn[j] = second ? t[half + pair] : -t[half + pair];
    }
  }

  const int32_t page = a.kv.page_table[(int64_t)b * a.kv.max_pages + (pos >> a.kv.log_page)];
  const int32_t slot = pos & (a.kv.page_tokens() - 1);
  uint8_t* pg = a.kv.pages + (int64_t)page * a.kv.page;
  const int32_t heads = 2 * a.kv.heads + a.q_heads;
  for (int32_t h = ((int32_t)blockIdx.y * (kAppendThreads / 32) + warp) * kHeads + lane / kLanes; h - lane / kLanes < heads;
       h += (int32_t)gridDim.y * (kAppendThreads / 32) * kHeads) {
    const bool live = h < heads;
    const bool is_k = h < a.kv.heads, is_v = !is_k && h < 2 * a.kv.heads;
    const int32_t head = is_k ? h : is_v ? h - a.kv.heads : h - 2 * a.kv.heads;
    const T* src = is_k ? static_cast<const T*>(a.k) + row * a.k_stride
                        : is_v ? static_cast<const T*>(a.v) + row * a.v_stride : static_cast<const T*>(a.q) + row * a.q_stride;
    src += (int64_t)head * D;
    float x[kChan] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (live) {
      load4(src + c0, x);
      if (!is_v) {
        float y[kChan];
#pragma unroll
        for (int j = 0; j < kChan; ++j) y[j] = turns[j] ? elem(src + other[j]) : 0.0f;
        // x1 cos - x2 sin and x2 cos + x1 sin, each product and sum rounded by itself
#pragma unroll
        for (int j = 0; j < kChan; ++j)
          if (turns[j]) x[j] = __fadd_rn(__fmul_rn(x[j], cs[j]), __fmul_rn(y[j], sn[j]));
      }
    }
    if (live && !is_k && !is_v) store4(static_cast<T*>(a.q_out) + (row * a.q_heads + head) * D + c0, x);
    // quantise: the largest magnitude over the group's eight lanes (fmaxf leaves a NaN out)
    float most = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    most = isnan(most) ? 0.0f : most;
#pragma unroll
    for (int o = 1; o < kKvGroup / kChan; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    const uint32_t sb = scale_byte(most);
    const float s = scale_value(sb);
    uint32_t w = 0u;
    const int base = (c0 & 4) ? 8 : 0;  // channels 4..7 of a word sit eight bits up
#pragma unroll
    for (int j = 0; j < kChan; ++j) {
      const float n = fminf(fmaxf(rintf(__fdiv_rn(x[j], s)), -7.0f), 7.0f);
      const uint32_t code = isnan(x[j]) ? 8u : (uint32_t)((int32_t)n + 8);
      w |= code << (base + 4 * (j / 2) + 16 * (j % 2));
    }
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 1);
    if (live && (is_k || is_v)) {
      uint8_t* blk = pg + ((int64_t)head * 2 + (is_v ? 1 : 0)) * a.kv.block;
      const int g = c0 / kKvGroup;
      if ((c0 & 4) == 0) *reinterpret_cast<uint32_t*>(blk + code_at(g, slot, a.kv.log_page) + (c0 % kKvGroup) / 8 * 4) = w;
      if ((c0 % kKvGroup) == 0) blk[scale_at<D>(g, slot, a.kv.log_page)] = (uint8_t)sb;
    }
  }
}

// ---- read -----------------------------------------------------------------------------

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 32;  // rows of a CTA

struct ReadArgs {
  KvView kv;
  KvSessions s;
  void *k_out, *v_out;
  const int32_t* status;
};

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp reads eight tokens of one head: the four words of a group of each, then the next group.
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadArgs a) {
  constexpr int kGroups = D / kKvGroup;
  __shared__ int64_t s_page[kReadTokens];  // byte offset of a row's page, -1: the row is zero
  __shared__ int32_t s_slot[kReadTokens];
  const int lane = (int)(threadIdx.x & 31u), warp = (int)(threadIdx.x >> 5);
  const int64_t row0 = (int64_t)blockIdx.x * kReadTokens;
  wait_for_previous();
  for (int r = warp; r < kReadTokens; r += kReadThreads / 32) {
    const int64_t row = row0 + r;
    int64_t at = -1;
    int32_t slot = 0;
    if (row < a.s.total) {
      const int32_t b = find_session(a.s.offsets, a.s.B, row, false);
      const int64_t i = row - a.s.offsets[b];
      if (a.status[b] == SDCP_S_OK && i >= 0 && row < a.s.offsets[b + 1]) {
        const int32_t pos = a.s.start[b] + (int32_t)i;
        at = (int64_t)a.kv.page_table[(int64_t)b * a.kv.max_pages + (pos >> a.kv.log_page)] * a.kv.page;
        slot = pos & (a.kv.page_tokens() - 1);
      }
    }
    if (lane == 0) {
      s_page[r] = at;
      s_slot[r] = slot;
    }
  }
  __syncthreads();
  const int word = lane & 3;
  for (int u = warp; u < kReadTokens / 8 * a.kv.heads * 2; u += kReadThreads / 32) {
    const int r = (u & 3) * 8 + (lane >> 2);
    const int which = (u >> 2) & 1, head = u >> 3;
    T* dst = static_cast<T*>(which ? a.v_out : a.k_out);
    if (dst == nullptr || row0 + r >= a.s.total) continue;
    dst += ((row0 + r) * a.kv.heads + head) * D;
    const int64_t page = s_page[r];
    const int32_t slot = s_slot[r];
    uint32_t w[kGroups], sb[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      w[g] = 0x88888888u;
      sb[g] = kScaleLow;
      if (page >= 0) {
        const uint8_t* blk = a.kv.pages + page + ((int64_t)head * 2 + which) * a.kv.block;
        w[g] = *reinterpret_cast<const uint32_t*>(blk + code_at(g, slot, a.kv.log_page) + word * 4);
        sb[g] = blk[scale_at<D>(g, slot, a.kv.log_page)];
      }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float s = scale_value(sb[g]);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (float)((int32_t)((w[g] >> (4 * (e / 2 + 4 * (e % 2)))) & 15u) - 8) * s;
      store8(dst + g * kKvGroup + word * 8, x);
    }
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace
}  // namespace sdcp

using namespace sdcp;

extern "C" size_t sdcp_kv_page_bytes(int32_t page_tokens, int32_t kv_heads, int32_t head_dim) {
  if (page_tokens < 16 || page_tokens > 1024 || (page_tokens & (page_tokens - 1)) != 0) return 0;
  if (kv_heads < 1 || kv_heads > 256 || (head_dim != 64 && head_dim != 128)) return 0;
  return (size_t)2 * (size_t)kv_heads * (size_t)page_tokens * (size_t)(head_dim / 2 + head_dim / kKvGroup);
}

extern "C" int sdcp_append_kv(const sdcp_kv_cache* cache, int32_t B, const int32_t* m_offsets,
                              int64_t total_drafts, const int32_t* kv_len, int dtype, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride,
                              const sdcp_rotary* rotary, const void* q, int64_t q_stride,
                              int32_t q_heads, void* q_out, int32_t* status, void* stream) {
  KvView kv;
  const int rc = kv_view(cache, &kv);
  if (rc != SDCP_OK) return rc;
  if (B < 0 || total_drafts < 0 || q_heads < 0) return SDCP_E_INVALID;
  if (dtype != SDCP_F32 && dtype != SDCP_BF16) return SDCP_E_INVALID;
  if (total_drafts + B > (int64_t)INT32_MAX / 2) return SDCP_E_TOO_LARGE;
  const int32_t D = cache->head_dim;
  if (rotary) {
    if (rotary->struct_size < sizeof(sdcp_rotary) || !rotary->table || rotary->n_positions < 1) return SDCP_E_INVALID;
    if (rotary->layout != SDCP_ROTARY_HALF && rotary->layout != SDCP_ROTARY_INTERLEAVED) return SDCP_E_INVALID;
    if (rotary->rot_dim < 2 || rotary->rot_dim > D || rotary->rot_dim % 2 != 0) return SDCP_E_INVALID;
    if (((uintptr_t)rotary->table & 3u) != 0) return SDCP_E_ALIGN;
  }
  if (B == 0) return SDCP_OK;
  if (!m_offsets || !kv_len || !k || !v || !status) return SDCP_E_INVALID;
  if ((q != nullptr) != (q_out != nullptr) || (q != nullptr && q_heads < 1)) return SDCP_E_INVALID;
  const int64_t kv_row = (int64_t)cache->kv_heads * D, q_row = (int64_t)q_heads * D;
  if (k_stride < kv_row || v_stride < kv_row || (q && q_stride < q_row)) return SDCP_E_INVALID;
  const int64_t per16 = dtype == SDCP_BF16 ? 8 : 4;
  if (!aligned16(k) || !aligned16(v) || k_stride % per16 != 0 || v_stride % per16 != 0) return SDCP_E_ALIGN;
  if (q && (!aligned16(q) || !aligned16(q_out) || q_stride % per16 != 0)) return SDCP_E_ALIGN;
  DeviceInfo di;
  if (!device_info(&di)) return SDCP_E_DEVICE;

  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const KvSessions s{B, m_offsets, total_drafts, 1, kv_len, -1, rotary ? rotary->n_positions : INT32_MAX};
  if (launch_kv_check(kv, s, status, st) != cudaSuccess) return SDCP_E_LAUNCH;
  const AppendArgs a{kv, s, k, v, q, k_stride, v_stride, q_stride, q ? q_heads : 0, q_out,
                     rotary ? rotary->table : nullptr, rotary ? rotary->rot_dim : 0,
                     rotary && rotary->layout == SDCP_ROTARY_INTERLEAVED ? 1 : 0, status};
  // heads of a row over several CTAs where there are few rows
  const int64_t rows = total_drafts + B;
  const int64_t per_cta = (int64_t)(kAppendThreads / 32) * (128 / D);
  const int64_t most = (2 * (int64_t)cache->kv_heads + a.q_heads + per_cta - 1) / per_cta;
  const int64_t y = min(most, (2 * (int64_t)di.sms + rows - 1) / rows);
  const dim3 grid((unsigned)rows, (unsigned)max(y, (int64_t)1));
  cudaError_t e;
  if (dtype == SDCP_BF16)
    e = D == 128 ? launch_after(append_kernel<__nv_bfloat16, 128>, grid, kAppendThreads, 0, st, a)
                 : launch_after(append_kernel<__nv_bfloat16, 64>, grid, kAppendThreads, 0, st, a);
  else
    e = D == 128 ? launch_after(append_kernel<float, 128>, grid, kAppendThreads, 0, st, a)
                 : launch_after(append_kernel<float, 64>, grid, kAppendThreads, 0, st, a);
  return e == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}

extern "C" int sdcp_read_kv(const sdcp_kv_cache* cache, int32_t B, const int32_t* offsets,
                            int64_t n_tokens, const int32_t* start, int dtype, void* k_out,
                            void* v_out, int32_t* status, void* stream) {
  KvView kv;
  const int rc = kv_view(cache, &kv);
  if (rc != SDCP_OK) return rc;
  if (B < 0 || n_tokens < 0) return SDCP_E_INVALID;
  if (dtype != SDCP_F32 && dtype != SDCP_BF16) return SDCP_E_INVALID;
  if (n_tokens > (int64_t)INT32_MAX / 2) return SDCP_E_TOO_LARGE;
  if (B == 0) return SDCP_OK;
  if (!offsets || !start || !status || (n_tokens > 0 && !k_out && !v_out)) return SDCP_E_INVALID;
  if (!aligned16(k_out) || !aligned16(v_out)) return SDCP_E_ALIGN;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const KvSessions s{B, offsets, n_tokens, 0, start, -1, INT32_MAX};
  if (launch_kv_check(kv, s, status, st) != cudaSuccess) return SDCP_E_LAUNCH;
  if (n_tokens == 0) return SDCP_OK;
  const ReadArgs a{kv, s, k_out, v_out, status};
  const dim3 grid((unsigned)((n_tokens + kReadTokens - 1) / kReadTokens));
  cudaError_t e;
  if (dtype == SDCP_BF16)
    e = cache->head_dim == 128 ? launch_after(read_kernel<__nv_bfloat16, 128>, grid, kReadThreads, 0, st, a)
                               : launch_after(read_kernel<__nv_bfloat16, 64>, grid, kReadThreads, 0, st, a);
  else
    e = cache->head_dim == 128 ? launch_after(read_kernel<float, 128>, grid, kReadThreads, 0, st, a)
                               : launch_after(read_kernel<float, 64>, grid, kReadThreads, 0, st, a);
  return e == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}
