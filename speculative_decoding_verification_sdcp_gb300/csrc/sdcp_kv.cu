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
  if (((uintptr_t)c->pages & 15u) != 0 || !on_words(c->page_table)) return SDCP_E_ALIGN;
  int log_page = 0;
  while ((1 << log_page) < c->page_tokens) ++log_page;
  *out = KvView{c->pages, c->page_table, c->n_pages, c->max_pages, c->kv_heads, log_page,
                (int32_t)(page / 2 / (size_t)c->kv_heads), (int64_t)page};
  return SDCP_OK;
}

namespace {

constexpr int kOffsetsThreads = 1024;
__global__ void __launch_bounds__(kOffsetsThreads) offsets_kernel(const int32_t* offsets, int32_t B, int32_t* status) {
  let_next_start();
  const bool bad = __syncthreads_or(!offsets_in_order(offsets, B)) != 0;
  const int64_t b = (int64_t)blockIdx.x * kOffsetsThreads + threadIdx.x;
  if (b < B) status[b] = bad ? SDCP_S_BAD_PARAMS : SDCP_S_OK;
}

}  // namespace

cudaError_t launch_offsets_check(const int32_t* offsets, int32_t B, int32_t* status, cudaStream_t stream) {
  if (B <= kScanSessions) return cudaSuccess;
  offsets_kernel<<<(unsigned)((B - 1) / kOffsetsThreads + 1), kOffsetsThreads, 0, stream>>>(offsets, B, status);
  return cudaGetLastError();
}

namespace {

__global__ void __launch_bounds__(kCheckThreads) kv_check_kernel(const KvView kv, const KvSessions s, int32_t* status) {
  let_next_start();
  const int32_t st = kv_session_status(kv, s, (int32_t)blockIdx.x, status);
  if (threadIdx.x == 0) status[blockIdx.x] = st;
}

cudaError_t launch_kv_check(const KvView& kv, const KvSessions& s, int32_t* status, cudaStream_t stream) {
  const cudaError_t e = launch_offsets_check(s.offsets, s.B, status, stream);
  if (e != cudaSuccess) return e;
  return launch_after_if(s.B > kScanSessions, kv_check_kernel, (unsigned)s.B, kCheckThreads, 0, stream, kv, s, status);
}

// ---- append ---------------------------------------------------------------------------

// Bound by latency: by its chain of loads (offsets, session, page, angles) in short rounds, and in long
// ones by the bytes it has in flight (15165 rows: DRAM at 55 % of its cycles, 38 % of the warps that an SM
// holds, three of four stalls wait for a load).  A warp has a row: it finds the row's session, position,
// page and angles once, behind its first loads, and goes over the heads, eight channels a lane (16 bytes
// of bfloat16, one word of codes), a few heads' loads in flight.  Short rounds share a row's heads among
// several warps.
// Measured: 15165 rows of 28 + 4 + 4 float heads of 64 channels, 256 MB read and written: 49 us, 5.3 TB/s;
// 2597 rows of 64 + 8 + 8 bfloat16 heads of 128 channels, 99 MB: 26 us, 3.8 TB/s; a few rows: the
// host's time for two launches (10 us on the GPU with a read of the rows).  With a CTA a row, each finding
// its session anew, these calls and a read of the rows took 114 and 81 us against 64 and 44.
constexpr int kAppendThreads = 128;
constexpr int kChan = 8;

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

__device__ __forceinline__ void load8(const float* p, float (&x)[kChan]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[kChan]) {
  uint32_t b[8];
  Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(p), b);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(b[j]);
}
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
__device__ __forceinline__ float elem(const float* p) { return *p; }
__device__ __forceinline__ float elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Eight channels as they are in memory.
template <typename T> struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) v[j] = reinterpret_cast<const uint4*>(p)[j];
  }
  __device__ __forceinline__ void values(float (&x)[kChan]) const { load8(reinterpret_cast<const T*>(v), x); }
};

// How a lane's channels turn: with their neighbours, with eight channels half a rotation away, or (a
// half that is no multiple of eight, or a table off its boundary) one by one.
enum { kStay, kNeighbours, kHalves, kOneByOne };
template <int kKind> struct Turn {
  float cs[kChan], sn[kChan];  // cosines, and sines with their signs
  int c0, rot;
  bool on;  // some of the lane's channels turn
  __device__ __forceinline__ Turn(const AppendArgs& a, int c) : c0(c), rot(a.rot), on(kKind != kStay && c < a.rot) {}
  __device__ __forceinline__ void angles(const AppendArgs& a, int64_t pos) {
    if (!on) return;
    const float* const row = a.table + pos * rot;
    const int half = rot / 2;
    if (kKind == kHalves) {
      const int pair = c0 >= half ? c0 - half : c0;
      load8(row + pair, cs);
      load8(row + half + pair, sn);
      if (c0 < half)
#pragma unroll
        for (int j = 0; j < kChan; ++j) sn[j] = -sn[j];
    } else {
#pragma unroll
      for (int j = 0; j < kChan; ++j) {
        const int c = c0 + j;
        const bool in = c < rot, second = a.interleaved ? (c & 1) != 0 : c >= half;
        const int pair = a.interleaved ? c >> 1 : second ? c - half : c;
        cs[j] = in ? row[pair] : 1.0f;
        const float s = in ? row[half + pair] : 0.0f;
        sn[j] = second ? s : -s;
      }
    }
  }
  // x1 cos - x2 sin and x2 cos + x1 sin, each product and sum rounded by itself; x: the lane's
  // channels of the head at src
  template <typename T> __device__ __forceinline__ void turn(const T* src, float (&x)[kChan]) const {
    if (!on) return;
    const int half = rot / 2;
    float y[kChan];
    if (kKind == kNeighbours) {
#pragma unroll
      for (int j = 0; j < kChan; ++j) y[j] = x[j ^ 1];
    } else if (kKind == kHalves) {
      load8(src + (c0 < half ? c0 + half : c0 - half), y);
    } else {
#pragma unroll
      for (int j = 0; j < kChan; ++j) {
        const int c = c0 + j;
        y[j] = c < rot ? elem(src + (c < half ? c + half : c - half)) : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < kChan; ++j)
      if (kKind == kHalves || c0 + j < rot) x[j] = __fadd_rn(__fmul_rn(x[j], cs[j]), __fmul_rn(y[j], sn[j]));
  }
};

// CTAs of an SM, each call with a read of its rows, us with 5 / 6 / 7 / 8: the calls above 70 / 70 / 66 / 67
// and 46 / 47 / 47 / 47; prompts of 16004 rows, 32 + 8 + 8 heads of 128 channels: bfloat16 in halves
// 131 / 125 / 123 / 119, with neighbours 120 / 112 / 105 / 104, float in halves 169 / 159 / 148 / 152;
// 28 + 4 + 4 bfloat16 heads of 64, 53 / 53 / 50 / 51.  (bfloat16 in halves spills 24 bytes with 7.)
// Channels that turn one by one need the registers of 5.
template <int kKind> constexpr int kAppendCtas = kKind == kOneByOne ? 5 : 7;
template <typename T, int D, int kKind>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas<kKind>) append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / kChan;               // lanes of a head
  constexpr int kHeads = 32 / kLanes;             // heads of a warp at once
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;  // and times that in flight
  const int lane = (int)(threadIdx.x & 31u);
  const int c0 = (lane % kLanes) * kChan, own = lane / kLanes;
  const int step = (int)gridDim.y * kHeads, h_first = (int)blockIdx.y * kHeads;
  const int64_t row = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  if (row >= a.s.total + a.s.B) return;
  wait_for_previous();

  // keys and values: head h below the cached heads is a key's, else a value's
  const int kv2 = 2 * a.kv.heads;
  const T* const k_row = static_cast<const T*>(a.k) + row * a.k_stride;
  const T* const v_row = static_cast<const T*>(a.v) + row * a.v_stride - (int64_t)a.kv.heads * D;
  Raw<T> raw[kBatch];
  auto load_kv = [&](int hs) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = hs + u * step + own;
      if (h < kv2) raw[u].load((h < a.kv.heads ? k_row : v_row) + h * D + c0);
    }
  };
  load_kv(h_first);

  const int32_t b = find_session(a.s.offsets, a.s.B, row, true);
  const int32_t off = a.s.offsets[b];
  const int64_t i = row - off - b;
  if (a.status[b] != SDCP_S_OK || i < 0 || i > (int64_t)a.s.offsets[b + 1] - off) return;
  const int32_t pos = a.s.start[b] + (int32_t)i;
  const int32_t page = a.kv.page_table[(int64_t)b * a.kv.max_pages + (pos >> a.kv.log_page)];
  Turn<kKind> t(a, c0);
  t.angles(a, pos);

  const int g = c0 / kKvGroup;
  const int32_t slot = pos & (a.kv.page_tokens() - 1);
  uint8_t* const pg = a.kv.pages + (int64_t)page * a.kv.page;
  const int32_t code = code_at(g, slot, a.kv.log_page) + (c0 % kKvGroup) / kChan * 4, scale = scale_at<D>(g, slot, a.kv.log_page);
  for (int hs = h_first; hs < kv2; hs += kBatch * step) {
    if (hs != h_first) load_kv(hs);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (hs + u * step >= kv2) break;
      const int h = hs + u * step + own;
      const bool live = h < kv2, is_k = h < a.kv.heads;
      float x[kChan];
      raw[u].values(x);
      if (is_k) t.turn(k_row + h * D, x);
      // the largest magnitude over the group's four lanes (fmaxf leaves a NaN out)
      float most = 0.0f;
#pragma unroll
      for (int j = 0; j < kChan; ++j) most = fmaxf(most, fabsf(x[j]));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      const uint32_t sb = scale_byte(most);
      const float s = scale_value(sb);
      uint32_t w = 0u;
#pragma unroll
      for (int j = 0; j < kChan; ++j) {
        const float n = fminf(fmaxf(rintf(__fdiv_rn(x[j], s)), -7.0f), 7.0f);
        const uint32_t c = isnan(x[j]) ? 8u : (uint32_t)((int32_t)n + 8);
        w |= c << (4 * (j / 2) + 16 * (j % 2));
      }
      if (live) {
        uint8_t* const blk = pg + ((int64_t)(is_k ? h : h - a.kv.heads) * 2 + (is_k ? 0 : 1)) * a.kv.block;
        *reinterpret_cast<uint32_t*>(blk + code) = w;
        if ((c0 % kKvGroup) == 0) blk[scale] = (uint8_t)sb;
      }
    }
  }
  // queries
  const T* const q_row = static_cast<const T*>(a.q) + row * a.q_stride;
  T* const q_to = static_cast<T*>(a.q_out) + row * a.q_heads * D + c0;
  for (int h = h_first + own; h < a.q_heads; h += kBatch * step) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (h + u * step < a.q_heads) raw[u].load(q_row + (int64_t)(h + u * step) * D + c0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (h + u * step < a.q_heads) {
        float x[kChan];
        raw[u].values(x);
        t.turn(q_row + (int64_t)(h + u * step) * D, x);
        store8(q_to + (int64_t)(h + u * step) * D, x);
      }
  }
}

template <typename T, int D>
cudaError_t launch_append(const AppendArgs& a, dim3 grid, cudaStream_t st) {
  if (a.table == nullptr) return launch_after(append_kernel<T, D, kStay>, grid, kAppendThreads, 0, st, a);
  if (a.interleaved) return launch_after(append_kernel<T, D, kNeighbours>, grid, kAppendThreads, 0, st, a);
  if (a.rot % (2 * kChan) == 0 && ((uintptr_t)a.table & 15u) == 0) return launch_after(append_kernel<T, D, kHalves>, grid, kAppendThreads, 0, st, a);
  return launch_after(append_kernel<T, D, kOneByOne>, grid, kAppendThreads, 0, st, a);
}

// ---- read -----------------------------------------------------------------------------

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 32;  // rows of a CTA, one per lane of its first warp

struct ReadArgs {
  KvView kv;
  KvSessions s;
  void *k_out, *v_out;
  const int32_t* status;
};

// A warp reads eight tokens of one head: the four words of a group of each, then the next group.
// Bound by memory: what is written is 3.8 times what is read, both in whole lines.  12 sessions of
// 8000 .. 24000 tokens, 8 heads of 128 channels to bfloat16: 152 us, 0.95 GB at 6.2 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadArgs a) {
  constexpr int kGroups = D / kKvGroup;
  __shared__ int64_t s_page[kReadTokens];  // byte offset of a row's page, -1: the row is zero
  __shared__ int32_t s_slot[kReadTokens];
  const int lane = (int)(threadIdx.x & 31u), warp = (int)(threadIdx.x >> 5);
  const int64_t row0 = (int64_t)blockIdx.x * kReadTokens;
  wait_for_previous();
  if (warp == 0) {  // the first row's session by a search, the others' from there on
    int32_t b = find_session(a.s.offsets, a.s.B, row0, false);
    const int64_t row = row0 + lane;
    int64_t at = -1;
    int32_t slot = 0;
    if (row < a.s.total) {
      while (b + 1 < a.s.B && a.s.offsets[b + 1] <= row) ++b;
      const int64_t i = row - a.s.offsets[b];
      if (a.status[b] == SDCP_S_OK && i >= 0 && row < a.s.offsets[b + 1]) {
        const int32_t pos = a.s.start[b] + (int32_t)i;
        at = (int64_t)a.kv.page_table[(int64_t)b * a.kv.max_pages + (pos >> a.kv.log_page)] * a.kv.page;
        slot = pos & (a.kv.page_tokens() - 1);
      }
    }
    s_page[lane] = at;
    s_slot[lane] = slot;
  }
  __syncthreads();
  const int word = lane & 3;
  for (int u = (int)blockIdx.y * (kReadThreads / 32) + warp; u < kReadTokens / 8 * a.kv.heads * 2; u += (int)gridDim.y * (kReadThreads / 32)) {
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
  if (total_drafts > (int64_t)INT32_MAX / 2 - B) return SDCP_E_TOO_LARGE;
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
  if (!on_words(m_offsets, kv_len, status)) return SDCP_E_ALIGN;
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
  // a row's heads over several warps where there are few rows
  const int64_t rows = total_drafts + B, per_warp = (int64_t)32 / (D / kChan);
  const int64_t most = (max(2 * (int64_t)cache->kv_heads, (int64_t)a.q_heads) + per_warp - 1) / per_warp;
  const int64_t y = max((int64_t)1, min(most, 24 * (int64_t)di.sms / rows));
  const dim3 grid((unsigned)((rows + kAppendThreads / 32 - 1) / (kAppendThreads / 32)), (unsigned)y);
  cudaError_t e;
  if (dtype == SDCP_BF16) e = D == 128 ? launch_append<__nv_bfloat16, 128>(a, grid, st) : launch_append<__nv_bfloat16, 64>(a, grid, st);
  else e = D == 128 ? launch_append<float, 128>(a, grid, st) : launch_append<float, 64>(a, grid, st);
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
  if (!aligned16(k_out) || !aligned16(v_out) || !on_words(offsets, start, status)) return SDCP_E_ALIGN;
  DeviceInfo di;
  if (!device_info(&di)) return SDCP_E_DEVICE;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const KvSessions s{B, offsets, n_tokens, 0, start, -1, INT32_MAX};
  if (launch_kv_check(kv, s, status, st) != cudaSuccess) return SDCP_E_LAUNCH;
  if (n_tokens == 0) return SDCP_OK;
  const ReadArgs a{kv, s, k_out, v_out, status};
  // heads over several CTAs where there are few tokens
  const int64_t chunks = (n_tokens + kReadTokens - 1) / kReadTokens;
  const dim3 grid((unsigned)chunks, (unsigned)max((int64_t)1, min((int64_t)cache->kv_heads, 8 * (int64_t)di.sms / chunks)));
  cudaError_t e;
  if (dtype == SDCP_BF16)
    e = cache->head_dim == 128 ? launch_after(read_kernel<__nv_bfloat16, 128>, grid, kReadThreads, 0, st, a)
                               : launch_after(read_kernel<__nv_bfloat16, 64>, grid, kReadThreads, 0, st, a);
  else
    e = cache->head_dim == 128 ? launch_after(read_kernel<float, 128>, grid, kReadThreads, 0, st, a)
                               : launch_after(read_kernel<float, 64>, grid, kReadThreads, 0, st, a);
  return e == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}
