// sdcp_attend.cu - sdcp_attend_kv: attention of a round's rows over the paged 4-bit cache.
//
//   out[row][h] = sum_t p_t value_t / sum_t p_t,   p_t = 2^(c q.key_t - m),  c = scale log2(e),
//
// in one pass over the tokens with a running reference m of the row.
#include <climits>
#include <math.h>

#include "sdcp_kv.cuh"

namespace sdcp {
namespace {

constexpr int kTile = 128;     // tokens of a tile, one per thread
constexpr int kCols = 8;       // query heads a CTA handles at a time

struct AttendArgs {
  KvView kv;
  KvSessions s;
  const __nv_bfloat16* q;
  int64_t q_stride;
  int32_t q_heads;
  float c;
  __nv_bfloat16* out;
  const int32_t* status;
};

// One CTA per row and cached head: thread t scores token t of a tile against the row's query heads,
// then thread d sums channel d over the tile's tokens.
template <int D>
__global__ void __launch_bounds__(kTile) attend_kernel(const AttendArgs a) {
  constexpr int kGroups = D / kKvGroup;
  __shared__ float s_q[kCols][D];
  __shared__ float s_p[kCols][kTile];
  __shared__ float s_red[kCols][kTile / 32];
  __shared__ float s_m[kCols], s_l[kCols], s_f[kCols];
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const int32_t kvh = (int32_t)blockIdx.y;
  const int32_t share = a.q_heads / a.kv.heads;
  wait_for_previous();
  const int32_t b = session_of(a.s.offsets, a.s.B, 1, row);
  const int64_t i = row - a.s.offsets[b] - b;
  __nv_bfloat16* out = a.out + (row * a.q_heads + (int64_t)kvh * share) * D;
  if (a.status[b] != SDCP_S_OK || i < 0 || i > (int64_t)a.s.offsets[b + 1] - a.s.offsets[b]) {
    for (int k = tid; k < share * D; k += kTile) out[k] = __float2bfloat16_rn(0.0f);
    return;
  }
  const int32_t last = a.s.start[b] + (int32_t)i;
  const int32_t first = a.s.window > 0 ? max(0, last - a.s.window + 1) : 0;
  for (int32_t h0 = 0; h0 < share; h0 += kCols) {
    const int n = min(kCols, share - h0);
    __syncthreads();
    for (int k = tid; k < n * D; k += kTile)
      s_q[k / D][k % D] = __bfloat162float(a.q[row * a.q_stride + ((int64_t)kvh * share + h0) * D + k]) * a.c;
    if (tid < kCols) {
      s_m[tid] = -INFINITY;
      s_l[tid] = 0.0f;
    }
    float o[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) o[j] = 0.0f;
    for (int32_t t0 = first; t0 <= last; t0 += kTile) {
      __syncthreads();
      const int32_t t = t0 + tid;
      float sc[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) sc[j] = 0.0f;
      if (t <= last) {
        const int64_t page = a.kv.page_table[(int64_t)b * a.kv.max_pages + (t >> a.kv.log_page)];
        const uint8_t* blk = a.kv.pages + page * a.kv.page + (int64_t)kvh * 2 * a.kv.block;
        const int32_t slot = t & (a.kv.page_tokens() - 1);
        for (int g = 0; g < kGroups; ++g) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(blk + code_at(g, slot, a.kv.log_page));
          const float s = scale_value(blk[scale_at<D>(g, slot, a.kv.log_page)]);
          for (int x = 0; x < 4; ++x)
            for (int e = 0; e < 8; ++e) {
              const float k = (float)((int32_t)((w[x] >> (4 * (e / 2 + 4 * (e % 2)))) & 15u) - 8) * s;
#pragma unroll
              for (int j = 0; j < kCols; ++j) sc[j] += k * s_q[j][g * kKvGroup + x * 8 + e];
            }
        }
      }
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        if (t > last) sc[j] = -INFINITY;
        float m = sc[j];
        for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
        if (lane == 0) s_red[j][warp] = m;
      }
      __syncthreads();
      if (tid < kCols) {
        const float m = fmaxf(fmaxf(s_red[tid][0], s_red[tid][1]), fmaxf(s_red[tid][2], s_red[tid][3]));
        const float to = fmaxf(s_m[tid], m);
        s_f[tid] = s_m[tid] == -INFINITY ? 0.0f : exp2f(s_m[tid] - to);
        s_m[tid] = to;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const float p = t <= last ? exp2f(sc[j] - s_m[j]) : 0.0f;
        s_p[j][tid] = p;
        float l = p;
        for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, k);
        if (lane == 0) s_red[j][warp] = l;
      }
      __syncthreads();
      if (tid < kCols) s_l[tid] = s_l[tid] * s_f[tid] + (s_red[tid][0] + s_red[tid][1]) + (s_red[tid][2] + s_red[tid][3]);
      if (tid < D) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) o[j] *= s_f[j];
        const int g = tid / kKvGroup, e = tid % 8, x = (tid % kKvGroup) / 8;
        for (int k = 0; k < min(kTile, last - t0 + 1); ++k) {
          const int32_t u = t0 + k;
          const int64_t page = a.kv.page_table[(int64_t)b * a.kv.max_pages + (u >> a.kv.log_page)];
          const uint8_t* blk = a.kv.pages + page * a.kv.page + ((int64_t)kvh * 2 + 1) * a.kv.block;
          const int32_t slot = u & (a.kv.page_tokens() - 1);
          const uint32_t w = reinterpret_cast<const uint32_t*>(blk + code_at(g, slot, a.kv.log_page))[x];
          const float v = (float)((int32_t)((w >> (4 * (e / 2 + 4 * (e % 2)))) & 15u) - 8) *
                          scale_value(blk[scale_at<D>(g, slot, a.kv.log_page)]);
#pragma unroll
          for (int j = 0; j < kCols; ++j) o[j] += s_p[j][k] * v;
        }
      }
    }
    __syncthreads();
    if (tid < D)
      for (int j = 0; j < n; ++j) out[(int64_t)(h0 + j) * D + tid] = __float2bfloat16_rn(o[j] / s_l[j]);
  }
}

}  // namespace
}  // namespace sdcp

using namespace sdcp;

extern "C" size_t sdcp_attend_workspace_bytes(int32_t B, int64_t total_drafts, int32_t q_heads,
                                              int32_t kv_heads, int32_t head_dim) {
  if (B < 0 || total_drafts < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  return 256;
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
  if (total_drafts + B > (int64_t)INT32_MAX / 2) return SDCP_E_TOO_LARGE;
  if (B == 0) return SDCP_OK;
  const int32_t D = cache->head_dim;
  if (!m_offsets || !kv_len || !q || !out || !status) return SDCP_E_INVALID;
  if (q_stride < (int64_t)q_heads * D) return SDCP_E_INVALID;
  if (((uintptr_t)q & 15u) != 0 || ((uintptr_t)out & 15u) != 0 || q_stride % 8 != 0) return SDCP_E_ALIGN;
  if (!workspace || ((uintptr_t)workspace & 255u) != 0 || workspace_bytes < need) return SDCP_E_WORKSPACE;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const KvSessions s{B, m_offsets, total_drafts, 1, kv_len, window, INT32_MAX};
  if (launch_kv_check(kv, s, status, st) != cudaSuccess) return SDCP_E_LAUNCH;
  const AttendArgs a{kv, s, static_cast<const __nv_bfloat16*>(q), q_stride, q_heads, scale * 1.4426950408889634f,
                     static_cast<__nv_bfloat16*>(out), status};
  const dim3 grid((unsigned)(total_drafts + B), (unsigned)cache->kv_heads);
  const cudaError_t e = D == 128 ? launch_after(attend_kernel<128>, grid, kTile, 0, st, a)
                                 : launch_after(attend_kernel<64>, grid, kTile, 0, st, a);
  return e == cudaSuccess ? SDCP_OK : SDCP_E_LAUNCH;
}
