// sdcp_tensor.cuh - what the attention kernels share: tcgen05 products and tensor memory, bounded waits,
// swizzled shared-memory matrices, and the turning of 4-bit codes into 16-bit numbers.
#pragma once

#include <math.h>

#include "sdcp_kv.cuh"

namespace sdcp {

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
__device__ __forceinline__ void tmem_ld32(uint32_t at, float (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
               : "r"(at)
               : "memory");
}
// The loads are done, and r is what they brought (named, so that no use of it is moved before).
__device__ __forceinline__ void tmem_loaded(float (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_loaded(float (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_loaded(float (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
               :
               : "memory");
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

}  // namespace sdcp
