// What the tensor-core attention kernels share (tq_kv8_tc.cuh, tq_prompt_tc.cu): batches of MMAs, packed arithmetic,
// tensor-memory accesses of whole rows, short waits.

#pragma once

#include "tq_tc.cuh"

#include <cuda_runtime.h>

#include <cstdint>

namespace tq {
namespace tcx {

// O (+)= w V: eight steps of 16 tokens (8 columns of weights, 2048 B or 128 descriptor units of values).
__device__ __forceinline__ void mma8_values(uint32_t d, uint32_t w, uint64_t v, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred e, t, p;\n .reg .b32 w1, w2, w3, w4, w5, w6, w7;\n .reg .b64 v1, v2, v3, v4, v5, v6, v7;\n"
      " add.u32 w1, %1, 8;\n add.u32 w2, %1, 16;\n add.u32 w3, %1, 24;\n add.u32 w4, %1, 32;\n add.u32 w5, %1, 40;\n"
      " add.u32 w6, %1, 48;\n add.u32 w7, %1, 56;\n"
      " add.u64 v1, %2, 128;\n add.u64 v2, %2, 256;\n add.u64 v3, %2, 384;\n add.u64 v4, %2, 512;\n"
      " add.u64 v5, %2, 640;\n add.u64 v6, %2, 768;\n add.u64 v7, %2, 896;\n"
      " setp.ne.b32 p, %4, 0;\n setp.ne.b32 t, 1, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w1], v1, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w2], v2, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w3], v3, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w4], v4, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w5], v5, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w6], v6, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [w7], v7, %3, t;\n}\n" ::"r"(d),
      "r"(w), "l"(v), "r"(idesc), "r"(acc)
      : "memory");
}
// MN-major operand, 128-byte swizzle: token rows of 64 channels, 8-row groups 1024 B apart, channel halves 16 KB apart
__device__ __forceinline__ uint64_t vdesc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(16384 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Pairs of fp32 in one 64-bit register (Blackwell's packed fp32 arithmetic).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 128 columns of this thread's lane: four loads in flight, one wait.  The values pass through an empty statement
// behind the wait, so that nothing uses them before it.
__device__ __forceinline__ void tld32_start(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void pin8(float* v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]));
}
__device__ __forceinline__ void tld32x4(uint32_t taddr, float (&v)[128]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) tld32_start(taddr + 32u * i, v + 32 * i);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) pin8(v + 8 * i);
}
// A bounded wait in few instructions, for the issuing warp: the tensor pipe's queue is short, and between two batches
// of MMAs every instruction of the wait is a gap in it.
__device__ __forceinline__ uint32_t wait_short(uint32_t b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, %3;\n"
      "W%=:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra D%=;\n"
      " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra W%=;\nD%=:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(b), "r"(parity), "n"(kWaitS)
      : "memory");
  return done;
}

// A value that is the same in the whole warp, by a reduction: its result is a uniform register, and so is what follows
// from it (the MMAs' operands, so that no issue waits for moves).
__device__ __forceinline__ int uniform(int v) {       // v >= 0
  return static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(v)));
}

__device__ __forceinline__ void stg256(void* p, const uint32_t* v) {   // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int DV>
__device__ __forceinline__ void rescale_o(uint32_t to, float alpha) {
#pragma unroll 1
  for (int c = 0; c < DV / 16; ++c) {
    float o[16];
    uint32_t u[16];
    tld16(to + 16u * c, o);
#pragma unroll
    for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] * alpha);
    tst16(to + 16u * c, u);
  }
}
}  // namespace tcx
}  // namespace tq
