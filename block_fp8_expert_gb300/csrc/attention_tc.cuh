// What the tensor-core attention kernels share: bf16 operand descriptors, the
// TMEM accesses of a softmax, and the waits of their warps.
#pragma once

#include "decoder_internal.h"
#include "tcgen05.cuh"

namespace moe {
namespace attn {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896341f;

// A running maximum is moved (and what was summed so far rescaled) only once a
// score exceeds it by this many powers of two: weights stay below 2^8, which
// fp32 sums and bf16 weights hold as well as ones below 1.
constexpr float kMaxSlack = 8.f;

// Instruction descriptor: bf16 A and B, fp32 D; A K-major, or M-major (its
// rows run along the contiguous axis of shared memory), B K-major or N-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return tc::idesc_f16_f32(M, N) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16);
}
// Descriptor of an operand whose M (or N) axis is contiguous, 128-byte
// swizzled: rows of one K each hold 64 elements of M, groups of 8 rows lie 1024
// bytes apart, and the next 64 elements of M `next` bytes further on.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t smem_addr, uint32_t next) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
  d |= (uint64_t)(next >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Rows lane / 4 and lane / 4 + 8 of the first 16 lanes of this warp's TMEM
// quadrant, 64 columns: r[4 i + u] is column 8 i + 2 (lane % 4) + u of the
// former, r[4 i + 2 + u] of the latter.
__device__ __forceinline__ void ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// 16 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A barrier of `threads` threads that tells whether any of them says yes.
__device__ __forceinline__ bool bar_any(int id, int threads, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred.aligned q, %2, %3, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)yes), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Warp-uniform bounded wait.  Once one wait of a CTA has run out, `abort_flag`
// is set and every other returns at once: the roles then run through the rest
// of their loops, whose results are reported as invalid, and keep their
// barriers matched.
__device__ __forceinline__ void role_wait(volatile int* abort_flag, uint64_t* bar, uint32_t parity,
                                          int32_t* status) {
  bool done = mbar_try_wait(bar, parity);
  if (__all_sync(kAll, done)) return;
  const WaitBudget b = wait_budget();
  for (uint32_t n = 1;; ++n) {
    if (__any_sync(kAll, done)) {
      // (the phase is complete: the others see it, too)
      for (int r = 0; !done && r < (1 << 16); ++r) done = mbar_try_wait(bar, parity);
      if (__all_sync(kAll, done)) return;
      break;
    }
    if ((n & 31) == 1) {
      const bool give_up = *abort_flag != 0 || budget_spent(b);
      if (__any_sync(kAll, give_up)) break;
    }
    done = mbar_try_wait(bar, parity);
  }
  if ((threadIdx.x & 31) == 0 && !*abort_flag) {
    *abort_flag = 1;
    raise_status(status, MOE_DEV_WAIT_TIMEOUT);
  }
  __syncwarp();
}

// The low n bits, 0 <= n <= 64.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
}

}  // namespace attn
}  // namespace moe
