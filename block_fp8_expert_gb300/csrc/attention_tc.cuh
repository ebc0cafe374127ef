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

// Instruction descriptor: bf16 A and B (HALF: fp16), fp32 D; A K-major, or M-major (its
// rows run along the contiguous axis of shared memory), B K-major or N-major.
template <bool HALF = false>
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return tc::idesc_f16_f32(M, N) | (HALF ? 0u : (1u << 7) | (1u << 10)) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16);
}
// Descriptors of 128-byte swizzled operands are built from their low words,
// which alone hold addresses, so that stepping through a tile is one addition
// (of bytes / 16).  K-major as tc::sw128_desc; with a contiguous M (or N) axis,
// rows of one K each hold 64 elements of M, groups of 8 rows lie 1024 bytes
// apart, and the next 64 elements of M `next` bytes further on.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t smem_addr) { return (smem_addr >> 4) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t smem_addr, uint32_t next) {
  return (smem_addr >> 4) | (next >> 4) << 16;
}
// The same value in every lane, in a form that tells the compiler so: the words
// of descriptors and TMEM addresses that change from tile to tile go through it
// (36 MMAs of 64 x 64 x 16, 32 cycles each, then follow one another without gaps;
// without it one took 51).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(kAll, v); }

// D[tmem] (+)= A[smem] B[smem]^T, descriptors by their low words.
__device__ __forceinline__ void mma_ss(uint32_t tmem_d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %5, 0;\n mov.b64 da, {%1, %3};\n"
      " mov.b64 db, {%2, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n}\n" ::"r"(tmem_d),
      "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]^T.
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %5, 0;\n mov.b64 db, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(accumulate)
      : "memory");
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
// The same of 32 columns.
__device__ __forceinline__ void ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
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

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
// Copies 4 bytes, or writes zeros when `valid` is false.
__device__ __forceinline__ void cp_async4_zfill(void* smem, const void* gmem, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(smem)), "l"(gmem),
               "r"(valid ? 4 : 0)
               : "memory");
}
// One arrival, counted by the barrier's initial number, once this thread's
// cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 A, B, C, R;\n mov.b64 A, {%2, %3};\n mov.b64 B, {%4, %5};\n mov.b64 C, {%6, %7};\n"
      " fma.rn.f32x2 R, A, B, C;\n mov.b64 {%0, %1}, R;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 A, B, R;\n mov.b64 A, {%2, %3};\n mov.b64 B, {%4, %5};\n add.rn.f32x2 R, A, B;\n"
      " mov.b64 {%0, %1}, R;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 A, B, R;\n mov.b64 A, {%2, %3};\n mov.b64 B, {%4, %5};\n mul.rn.f32x2 R, A, B;\n"
      " mov.b64 {%0, %1}, R;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// Whether a pair of bf16 (of fp16) values holds an infinity or a NaN.
template <bool HALF>
__device__ __forceinline__ bool nonfinite_16x2(uint32_t v) {
  constexpr uint32_t lo = HALF ? 0x7C00u : 0x7F80u, hi = lo << 16;
  return (v & lo) == lo || (v & hi) == hi;
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

// mbar_try_wait that may sleep for kNap nanoseconds.
constexpr uint32_t kNap = 20000;
__device__ __forceinline__ bool mbar_nap(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(kNap)
      : "memory");
  return ok != 0;
}
// Warp-uniform bounded wait; whether the phase has come (the same answer in every
// lane, which a read of `abort_flag` is not: another warp may raise it between two
// lanes' reads).  Once one wait of a CTA has run out, `abort_flag`
// is set and the others return after a nap: the roles then run through the rest
// of their loops, whose results are reported as invalid, and keep their
// barriers matched.  (Clocks and flag are only read once a nap is over: reading
// them takes as long as most waits, and a warp that polls takes issue slots and
// shared-memory cycles from those that work.)
// (out of line: every wait is in the way of the code that a first call fetches)
static __device__ __noinline__ bool role_wait_on(volatile int* abort_flag, uint64_t* bar, uint32_t parity,
                                                 int32_t* status) {
  const WaitBudget b = wait_budget();
  while (true) {
    bool done = mbar_nap(bar, parity);
    if (__any_sync(kAll, done)) {
      // (the phase is complete: the others see it, too)
      for (int r = 0; !done && r < (1 << 16); ++r) done = mbar_try_wait(bar, parity);
      if (__all_sync(kAll, done)) return true;
      break;
    }
    if (__any_sync(kAll, *abort_flag != 0 || budget_spent(b))) break;
  }
  if ((threadIdx.x & 31) == 0 && !*abort_flag) {
    *abort_flag = 1;
    raise_status(status, MOE_DEV_WAIT_TIMEOUT);
  }
  __syncwarp();
  return false;
}
__device__ __forceinline__ bool role_wait(volatile int* abort_flag, uint64_t* bar, uint32_t parity,
                                          int32_t* status) {
  return __all_sync(kAll, mbar_try_wait(bar, parity)) || role_wait_on(abort_flag, bar, parity, status);
}

// Three waits at once: a wait for what has long come still takes 180 cycles, which
// here pass side by side.
__device__ __forceinline__ void role_wait3(volatile int* abort_flag, uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                           uint64_t* c, uint32_t pc, int32_t* status) {
  const bool da = mbar_try_wait(a, pa), db = mbar_try_wait(b, pb), dc = mbar_try_wait(c, pc);
  if (__all_sync(kAll, da && db && dc)) return;
  role_wait(abort_flag, a, pa, status);
  role_wait(abort_flag, b, pb, status);
  role_wait(abort_flag, c, pc, status);
}

// The same by a thread on its own.
__device__ __forceinline__ void lane_wait(volatile int* abort_flag, uint64_t* bar, uint32_t parity,
                                          int32_t* status) {
  if (mbar_nap(bar, parity)) return;
  const WaitBudget b = wait_budget();
  while (!mbar_nap(bar, parity)) {
    if (*abort_flag) return;
    if (budget_spent(b)) {
      *abort_flag = 1;
      raise_status(status, MOE_DEV_WAIT_TIMEOUT);
      return;
    }
  }
}

// The low n bits, 0 <= n <= 64.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
}

}  // namespace attn
}  // namespace moe
