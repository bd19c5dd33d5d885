// tcgen05 matrix instructions, tensor memory and tensor-map loads (sm_103a), as
// the kernels over bf16 pages use them.
//
// Operands lie in shared memory as tensor-map loads with 128-byte swizzle leave
// them: a tile [rows][128] of bf16 is two halves of 64 columns, each [rows] of
// 128 bytes (rows * 128 bytes long), 1024 bytes per 8 rows.  Such a tile is
// either operand with its columns as the summed dimension ("K-major": queries
// times keys), or the second operand with its rows as the summed dimension
// ("MN-major": weights times values).
#pragma once

#include <cuda.h>

#include "locks_common.cuh"

namespace locks {

// ---- descriptors ------------------------------------------------------------
// Shared-memory matrix descriptor, 128-byte swizzle, 1024 bytes from 8 rows to the next: the low
// word (start address and leading byte offset in 16-byte units); the high word is the same for all
// (stride 1024, version 1 at bit 46, swizzle 2 at bit 61).
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t smem_desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFF) | ((lbo >> 4) & 0x3FFF) << 16;
}
// A value that all lanes have, in a form that the compiler keeps in a uniform register: a matrix
// instruction takes its operands from those, and five moves for each one cost more issue slots
// beside busy warps than the instruction lasts.
__device__ __forceinline__ uint32_t warp_uniform(uint32_t x) { return __shfl_sync(kFull, x, 0); }

// instruction descriptor of kind::f16: bf16 operands, float accumulators, M x N;
// the second operand MN-major if bit 16 is set
__host__ __device__ constexpr uint32_t mma_idesc(int m, int n, bool b_rows_summed) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_rows_summed ? 1u << 16 : 0u) |
         uint32_t(n >> 3) << 17 | uint32_t(m >> 4) << 24;
}

// ---- tensor memory ------------------------------------------------------------
// a whole warp; the base address lands in *slot (shared memory)
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(slot)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns)
               : "memory");
}

// 32 (16) columns of the warp's 32 lanes: thread = lane, one word a column
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// this thread's writes to shared memory become visible to matrix instructions
__device__ __forceinline__ void proxy_fence_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// one lane of a converged warp, always the same
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(yes));
  return yes != 0;
}

// ---- matrix instructions (one thread issues) ----------------------------------
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(add), "n"(kDescHi)
      : "memory");
}
// The eight instructions of a product of depth 128 in one piece, descriptors stepped in 64 bits:
// the issuing thread shares its scheduler with busy warps, where every instruction that it needs
// beside the products costs some 25 cycles.
// D = A B, A and B in shared memory, both with the summed dimension along the rows' 256 bytes
__device__ __forceinline__ void mma_ss_128(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.u32 p, 0, 0;\n setp.eq.u32 q, 0, 0;\n"
      " mov.b64 a, {%1, %4};\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n add.s64 a, a, 2;\n add.s64 b, b, 2;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n add.s64 a, a, 2;\n add.s64 b, b, 2;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n add.s64 a, a, 2;\n add.s64 b, b, 2;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n add.s64 a, a, %5;\n add.s64 b, b, %5;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n add.s64 a, a, 2;\n add.s64 b, b, 2;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n add.s64 a, a, 2;\n add.s64 b, b, 2;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n add.s64 a, a, 2;\n add.s64 b, b, 2;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kDescHi), "n"(16384 / 16 - 6)
      : "memory");
}
// D (+)= A B, A in tensor memory (two values a column; its second half 64 columns on), B's summed
// dimension its rows: 16 rows of 128 bytes a step
__device__ __forceinline__ void mma_ts_128(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                           uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 b;\n .reg .b32 x;\n setp.ne.u32 p, %4, 0;\n"
      " setp.eq.u32 q, 0, 0;\n mov.b64 b, {%2, %5};\n mov.b32 x, %1;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, p;\n add.u32 x, x, 8;\n add.s64 b, b, 128;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n add.u32 x, x, 8;\n add.s64 b, b, 128;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n add.u32 x, x, 8;\n add.s64 b, b, 128;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n add.u32 x, x, 40;\n add.s64 b, b, 128;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n add.u32 x, x, 8;\n add.s64 b, b, 128;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n add.u32 x, x, 8;\n add.s64 b, b, 128;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n add.u32 x, x, 8;\n add.s64 b, b, 128;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(add), "n"(kDescHi)
      : "memory");
}
// `bar` gets an arrival once everything this thread has issued so far is done
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// ---- tensor-map loads -----------------------------------------------------------
__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* map, int x, int y, int z,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- waits ------------------------------------------------------------------------
// Wait for phase `parity` of `bar`.  False, and *dead set, if the limit ran out or another
// thread of the block gave up: every role then leaves its loop.
__device__ __forceinline__ bool mbar_wait_or_dead(uint64_t* bar, uint32_t parity, volatile int* dead) {
  unsigned long long t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if (i & 255) continue;
    if (*dead) return false;
    const unsigned long long now = global_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      *dead = 1;
      return false;
    }
  }
  return true;
}

// The same for a whole warp: all of its lanes go on, or none.
__device__ __forceinline__ bool warp_wait_or_dead(uint64_t* bar, uint32_t parity, volatile int* dead) {
  return __all_sync(kFull, mbar_wait_or_dead(bar, parity, dead));
}

}  // namespace locks
