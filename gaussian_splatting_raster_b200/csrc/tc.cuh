// tcgen05, TMEM, mbarrier and bulk-copy instructions as used by the feed-forward kernels.
//
// Operand tiles lie in shared memory as blocks of [rows][64] 16-bit elements, 128 bytes a row, the
// 16-byte pieces of a row exchanged by the 128-byte swizzle (piece c of row r at c ^ (r & 7)). The
// same block serves as a K-major operand (rows along M or N, columns along K) and as an MN-major
// one (columns along M or N, rows along K), so a transposed product needs no second copy.
//
// Every wait is bounded: after kWaitClocks a wait sets the failure flag and returns, later waits
// return at once, the kernel runs to its end (on meaningless values, within its buffers) and the
// status word tells the host.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace splat {
namespace tc {

constexpr long long kWaitClocks = 8000000000LL;  // about four seconds

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// arrivals that were pending before this one
__device__ __forceinline__ unsigned mbar_arrive_pending(uint32_t bar) {
  unsigned n;
  asm volatile(
      "{\n.reg .b64 s;\n"
      "mbarrier.arrive.shared::cta.b64 s, [%1];\n"
      "mbarrier.pending_count.b64 %0, s;\n}\n"
      : "=r"(n)
      : "r"(bar)
      : "memory");
  return n;
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// more bytes for the open phase, without an arrival
__device__ __forceinline__ void mbar_expect_more(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Whether the phase is complete, without the suspension that try_wait may take (for a thread that
// looks at several barriers in turn).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for the completion of the phase of the given parity, by whole warps: true where the phase is
// over (and, SURE, no wait of the CTA has failed so far). `failed` is the CTA's failure flag. A
// warp leaves together and with one result, a vote: its lanes may read the flag on either side of
// its being set.
template <bool SURE = false>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* failed,
                                          unsigned int* status) {
  bool over = mbar_try(bar, parity);
  if (!over) {
    const long long t0 = clock64();
    while (!(over = mbar_try(bar, parity))) {
      if (*failed) break;
      if (clock64() - t0 > kWaitClocks) {
        *failed = 1;
        atomicOr(status, 1u);
        break;
      }
    }
  }
  if (SURE) over = over && !*failed;
  return __all_sync(0xffffffffu, over);
}

// For what must be over before a CTA ends, also after a failed wait: copies and MMAs in flight,
// which end by themselves. It lasts twice as long as a wait, which may have run out shortly before.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity, unsigned int* status) {
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (clock64() - t0 > 2 * kWaitClocks) {
      atomicOr(status, 1u);
      break;
    }
  }
  __syncwarp();
}

// contiguous copy global -> shared, completing on the barrier (16-byte aligned, multiple of 16)
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// contiguous copy shared -> global (16-byte aligned, multiple of 16), in the thread's bulk group
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
}

// a box of a two-dimensional tensor map: column x (a multiple of 16 bytes), row y
__device__ __forceinline__ void tile_load(uint32_t dst, const void* map, int x, int y,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: its low word (start address and leading
// offset, in 16 bytes); the high word is the same for all tiles. K-major: groups of 8 rows lie
// 1,024 bytes apart (stride offset), the leading offset is not used. MN-major: groups of 8 K rows
// lie 1,024 bytes apart (stride offset), blocks of 64 columns `block_bytes` apart (leading offset).
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t block_bytes) {
  return ((addr & 0x3FFFF) >> 4) | ((block_bytes >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc(uint32_t lo) {
  constexpr uint32_t hi = (1024 >> 4) | (1u << 14) | (2u << 29);
  return ((uint64_t)hi << 32) | lo;
}

// Instruction descriptor: fp32 accumulator, both operands bf16 or both fp16, M = 128.
__device__ __forceinline__ uint32_t idesc(bool bf16, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
         ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((128u >> 4) << 24);
}

// One lane of a converged warp (the same one each time). Blocks that issue MMAs are entered under
// it, in loops with fixed counts and descriptors formed beforehand: an MMA of 128 x 128 x 16 takes
// 64 cycles, and with the lane chosen by an ordinary comparison and the descriptors formed inside
// a counted loop its issue alone took 105.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n.reg .pred P;\n"
      "elect.sync _|P, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, P;\n}\n"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id,
                                    bool add) {
  const uint64_t a = desc(a_lo), b = desc(b_lo);
  asm volatile(
      "{\n.reg .pred p;\n"
      "setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)add)
      : "memory");
}

// 32 lanes x 16 (8, 4) columns of fp32 from TMEM; lane = the warp's quadrant of rows
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr));
}
// Wait for this thread's TMEM loads. The loaded registers pass through, so that no use of them is
// moved before the wait.
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[N]) {
  static_assert(N == 4 || N == 8 || N == 16, "");
  if constexpr (N == 4)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3])
                 :
                 : "memory");
  else if constexpr (N == 16)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
  else
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7])
                 :
                 : "memory");
}

}  // namespace tc
}  // namespace splat
