// The 5th-generation tensor cores' building blocks (sm_103a): shared-memory
// barriers with bounded waits, tiled copies, tensor memory, descriptors.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "arx_device.cuh"

namespace arx {

// ---- mbarriers --------------------------------------------------------------------

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}

// Makes the initialisations visible to the copy engine and the cluster.
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
               " selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}

// Bound of every wait: `limit_ns` (two seconds unless a call says less) of the
// global timer, as far as the block was running: what passes between two looks
// at the timer, 64 polls that suspend the thread for 4 us each, counts as half a
// millisecond at most, so that a block that is suspended in between (time
// slices, a debugger) does not run out of time standing still (beside a busy
// process waits of 2.4 ms ran out of 6 ms of the timer alone, none of 4.5 ms so),
// and as a microsecond at least, in case the timer stood still.  A wait that
// runs out raises the block's abort flag, which ends its other waits too.
// (32 bits, and no count of the polls: the threads that load operands have no
// registers to spare around the call.)
constexpr uint32_t kWaitNs = 2000000000u, kPollsToLook = 64, kLeastNs = 1000, kMostNs = 500000;

struct Waits {
  uint32_t limit_ns, abort;
};

__device__ __forceinline__ uint32_t global_timer_low_ns() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}

__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile Waits* w) {
  uint32_t last = global_timer_low_ns(), waited = 0;
  do {
    for (uint32_t i = 0; i < kPollsToLook; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    const uint32_t now = global_timer_low_ns(), passed = now - last;
    last = now;
    waited += passed < kLeastNs ? kLeastNs : passed < kMostNs ? passed : kMostNs;
  } while (!w->abort && waited <= w->limit_ns);
  w->abort = 1;
  return false;
}

// True once the barrier's phase `parity` has completed, false when the block
// gave up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile Waits* w) {
  if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_slow(bar, parity, w);
}

// Counts `bytes` of a phase as arrived.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}

// ---- tiled copies (TMA) -----------------------------------------------------------

__device__ __forceinline__ void prefetch_tensor_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" :: "l"(m) : "memory");
}

// Box at (x, y) of a two-dimensional map to shared memory; the bytes count on
// `bar`.  x is a multiple of 8 elements of 16 bits; parts of the box outside
// the matrix are filled with zeros.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t x, uint32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
}

// Box at (0, y, z) of a three-dimensional map (see copy_operand).
template <bool kPair>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t y, uint32_t z, uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(m), "r"(0u), "r"(y), "r"(z), "r"(bar) : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(m), "r"(0u), "r"(y), "r"(z), "r"(bar) : "memory");
}

// The same by a block of a pair, counted on a barrier that may be the other
// block's (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m, uint32_t x, uint32_t y,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
}

// Box at (x, y) from shared memory to a map's matrix, the parts inside it; one
// bulk group.  x is a multiple of 8 elements of 16 bits, neither is negative.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t x, uint32_t y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
               :: "l"(m), "r"(x), "r"(y), "r"(src) : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// All but the thread's last kGroups bulk groups have read shared memory.
template <int kGroups>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" :: "n"(kGroups) : "memory");
}

// The thread's bulk groups are complete.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Arrival on a barrier of another block of the cluster.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_bar) : "memory");
}

// Orders this thread's shared-memory stores before later reads by the tensor
// cores and the copy engine.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tensor memory ------------------------------------------------------------------

// One whole warp (of each block of a pair); columns a power of two, 32..512.
// The address is stored to shared memory.
template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t columns) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}

template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(columns) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(columns) : "memory");
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of the warp's 32 lanes: thread l gets lane l's 16 values, valid
// after tmem_load_wait.
__device__ __forceinline__ void tmem_load16_start(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr) : "memory");
}

// Waits for the warp's loads; `r` passes through, so that no use of it moves
// above the wait.
__device__ __forceinline__ void tmem_load_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  tmem_load16_start(addr, r);
  tmem_load_wait(r);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// ---- matrix instructions ------------------------------------------------------------

// Shared-memory descriptor of an operand tile in 128-byte swizzle: rows of 64
// 16-bit elements, eight rows to a 1024-byte atom.
//  K-major  (rows are matrix rows, 64 contraction elements each): atoms of 8
//           matrix rows 1024 bytes apart; the other offset is unused.
//  MN-major (rows are contraction steps, 64 matrix rows each): `leading` is
//           the distance between blocks of 64 matrix rows, 1024 bytes that
//           between groups of 8 contraction steps.
__device__ __forceinline__ uint64_t operand_descriptor(uint32_t addr, uint32_t leading) {
  return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t((leading >> 4) & 0x3FFFu) << 16) |
         (uint64_t(1024u >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// D[tmem] (+)= A B over 16 contraction steps (one thread issues it).  In a
// pair, each block's shared memory holds its half of A's rows and of B's, at
// the same addresses, and each block's tensor memory receives its rows.
template <bool kPair>
__device__ __forceinline__ void mma_f16(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
        :: "r"(tmem), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate)) : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
        :: "r"(tmem), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate)) : "memory");
}

// Arrives on `bar` (of both blocks of a pair) when every matrix instruction
// this thread issued is done.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        :: "r"(bar), "h"(uint16_t(3)) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}

// The same on this block's `bar` alone.
template <bool kPair>
__device__ __forceinline__ void mma_commit_own(uint32_t bar) {
  if constexpr (kPair)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
  else
    mma_commit<false>(bar);
}

// Instruction descriptor: fp32 accumulators, both operands bf16 or both fp16.
inline uint32_t mma_descriptor(bool bf16, bool a_mn, bool b_mn, uint32_t m, uint32_t n) {
  return (1u << 4) | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10) | (uint32_t(a_mn) << 15) |
         (uint32_t(b_mn) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// ---- distributed shared memory -----------------------------------------------------

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

}  // namespace arx
