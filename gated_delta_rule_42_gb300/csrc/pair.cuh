// Helpers of the two-SM tensor-core kernel: tcgen05 with cta_group::2, whose
// operands lie half in each CTA of a pair and whose accumulator rows are split
// between the two tensor memories, TMA loads that report to the leader CTA's
// mbarrier, and arrivals across the pair.
#pragma once

#include "umma.cuh"

namespace kda {
namespace pair {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// Address, in the cluster's shared window, of the CTA `rank`'s copy of a shared variable.
__device__ __forceinline__ uint32_t at_rank(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(umma::smem_u32(p)), "r"(rank));
  return a;
}
// Hands back tensor memory that has been read (the loads waited for, then
// tcgen05.fence::before_thread_sync).  The release is the default one, of this
// CTA's scope: a release at cluster scope would also wait for the warp's global
// stores to arrive, 1200 clocks a tile, and the waiter reads none of them.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(umma::smem_u32(bar)), "r"(bytes)
               : "memory");
}
// Counts bytes that no copy will bring (the peer CTA ended before it issued its own).
__device__ __forceinline__ void complete_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(umma::smem_u32(bar)), "r"(bytes)
               : "memory");
}
// A word of the CTA `rank`'s shared memory.
__device__ __forceinline__ void store_at(uint32_t *p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(at_rank(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t load_at(const uint32_t *p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(at_rank(p, rank)) : "memory");
  return v;
}
// Bounded wait that also acquires what the peer CTA released (tensor memory
// handed back, barriers of the pair).
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, int polls) {
  for (int it = 0; it < polls; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(umma::smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}

// One lane of a converged warp, chosen by the hardware.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xffffffff;\nselp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}
// One look at the phase, without waiting.
__device__ __forceinline__ bool peek(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(umma::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A 2-D box into this CTA's shared memory; its bytes are counted on `bar`, an
// mbarrier of either CTA of the pair (an address of the cluster's window).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(umma::smem_u32(slot)),
               "r"(ncols));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
}
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols));
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

// D (+)= A B^T over the pair: A 256 x 16 (128 rows in each CTA), B 256 x 16 (128 rows in each).
__device__ __forceinline__ void mma(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// Arrives on `bar` in both CTAs once every tcgen05 operation issued so far is done.
__device__ __forceinline__ void commit_both(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
          umma::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// The same in this CTA alone.
__device__ __forceinline__ void commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(
                   umma::smem_u32(bar))
               : "memory");
}

// Operand with its rows contiguous (MN-major), 128-byte swizzle: blocks of 64
// rows x 64 k, each k one 128-byte line; 8-k groups 1024 bytes apart, 64-row
// blocks 8192 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(8192 >> 4) << 16;  // leading byte offset: the next 64 rows
  d |= (uint64_t)(1024 >> 4) << 32;  // stride byte offset: the next 8 k
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;  // SWIZZLE_128B
  return d;
}

}  // namespace pair
}  // namespace kda
