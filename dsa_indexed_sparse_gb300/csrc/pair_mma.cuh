// What the attention kernels on pairs of CTAs share: cluster and pair (cta_group::2)
// instructions, and a quick division.
#pragma once

#include <cuda.h>

#include "dsa_device.cuh"

namespace dsa {

// floor(n / d) for 0 <= n < 2^31 as (2 n mul) >> (32 + s): with 2^(s - 1) < d <= 2^s and mul =
// ceil(2^(31 + s) / d) < 2^32, the error mul d - 2^(31 + s) < d <= 2^s is too small to reach the next quotient.
struct Divisor {
  uint32_t mul, s;
  explicit Divisor(int64_t d) : s(0) {
    while ((1ll << s) < d) ++s;
    mul = static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>(__umulhi(static_cast<uint32_t>(n) << 1, mul) >> s);
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `bar` in the leader CTA (rank 0) of the cluster.
__device__ __forceinline__ uint32_t leader_addr(const uint64_t* bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
  return r;
}
// Arrival on a barrier of either CTA.  At CTA scope: what the arrival announces -- rows,
// P and logits read -- lies in this CTA's own shared memory and TMEM and is handed to
// the tensor cores by the proxy and tcgen05 fences before it.  A release at cluster
// scope waited for the warp's global loads as well: 4000 clocks a tile.
__device__ __forceinline__ void arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Whether a phase of `bar` is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
template <int kRegs>
__device__ __forceinline__ void shrink_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void grow_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// One arrival on `bar` of both CTAs when every MMA issued so far by this thread is complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// A barrier of `nthreads` threads that tells each whether any of them gave true.
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t nthreads, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(nthreads), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return any != 0;
}

// Tiled load of 64 values of rows from `row` on, atoms (64 values each) from `atom` on, into this
// CTA; its bytes are counted on a barrier of either CTA of the pair (bar: an address in the
// cluster's window).
__device__ __forceinline__ void tma_load_atoms_pair(void* smem_dst, const void* map, uint32_t bar, int32_t row, int32_t atom) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(map), "r"(bar), "r"(0), "r"(row), "r"(atom)
      : "memory");
}
// Stores a box of one atom of heads from `head` on of a token, from shared memory; part of the
// thread's bulk group.
__device__ __forceinline__ void tma_store_heads(const void* map, const void* smem_src, int32_t head, int32_t token,
                                                int32_t atom) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(map),
               "r"(smem_u32(smem_src)), "r"(0), "r"(head), "r"(token), "r"(atom)
               : "memory");
}
// Closes the thread's bulk group; waits until what its groups store has been read from shared
// memory, or has been written.
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Asks the L2 for `bytes` (a multiple of 16) from a 16-byte boundary on.
__device__ __forceinline__ void prefetch_l2_bulk(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

}  // namespace dsa
