// pair.cuh -- tcgen05 cta_group::2: two CTAs of a cluster (ranks 2p and 2p + 1)
// working on one tile.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "sm100.cuh"

namespace tidar {

// One copy into this CTA's shared memory, counted on a barrier of either CTA of
// the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// Issued by one thread of the pair's first CTA: A rows and B rows are halves in
// the two shared memories (at the same offsets), D the same columns of both TMEMs.
// A 64-deep slice: four MMAs (the K-major descriptors step by 32 bytes, 2 in their
// address field) as one asm block, so that the issuing thread spends its
// instructions on the MMAs.  The first accumulates when acc != 0.
__device__ __forceinline__ void mma_pair_x4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %10, 0;\n\tsetp.eq.b32 q, %10, %10;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %5, %9, p;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %2, %6, %9, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %3, %7, %9, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %4, %8, %9, q;\n\t}"
      ::"r"(d), "l"(a), "l"(a + 2), "l"(a + 4), "l"(a + 6), "l"(b), "l"(b + 2), "l"(b + 4), "l"(b + 6), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives on the barrier at the same offset in the CTAs of `mask` (cluster
// ranks) once every MMA issued so far is complete.
__device__ __forceinline__ void commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"(mask)
      : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

}  // namespace tidar
