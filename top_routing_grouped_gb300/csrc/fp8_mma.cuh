// fp8_mma.cuh -- inline PTX of the block-scaled e4m3 MMA (kind::mxf8f6f4) and of its factors in
// TMEM, shared by the 8-bit products.
#pragma once
#include <stdint.h>

namespace moe {
namespace fp8 {

// Instruction descriptor of kind::mxf8f6f4 with e4m3 A and B (both K-major), e8m0 factors, fp32
// D: bits 4-5 B's factor byte, 7-9 / 10-12 the types (0 = e4m3), 17-22 N >> 3, 23 factor type
// (1 = e8m0), 24-28 M >> 4, 29-30 A's factor byte.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, uint32_t byte) {
  return (byte << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) | (byte << 29);
}
// One more in either factor byte.
__host__ __device__ constexpr uint32_t idesc_byte() { return (1u << 4) | (1u << 29); }

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// D (+)= A * B^T with block factors: a CTA pair (M = 256) or one CTA (M = 128).
__device__ __forceinline__ void mma_mxf8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// This lane's words to 4 or 8 columns of its warp's TMEM lane quarter.
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrives on a barrier of any CTA of the cluster after TMEM has been written or read (waited for, then
// tc_fence_before, which is all the order this needs).  A release to the cluster also waits for the
// warp's other accesses to memory, some 2000 clocks each time: with it 8192 x 2048 x 8192 took 94 us, not 86.
__device__ __forceinline__ void arrive_relaxed_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

}  // namespace fp8
}  // namespace moe
