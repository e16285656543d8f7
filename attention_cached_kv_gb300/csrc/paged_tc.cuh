// paged_tc.cuh -- tcgen05 wrappers of the paged kernels beside those of tcgen05.cuh:
// products of 8-bit operands, and one lane to issue them.
#pragma once

#include "tcgen05.cuh"

namespace gattn {
namespace tc {

// One lane of a converged warp, the same one every time.  The compiler knows the code
// under it to be a single thread's and keeps descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// Instruction descriptor for kind::f8f6f4 with E4M3 A and B, fp32 accumulate.
// a_mn_major: A stored with M contiguous.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N, uint32_t a_mn_major) {
  return (1u << 4)                 // D format: f32 (A and B format 0: E4M3)
         | (a_mn_major << 15)      // A major-ness
         | ((N >> 3) << 17)        // N / 8
         | ((M >> 4) << 24);       // M / 16
}

// 8-bit operands.
__device__ __forceinline__ void mma_ss_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

}  // namespace tc
}  // namespace gattn
