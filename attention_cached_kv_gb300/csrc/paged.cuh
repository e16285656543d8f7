// paged.cuh -- device helpers of the ragged serving step (paged_*.cu): rotation
// angles in fixed point, E4M3 conversions, the walk over requests.
#pragma once

#include "common.cuh"

namespace gattn {

// Angle of position `pos` at frequency `turn` (theta / 2 pi modulo 1, in units of
// 2^-64): the product modulo 2^64 is the angle modulo a whole turn, so nothing is
// lost at far positions (off by at most pos 2^-53 turns, the double that `turn`
// came from) and no range reduction is left.  In [-pi, pi).
__device__ __forceinline__ float turn_angle(int pos, uint64_t turn) {
  const uint64_t a = (uint64_t)(int64_t)pos * turn;
  return (float)(int32_t)(a >> 32) * 1.4629180792671596e-09f;  // 2 pi / 2^32
}

// Two floats to two E4M3 codes (nearest even, saturating at 448; `lo` in the low byte).
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes to an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t v) {
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(v));
  return f;
}

}  // namespace gattn
