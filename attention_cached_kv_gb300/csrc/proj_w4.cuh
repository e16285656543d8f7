// proj_w4.cuh -- what the two kernels of the 4-bit projections share: their parameters,
// the conversion of codes, and the end of a result (rotation and its place).
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace gattn {

struct W4Params {
  const bf16* x;
  const uint8_t* w;
  const bf16* scale;
  bf16* out[3];           // q, k_new, v_new; or y
  const int32_t* position;  // nullptr: output projection
  int32_t* status;
  int T, N, K, group, tiles, slice;  // slice: inputs of a CTA
  int Hq, Hkv, d, shift;  // d = 1 << shift
  uint64_t turn[64];
};

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// Bytes of x (0-3) and y (4-7) by a selector; with bit 3 of a selector's digit set, the byte's sign.
__device__ __forceinline__ uint32_t permute(uint32_t x, uint32_t y, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(sel));
  return r;
}
// Less 8 as bf16: 128 + c (c in the lower bits of the mantissa) is exact, and so is the difference.
__device__ __forceinline__ uint32_t less136(uint32_t v) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0x3f803f80u), "r"(0xc308c308u));  // 1 v - 136
  return r;
}
// Two codes (bits 0..3 and 16..19) less 8, as bf16.
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t c) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(c), "r"(0x000f000fu), "r"(0x43004300u));  // (c & mask) | 128.0
  return less136(v);
}
// The eight codes of a word less 8, over 64, as bf16 pairs in their order: ten instructions.
// Up to its lowest exponent a bf16 is a count of 2^-133, so that a code in bits 0-3 is c 2^-133
// and one in bits 4-7 is c 2^-129; one fma takes both, times 2^127 and 2^123, to (c - 8) / 64, exactly.
__device__ __forceinline__ void word_to_bf16(uint32_t u, uint32_t* a) {
  const uint32_t even = u & 0x0f0f0f0fu, odd = u & 0xf0f0f0f0u;
  constexpr uint32_t sel[4] = {0x8480, 0x9591, 0xa6a2, 0xb7b3};  // byte j of both, zeros (the signs of even's) between
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(a[j]) : "r"(permute(even, odd, sel[j])), "r"(0x7d007f00u), "r"(0xbe00be00u));
}

// Where row n of the QKV projection goes for token t (heads of d = 1 << shift).
__device__ __forceinline__ bf16* qkv_place(const W4Params& p, int t, int n) {
  int head = n >> p.shift, heads = p.Hq;
  bf16* out = p.out[0];
  if (head >= p.Hq) {
    head -= p.Hq;
    heads = p.Hkv;
    out = p.out[1];
    if (head >= p.Hkv) {
      head -= p.Hkv;
      out = p.out[2];
    }
  }
  return out + ((((int64_t)t * heads + head) << p.shift) + (n & (p.d - 1)));
}

// Results a of row n and b of row n + far of token t: rows half a head apart for the QKV
// projection, whose q and k are rotated.
__device__ __forceinline__ void finish_pair(const W4Params& p, int t, int n, int far, float a, float b) {
  if (!p.position) {
    bf16* y = p.out[0] + (int64_t)t * p.N + n;
    y[0] = __float2bfloat16(a);
    if (n + far < p.N) y[far] = __float2bfloat16(b);
    return;
  }
  const int pos = p.position[t];
  if (pos < 0) return;
  if (n < (p.Hq + p.Hkv) << p.shift) {
    const uint32_t angle = turn_part(pos, p.turn[n & (p.d - 1)]);
    uint64_t sn2, cs2;
    sincos_turns(angle, angle, sn2, cs2);
    float sn, cs, same;
    f2_split(sn2, sn, same);
    f2_split(cs2, cs, same);
    const float x = a;
    a = x * cs - b * sn;
    b = b * cs + x * sn;
  }
  bf16* y = qkv_place(p, t, n);
  y[0] = __float2bfloat16(a);
  y[far] = __float2bfloat16(b);
}

// Many tokens (proj_w4_tc.cu), and the chunks of 128 inputs that a CTA of it has.
int launch_w4_tc(const W4Params& p, int sms, cudaStream_t stream);
int w4_tc_chunks(const W4Params& p, int sms);

}  // namespace gattn
