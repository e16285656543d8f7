// paged.cuh -- device helpers of the ragged serving step (paged_*.cu): rotation
// angles in fixed point, E4M3 conversions, the walk over requests.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace gattn {

// Angle of position `pos` at frequency `turn` (theta / 2 pi modulo 1, in units of 2^-64,
// its lower half signed: the upper one is one more where that is negative): the product
// modulo 2^64 is the angle modulo a whole turn, so nothing is lost at far positions (off by
// at most pos 2^-53 turns, the double that `turn` came from) and no range reduction is left.
// In units of 2^-32 turns.
__device__ __forceinline__ uint32_t turn_part(int pos, uint64_t turn) {
  return (uint32_t)pos * (uint32_t)(turn >> 32) + (uint32_t)__mulhi(pos, (int)(uint32_t)turn);
}
constexpr float kTurnUnit = 1.4629180792671596e-09f;  // 2 pi / 2^32
// The same in radians, in [-pi, pi).
__device__ __forceinline__ float turn_angle(int pos, uint64_t turn) {
  return (float)(int32_t)turn_part(pos, turn) * kTurnUnit;
}

// Sines and cosines of two angles in units of 2^-32 turns, off by about 2^-24: an angle
// is brought within an eighth of a turn of a quarter's multiple (exact, in integers), x;
// there sin x = x + x z S(z) and cos x = 1 - z / 2 + z^2 C(z), z = x^2, with S and C the
// polynomials of degree 2 that interpolate at Chebyshev's nodes.
__device__ __forceinline__ void sincos_turns(uint32_t a0, uint32_t a1, uint64_t& sn, uint64_t& cs) {
  const uint32_t b[2] = {a0 + 0x20000000u, a1 + 0x20000000u};  // upper two bits: quarters
  auto rest = [](uint32_t v) { return (float)((int)(v & 0x3fffffffu) - 0x20000000); };
  auto both = [](float v) { return f2_make(v, v); };
  const uint64_t x = f2_mul(f2_make(rest(b[0]), rest(b[1])), both(kTurnUnit)), z = f2_mul(x, x);
  uint64_t s = f2_fma(both(-0.00019587890880412386f), z, both(0.008332748270629749f));
  s = f2_fma(s, z, both(-0.1666666466231438f));
  s = f2_fma(f2_mul(s, z), x, x);
  uint64_t c = f2_fma(both(2.4547942085071572e-05f), z, both(-0.0013888303035894866f));
  c = f2_fma(c, z, both(0.04166666465950221f));
  c = f2_fma(f2_fma(c, z, both(-0.5f)), z, both(1.f));
  float sv[2], cv[2], so[2], co[2];
  f2_split(s, sv[0], sv[1]);
  f2_split(c, cv[0], cv[1]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const bool odd = b[e] & 0x40000000u;
    so[e] = __uint_as_float(__float_as_uint(odd ? cv[e] : sv[e]) ^ (b[e] & 0x80000000u));
    co[e] = __uint_as_float(__float_as_uint(odd ? sv[e] : cv[e]) ^ ((b[e] ^ (b[e] << 1)) & 0x80000000u));
  }
  sn = f2_make(so[0], so[1]);
  cs = f2_make(co[0], co[1]);
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

// Two floats (magnitudes below 448) as the sums of four E4M3 pairs, each the rounded
// remainder of the ones before: off by at most 2^-16 of a value or 2^-10, and 2^-19 of a
// value where the second remainder goes on in f16.
__device__ __forceinline__ void terms4(float lo, float hi, uint16_t& t0, uint16_t& t1, uint16_t& t2, uint16_t& t3) {
  auto rest = [&](uint16_t t) {  // exact
    const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(t));
    lo -= f.x;
    hi -= f.y;
  };
  t0 = e4m3x2(lo, hi);
  rest(t0);
  t1 = e4m3x2(lo, hi);
  rest(t1);
  asm("{\n\t.reg .b32 x, f;\n\t"
      "cvt.rn.f16x2.f32 x, %3, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %0, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 f, %0;\n\t"
      "sub.rn.f16x2 x, x, f;\n\t"  // exact
      "cvt.rn.satfinite.e4m3x2.f16x2 %1, x;\n\t}"
      : "=&h"(t2), "=&h"(t3)
      : "f"(lo), "f"(hi));
}

// The attention kernels hold exp2(s + log2 |v| - m), v the V scale of a key's block and m the
// running maximum of s + log2 |v| (which may stay 12 behind), and sum exp2(s - m) apart.
// With |v| from 2^-96 to 2^100 that sum stays in fp32's range: 2^19 keys of the least scale
// come to 2^(96 + 12 + 19) at most, and beside a key of the largest all of at least 2^-26 of
// its weight count.  Smaller scales count as zero, larger ones are reported.
constexpr float kLeastScale = 1.262177448353619e-29f, kMostScale = 1.2676506002282294e+30f;
__device__ __forceinline__ float scale_log2(float v) {
  const float a = fabsf(v);
  return a < kLeastScale ? -96.f : log2f(a);
}

// The requests of a step, as the attention kernels walk them.
struct Requests {
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* block_table;
  int B, T, max_new, G, Hkv, W, block_len;
  int max_rows;  // requests of more rows (new tokens x G) are another kernel's

  // A request's cached tokens; -1 where the table cannot hold them.
  __device__ __forceinline__ int length(int r) const {
    const int kv = kv_len[r];
    return kv > W * block_len ? -1 : max(kv, 0);
  }
  // New tokens of request r, 0 where its token rows are out of order or range.
  __device__ __forceinline__ int tokens(int r, bool* bad = nullptr) const {
    const int a = q_start[r], b = q_start[r + 1];
    if (a < 0 || b > T || b < a || b - a > max_new) {
      if (bad) *bad = true;
      return 0;
    }
    return b - a;
  }
  // Tiles of KT keys of request r for one KV head, 0 if this kernel has nothing
  // to do for it; one where it sees no key (its rows are zeros).
  template <int KT>
  __device__ __forceinline__ int tiles(int r, bool* bad = nullptr) const {
    const int n = tokens(r, bad);
    if (n == 0 || n > max_rows / G) return 0;
    const int kv = length(r);
    if (bad && kv < 0) *bad = true;
    return max(1, (kv + KT - 1) / KT);
  }
};

// Sums count(r) over the requests (the NT threads of a CTA, all of them), finds the
// request that holds unit at(total) of the running sum and the units before it.
// *start_r is -1 where there is no such unit.  Thread t's requests are the t-th (B + NT - 1) / NT ones; the
// units before them go to before_thread[t], if it is given.
template <int NT, class Int, class Count, class At>
__device__ __forceinline__ void scan_requests(int B, Count count, Int* warp_sum, int* start_r, Int* start_pre,
                                              Int* total, At at, Int* before_thread = nullptr) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (B + NT - 1) / NT;
  const int r0 = min(tid * per, B), r1 = min(r0 + per, B);
  Int own = 0;
  for (int r = r0; r < r1; ++r) own += count(r);
  Int inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sum[warp] = inc;
  if (tid == 0) *start_r = -1;
  __syncthreads();
  Int before = inc - own, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const Int s = warp_sum[w];
    if (w < warp) before += s;
    all += s;
  }
  if (tid == 0) *total = all;
  if (before_thread) before_thread[tid] = before;
  const Int x = at(all);
  if (x >= before && x < before + own) {
    for (int r = r0; r < r1; ++r) {
      const Int n = count(r);
      if (x < before + n) {
        *start_r = r;
        *start_pre = before;
        break;
      }
      before += n;
    }
  }
  __syncthreads();
}

// Whether one of four E4M3 codes is a NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

inline Requests requests_of(const PagedProblem& pb) {
  return Requests{pb.q_start, pb.kv_len, pb.block_table, pb.B, pb.T, pb.max_new, pb.G, pb.Hkv, pb.W, pb.block_len, 0};
}

}  // namespace gattn
