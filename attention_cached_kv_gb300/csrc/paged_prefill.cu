// paged_prefill.cu -- many query rows a request (prompt chunks) against its E4M3
// paged cache, causal ([KV page, "Reusable-state"]; [Suffix page, §2, §5, §6 问题四]).
//
// A CTA takes one KV head and up to 256 query rows of a request: two row tiles of
// floor(128 / G) tokens x G heads.  Its keys stream by in tiles of 128, one pass,
//     S = q K^T, P = exp2(S - m), O += P V       (tcgen05 kind::f16, TMEM)
// with m the row's running maximum, moved only when a tile's maximum passes it by
// more than 8 (log2 units).  Twelve warps with registers to spare:
//   * 0-3, 4-7: a thread a row of each row tile, softmax and output; P goes back
//     into S's columns as f16 (11 bits), A operand of the second product;
//   * 8-11: cached rows from global memory through registers into f16 tiles.  E4M3
//     to f16 is exact; values are also divided by the largest V scale of the
//     request (exact for powers of two), K's block scales multiply the fp32 scores;
//   * 12: the MMAs, alternating between the row tiles, so that one's products run
//     while the other's softmax does.
// One conversion of a key serves 256 rows, against 256 exponentials for it: that is
// why rows are taken in pairs of tiles here and cached bytes are used as they are
// where there are few rows (paged_decode.cu).  q is scaled by a power of two a row
// before its one rounding to f16.
//
// Few CTAs (a short chunk behind a long context): the keys are split in `splits`
// equal runs, whose parts join_kernel adds up in order.
// Bound: exponentials and tensor work, about equally.
//
// Pages: [KV page] "为什么自回归推理缓存 KV，而不缓存历史 Q？";
//        [Suffix page] icman.com.cn news 64898.
#include <math.h>

#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "tcgen05.cuh"

namespace gattn {
namespace {

constexpr int kThreads = 416;         // 8 softmax + 4 converting + 1 MMA warp
constexpr int kKT = 128;              // keys a tile
constexpr float kNone = -3.0e38f;     // running maximum before any key
constexpr float kSlack = 8.f;         // log2 units a score may pass it by

struct PrefillParams {
  const bf16* q;
  bf16* out;
  const uint8_t* pool;
  const float* scale;
  float* parts;
  int32_t* status;
  Requests rq;
  int Hq, L, layer, num_blocks, min_new, Tm, splits;
  float scale_log2;
  uint64_t turn[64];
};

template <int D>
struct PCfg {
  static constexpr uint32_t kTile = 128 * D * 2;        // bytes of a 128-row f16 tile
  static constexpr uint32_t kPanel = 128 * 128;
  static constexpr uint32_t offK = 2 * kTile, offV = 4 * kTile, offMisc = 6 * kTile;
  static constexpr int kS = 0, kO = 256;  // TMEM columns: S (P) of the row tiles, O
};

template <int D>
struct PMisc {
  uint64_t kready[2], kfree[2], vready[2], vfree[2], sfull[2], pfull[2], qready, drain;
  uint32_t tmem;
  int bad, any_nan;
  int warp_sum[kThreads / 32 + 1];
  int start_r, start_pre, total;
  // by tile (modulo 4) and 16-key group: K and V scale, first byte of the K rows in
  // the pool (-1: no key that is seen, or a block outside the pool)
  alignas(16) float ksc[4][8], vsc[4][8];
  int64_t at[4][8];
  int even[4];  // the groups' K scales are equal in pairs
  float vref, vpart[4];
  int nankey[D];  // first key past the first row's whose V is NaN, by element
};

__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// As ld32, waited for, the maximum only.
__device__ __forceinline__ float ld32_max(uint32_t taddr) {
  uint32_t r[32];
  float m;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(m)
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(m)::"memory");
  return m;
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint32_t to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillParams prm) {
  using C = PCfg<D>;
  using M = PMisc<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  M& ms = *reinterpret_cast<M*>(smem + C::offMisc);
  const Requests& rq = prm.rq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = rq.G, Tm = prm.Tm;

  // ---- this CTA's request, KV head, row tiles and keys; the longest runs first
  const int g = blockIdx.y, z = blockIdx.z;
  scan_requests<kThreads>(
      rq.B,
      [&](int r) {
        const int n = rq.tokens(r);
        return n >= prm.min_new ? (n + 2 * Tm - 1) / (2 * Tm) : 0;
      },
      ms.warp_sum, &ms.start_r, &ms.start_pre, &ms.total,
      [&](int all) { return min(all, (int)gridDim.x) - 1 - (int)blockIdx.x; });
  const int item = min(ms.total, (int)gridDim.x) - 1 - (int)blockIdx.x, r = ms.start_r;
  if (item < 0 || r < 0) return;
  const int n = rq.q_start[r + 1] - rq.q_start[r], kv = rq.length(r);
  const int tok0 = (item - ms.start_pre) * 2 * Tm, toks = min(2 * Tm, n - tok0);
  const int q0 = rq.q_start[r] + tok0;             // the CTA's first token row
  const int pos0 = max(kv, 0) - n + tok0;          // position of the first token
  const int kend = max(0, pos0 + toks);            // keys that the last token sees
  const int all_tiles = (kend + kKT - 1) / kKT;
  const int kt0 = (int)((int64_t)all_tiles * z / prm.splits);
  const int nt = (int)((int64_t)all_tiles * (z + 1) / prm.splits) - kt0;
  const bool two = toks > Tm;

  if (warp == 12) {
    tc::tmem_alloc(smem_u32(&ms.tmem), 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms.kready[s], 128);
      mbar_init(&ms.kfree[s], 1);
      mbar_init(&ms.vready[s], 128);
      mbar_init(&ms.vfree[s], 1);
      mbar_init(&ms.sfull[s], 1);
      mbar_init(&ms.pfull[s], 128);
    }
    mbar_init(&ms.qready, 256);
    mbar_init(&ms.drain, 1);
    fence_mbar_init();
    ms.bad = kv < 0;
    ms.any_nan = 0;
    if (kv < 0) report(prm.status, GIST_ATTN_STATUS_BAD_BLOCK);
  }
  for (int i = tid; i < D; i += kThreads) ms.nankey[i] = INT32_MAX;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ms.tmem;
  bool failed = false;

  if (warp == 12) {
    // ================================================== tcgen05
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (failed || __any_sync(0xffffffffu, !mbar_wait(bar, parity))) failed = true;
      tc::fence_after_sync();
      return !failed;
    };
    auto issue_s = [&](int x, int i) {  // S of row tile x and the CTA's i-th key tile
      if (lane == 0) {
        const uint32_t qb = sbase + x * C::kTile, kb = sbase + C::offK + (i & 1) * C::kTile;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(tmem + C::kS + x * 128, tc::smem_desc_sw128(qb + (k / 4) * C::kPanel + (k % 4) * 32, 16, 1024),
                     tc::smem_desc_sw128(kb + (k / 4) * C::kPanel + (k % 4) * 32, 16, 1024),
                     tc::idesc_f16_f32(128, 128, 0), k > 0);
        tc::commit(smem_u32(&ms.sfull[x]));
      }
      __syncwarp();
    };
    auto issue_pv = [&](int x, int i) {
      if (lane == 0) {
        const uint32_t vb = sbase + C::offV + (i & 1) * C::kTile;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc::mma_ts(tmem + C::kO + x * D, tmem + C::kS + x * 128 + k * 8,
                     tc::smem_desc_sw128(vb + k * 2048, C::kPanel, 1024), tc::idesc_f16_f32(128, D, 1), i > 0 || k > 0);
      }
      __syncwarp();
    };
    auto arrive = [&](uint64_t* bar) {
      if (lane == 0) tc::commit(smem_u32(bar));
      __syncwarp();
    };
    if (nt > 0 && wait(&ms.qready, 0) && wait(&ms.kready[0], 0)) {
      issue_s(0, 0);
      if (two) issue_s(1, 0);
      arrive(&ms.kfree[0]);
      for (int i = 0; i < nt; ++i) {
        const uint32_t ph = (uint32_t)i & 1u;
        const bool more = i + 1 < nt;
        if (!wait(&ms.vready[i & 1], (uint32_t)(i >> 1) & 1u) || !wait(&ms.pfull[0], ph)) break;
        issue_pv(0, i);
        if (!two) arrive(&ms.vfree[i & 1]);
        if (more) {
          if (!wait(&ms.kready[(i + 1) & 1], (uint32_t)((i + 1) >> 1) & 1u)) break;
          issue_s(0, i + 1);
          if (!two) arrive(&ms.kfree[(i + 1) & 1]);
        } else {
          arrive(&ms.sfull[0]);  // the last P V is done
        }
        if (two) {
          if (!wait(&ms.pfull[1], ph)) break;
          issue_pv(1, i);
          arrive(&ms.vfree[i & 1]);
          if (more) {
            issue_s(1, i + 1);
            arrive(&ms.kfree[(i + 1) & 1]);
          } else {
            arrive(&ms.sfull[1]);
          }
        }
      }
    }
    if (lane == 0) tc::commit(smem_u32(&ms.drain));
    __syncwarp();
    if (!mbar_wait(&ms.drain, 0)) failed = true;
  } else if (warp >= 8) {
    // ================================================== cached rows into f16 tiles
    constexpr int kLanes = D / 16;             // threads of a row (16 bytes each)
    constexpr int kRows = 128 / kLanes;        // rows of a pass
    constexpr int kPass = 128 / kRows;
    const int ct = tid - 256, c = ct % kLanes, row0 = ct / kLanes;
    const int32_t* table = rq.block_table + (int64_t)r * rq.W;
    const int64_t vstep = (int64_t)rq.Hkv * rq.block_len * D;
    // the largest V scale among the blocks that the rows see
    float top = 0.f;
    const int blocks = kv < 0 ? 0 : (kend + rq.block_len - 1) / rq.block_len;
    for (int b = ct; b < blocks; b += 128) {
      const int blk = table[b];
      if (blk >= 0 && blk < prm.num_blocks)
        top = fmaxf(top, prm.scale[(((int64_t)blk * prm.L + prm.layer) * 2 + 1) * rq.Hkv + g]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) ms.vpart[warp - 8] = top;
    named_bar_sync(2, 128);
    const float vref = fmaxf(fmaxf(fmaxf(ms.vpart[0], ms.vpart[1]), fmaxf(ms.vpart[2], ms.vpart[3])), 7.5e-37f);
    if (ct == 0) ms.vref = vref;  // (read by the softmax after vready -> pfull -> sfull)
    const float rvref = 1.f / vref;
    // Threads 0 .. 7 look up the groups of the tiles ahead: an id four tiles ahead of
    // its use, the scales three, in shared memory two.
    float gk = 0.f, gv = 0.f;
    int64_t ga = -1;
    int gid = -1;
    bool want = false;  // there are such keys
    auto look_up = [&](int i) {
      const int key = (kt0 + i) * kKT + ct * 16;
      want = i < nt && key < kend && kv >= 0;
      gid = want ? table[key / rq.block_len] : -1;
    };
    auto scales_of = [&](int kt) {
      gk = gv = 0.f;
      ga = -1;
      if (want && gid >= 0 && gid < prm.num_blocks) {
        const int64_t plane = ((int64_t)gid * prm.L + prm.layer) * 2 * rq.Hkv + g;
        ga = (plane * rq.block_len + (kt * kKT + ct * 16) % rq.block_len) * D;
        gk = prm.scale[plane];
        gv = prm.scale[plane + rq.Hkv];
      } else if (want) {
        ms.bad = 1;
        report(prm.status, GIST_ATTN_STATUS_BAD_BLOCK);
      }
    };
    auto publish = [&](int i) {
      ms.ksc[i & 3][ct] = gk;
      ms.vsc[i & 3][ct] = gv;
      ms.at[i & 3][ct] = ga;
      const bool same = __shfl_xor_sync(0xffu, gk, 1) == gk;
      const bool all = __all_sync(0xffu, same);
      if (ct == 0) ms.even[i & 3] = all;
    };
    if (ct < 8) {
      for (int i = 0; i < 2; ++i) {
        look_up(i);
        scales_of(kt0 + i);
        publish(i);
      }
      look_up(2);
      scales_of(kt0 + 2);
      look_up(3);
    }
    named_bar_sync(2, 128);
    uint4 kx[kPass], vx[kPass];
    auto fetch = [&](int i, uint4 (&x)[kPass], int64_t more) {
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        const int row = p * kRows + row0;
        const int64_t at = ms.at[i & 3][row >> 4];
        x[p] = make_uint4(0, 0, 0, 0);
        if (at >= 0 && (kt0 + i) * kKT + row < kend) x[p] = ldg16(prm.pool + at + (row & 15) * D + c * 16 + more);
      }
    };
    // 16 codes as two 16-byte chunks of f16 of tile row `row`; the second half of a
    // row's threads stores its chunks in the other order (bank conflicts)
    auto put = [&](uint32_t tile, int row, uint4 x, uint32_t mul, bool scaled) {
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[2 * e] = e4m3x2_to_f16x2((uint16_t)w[e]);
        h[2 * e + 1] = e4m3x2_to_f16x2((uint16_t)(w[e] >> 16));
        if (scaled) {
          h[2 * e] = mul_f16x2(h[2 * e], mul);
          h[2 * e + 1] = mul_f16x2(h[2 * e + 1], mul);
        }
      }
      const uint32_t base = tile + (c / 4) * C::kPanel;
      const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
      const int odd = (c >> 2) & 1, ch = 2 * (c % 4);
      sts16(base + swz128(row, ch + odd), odd ? hi : lo);
      sts16(base + swz128(row, ch + 1 - odd), odd ? lo : hi);
    };
    if (nt > 0) fetch(0, kx, 0), fetch(0, vx, vstep);
    for (int i = 0; i < nt && !failed; ++i) {
      const int kt = kt0 + i, b = i & 1;
      if (i >= 2 && !mbar_wait(&ms.kfree[b], ((uint32_t)(i >> 1) & 1u) ^ 1u)) {
        failed = true;
        break;
      }
#pragma unroll
      for (int p = 0; p < kPass; ++p) put(sbase + C::offK + b * C::kTile, p * kRows + row0, kx[p], 0, false);
      fence_proxy_async_smem();
      mbar_arrive(&ms.kready[b]);
      if (i + 1 < nt) fetch(i + 1, kx, 0);
      if (i >= 2 && !mbar_wait(&ms.vfree[b], ((uint32_t)(i >> 1) & 1u) ^ 1u)) {
        failed = true;
        break;
      }
      if (kt * kKT + kKT > pos0 + 1) {
        // keys that not every row sees: a NaN would reach the others (0 x NaN), so it
        // is noted for the rows that see it and cleared
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
          const int key = kt * kKT + p * kRows + row0;
          const uint32_t any = e4m3_nan(vx[p].x) | e4m3_nan(vx[p].y) | e4m3_nan(vx[p].z) | e4m3_nan(vx[p].w);
          if (key > pos0 && any) {
            uint32_t w[4] = {vx[p].x, vx[p].y, vx[p].z, vx[p].w};
            ms.any_nan = 1;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (((w[e >> 2] >> (8 * (e & 3))) & 0x7fu) == 0x7fu) {
                w[e >> 2] &= ~(0xffu << (8 * (e & 3)));
                atomicMin(&ms.nankey[c * 16 + e], key);
              }
            vx[p] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        const float f = ms.vsc[i & 3][(p * kRows + row0) >> 4] * rvref;
        put(sbase + C::offV + b * C::kTile, p * kRows + row0, vx[p], to_f16x2(f, f), true);
      }
      fence_proxy_async_smem();
      mbar_arrive(&ms.vready[b]);
      if (i + 1 < nt) fetch(i + 1, vx, vstep);
      if (ct < 8) {
        publish(i + 2);
        scales_of(kt + 3);
        look_up(i + 4);
      }
      named_bar_sync(2, 128);
    }
  } else {
    // ================================================== q rows, softmax, output
    const int x = warp >> 2, row = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + C::kS + x * 128, to = tmem + lane_base + C::kO + x * D;
    const int tok = x * Tm + row / G, head = row % G;
    const bool valid = row < Tm * G && tok < toks;
    const int lim = valid ? pos0 + tok + 1 : 0;         // keys the row sees
    const int lim_all = pos0 + x * Tm + 1;              // keys every row of the tile sees
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!failed && !mbar_wait(bar, parity)) failed = true;
    };
    float rs;  // softmax scale (log2) x the row's power of two
    {
      const bf16* src = prm.q + ((int64_t)(q0 + tok) * prm.Hq + g * G + head) * D;
      uint4 v[D / 8];
#pragma unroll
      for (int j = 0; j < D / 8; ++j) v[j] = valid ? ldg16(src + j * 8) : make_uint4(0, 0, 0, 0);
      uint32_t* w = reinterpret_cast<uint32_t*>(v);
      float top = 0.f;
      // two passes over the pairs (j, j + D/2): the largest magnitude bounds the
      // rotated ones by sqrt 2, which the power of two leaves room for
#pragma unroll
      for (int j = 0; j < D / 2; ++j) {
        const float2 f = bf16x2_to_float2(w[j]);
        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        if (!(fabsf(f.x) <= 3.4e38f) || !(fabsf(f.y) <= 3.4e38f)) top = INFINITY;
      }
      const uint32_t tb = __float_as_uint(top);
      const int ex = min(max((int)(tb >> 23) - 127, -119), 126);
      const float down = __uint_as_float((uint32_t)(127 - ex) << 23);  // largest to [1, 2)
      rs = tb >= 0x7f800000u ? __int_as_float(0x7fc00000) : prm.scale_log2 * __uint_as_float((uint32_t)(ex + 127) << 23);
      const int pos = pos0 + tok;
      const uint32_t tile = sbase + x * C::kTile;
#pragma unroll
      for (int ch = 0; ch < D / 16; ++ch) {  // 8 pairs: elements 8 ch .. and D/2 + 8 ch ..
        uint32_t a[4], b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 u = bf16x2_to_float2(w[ch * 4 + e]), y = bf16x2_to_float2(w[D / 4 + ch * 4 + e]);
          float s0, c0, s1, c1;
          __sincosf(turn_angle(pos, prm.turn[ch * 8 + 2 * e]), &s0, &c0);
          __sincosf(turn_angle(pos, prm.turn[ch * 8 + 2 * e + 1]), &s1, &c1);
          const float u0 = u.x * down, u1 = u.y * down, y0 = y.x * down, y1 = y.y * down;
          a[e] = to_f16x2(u0 * c0 - y0 * s0, u1 * c1 - y1 * s1);
          b[e] = to_f16x2(y0 * c0 + u0 * s0, y1 * c1 + u1 * s1);
        }
        const int c2 = ch + D / 16;  // 16-byte chunk of the second half
        sts16(tile + (ch / 8) * C::kPanel + swz128(row, ch % 8), make_uint4(a[0], a[1], a[2], a[3]));
        sts16(tile + (c2 / 8) * C::kPanel + swz128(row, c2 % 8), make_uint4(b[0], b[1], b[2], b[3]));
      }
      fence_proxy_async_smem();
      mbar_arrive(&ms.qready);
    }
    float m = kNone;
    uint64_t acc = f2_make(0.f, 0.f), acc2 = acc;
    const bool live = x == 0 || two;
    for (int i = 0; live && i < nt; ++i) {
      const int key0 = (kt0 + i) * kKT;
      const bool edge = key0 + kKT > lim_all;
      wait(&ms.sfull[x], (uint32_t)i & 1u);
      tc::fence_after_sync();
      const float* ksc = ms.ksc[i & 3];
      float mx = kNone;
      if (!edge && ms.even[i & 3]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) mx = fmaxf(mx, ld32_max(ts + c * 32) * (ksc[2 * c] * rs));
      } else {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          ld32(ts + c * 32, v);
          tc::wait_ld();
          const int left = lim - key0 - c * 32;  // columns of these that the row sees
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float t = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e) t = fmaxf(t, h * 16 + e < left || !edge ? __uint_as_float(v[h * 16 + e]) : -INFINITY);
            mx = fmaxf(mx, t * (ksc[2 * c + h] * rs));
          }
        }
      }
      // a row whose maximum jumps scales its O and sum down first; the TMEM load and
      // store are warp-collective, so the warp does it for any of its rows
      const bool move = mx - m > kSlack;
      if (__any_sync(0xffffffffu, move)) {
        const float fm = move ? ex2_approx(m - mx) : 1.f;
        if (move) m = mx;
        const uint64_t f2 = f2_make(fm, fm);
        acc = f2_mul(acc, f2);
        acc2 = f2_mul(acc2, f2);
        if (i > 0) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t ov[16];
            tc::ld16(to + c * 16, ov);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * fm);
            st16(to + c * 16, ov);
          }
        }
      }
      // 32 scores in registers, the next 32 on their way
      const uint64_t nm2 = f2_make(-m, -m);
      uint32_t va[32], vb[32];
      auto weights = [&](int c, uint32_t (&v)[32], auto masked) {
        uint32_t pk[16];
        const float2 k2 = *reinterpret_cast<const float2*>(ksc + 2 * c);
        const float f0 = k2.x * rs, f1 = k2.y * rs;
        const uint64_t g0 = f2_make(f0, f0), g1 = f2_make(f1, f1);
        const int left = lim - key0 - c * 32;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float a, b;
          f2_split(f2_fma(f2_make(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), e < 8 ? g0 : g1, nm2), a, b);
          if (masked) {
            if (2 * e >= left) a = -INFINITY;
            if (2 * e + 1 >= left) b = -INFINITY;
          }
          const float pa = ex2_approx(a), pb = ex2_approx(b);
          if (e & 1) acc = f2_add(acc, f2_make(pa, pb));
          else acc2 = f2_add(acc2, f2_make(pa, pb));
          pk[e] = to_f16x2(pa, pb);
        }
        st16(ts + c * 16, pk);
      };
      if (!edge) {
        ld32(ts, va);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          ld32(ts + c * 32 + 32, vb);
          weights(c, va, std::false_type{});
          tc::wait_ld();
          if (c + 2 < 4) ld32(ts + c * 32 + 64, va);
          weights(c + 1, vb, std::false_type{});
          tc::wait_ld();
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          ld32(ts + c * 32, va);
          tc::wait_ld();
          weights(c, va, std::true_type{});
        }
      }
      tc::wait_st();
      tc::fence_before_sync();
      mbar_arrive(&ms.pfull[x]);
    }
    if (live) {
      if (nt > 0) wait(&ms.sfull[x], (uint32_t)nt & 1u);
      tc::fence_after_sync();
      float a0, a1, b0, b1;
      f2_split(acc, a0, a1);
      f2_split(acc2, b0, b1);
      const float sum = (a0 + a1) + (b0 + b1);
      const bool none = lim <= 0 || ms.bad, whole = prm.splits == 1, nan = nt > 0 && ms.any_nan;
      const float vref = nt > 0 ? ms.vref : 0.f;
      if (valid && whole && !none && !(sum <= 3.0e38f)) report(prm.status, GIST_ATTN_STATUS_RANGE);
      const float inv = whole ? (none ? 0.f : vref / sum) : vref;
      const int64_t dst = ((int64_t)(q0 + tok) * prm.Hq + g * G + head) * D;
      float* part = prm.parts + ((((int64_t)item * rq.Hkv + g) * prm.splits + z) * 256 + tid) * (D + 2);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        float o[16];
        if (nt > 0) {
          uint32_t ov[16];
          tc::ld16(to + c * 16, ov);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = none ? 0.f : __uint_as_float(ov[e]) * inv;
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0.f;
        }
        if (nan && !none) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (ms.nankey[c * 16 + e] < lim) o[e] = __int_as_float(0x7fc00000);
        }
        if (valid && whole) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = float2_to_bf16x2(o[2 * e], o[2 * e + 1]);
          stg16(prm.out + dst + c * 16, make_uint4(w[0], w[1], w[2], w[3]));
          stg16(prm.out + dst + c * 16 + 8, make_uint4(w[4], w[5], w[6], w[7]));
        } else if (valid) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) *reinterpret_cast<float2*>(part + c * 16 + e) = make_float2(o[e], o[e + 1]);
        }
      }
      if (valid && !whole) {
        part[D] = m;
        part[D + 1] = ms.bad ? -1.f : sum;
      }
    }
  }
  if (failed) report(prm.status, GIST_ATTN_STATUS_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 12) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Adds up the splits' parts of a row, a warp a row: O, m and sum in key order.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ PrefillParams prm) {
  __shared__ int warp_sum[8], start_r, start_pre, total;
  const Requests& rq = prm.rq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = rq.G, Tm = prm.Tm, g = blockIdx.y;
  scan_requests<256>(
      rq.B,
      [&](int r) {
        const int n = rq.tokens(r);
        return n >= prm.min_new ? (n + 2 * Tm - 1) / (2 * Tm) : 0;
      },
      warp_sum, &start_r, &start_pre, &total, [&](int) { return (int)blockIdx.x; });
  if ((int)blockIdx.x >= total || start_r < 0) return;
  const int r = start_r, n = rq.q_start[r + 1] - rq.q_start[r];
  const int tok0 = ((int)blockIdx.x - start_pre) * 2 * Tm, toks = min(2 * Tm, n - tok0);
  const int q0 = rq.q_start[r] + tok0;
  const int pos0 = max(rq.length(r), 0) - n + tok0;
  const int row = blockIdx.z * 8 + warp, x = row >> 7, in = row & 127;
  const int tok = x * Tm + in / G, head = in % G;
  if (in >= Tm * G || tok >= toks) return;
  const float* part = prm.parts + (((int64_t)blockIdx.x * rq.Hkv + g) * prm.splits * 256 + row) * (D + 2);
  const int64_t step = 256 * (D + 2);
  float m = kNone, sum = 0.f, o[D / 32];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  for (int z = lane; z < prm.splits; z += 32) m = fmaxf(m, part[z * step + D]);
#pragma unroll
  for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
#pragma unroll 4
  for (int z = 0; z < prm.splits; ++z) {
    const float* p = part + z * step;
    const float f = exp2f(p[D] - m), s = p[D + 1];
    bad |= s < 0.f;
    sum += s * f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] += f * p[lane + 32 * e];
  }
  const bool none = bad || pos0 + tok < 0;
  if (lane == 0 && !none && !(sum <= 3.0e38f)) report(prm.status, GIST_ATTN_STATUS_RANGE);
  bf16* dst = prm.out + ((int64_t)(q0 + tok) * prm.Hq + g * G + head) * D + lane;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) dst[32 * e] = __float2bfloat16(none ? 0.f : o[e] / sum);
}

// Row-tile pairs at most: every request with min_new tokens or more may end in a
// pair that is not full.
int64_t pairs_of(const PagedProblem& pb, int min_new) {
  const int Tm = 128 / pb.G;
  const int64_t requests = pb.T / min_new < pb.B ? pb.T / min_new : pb.B;
  return pb.T / (2 * Tm) + requests;
}

// Runs that the keys are cut into: one unless the pairs leave SMs idle; a run has
// 8 tiles (1024 keys) or more of the longest request that the table can hold.
int splits_of(const PagedProblem& pb, int min_new, int sms) {
  const int64_t ctas = pairs_of(pb, min_new) * pb.Hkv;
  const int64_t tiles = ((int64_t)pb.W * pb.block_len + kKT - 1) / kKT;
  int64_t s = ctas > 0 ? sms / ctas : 1;
  s = s < tiles / 8 ? s : tiles / 8;
  return s < 1 ? 1 : (int)s;
}

template <int D>
int launch(const PagedProblem& pb, void* workspace, int min_new, int sms, cudaStream_t stream) {
  const int64_t pairs = pairs_of(pb, min_new);
  if (pairs == 0) return GIST_ATTN_OK;
  PrefillParams prm{};
  prm.q = static_cast<const bf16*>(pb.q);
  prm.out = static_cast<bf16*>(pb.out);
  prm.pool = pb.pool;
  prm.scale = pb.scale;
  prm.parts = static_cast<float*>(workspace);
  prm.status = pb.status;
  prm.rq = requests_of(pb);
  prm.Hq = pb.Hq;
  prm.L = pb.L;
  prm.layer = pb.layer;
  prm.num_blocks = pb.num_blocks;
  prm.min_new = min_new;
  prm.Tm = 128 / pb.G;
  prm.splits = splits_of(pb, min_new, sms);
  prm.scale_log2 = pb.scale_log2;
  for (int j = 0; j < 64; ++j) prm.turn[j] = pb.turn[j];
  constexpr int smem = (int)(PCfg<D>::offMisc + sizeof(PMisc<D>));
  static_assert(smem <= 227 * 1024, "shared memory");
  if (cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  prefill_kernel<D><<<dim3((unsigned)pairs, pb.Hkv, prm.splits), kThreads, smem, stream>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return GIST_ATTN_ERR_LAUNCH;
  if (prm.splits > 1) join_kernel<D><<<dim3((unsigned)pairs, pb.Hkv, 32), 256, 0, stream>>>(prm);
  return cudaGetLastError() == cudaSuccess ? GIST_ATTN_OK : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace

size_t paged_prefill_workspace(const PagedProblem& pb, int min_new, int sms) {
  const int splits = splits_of(pb, min_new, sms);
  return splits == 1 ? 0 : (size_t)pairs_of(pb, min_new) * pb.Hkv * splits * 256 * (pb.d + 2) * sizeof(float);
}

int launch_paged_prefill(const PagedProblem& pb, void* workspace, int min_new, int sms, cudaStream_t stream) {
  return pb.d == 64 ? launch<64>(pb, workspace, min_new, sms, stream) : launch<128>(pb, workspace, min_new, sms, stream);
}

}  // namespace gattn
