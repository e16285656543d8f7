// paged_decode.cu -- few query rows a request (new tokens x heads of a KV group)
// against its E4M3 paged cache: the decoding step and the check of drafted tokens
// ([KV page, "Reusable-state"]; [Suffix page, §2, §5, §6 问题四]).
//
// The pool's bytes go to the tensor core as they lie in the cache.  A tile is 128
// rows of 128 bytes of one KV head (128 keys for d = 128; 256 for d = 64, a row
// then holding an even and an odd key).  Per tile
//     S^T = K q^T      tcgen05 kind::f8f6f4, keys as M, the query rows as N
//     O^T = V^T P^T    the V tile read transposed (M contiguous), P as N
// so no cached element is ever converted.  q and P keep their precision as sums
// of E4M3 terms, each the rounded remainder of the last.  q has four, added in TMEM, one
// product after the other: it is scaled by a power of two a row, its largest value to 128
// and more, and the terms leave 2^-16 of a value or 2^-17 of that (a score is off by as
// much of |q| |k|: after a rounding to f16, 2^-11, outputs of logits in the tens were off
// by more than their rounding to bf16).  P, whose rounding moves an output by as little of
// itself, has three of 11 bits or more; its small weights matter (they are many), so they
// are kept apart, p0 + p1 / 16 + p2 / 256, side by side as columns of N: the few query rows
// leave N room that costs nothing.
//
// The K scale of a key's block multiplies its fp32 scores s, the logarithm of its V scale is
// added to them: a weight with its V scale is P = exp2(s + log2 v - m), without it
// exp2(s - m), and a row's output is the quotient of the two sums (over P x V codes, and
// over the second).  So P's bits go by what a key adds to the row, and a large V scale of a
// key that the row hardly weighs, or does not see, takes none away.
//
// A softmax thread owns one tile row (TMEM lane): its scores for all query rows,
// the running maximum (of s + log2 v, less kPUnit) m of each (the same in all threads),
// its own part of the sums.  m moves only when a score passes it by more than 2 (log2
// units), all threads together; then O in TMEM is rescaled.  P is at most 2^2 x 64 of 448.
//
// Work is the sequence of tiles of all (request, KV head) units; each of at most
// two CTAs an SM takes an equal run of it, so one long request spreads over the
// machine.  A unit that crosses CTAs leaves parts (O, m, sum) in the workspace;
// combine_kernel joins them in key order, the same way every time.  Where no unit can
// have more than four tiles the runs are of whole units, and that launch falls away.
//
// Bound: HBM (a byte a cached element) where the contexts are long: 32 x ~4050 keys,
// 32 heads of 128 with a KV head each, 167 us = 6.4 TB/s; in groups of four, 54 us =
// 5.1 TB/s, of which about 10 us start, tail and join.  Few tiles a CTA: the chain
// copy - scores - softmax - output, 1 to 6 us a tile; 16 requests of 2-5 tokens behind
// 500-3000 keys 40 us, one of 131000 keys 21 us, four of 20-200 keys 8.3 us.
// Eight warps: 0-3 softmax, 4 TMA and scales, 5 tcgen05, 6-7 q rows.
//
// Pages: [KV page] "为什么自回归推理缓存 KV，而不缓存历史 Q？";
//        [Suffix page] icman.com.cn news 64898.
#include <math.h>
#include <stddef.h>

#include "kernels.h"
#include "paged.cuh"
#include "paged_tc.cuh"

namespace gattn {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kStage = 128 * 128;  // bytes of a K or V tile
constexpr float kNone = -3.0e38f;       // running maximum before any key
constexpr float kSlack = 2.f;           // log2 units a score may pass it by
constexpr float kPUnit = 6.f;           // log2 of P's scale into E4M3
// Short caches: two to four tiles one after the other (about 1.5 us each) against a
// second launch and its loads (2 us on the GPU, 3 to 4 on the host).
constexpr int kWhole = 4;

// What the join needs of a unit that crosses CTAs, left by the CTA in whose run the
// unit's second part begins (parts 0: nothing to join there).
struct JoinUnit {
  int parts, rows, q0, pos0, g, second;  // second: part 0 is the second of its CTA
  int pad[2];
};
struct DecodeParams {
  const bf16* q;
  bf16* out;
  const float* scale;
  JoinUnit* join;  // workspace: [CTAs], then the parts
  float* parts;
  int32_t* status;
  Requests rq;
  int Hq, L, layer, num_blocks;
  int box_rows, box_shift;  // tile rows of one TMA box: 2^box_shift
  float scale_log2;
  uint32_t per_g;  // 2^16 / G rounded up: j / G = j per_g >> 16 for the rows there are
  int join_rows;   // rows that a block of the join takes
  int whole;       // runs are of whole units
  uint64_t turn[64];
};

template <int D, int CH>
struct Cfg {
  static constexpr int KPR = 128 / D;           // keys a tile row
  static constexpr int KT = 128 * KPR;          // keys a tile
  static constexpr int ROWS = 8 * CH;           // query rows at most
  static constexpr int NPB = CH <= 2 ? 2 : 1;   // P buffers (q tiles: two, one made ahead)
  static constexpr int SP = (8 * CH + 15) & ~15;   // S columns a parity
  static constexpr int OC = (KPR * 24 * CH + 15) & ~15;  // O columns
  static constexpr int SB = 2 * KPR * SP + OC <= 256 ? 2 : 1;  // S buffers
  static constexpr uint32_t QT = 1024 * CH, QB = 4 * QT, PB = KPR * 3 * QT;
  static constexpr int NK = D == 128 && CH <= 2 ? 3 : D == 64 && CH == 1 ? 3 : 2;
  static constexpr int NV = D == 128 && CH == 1 ? 3 : 2;
  static constexpr uint32_t kO = SB * KPR * SP;  // O's first TMEM column
  static constexpr uint32_t offV = NK * kStage, offQ = offV + NV * kStage, offP = offQ + 2 * QB,
                            offMisc = offP + NPB * PB + 1024;  // (an MMA's N may run 8 rows past a tile)
  static_assert(QB >= ROWS * 512, "a segment's outputs leave through its q");
  static_assert(kO + OC <= 256, "TMEM columns");
};

struct Seg {  // one unit's share of a CTA
  int r, g, rows, q0, pos0, kv, kt0, kt1, nt, pad;
};

template <int D, int CH>
struct Misc {
  using C = Cfg<D, CH>;
  uint64_t kfull[3], kfree[3], vfull[3], vfree[3], scfull[3];
  uint64_t qfull[2], qfree[2], sfull[2], sfree[2], pfull[2], pfree[2], drain;
  uint32_t tmem;
  int bad[8];  // by segment: a block id outside the pool
  Seg seg[2];
  alignas(16) float rs[2][C::ROWS];  // softmax scale (log2) x q's power of two, by row
  alignas(16) float wmax[4][C::ROWS];  // by warp: a tile's maxima, a segment's sums
  alignas(16) float mrow[4][C::ROWS];  // running maxima, a copy a warp
  float ksc[3][16], vsc[3][16], vlog[3][16];  // scales of a tile's boxes, log2 of V's
  alignas(16)
  int nankey[D];  // first key past the first row's whose V is NaN, by element
  // the scan
  int warp_sum[kThreads / 32];
  int start_r, start_pre, total;
};

template <int D, int CH>
constexpr uint32_t smem_bytes() {
  using M = Misc<D, CH>;
  static_assert(offsetof(M, rs) % 16 == 0 && offsetof(M, wmax) % 16 == 0 && offsetof(M, mrow) % 16 == 0 &&
                    offsetof(M, nankey) % 16 == 0,
                "read as float4");
  return Cfg<D, CH>::offMisc + (uint32_t)sizeof(Misc<D, CH>);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void sts8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// The largest of the warp's values (all lanes; NaN counts as no value).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// An f16 pair (magnitudes at most 448) as three E4M3 pairs: x0 + x1 / 16 + x2 / 256.
__device__ __forceinline__ void split3(uint32_t x, uint16_t& t0, uint16_t& t1, uint16_t& t2) {
  asm("{\n\t.reg .b32 f, r, m, s;\n\t"
      "mov.b32 m, 0xcc00cc00;\n\t"  // -16, -16
      "mov.b32 s, 0x4c004c00;\n\t"  // 16, 16
      "cvt.rn.satfinite.e4m3x2.f16x2 %0, %3;\n\t"
      "cvt.rn.f16x2.e4m3x2 f, %0;\n\t"
      "mul.rn.f16x2 r, %3, s;\n\t"
      "fma.rn.f16x2 r, f, m, r;\n\t"  // 16 (x - x0), exact
      "cvt.rn.satfinite.e4m3x2.f16x2 %1, r;\n\t"
      "cvt.rn.f16x2.e4m3x2 f, %1;\n\t"
      "mul.rn.f16x2 r, r, s;\n\t"
      "fma.rn.f16x2 r, f, m, r;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %2, r;\n\t}"
      : "=&h"(t0), "=&h"(t1), "=&h"(t2)
      : "r"(x));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The walk over a CTA's segments; every role makes it for itself.  A unit counts for
// its tiles, or for one where runs are of whole units.
template <int KT>
struct Walk {
  int x, x_end, r, pre, g, nt, whole;
  __device__ int count() const { return whole ? 1 : nt; }
  __device__ int unit(const Requests& rq) const { return rq.Hkv * pre + g * count(); }
  __device__ void init(const Requests& rq, int x0, int x1, int r0, int pre0, int whole_units) {
    x = x0;
    x_end = x1;
    r = r0;
    pre = pre0;
    whole = whole_units;
    nt = rq.tiles<KT>(r);
    g = (x - rq.Hkv * pre) / count();
  }
  __device__ bool more() const { return x < x_end; }
  __device__ void get(int& kt0, int& kt1, const Requests& rq) const {
    kt0 = whole ? 0 : x - unit(rq);
    kt1 = whole ? nt : min(nt, x_end - unit(rq));
  }
  __device__ void next(const Requests& rq) {
    x = min(unit(rq) + count(), x_end);
    if (x >= x_end) return;
    if (++g == rq.Hkv) {
      g = 0;
      pre += count();
      do nt = ++r < rq.B ? rq.tiles<KT>(r) : 0;
      while (nt == 0 && r < rq.B);
      if (r >= rq.B) x = x_end;  // (lengths that changed under the kernel)
    }
  }
};

// The run of CTA w among W is tiles [first(w), first(w + 1)): the lower ones are one
// longer where W does not divide the total.
struct Share {
  int base, rest;
  __device__ __forceinline__ Share(int total, int W) : base(total / W), rest(total % W) {}
  __device__ __forceinline__ int first(int w) const { return w * base + min(w, rest); }
  __device__ __forceinline__ int of(int x) const {  // the CTA that has tile x
    const int cut = rest * (base + 1);
    return x < cut ? x / (base + 1) : rest + (x - cut) / base;
  }
};

template <int D, int CH>
__global__ void __launch_bounds__(kThreads, 2)
    decode_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ DecodeParams prm) {
  using C = Cfg<D, CH>;
  using M = Misc<D, CH>;
  constexpr int KPR = C::KPR, KT = C::KT, ROWS = C::ROWS, NK = C::NK, NV = C::NV, NPB = C::NPB, SB = C::SB;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  M& ms = *reinterpret_cast<M*>(smem + C::offMisc);
  const Requests& rq = prm.rq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = rq.G;
  auto token_of = [&](int row) { return (int)((uint32_t)row * prm.per_g >> 16); };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int W = gridDim.x, me = blockIdx.x;
  if (warp == 5) {
    tc::tmem_alloc(smem_u32(&ms.tmem), 256);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < 3; ++s) {
      mbar_init(&ms.kfull[s], 1);
      mbar_init(&ms.kfree[s], 1);
      mbar_init(&ms.vfull[s], 1);
      mbar_init(&ms.vfree[s], 1);
      mbar_init(&ms.scfull[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms.qfull[s], 2);
      mbar_init(&ms.qfree[s], 2);
      mbar_init(&ms.sfull[s], 1);
      mbar_init(&ms.sfree[s], 128);
      mbar_init(&ms.pfull[s], 128);
      mbar_init(&ms.pfree[s], 1);
    }
    mbar_init(&ms.drain, 1);
    fence_mbar_init();
  }
  for (int i = tid; i < D; i += kThreads) ms.nankey[i] = INT32_MAX;
  tc::fence_before_sync();
  bool odd = false;
  scan_requests<kThreads>(  // (its barriers publish the above too)
      rq.B,
      [&](int r) {
        const int n = rq.tiles<KT>(r, &odd);
        return prm.whole ? min(n, 1) : n;
      },
      ms.warp_sum, &ms.start_r, &ms.start_pre, &ms.total,
      [&](int all) { return Share(all * rq.Hkv, W).first(me) / rq.Hkv; });
  if (me == 0 && odd) report(prm.status, GIST_ATTN_STATUS_BAD_BLOCK);
  tc::fence_after_sync();
  const uint32_t tmem = ms.tmem;
  const Share sh(ms.total * rq.Hkv, W);
  const int x0 = sh.first(me), x1 = sh.first(me + 1);
  if (x0 >= x1 || ms.start_r < 0) {
    if (tid == 0) prm.join[me].parts = 0;
    if (warp == 5) tc::tmem_dealloc(tmem, 256);
    return;
  }
  Walk<KT> wk;
  wk.init(rq, x0, x1, ms.start_r, ms.start_pre, prm.whole);
  if (tid == 0 && !prm.whole) {
    const int a = wk.unit(rq);  // the unit of this run's first tile
    JoinUnit u{};
    if (x0 > a && sh.first(me - 1) <= a) {
      const int q0 = rq.q_start[wk.r], n = rq.q_start[wk.r + 1] - q0;
      u.parts = sh.of(a + wk.nt - 1) - me + 2;
      u.rows = n * G;
      u.q0 = q0;
      u.pos0 = max(rq.length(wk.r), 0) - n;
      u.g = wk.g;
      u.second = sh.first(me - 1) < a;
    }
    prm.join[me] = u;
  }
  bool failed = false;

  if (warp == 4) {
    // ================================================== K, V tiles and their scales
    if (lane == 0) tma_prefetch_map(&tm);
    const int br = prm.box_rows, vbl = rq.block_len / KPR, boxes = 128 / br;
    int i = 0, seg = 0;
    for (; wk.more() && !failed; wk.next(rq), ++seg) {
      int kt0, kt1;
      wk.get(kt0, kt1, rq);
      const int kv = rq.length(wk.r);
      const int32_t* table = rq.block_table + (int64_t)wk.r * rq.W;
      auto block_of = [&](int kt) {  // this lane's box of tile kt: block id, -1 if there is none
        const int row = kt * 128 + lane * br;
        return lane < boxes && (int64_t)row * KPR < kv ? table[row / vbl] : -1;
      };
      // ids are loaded two tiles ahead of their copies, scales one: no copy waits for
      // either but a segment's first
      auto plane_of = [&](int blk) {
        return ((blk >= 0 && blk < prm.num_blocks ? blk : 0) * prm.L + prm.layer) * 2 * rq.Hkv + wk.g;
      };
      int blk = block_of(kt0), blk1 = kt0 + 1 < kt1 ? block_of(kt0 + 1) : -1;
      int plane = plane_of(blk);
      float k_scale = lane < boxes ? __ldg(prm.scale + plane) : 0.f;
      float v_scale = lane < boxes ? __ldg(prm.scale + plane + rq.Hkv) : 0.f;
      if (lane == 0) ms.bad[seg & 7] = kv < 0;
      __syncwarp();
      for (int kt = kt0; kt < kt1; ++kt, ++i) {
        const int ks = i % NK, vs = i % NV;
        const int row = kt * 128 + lane * br;
        const bool want = lane < boxes && (int64_t)row * KPR < kv;
        const bool ok = want && blk >= 0 && blk < prm.num_blocks;
        if (want && !ok) {
          ms.bad[seg & 7] = 1;
          report(prm.status, GIST_ATTN_STATUS_BAD_BLOCK);
        }
        if (ok && fabsf(v_scale) > kMostScale) report(prm.status, GIST_ATTN_STATUS_RANGE);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, ok)) * br * 128;
        const int inner = row % vbl;
        if (__any_sync(0xffffffffu, (i >= NK && !mbar_wait(&ms.kfree[ks], ((uint32_t)(i / NK) & 1u) ^ 1u)))) {
          failed = true;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&ms.kfull[ks], bytes);
        __syncwarp();
        if (ok) tma_load_3d(sbase + ks * kStage + lane * br * 128, &tm, &ms.kfull[ks], 0, inner, plane);
        const int plane1 = plane_of(blk1);
        const float k1 = lane < boxes ? __ldg(prm.scale + plane1) : 0.f;
        const float v1 = lane < boxes ? __ldg(prm.scale + plane1 + rq.Hkv) : 0.f;
        const int blk2 = kt + 2 < kt1 ? block_of(kt + 2) : -1;
        if (__any_sync(0xffffffffu, (i >= NV && !mbar_wait(&ms.vfree[vs], ((uint32_t)(i / NV) & 1u) ^ 1u)))) {
          failed = true;
          ++i;  // its K load is in flight
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&ms.vfull[vs], bytes);
        __syncwarp();
        if (ok) tma_load_3d(sbase + C::offV + vs * kStage + lane * br * 128, &tm, &ms.vfull[vs], 0, inner, plane + rq.Hkv);
        if (lane < 16) {
          ms.ksc[vs][lane] = ok ? k_scale : 0.f;
          ms.vsc[vs][lane] = ok ? v_scale : 0.f;
          ms.vlog[vs][lane] = ok ? scale_log2(v_scale) : 0.f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.scfull[vs]);
        blk = blk1;
        blk1 = blk2;
        plane = plane1;
        k_scale = k1;
        v_scale = v1;
      }
    }
    if (failed) {  // the copies issued land before the CTA leaves
      for (int s = 0; s < NK && s < i; ++s) mbar_wait(&ms.kfull[(i - 1 - s) % NK], (uint32_t)((i - 1 - s) / NK) & 1u);
      for (int s = 0; s < NV && s < i; ++s) mbar_wait(&ms.vfull[(i - 1 - s) % NV], (uint32_t)((i - 1 - s) / NV) & 1u);
    }
  } else if (warp == 5) {
    // ================================================== tcgen05
    int i = 0, seg = 0;
    bool pending = false, first = false;  // P V of tile i - 1 to issue; the first of its segment
    int nch = 1;
    auto issue_pv = [&]() {
      const int t = i - 1, pb = t % NPB, vs = t % NV;
      if (__any_sync(0xffffffffu, !mbar_wait(&ms.pfull[pb], (uint32_t)(t / NPB) & 1u) ||
                                      !mbar_wait(&ms.vfull[vs], (uint32_t)(t / NV) & 1u))) {
        failed = true;
        return;
      }
      tc::fence_after_sync();
      if (tc::elect_one()) {
        const uint32_t id = tc::idesc_e4m3_f32(128, (KPR * 24 * nch + 15) & ~15, 1);
        const uint32_t vb = sbase + C::offV + vs * kStage, pp = sbase + C::offP + pb * C::PB;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc::mma_ss_f8(tmem + C::kO, tc::smem_desc_sw128(vb + k * 4096, kStage, 1024),
                 tc::smem_desc_sw128(pp + k * 32, 16, 1024), id, !first || k > 0);
        tc::commit(smem_u32(&ms.pfree[pb]));
        tc::commit(smem_u32(&ms.vfree[vs]));
      }
      __syncwarp();
    };
    for (; wk.more() && !failed; wk.next(rq), ++seg) {
      int kt0, kt1;
      wk.get(kt0, kt1, rq);
      if (pending) issue_pv();
      pending = false;
      const int qs = seg & 1;
      if (failed || __any_sync(0xffffffffu, !mbar_wait(&ms.qfull[qs], (uint32_t)(seg >> 1) & 1u))) {
        failed = true;
        break;
      }
      nch = (ms.seg[qs].rows + 7) >> 3;
      const uint32_t id = tc::idesc_e4m3_f32(128, (8 * nch + 15) & ~15, 0);
      const uint32_t qb = sbase + C::offQ + qs * C::QB;
      for (int kt = kt0; kt < kt1; ++kt) {
        const int ks = i % NK, sb = i % SB;
        if (__any_sync(0xffffffffu, !mbar_wait(&ms.kfull[ks], (uint32_t)(i / NK) & 1u) ||
                                        (i >= SB && !mbar_wait(&ms.sfree[sb], ((uint32_t)(i / SB) & 1u) ^ 1u)))) {
          failed = true;
          break;
        }
        tc::fence_after_sync();
        if (tc::elect_one()) {
          const uint32_t kb = sbase + ks * kStage;
#pragma unroll
          for (int p = 0; p < KPR; ++p)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                tc::mma_ss_f8(tmem + (sb * KPR + p) * C::SP, tc::smem_desc_sw128(kb + p * 64 + k * 32, 16, 1024),
                              tc::smem_desc_sw128(qb + t * C::QT + k * 32, 16, 1024), id, t > 0 || k > 0);
          tc::commit(smem_u32(&ms.sfull[sb]));
          tc::commit(smem_u32(&ms.kfree[ks]));
          if (kt == kt1 - 1) tc::commit(smem_u32(&ms.qfree[qs]));
        }
        __syncwarp();
        if (pending) issue_pv();
        if (failed) break;
        first = kt == kt0;
        pending = true;
        ++i;
      }
    }
    if (pending && !failed) issue_pv();
    if (tc::elect_one()) tc::commit(smem_u32(&ms.drain));
    __syncwarp();
    if (!mbar_wait(&ms.drain, 0)) failed = true;
  } else if (warp >= 6) {
    // ================================================== q rows
    // D / 16 lanes a row, each with elements j .. j + 7 and their partners j + D/2 ..
    constexpr int LR = D / 16, RP = 32 / LR;
    const int l = lane % LR, rl = lane / LR;
    uint64_t turn[8];  // into registers once: a constant read at LR places by a warp is slow
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      turn[e] = prm.turn[l * 8 + e];
      asm volatile("" : "+l"(turn[e]));
    }
    for (int seg = 0; wk.more() && !failed; wk.next(rq), ++seg) {
      int kt0, kt1;
      wk.get(kt0, kt1, rq);
      const int qs = seg & 1;
      const int q0 = rq.q_start[wk.r], n = rq.q_start[wk.r + 1] - q0, kv = rq.length(wk.r);
      const int rows = n * G, pos0 = max(kv, 0) - n;
      if (__any_sync(0xffffffffu, seg >= 2 && !mbar_wait(&ms.qfree[qs], ((uint32_t)(seg >> 1) & 1u) ^ 1u))) {
        failed = true;
        break;
      }
      const bf16* src = prm.q + ((int64_t)q0 * prm.Hq + wk.g * G) * D + l * 8;
      uint4 u, v;
      auto fetch = [&](int row) {
        const int rr = min(row, rows - 1), tok = token_of(rr);
        const bf16* p = src + ((int64_t)tok * prm.Hq + rr - tok * G) * D;
        u = ldg16(p);
        v = ldg16(p + D / 2);
      };
      const int padded = (rows + 7) & ~7, mine = (warp - 6) * RP;
      fetch(mine + rl);
#pragma unroll 1
      for (int j0 = mine; j0 < padded; j0 += 2 * RP) {
        const int row = j0 + rl;
        const bool real = row < rows;
        const int pos = pos0 + token_of(row);
        const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
        if (j0 + 2 * RP < padded) fetch(row + 2 * RP);
        float a[8], b[8], top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = real ? __uint_as_float(e & 1 ? uw[e >> 1] & 0xffff0000u : uw[e >> 1] << 16) : 0.f;
          const float y = real ? __uint_as_float(e & 1 ? vw[e >> 1] & 0xffff0000u : vw[e >> 1] << 16) : 0.f;
          float sn, cs;
          __sincosf(turn_angle(pos, turn[e]), &sn, &cs);  // off by 2^-21: under the terms' rounding
          a[e] = x * cs - y * sn;
          b[e] = y * cs + x * sn;
          top = fmaxf(top, fmaxf(fabsf(a[e]), fabsf(b[e])));
          if (!(fabsf(a[e]) <= 3.4e38f) || !(fabsf(b[e]) <= 3.4e38f)) top = INFINITY;
        }
#pragma unroll
        for (int o = LR / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t tb = __float_as_uint(top);
        const int ex = max((int)(tb >> 23) - 127 - 7, -119);  // the row's largest lands in [128, 256)
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        if (l == 0)
          ms.rs[qs][row] = !real                ? 0.f
                           : tb >= 0x7f800000u ? __int_as_float(0x7fc00000)
                                               : prm.scale_log2 * __uint_as_float((uint32_t)max(ex + 127, 1) << 23);
        const uint32_t base = sbase + C::offQ + qs * C::QB + row * 128;
        const uint32_t at = (uint32_t)(l * 8) ^ ((row & 7) << 4), bt = (uint32_t)(D / 2 + l * 8) ^ ((row & 7) << 4);
        uint16_t ta[4][4], tb2[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          terms4(a[2 * e] * down, a[2 * e + 1] * down, ta[0][e], ta[1][e], ta[2][e], ta[3][e]);
          terms4(b[2 * e] * down, b[2 * e + 1] * down, tb2[0][e], tb2[1][e], tb2[2][e], tb2[3][e]);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          sts64(base + s * C::QT + at, (uint32_t)ta[s][0] | (uint32_t)ta[s][1] << 16, (uint32_t)ta[s][2] | (uint32_t)ta[s][3] << 16);
          sts64(base + s * C::QT + bt, (uint32_t)tb2[s][0] | (uint32_t)tb2[s][1] << 16, (uint32_t)tb2[s][2] | (uint32_t)tb2[s][3] << 16);
        }
      }
      if (warp == 6 && lane == 0) ms.seg[qs] = Seg{wk.r, wk.g, rows, q0, pos0, max(kv, 0), kt0, kt1, wk.nt, 0};
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.qfull[qs]);
    }
  } else {
    // ================================================== softmax, output
    const int t = tid;  // tile row == TMEM lane
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    uint32_t pof[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) pof[j] = sbase + C::offP + j * 128 + (t ^ (j << 4));
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!failed && !mbar_wait(bar, parity)) failed = true;
    };
    int i = 0, seg = 0;
    for (; wk.more(); wk.next(rq), ++seg) {
      int kt0, kt1;
      wk.get(kt0, kt1, rq);
      const int qs = seg & 1;
      wait(&ms.qfull[qs], (uint32_t)(seg >> 1) & 1u);
      // a role that gave up ends this one's waits too: leave together
      if (named_bar_or(1, 128, failed)) {
        failed = true;
        break;
      }
      const Seg sg = ms.seg[qs];
      const int nch = (sg.rows + 7) >> 3;
      // running maxima: registers, or, where scores and sums fill those, a warp's own
      // copy in shared memory
      constexpr bool kHeld = CH * KPR < 4;
      float m[kHeld ? ROWS : 1], l[ROWS];
      auto maxima = [&](int c, float (&v)[8]) {
        if constexpr (kHeld) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = m[c * 8 + j];
        } else {
          const float4* at = reinterpret_cast<const float4*>(&ms.mrow[warp][c * 8]);
          const float4 a = at[0], b = at[1];
          v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
      };
#pragma unroll
      for (int j = 0; j < ROWS; ++j) l[j] = 0.f;
      if constexpr (kHeld) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) m[j] = kNone;
      } else {
        if (lane < ROWS) ms.mrow[warp][lane] = kNone;
        __syncwarp();
      }
      for (int kt = kt0; kt < kt1; ++kt, ++i) {
        const int sb = i % SB, vs = i % NV, pb = i % NPB;
        const int key0 = kt * KT + t * KPR;  // this thread's first key
        const bool edge = kt * KT + KT > sg.pos0 + 1;  // some row does not see all of the tile
        float s[ROWS * KPR];
        wait(&ms.scfull[vs], (uint32_t)(i / NV) & 1u);
        const int box = t >> prm.box_shift;
        const float ks = ms.ksc[vs][box], vlog = ms.vlog[vs][box];
        wait(&ms.sfull[sb], (uint32_t)(i / SB) & 1u);
        tc::fence_after_sync();
        bool over = false;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (c < nch) {
            uint32_t v[KPR][8];
#pragma unroll
            for (int p = 0; p < KPR; ++p) ld8(tmem + lane_base + (sb * KPR + p) * C::SP + c * 8, v[p]);
            tc::wait_ld();
            const float4* rp = reinterpret_cast<const float4*>(&ms.rs[qs][c * 8]);
            const float4 ra = rp[0], rb = rp[1];
            const float rs[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
            float mv[8];
            maxima(c, mv);
#pragma unroll
            for (int p = 0; p < KPR; ++p)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                float x = fmaf(__uint_as_float(v[p][j]), ks * rs[j], vlog);
                if (edge && key0 + p > sg.pos0 + token_of(c * 8 + j)) x = -INFINITY;
                over |= x - mv[j] > kSlack + kPUnit;
                s[(c * KPR + p) * 8 + j] = x;
              }
          }
        }
        tc::fence_before_sync();
        mbar_arrive(&ms.sfree[sb]);
        if (named_bar_or(1, 128, over)) {
          // new maxima, the same in all threads; the sums and O follow
#pragma unroll
          for (int c = 0; c < CH; ++c)
            if (c < nch) {
              float w[8];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                w[j] = warp_max(fmaxf(s[c * KPR * 8 + j], s[(c * KPR + KPR - 1) * 8 + j]));
              if (lane == 0) {
                float4* at = reinterpret_cast<float4*>(&ms.wmax[warp][c * 8]);
                at[0] = make_float4(w[0], w[1], w[2], w[3]);
                at[1] = make_float4(w[4], w[5], w[6], w[7]);
              }
            }
          named_bar_sync(1, 128);
          if (kt > kt0) wait(&ms.pfree[(i - 1) % NPB], (uint32_t)((i - 1) / NPB) & 1u);
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < CH; ++c)
            if (c < nch) {
              float f[8], mv[8];
              maxima(c, mv);
#pragma unroll
              for (int j = 0; j < 8; j += 4) {
                float4 w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const float4*>(&ms.wmax[k][c * 8 + j]);
                const float top[4] = {fmaxf(fmaxf(w[0].x, w[1].x), fmaxf(w[2].x, w[3].x)),
                                      fmaxf(fmaxf(w[0].y, w[1].y), fmaxf(w[2].y, w[3].y)),
                                      fmaxf(fmaxf(w[0].z, w[1].z), fmaxf(w[2].z, w[3].z)),
                                      fmaxf(fmaxf(w[0].w, w[1].w), fmaxf(w[2].w, w[3].w))};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int q = c * 8 + j + k;
                  // (in two steps: where the maximum moves by V scales the sum may be far from 1)
                  const float mn = fmaxf(mv[j + k], top[k] - kPUnit), half = ex2_approx(0.5f * (mv[j + k] - mn));
                  f[j + k] = half * half;
                  l[q] = l[q] * half * half;
                  mv[j + k] = mn;
                }
              }
              if constexpr (kHeld) {
#pragma unroll
                for (int j = 0; j < 8; ++j) m[c * 8 + j] = mv[j];
              } else {
                __syncwarp();  // (all lanes have read the old ones)
                if (lane == 0) {
                  float4* at = reinterpret_cast<float4*>(&ms.mrow[warp][c * 8]);
                  at[0] = make_float4(mv[0], mv[1], mv[2], mv[3]);
                  at[1] = make_float4(mv[4], mv[5], mv[6], mv[7]);
                }
                __syncwarp();
              }
              bool moved = false;  // (the same in all threads)
#pragma unroll
              for (int j = 0; j < 8; ++j) moved |= f[j] != 1.f;
              if (kt > kt0 && moved) {
#pragma unroll
                for (int p = 0; p < KPR; ++p) {
                  const uint32_t a = tmem + lane_base + C::kO + p * 24 * nch + c * 24;
                  uint32_t v[3][8];
#pragma unroll
                  for (int k = 0; k < 3; ++k) ld8(a + k * 8, v[k]);
                  tc::wait_ld();
#pragma unroll
                  for (int k = 0; k < 3; ++k) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[k][j] = __float_as_uint(__uint_as_float(v[k][j]) * f[j]);
                    tc::st8(a + k * 8, v[k]);
                  }
                }
              }
            }
          tc::wait_st();
        }
        if (i >= NPB) wait(&ms.pfree[pb], (uint32_t)(i / NPB - 1) & 1u);
        // the V scale's sign goes to P, and a scale of zero makes P zero
        // (a NaN logarithm is in the scores of the rows that see the key; the others' weights
        // stay 0)
        const float vsc = ms.vsc[vs][box], vback = vlog == vlog ? vlog : 0.f;
        const uint32_t sign = fabsf(vsc) < kLeastScale ? 0u : vsc < 0.f ? 0xbc00bc00u : 0x3c003c00u;  // 0, -1 or 1, twice
#pragma unroll
        for (int c = 0; c < CH; ++c)
          if (c < nch) {
            float mv[8];
            maxima(c, mv);
#pragma unroll
            for (int p = 0; p < KPR; ++p) {
              const uint32_t at = pb * C::PB + (p * 3 * nch + c * 3) * 1024;
#pragma unroll
              for (int j = 0; j < 8; j += 2) {
                const int q = c * 8 + j;
                const float x0 = s[(c * KPR + p) * 8 + j] - mv[j], x1 = s[(c * KPR + p) * 8 + j + 1] - mv[j + 1];
                l[q] += ex2_approx(x0 - vback);
                l[q + 1] += ex2_approx(x1 - vback);
                uint16_t u[3];
                split3(mul_f16x2(to_f16x2(ex2_approx(x0), ex2_approx(x1)), sign), u[0], u[1], u[2]);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                  sts8(pof[j] + at + k * 1024, u[k]);
                  sts8(pof[j + 1] + at + k * 1024, u[k] >> 8);
                }
              }
            }
          }
        if (edge) {
          // V rows that not every query row sees: those past the end are cleared, and
          // a NaN in the others too (0 x NaN would reach rows that do not see it),
          // noted for the rows that do
          wait(&ms.vfull[vs], (uint32_t)(i / NV) & 1u);
          if (key0 + KPR - 1 > sg.pos0) {
            const uint32_t vrow = sbase + C::offV + vs * kStage + t * 128;
#pragma unroll 1
            for (int ch = 0; ch < 8; ++ch) {
              const int key = key0 + (KPR == 2 ? ch >> 2 : 0);
              const uint32_t a = vrow + ((ch ^ (t & 7)) << 4);
              if (key >= sg.kv) {
                sts16(a, make_uint4(0, 0, 0, 0));
              } else if (key > sg.pos0) {
                const uint4 w = lds16(a);
                if (e4m3_nan(w.x) | e4m3_nan(w.y) | e4m3_nan(w.z) | e4m3_nan(w.w)) {
#pragma unroll 1
                  for (int e = 0; e < 16; ++e)
                    if ((lds8(a + e) & 0x7fu) == 0x7fu) {
                      sts8(a + e, 0);
                      atomicMin(&ms.nankey[(ch * 16 + e) % D], key);
                    }
                }
              }
            }
          }
        }
        fence_proxy_async_smem();
        tc::fence_before_sync();
        mbar_arrive(&ms.pfull[pb]);
      }
      // ---- the segment's O, m and sums
      wait(&ms.pfree[(i - 1) % NPB], (uint32_t)((i - 1) / NPB) & 1u);
      tc::fence_after_sync();
      // through shared memory (the segment's q is used no more), a warp a row then
      float* stage = reinterpret_cast<float*>(smem + C::offQ + qs * C::QB);  // [ROWS][128]
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (c < nch) {
          uint32_t v[24];
#pragma unroll
          for (int k = 0; k < 3; ++k)
            ld8(tmem + lane_base + C::kO + (KPR == 2 ? (t >> 6) * 24 * nch : 0) + c * 24 + k * 8, v + k * 8);
          tc::wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float x = __uint_as_float(v[j]);
            x = fmaf(__uint_as_float(v[8 + j]), 0.0625f, x);
            x = fmaf(__uint_as_float(v[16 + j]), 0.00390625f, x);
            stage[(c * 8 + j) * 128 + t] = x;
          }
          // the warp's sums of 8 rows: halves, quarters, eighths of the rows a lane
          float h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float keep = lane & 16 ? l[c * 8 + 4 + k] : l[c * 8 + k], send = lane & 16 ? l[c * 8 + k] : l[c * 8 + 4 + k];
            h[k] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float keep = lane & 8 ? h[2 + k] : h[k], send = lane & 8 ? h[k] : h[2 + k];
            h[k] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
          }
          float y = (lane & 4 ? h[1] : h[0]) + __shfl_xor_sync(0xffffffffu, lane & 4 ? h[0] : h[1], 4);
          y += __shfl_xor_sync(0xffffffffu, y, 2);
          y += __shfl_xor_sync(0xffffffffu, y, 1);
          if ((lane & 3) == 0) ms.wmax[warp][c * 8 + (lane >> 4) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1)] = y;
          if (kHeld && t == 0) {
            float mv[8];
            maxima(c, mv);
            float4* at = reinterpret_cast<float4*>(&ms.mrow[0][c * 8]);
            at[0] = make_float4(mv[0], mv[1], mv[2], mv[3]);
            at[1] = make_float4(mv[4], mv[5], mv[6], mv[7]);
          }
        }
      tc::fence_before_sync();
      named_bar_sync(1, 128);
      const bool whole = kt0 == 0 && kt1 == sg.nt, bad = ms.bad[seg & 7] != 0;
      float* part = prm.parts + (int64_t)(2 * me + (x0 == wk.x ? 0 : 1)) * ROWS * (D + 2);
      constexpr int E = D / 32;  // elements a lane
#pragma unroll 1
      for (int q = warp; q < sg.rows; q += 4) {
        const int tok = token_of(q), pos = sg.pos0 + tok;
        float x[E];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 a = *reinterpret_cast<const float2*>(&stage[q * 128 + lane * E + e]);
          x[e] = a.x;
          x[e + 1] = a.y;
          if (KPR == 2) {
            const float2 b = *reinterpret_cast<const float2*>(&stage[q * 128 + 64 + lane * E + e]);
            x[e] += b.x;
            x[e + 1] += b.y;
          }
          const int2 nk = *reinterpret_cast<const int2*>(&ms.nankey[lane * E + e]);
          if (nk.x <= pos) x[e] = __int_as_float(0x7fc00000);
          if (nk.y <= pos) x[e + 1] = __int_as_float(0x7fc00000);
        }
        const float sum = (ms.wmax[0][q] + ms.wmax[1][q]) + (ms.wmax[2][q] + ms.wmax[3][q]);
        if (whole) {
          const bool none = bad || pos < 0;
          if (lane == 0 && !none && !(sum <= 3.0e38f)) report(prm.status, GIST_ATTN_STATUS_RANGE);
          const float inv = 1.f / sum;
          bf16* dst = prm.out + ((int64_t)(sg.q0 + tok) * prm.Hq + sg.g * G + q - tok * G) * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; e += 2)
            *reinterpret_cast<uint32_t*>(dst + e) = none ? 0u : float2_to_bf16x2(x[e] * inv, x[e + 1] * inv);
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(part + q * D + lane * E + e) = make_float2(x[e], x[e + 1]);
          if (lane == 0) {
            part[ROWS * D + q] = ms.mrow[0][q];
            part[ROWS * D + ROWS + q] = bad ? -1.f : sum;
          }
        }
      }
      named_bar_sync(1, 128);  // the stage, the sums and nankey are read
      if (t < D) ms.nankey[t] = INT32_MAX;
      if (t == 0) mbar_arrive(&ms.qfree[qs]);
    }
  }
  if (failed) report(prm.status, GIST_ATTN_STATUS_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 256);
  }
}

// Joins the parts of the units that cross CTAs, a block of the grid a CTA w that may
// hold a unit's second part.  A warp (several, if there are fewer rows than warps)
// takes a row: all parts' maxima and sums at once, then their O with the final
// weights, so that no load waits for another's result; the order of the sums is
// fixed.
constexpr int kJoinThreads = 32 * 32, kJoinHeld = 2048;
template <int D, int CH>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const __grid_constant__ DecodeParams prm) {
  constexpr int ROWS = Cfg<D, CH>::ROWS, E = D / 32;  // E elements a lane
  __shared__ float2 held[kJoinHeld];                  // [row][part]: maximum and sum
  __shared__ float acc[kJoinThreads / 32][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, w = blockIdx.x + 1;
  const int G = prm.rq.G, threads = blockDim.x, warps = threads / 32;
  const int row0 = blockIdx.y * prm.join_rows;  // this block's rows
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinUnit u = prm.join[w];
  const int rows = min(u.rows - row0, prm.join_rows);
  if (u.parts == 0 || rows <= 0) return;
  int wpr = warps;  // warps a row
  while (wpr > 1 && warps / wpr < rows) wpr >>= 1;
  const int sub = warp % wpr, local = warp / wpr, q = row0 + local;
  const bool mine = local < rows;
  auto part = [&](int v) {
    return prm.parts + (int64_t)(2 * (w - 1 + v) + (v == 0 ? u.second : 0)) * ROWS * (D + 2);
  };
  float m = kNone, sum = 0.f, o[E];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const int most = kJoinHeld / rows;
  for (int v0 = 0; v0 < u.parts; v0 += most) {
    const int nv = min(most, u.parts - v0);
    for (int i = tid; i < nv * rows; i += threads) {
      const int v = i / rows, row = i - v * rows;
      const float* p = part(v0 + v) + ROWS * D + row0 + row;
      held[row * most + v] = make_float2(p[0], p[ROWS]);
    }
    __syncthreads();
    if (mine) {
      const float2* h = held + local * most;
      float top = kNone;
      for (int v = lane; v < nv; v += 32) top = fmaxf(top, h[v].x);
#pragma unroll
      for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
      top = fmaxf(top, m);
      const float half = exp2f(0.5f * (m - top)), f = half * half;
      m = top;
      sum = sum * half * half;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
      for (int v = lane; v < nv; v += 32) {
        const float2 x = h[v];
        const float half = exp2f(0.5f * (x.x - m));
        sum += x.y * half * half;
        bad |= x.y < 0.f;
      }
#pragma unroll 8
      for (int v = sub; v < nv; v += wpr) {
        const float* p = part(v0 + v) + q * D + lane * E;
        const float fv = exp2f(h[v].x - m);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 x = *reinterpret_cast<const float2*>(p + e);
          o[e] += fv * x.x;
          o[e + 1] += fv * x.y;
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  bad = __any_sync(0xffffffffu, bad);
  if (wpr > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[warp][lane * E + e] = o[e];
    __syncthreads();
    if (sub == 0)
      for (int k = 1; k < wpr; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += acc[warp + k][lane * E + e];
  }
  if (mine && sub == 0) {
    const int tok = q / G;
    const bool none = bad || u.pos0 + tok < 0;
    if (lane == 0 && !none && !(sum <= 3.0e38f)) report(prm.status, GIST_ATTN_STATUS_RANGE);
    const float inv = 1.f / sum;
    bf16* dst = prm.out + ((int64_t)(u.q0 + tok) * prm.Hq + u.g * G + q - tok * G) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = none ? 0u : float2_to_bf16x2(o[e] * inv, o[e + 1] * inv);
  }
}

// The pool as {128 bytes, rows of 128 bytes a plane, planes}, boxes of `rows` rows.
int encode_pool(CUtensorMap* m, const PagedProblem& pb, int rows) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return GIST_ATTN_ERR_LAUNCH;
  const cuuint64_t plane_rows = (cuuint64_t)pb.block_len * pb.d / 128;
  const cuuint64_t dims[3] = {128, plane_rows, (cuuint64_t)pb.num_blocks * pb.L * 2 * pb.Hkv};
  const cuuint64_t strides[2] = {128, plane_rows * 128};
  const cuuint32_t box[3] = {128, (cuuint32_t)rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(pb.pool), dims, strides, box,
                         estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GIST_ATTN_OK : GIST_ATTN_ERR_UNSUPPORTED;
}

// CTAs: two an SM, or one a tile where the table cannot hold that many.
int grid_of(const PagedProblem& pb, int sms) {
  const double tiles = (double)pb.B * pb.Hkv * (((int64_t)pb.W * pb.block_len * pb.d + 16383) / 16384);
  return tiles < 2.0 * sms ? (int)tiles : 2 * sms;
}

template <int D, int CH>
int launch(const PagedProblem& pb, void* workspace, int sms, cudaStream_t stream) {
  DecodeParams prm{};
  prm.q = static_cast<const bf16*>(pb.q);
  prm.out = static_cast<bf16*>(pb.out);
  prm.scale = pb.scale;
  const int grid = grid_of(pb, sms);
  prm.whole = ((int64_t)pb.W * pb.block_len + Cfg<D, CH>::KT - 1) / Cfg<D, CH>::KT <= kWhole;
  prm.join = static_cast<JoinUnit*>(workspace);
  prm.parts = reinterpret_cast<float*>(prm.join + grid);
  prm.status = pb.status;
  prm.rq = requests_of(pb);
  prm.rq.max_rows = Cfg<D, CH>::ROWS;
  prm.Hq = pb.Hq;
  prm.L = pb.L;
  prm.layer = pb.layer;
  prm.num_blocks = pb.num_blocks;
  prm.scale_log2 = pb.scale_log2;
  prm.per_g = (65536u + pb.G - 1) / pb.G;
  for (int j = 0; j < 64; ++j) prm.turn[j] = pb.turn[j];
  const int plane_rows = pb.block_len * D / 128;
  prm.box_shift = 7;
  while (plane_rows & ((1 << prm.box_shift) - 1)) --prm.box_shift;
  prm.box_rows = 1 << prm.box_shift;
  // The join: a block a unit, a warp a row; where units are few their parts are many, and
  // several warps take a row, blocks of eight warps a row or four.
  const bool many = (int64_t)pb.B * pb.Hkv * 4 < grid;
  prm.join_rows = !many ? Cfg<D, CH>::ROWS : CH == 1 ? 1 : 4;
  alignas(64) CUtensorMap tm;
  const int rc = encode_pool(&tm, pb, prm.box_rows);
  if (rc != GIST_ATTN_OK) return rc;
  constexpr uint32_t smem = smem_bytes<D, CH>();
  static_assert(smem <= 113 * 1024, "two CTAs an SM");
  if (cudaFuncSetAttribute(decode_kernel<D, CH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  decode_kernel<D, CH><<<grid, kThreads, smem, stream>>>(tm, prm);
  if (cudaGetLastError() != cudaSuccess) return GIST_ATTN_ERR_LAUNCH;
  if (grid == 1 || prm.whole) return GIST_ATTN_OK;
  // the combine's CTAs may start while the last tiles run (and then wait for them)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid - 1, many ? (Cfg<D, CH>::ROWS + prm.join_rows - 1) / prm.join_rows : 1);
  cfg.blockDim = dim3(many ? 256 : 32 * Cfg<D, CH>::ROWS);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<D, CH>, prm) == cudaSuccess ? GIST_ATTN_OK : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace

// Rows (new tokens x group) the kernel takes for a request.
int paged_decode_rows(const PagedProblem& pb) { return pb.d / 4; }

size_t paged_decode_workspace(const PagedProblem& pb, int sms) {
  return (size_t)grid_of(pb, sms) * (sizeof(JoinUnit) + 2 * paged_decode_rows(pb) * (pb.d + 2) * sizeof(float));
}

int launch_paged_decode(const PagedProblem& pb, void* workspace, int sms, cudaStream_t stream) {
  const int64_t rows = (int64_t)pb.max_new * pb.G;
  if (pb.d == 64)
    return rows <= 8 ? launch<64, 1>(pb, workspace, sms, stream) : launch<64, 2>(pb, workspace, sms, stream);
  return rows <= 8    ? launch<128, 1>(pb, workspace, sms, stream)
         : rows <= 16 ? launch<128, 2>(pb, workspace, sms, stream)
                      : launch<128, 4>(pb, workspace, sms, stream);
}

}  // namespace gattn
