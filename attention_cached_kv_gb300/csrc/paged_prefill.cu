// paged_prefill.cu -- many query rows a request (prompt chunks) against its E4M3
// paged cache, causal ([KV page, "Reusable-state"]; [Suffix page, §2, §5, §6 问题四]).
//
// A CTA takes one KV head and up to 256 query rows of a request: two row tiles of
// floor(128 / G) tokens x G heads.  Its keys stream by in tiles of 128, one pass,
//     S = q K^T, P = exp2(S + log2 v - m), O += P V       (tcgen05 kind::f16, TMEM)
// with v the V scale of a key's block, V its codes, and m the row's running maximum of
// S + log2 v, moved only when a tile's maximum passes it by more than 12 (log2 units).
// The sum of weights is of P / v.  So P's bits go by what a key adds to the row, and the
// values are exact.  The warps:
//   * 0-3, 4-7: a thread a row of each row tile, softmax and output; P goes back
//     into S's columns as f16 (11 bits), A operand of the second product;
//   * 8-11: cached rows from global memory through registers into f16 tiles, exactly
//     (K's block scales multiply the fp32 scores);
//   * 12: the MMAs, alternating between the row tiles, so that one's products run
//     while the other's softmax does;
//   * 13: block ids and scales, four tiles at a time, ahead of the copies;
//   * 14: the softmax warps' segments, one ahead.
// One conversion of a key serves 256 rows: that is why rows are taken in pairs of tiles
// here and cached bytes are used as they are where there are few rows (paged_decode.cu).
// q is scaled by a power of two a row and rounded to f16, and what that leaves of it to f16
// again: the low part, which takes part only in tiles where scores may be so large that the
// first rounding shows (kFine).  Its room is why values have one buffer if D = 128: they are
// converted a tile behind the keys.  All that costs 10 us of the chunks below, the low
// products, where scores are large, 30 more (as four E4M3 terms against unconverted keys,
// with two buffers for values, they were always there and cost 54).
//
// Work is the sequence of (request, KV head, row-tile pair) units, each worth the keys
// it sees and a constant for its start; each SM's CTA takes an equal run of it, cut
// inside a unit between key tiles.  Units that cross CTAs leave parts (O, m, sum) in
// the workspace and join_kernel adds them up in key order: chunks of unlike lengths,
// or one short chunk behind a long context, spread evenly.  A start and an end (rows of q
// in and rotated, rows of O out) run a few times a CTA, mostly out of a cold instruction
// cache, so their loops stay rolled: unrolled they took 11 us together, rolled 9.
// Bound: per key tile (2.1 us) the chain scores - softmax - output of a row tile; the
// converting warps (1.6 us) and the products (1.5 us) are not far below.  Four chunks of
// 700-1024 tokens behind 1000-6000 cached ones, 32 / 8 heads of 128: 264 us = 884 TFLOP/s;
// 293 us where every tile needs q's low part.  (Tried: a warp a row tile for the products;
// a warpgroup each for keys and values with a register split; half the keys widened by
// integer operations; the copies ahead into L2.  None gained, some lost up to a tenth.)
//
// Pages: [KV page] "为什么自回归推理缓存 KV，而不缓存历史 Q？";
//        [Suffix page] icman.com.cn news 64898.
#include <math.h>

#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "paged_tc.cuh"

namespace gattn {
namespace {

constexpr int kThreads = 480;         // 8 softmax, 4 converting, MMA, look-up, segment warp
constexpr int kRing = 8;              // tiles whose look-ups are held, in two halves
constexpr int kKT = 128;              // keys a tile
constexpr float kNone = -3.0e38f;     // running maximum before any key
// Log2 units that a score may pass it by (P stays below f16's 2^16).  A tile that passes it
// is done twice: with 8, where V scales differ by 2^2, the chunks below took 295 us for 252.
constexpr float kSlack = 12.f;
// Where |q| |k| (log2 units, k all of 448) is above this, q's scores take its low part as well.
// Below it what f16 rounds off q, 2^-11 at most of an element, moves a score by 160 2^-11 /
// sqrt(3 d) rms even then, a weight by no more than an output's half step in bf16.
constexpr float kFine = 160.f;

// While no V scale is outside 2^+-45 the sum's terms are P / v: P is at least 2^-126 for all
// keys of 2^-36 of the largest weight and more.  Otherwise they are exponentials of their own.
constexpr float kPlain = 45.f;

constexpr int kStartCost = 512;       // keys that a unit's start is worth

// What the join needs of a unit that crosses CTAs, left by the CTA whose run starts in
// it first (cost 0: nothing to join there).
struct JoinRun {
  int64_t at, share, rest;  // the unit's first place in the sequence of costs; total / CTAs, total % CTAs
  int cost, tiles, q0, toks, pos0, g;
  int pad[4];
};
static_assert(sizeof(JoinRun) == 64, "the parts behind the headers are read 16 bytes at a time");

struct PrefillParams {
  const bf16* q;
  bf16* out;
  const uint8_t* pool;
  const float* scale;
  JoinRun* join;  // workspace: [CTAs], then the parts, two a CTA
  float* parts;
  int32_t* status;
  Requests rq;
  int Hq, L, layer, num_blocks, min_new, Tm;
  float scale_log2;
  float largest;  // |k| of codes all 448 (0 where q has no low parts)
  uint32_t per_g;  // 2^16 / G rounded up: j / G = j per_g >> 16 for j < 128
  uint64_t turn[64];
};

template <int D>
struct PCfg {
  static constexpr uint32_t kTile = 128 * D * 2;        // bytes of a 128-row f16 tile
  static constexpr uint32_t kPanel = 128 * 128;         // 64 columns of it
  static constexpr int NV = D == 64 ? 2 : 1;            // V buffers
  static constexpr int kSlots = 2 * NV;                 // segments that are apart: see nankey
  static constexpr uint32_t offL = 2 * kTile, offK = 4 * kTile, offV = 6 * kTile, offMisc = (6 + NV) * kTile;
  static constexpr int kS = 0, kO = 256;  // TMEM columns: S (P) of the row tiles, O
};

// One unit's share of a CTA.
struct PSeg {
  int r, g, q0, toks, pos0, kend, kt0, nt, slot;
  bool two, whole;
};

// The walk over a CTA's segments; every role makes it for itself.  In a request
// whose rows end at key `base` + n, pair p of row tiles (w tokens) costs
// kStartCost + base + w (p + 1).
struct PWalk {
  int64_t x, x_end, pre;
  int r, g, p;
  int n, kv, base, np, w;
  __device__ int64_t before(int q) const { return (int64_t)q * (kStartCost + base) + (int64_t)w * q * (q + 1) / 2; }
  __device__ int64_t unit() const { return pre + g * before(np) + before(p); }
  __device__ int cost() const { return kStartCost + base + w * (p + 1); }
  __device__ void request(const PrefillParams& prm) {
    const Requests& rq = prm.rq;
    n = r < rq.B ? rq.tokens(r) : 0;
    if (n < prm.min_new) n = 0;
    kv = n > 0 ? rq.length(r) : 0;
    base = max(max(kv, 0) - n, 0);
    np = (n + w - 1) / w;
  }
  __device__ void init(const PrefillParams& prm, int64_t x0, int64_t x1, int r0, int64_t pre0) {
    x = x0;
    x_end = x1;
    r = r0;
    pre = pre0;
    w = 2 * prm.Tm;
    request(prm);
    int64_t rem = x - pre;
    const int64_t head = before(np);
    g = (int)(rem / head);
    rem -= g * head;
    // before(p) <= rem < before(p + 1): a root in fp32, then the step or two it is off
    const float b = (float)(kStartCost + base) + 0.5f * w;
    p = max(0, min(np - 1, (int)((sqrtf(b * b + 2.f * w * (float)rem) - b) / w)));
    while (p > 0 && before(p) > rem) --p;
    while (p + 1 < np && before(p + 1) <= rem) ++p;
  }
  __device__ bool more() const { return x < x_end; }
  // The segment at x; false where the run holds none of the unit's key tiles.
  __device__ bool get(const PrefillParams& prm, PSeg& s) const {
    const int64_t u = unit();
    const int c = cost(), tok0 = p * w;
    s.r = r;
    s.g = g;
    s.toks = min(w, n - tok0);
    s.q0 = prm.rq.q_start[r] + tok0;         // first token row
    s.pos0 = max(kv, 0) - n + tok0;          // position of the first token
    s.kend = max(0, s.pos0 + s.toks);        // keys that the last token sees
    s.two = s.toks > prm.Tm;
    const int all = (s.kend + kKT - 1) / kKT;
    const int64_t o0 = x - u, o1 = x_end - u;
    s.kt0 = (int)(all * o0 / c);
    s.nt = (o1 >= c ? all : (int)(all * o1 / c)) - s.kt0;
    s.whole = s.nt == all && o0 == 0;
    if (s.kt0 == 0 && s.nt == all && all > 0) s.whole = true;  // (the cut fell before the first tile)
    s.slot = o0 > 0 ? 0 : 1;
    return s.nt > 0 || (all == 0 && o0 == 0);
  }
  __device__ void next(const PrefillParams& prm) {
    x = min(unit() + cost(), x_end);
    if (x >= x_end || ++p < np) return;
    p = 0;
    if (++g < prm.rq.Hkv) return;
    g = 0;
    pre += prm.rq.Hkv * before(np);
    do {
      ++r;
      request(prm);
    } while (n == 0 && r < prm.rq.B);
    if (n == 0) x = x_end;  // (lengths that changed under the kernel)
  }
};

// A key tile of the CTA's sequence, for the converting warps.
struct Tile {
  int left;  // rows that some query row sees (INT32_MIN: past the last tile)
  int all;   // rows that every query row sees
  int key0;  // its first key
  int sl;    // its segment's slot
  int full;  // all of its rows are seen, and all in the pool
  int odd;   // some are in a block outside the pool, or of V scale zero or negative
};

// Of a 16-key group.
struct alignas(16) Scales {
  float k, vlog;  // K scale, log2 of the V scale
  float vinv;     // the V scale's inverse (infinite: a scale that counts as zero)
  uint32_t tile;  // of the tile: in its first group 1 or 2 where a V scale is outside
};                // 2^+-kPlain (2: above), in the others the largest magnitude of a K scale

template <int D>
struct PMisc {
  static constexpr int kSlots = PCfg<D>::kSlots;
  uint64_t kready[2], kfree[2], vready[2], vfree[2], sfull[2], pfull[2], gready[2], gfree[2], qready, drain;
  uint32_t tmem;
  float qpart[8];  // the largest bound on a row's scores by a key of scale 1, by warp
  int bad[kSlots], any_nan[kSlots];  // by segment (modulo kSlots), as nankey
  int64_t warp_sum[kThreads / 32], start_pre, total;
  int start_r;
  PSeg seg[2];  // the softmax warps' segments
  int any_seg[2];  // 0: there is no further one
  // by tile (modulo kRing) and 16-key group: scales; the K rows' place in the pool, counted
  // in groups (32 bits: 2 TB or more; -1: no key that is seen, -2: a block outside the pool)
  Scales scales[kRing][8];
  int at[kRing][8];
  Tile tile[kRing];
  // First key past the first row's whose V is NaN, by element.  Values of a segment's tile are
  // written when the softmax of NV tiles before is done, so at most NV segments ahead of it;
  // a segment's start clears the slot of the NV-th after it.
  int nankey[kSlots][D];
};

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
// Two floats as f16 pairs: rounded, and what that leaves.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = to_f16x2(a, b);
  const float2 f = f16x2_to_float2(hi);
  lo = to_f16x2(a - f.x, b - f.y);
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 16 bytes from global memory where `ok`, else zeros (no branch: the loads of a pass
// go out together).
__device__ __forceinline__ uint4 ldg16_if(const void* p, bool ok) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@q ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)ok));
  return v;
}

__device__ __forceinline__ int64_t cut(int64_t total, int w, int W) {
  return total / W * w + min((int64_t)w, total % W);
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
  const int G = rq.G, Tm = prm.Tm, W = gridDim.x, me = blockIdx.x;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
      mbar_init(&ms.gready[s], 1);
      mbar_init(&ms.gfree[s], 1);
    }
    mbar_init(&ms.qready, 256);
    mbar_init(&ms.drain, 1);
    fence_mbar_init();
    for (int s = 0; s < C::kSlots; ++s) ms.bad[s] = ms.any_nan[s] = 0;
  }
  for (int i = tid; i < C::kSlots * D; i += kThreads) ms.nankey[i / D][i % D] = INT32_MAX;
  tc::fence_before_sync();
  // ---- this CTA's run of the sequence (the scan's barriers publish the above too)
  bool odd = false;
  scan_requests<kThreads>(
      rq.B,
      [&](int r) {
        PWalk k;
        const int n = rq.tokens(r, &odd);
        if (n < prm.min_new) return (int64_t)0;
        const int kv = rq.length(r);
        odd |= kv < 0;
        k.base = max(max(kv, 0) - n, 0);
        k.w = 2 * Tm;
        return rq.Hkv * k.before((n + k.w - 1) / k.w);
      },
      ms.warp_sum, &ms.start_r, &ms.start_pre, &ms.total, [&](int64_t all) { return cut(all, me, W); });
  if (me == 0 && odd) report(prm.status, GIST_ATTN_STATUS_BAD_BLOCK);
  tc::fence_after_sync();
  const uint32_t tmem = ms.tmem;
  const int64_t total = ms.total, x0 = cut(total, me, W), x1 = cut(total, me + 1, W);
  if (x0 >= x1 || ms.start_r < 0) {
    if (tid == 0) prm.join[me].cost = 0;
    if (warp == 12) tc::tmem_dealloc(tmem, 512);
    return;
  }
  PWalk wk;
  wk.init(prm, x0, x1, ms.start_r, ms.start_pre);
  if (tid == 0) {
    JoinRun j{};
    if (x0 > wk.unit() && cut(total, me - 1, W) <= wk.unit()) {
      PSeg s;
      wk.get(prm, s);
      j = JoinRun{wk.unit(), total / W, total % W, wk.cost(), (s.kend + kKT - 1) / kKT, s.q0, s.toks, s.pos0, s.g, {}};
    }
    prm.join[me] = j;
  }
  bool failed = false;

  if (warp == 12) {
    // ================================================== tcgen05
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (failed || __any_sync(0xffffffffu, !mbar_wait(bar, parity))) failed = true;
      tc::fence_after_sync();
      return !failed;
    };
    // S of row tile x and the CTA's i-th key tile; q's low parts where scores may be large
    auto issue_s = [&](int x, int i, float bound) {
      const bool low = bound * __uint_as_float(ms.scales[i & (kRing - 1)][1].tile) > kFine;
      if (tc::elect_one()) {
        const uint32_t qb = sbase + x * C::kTile, kb = sbase + C::offK + (i & 1) * C::kTile;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(tmem + C::kS + x * 128, tc::smem_desc_sw128(qb + (k / 4) * C::kPanel + (k % 4) * 32, 16, 1024),
                     tc::smem_desc_sw128(kb + (k / 4) * C::kPanel + (k % 4) * 32, 16, 1024),
                     tc::idesc_f16_f32(128, 128, 0), k > 0);
        if (low) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_ss(tmem + C::kS + x * 128,
                       tc::smem_desc_sw128(qb + C::offL + (k / 4) * C::kPanel + (k % 4) * 32, 16, 1024),
                       tc::smem_desc_sw128(kb + (k / 4) * C::kPanel + (k % 4) * 32, 16, 1024),
                       tc::idesc_f16_f32(128, 128, 0), 1);
        }
        tc::commit(smem_u32(&ms.sfull[x]));
      }
      __syncwarp();
    };
    auto issue_pv = [&](int x, int i, bool first) {
      if (tc::elect_one()) {
        const uint32_t vb = sbase + C::offV + i % C::NV * C::kTile;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc::mma_ts(tmem + C::kO + x * D, tmem + C::kS + x * 128 + k * 8,
                     tc::smem_desc_sw128(vb + k * 2048, C::kPanel, 1024), tc::idesc_f16_f32(128, D, 1), !first || k > 0);
      }
      __syncwarp();
    };
    auto arrive = [&](uint64_t* bar) {
      if (tc::elect_one()) tc::commit(smem_u32(bar));
      __syncwarp();
    };
    int i0 = 0, seg = 0;       // tiles and segments so far
    uint32_t np0 = 0, np1 = 0;  // P tiles so far of each row tile
    for (; wk.more() && !failed; wk.next(prm)) {
      PSeg sg;
      if (!wk.get(prm, sg) || sg.nt == 0) continue;  // (without tiles there is no q either)
      if (!wait(&ms.qready, (uint32_t)seg++ & 1u)) break;
      float qnorm[2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        qnorm[x] = fmaxf(fmaxf(ms.qpart[4 * x], ms.qpart[4 * x + 1]), fmaxf(ms.qpart[4 * x + 2], ms.qpart[4 * x + 3]));
      if (!wait(&ms.kready[i0 & 1], (uint32_t)(i0 >> 1) & 1u)) continue;
      const bool two = sg.two;
      issue_s(0, i0, qnorm[0]);
      if (two) issue_s(1, i0, qnorm[1]);
      arrive(&ms.kfree[i0 & 1]);
      for (int e = 0; e < sg.nt; ++e) {
        const int i = i0 + e;
        const bool more = e + 1 < sg.nt;
        auto free_v = [&]() {
          arrive(&ms.vfree[i % C::NV]);
          if ((i & 3) == 3) arrive(&ms.gfree[(i >> 2) & 1]);  // (the tile's softmax is done too)
        };
        if (!wait(&ms.vready[i % C::NV], (uint32_t)(i / C::NV) & 1u) || !wait(&ms.pfull[0], np0++ & 1u)) break;
        issue_pv(0, i, e == 0);
        if (!two) free_v();
        if (more) {
          if (!wait(&ms.kready[(i + 1) & 1], (uint32_t)((i + 1) >> 1) & 1u)) break;
          issue_s(0, i + 1, qnorm[0]);
          if (!two) arrive(&ms.kfree[(i + 1) & 1]);
        } else {
          arrive(&ms.sfull[0]);  // the last P V is done
        }
        if (two) {
          if (!wait(&ms.pfull[1], np1++ & 1u)) break;
          issue_pv(1, i, e == 0);
          free_v();
          if (more) {
            issue_s(1, i + 1, qnorm[1]);
            arrive(&ms.kfree[(i + 1) & 1]);
          } else {
            arrive(&ms.sfull[1]);
          }
        }
      }
      i0 += sg.nt;
    }
    if (tc::elect_one()) tc::commit(smem_u32(&ms.drain));
    __syncwarp();
    if (!mbar_wait(&ms.drain, 0)) failed = true;
  } else if (warp == 13) {
    // ================================================== look-ups, a lane a 16-key group
    // lane group t walks to tiles t, t + 4, ... of the CTA's sequence by itself
    const int t = lane >> 3, gr = lane & 7;
    PSeg sg;
    int e = t, passed = 0;  // the tile within the segment; segments with tiles before
    bool have = false, want = false;
    auto settle = [&]() {  // to the segment that tile e of this or a later one lies in
      while (wk.more()) {
        if (have && e < sg.nt) return;
        if (have) {
          e -= sg.nt;
          passed += sg.nt > 0;
          wk.next(prm);
        }
        have = false;
        while (wk.more() && !(have = wk.get(prm, sg))) wk.next(prm);
      }
      have = false;
    };
    int blk = -1, key = 0, g = 0;
    Tile tl;
    auto look_up = [&]() {
      settle();
      want = false;
      blk = -1;
      tl = Tile{INT32_MIN, 0, 0, 0, 0, 0};
      if (have) {
        const int key0 = (sg.kt0 + e) * kKT;
        key = key0 + gr * 16;
        tl = Tile{sg.kend - key0, sg.pos0 + 1 - key0, key0, passed & (C::kSlots - 1), 0, 0};
        g = sg.g;
        want = key < sg.kend;
        if (want) blk = rq.block_table[(int64_t)sg.r * rq.W + key / rq.block_len];
        e += 4;
      }
    };
    look_up();
    for (int i = 0;; i += 4) {
      const bool last = __any_sync(0xffffffffu, !have);  // this half ends the sequence
      Tile now = tl;
      const int half = (i >> 2) & 1;
      const bool ok = want && blk >= 0 && blk < prm.num_blocks, lost = want && !ok;
      if (lost) report(prm.status, GIST_ATTN_STATUS_BAD_BLOCK);
      const int64_t plane = ((int64_t)(ok ? blk : 0) * prm.L + prm.layer) * 2 * rq.Hkv + g;
      const int at = ok ? (int)((plane * rq.block_len + key % rq.block_len) >> 4) : lost ? -2 : -1;
      const float ks = ok ? prm.scale[plane] : 0.f, vs = ok ? prm.scale[plane + rq.Hkv] : 1.f;
      const float vlog = scale_log2(vs), vinv = fabsf(vs) < kLeastScale ? INFINITY : 1.f / vs;
      if (fabsf(vs) > kMostScale) report(prm.status, GIST_ATTN_STATUS_RANGE);
      auto in_tile = [&](bool p) { return __ballot_sync(0xffffffffu, p) >> (8 * t) & 0xffu; };
      now.full = in_tile(ok) == 0xffu && now.left >= kKT;
      now.odd = in_tile(lost || vs < kLeastScale) != 0;
      const uint32_t above = in_tile(vlog > kPlain), below = in_tile(vlog < -kPlain);
      float kmax = fabsf(ks);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) kmax = fmaxf(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
      const uint32_t of_tile = gr > 0 ? __float_as_uint(kmax) : above ? 2u : below ? 1u : 0u;
      if (!last) look_up();  // its load runs while this half is waited for
      if (__any_sync(0xffffffffu, i >= kRing && !mbar_wait(&ms.gfree[half], ((uint32_t)(i >> 3) & 1u) ^ 1u))) {
        failed = true;
        break;
      }
      const int slot = (i + t) & (kRing - 1);
      ms.scales[slot][gr] = Scales{ks, vlog, vinv, of_tile};
      ms.at[slot][gr] = at;
      if (gr == 0) ms.tile[slot] = now;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.gready[half]);
      if (last) break;
    }
  } else if (warp == 14) {
    // ================================================== the softmax warps' segments
    for (int now = 0;; now ^= 1) {
      bool any = false;
      if (lane == 0) {
        PSeg s;
        while (wk.more() && !any) {
          any = wk.get(prm, s);
          wk.next(prm);
        }
        if (any) ms.seg[now] = s;
        ms.any_seg[now] = any;
      }
      named_bar_sync(3, 288);  // nothing of the segment before is still read
      if (!__shfl_sync(0xffffffffu, any, 0)) break;
    }
  } else if (warp >= 8) {
    // ================================================== cached rows into f16 tiles
    constexpr int kLanes = D / 16;             // threads of a row (16 bytes each)
    constexpr int kRows = 128 / kLanes;        // rows of a pass
    constexpr int kPass = 128 / kRows;
    const int ct = tid - 256, c = ct % kLanes, row0 = ct / kLanes;
    const int64_t vstep = (int64_t)rq.Hkv * rq.block_len * D;
    uint4 kx[kPass], vx[kPass];
    auto fetch = [&](int i, uint4 (&x)[kPass], int64_t more) {
      const int left = ms.tile[i & (kRing - 1)].left;  // rows of the tile that are seen
      const uint8_t* src = prm.pool + (row0 & 15) * D + c * 16 + more;
      if (ms.tile[i & (kRing - 1)].full) {
#pragma unroll
        for (int p = 0; p < kPass; ++p) x[p] = ldg16(src + (int64_t)ms.at[i & (kRing - 1)][(p * kRows + row0) >> 4] * (16 * D));
        return;
      }
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        const int row = p * kRows + row0;
        const int at = ms.at[i & (kRing - 1)][row >> 4];
        x[p] = ldg16_if(src + (int64_t)at * (16 * D), at >= 0 && row < left);
      }
    };
    auto looked_up = [&](int i) {
      if ((i & 3) == 0 && !mbar_wait(&ms.gready[(i >> 2) & 1], (uint32_t)(i >> 3) & 1u)) failed = true;
      return !failed;
    };
    // 16 elements as two 16-byte chunks of f16 of tile row `row`; the second half of a
    // row's threads stores its chunks in the other order (bank conflicts)
    auto put = [&](uint32_t tile, int row, const uint32_t (&h)[8]) {
      const uint32_t base = tile + (c / 4) * C::kPanel;
      const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
      const int odd = (c >> 2) & 1, ch = 2 * (c % 4);
      sts16(base + swz128(row, ch + odd), odd ? hi : lo);
      sts16(base + swz128(row, ch + 1 - odd), odd ? lo : hi);
    };
    // address of f16 element k % 16 of this thread's row of pass k / 16
    auto element = [&](uint32_t tile, int k) {
      return tile + (c / 4) * C::kPanel + swz128((k >> 4) * kRows + row0, 2 * (c % 4) + ((k >> 3) & 1)) + (k & 7) * 2;
    };
    // Keys go a tile ahead of values: those have one buffer (two if D = 64), free only when
    // the tile before is done.
    auto keys = [&](int i) {  // tile i's into their buffer, the next one's from memory
      const int b = i & 1;
      if (i >= 2 && !mbar_wait(&ms.kfree[b], ((uint32_t)(i >> 1) & 1u) ^ 1u)) {
        failed = true;
        return;
      }
      const uint32_t ktile = sbase + C::offK + b * C::kTile;
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        const uint32_t w[4] = {kx[p].x, kx[p].y, kx[p].z, kx[p].w};
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[2 * e] = e4m3x2_to_f16x2((uint16_t)w[e]);
          h[2 * e + 1] = e4m3x2_to_f16x2((uint16_t)(w[e] >> 16));
        }
        put(ktile, p * kRows + row0, h);
      }
      fence_proxy_async_smem();
      mbar_arrive(&ms.kready[b]);
      if (looked_up(i + 1)) fetch(i + 1, kx, 0);
    };
    auto past = [&](int i) { return ms.tile[i & (kRing - 1)].left == INT32_MIN; };
    if (looked_up(0)) {
      fetch(0, kx, 0);
      fetch(0, vx, vstep);
      if (!past(0)) keys(0);
    }
#pragma unroll 1
    for (int i = 0; !failed && !past(i); ++i) {
      if (!past(i + 1)) keys(i + 1);
      if (failed) break;
      const Tile& tl = ms.tile[i & (kRing - 1)];
      const int sl = tl.sl;
      const uint32_t vtile = sbase + C::offV + i % C::NV * C::kTile;
      if (i >= C::NV && !mbar_wait(&ms.vfree[i % C::NV], ((uint32_t)(i / C::NV) & 1u) ^ 1u)) {
        failed = true;
        break;
      }
      if (tl.odd) {
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
          const int gr = (p * kRows + row0) >> 4;
          if (ms.at[i & (kRing - 1)][gr] == -2) ms.bad[sl] = 1;
          const float inv = ms.scales[i & (kRing - 1)][gr].vinv;
          auto turn = [&](uint32_t w) {  // the scale's sign; zeros but for NaN
            const uint32_t nan = e4m3_nan(w);
            return isinf(inv) ? nan - (nan >> 7) : signbit(inv) ? w ^ 0x80808080u : w;
          };
          vx[p] = make_uint4(turn(vx[p].x), turn(vx[p].y), turn(vx[p].z), turn(vx[p].w));
        }
      }
      // keys that not every row sees: a NaN would reach the others (0 x NaN)
      const int all = tl.all;
      bool nan = false;
      if (all < kKT) {
#pragma unroll
        for (int p = 0; p < kPass; ++p)
          nan |= p * kRows + row0 >= all && (e4m3_nan(vx[p].x) | e4m3_nan(vx[p].y) | e4m3_nan(vx[p].z) | e4m3_nan(vx[p].w));
      }
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        const uint32_t w[4] = {vx[p].x, vx[p].y, vx[p].z, vx[p].w};
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[2 * e] = e4m3x2_to_f16x2((uint16_t)w[e]);
          h[2 * e + 1] = e4m3x2_to_f16x2((uint16_t)(w[e] >> 16));
        }
        put(vtile, p * kRows + row0, h);
      }
      if (nan) {  // noted for the rows that see it, and cleared
        ms.any_nan[sl] = 1;
#pragma unroll 1
        for (int k = 0; k < kPass * 16; ++k) {
          const int row = (k >> 4) * kRows + row0, e = k & 15;
          const uint32_t a = element(vtile, k);
          if (row >= all && (lds_u16(a) & 0x7fffu) > 0x7c00u) {
            sts_u16(a, 0);
            atomicMin(&ms.nankey[sl][c * 16 + e], tl.key0 + row);
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&ms.vready[i % C::NV]);
      if (!failed) fetch(i + 1, vx, vstep);
    }
  } else {
    // ================================================== q rows, softmax, output
    const int x = warp >> 2, row = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + C::kS + x * 128, to = tmem + lane_base + C::kO + x * D;
    auto token_of = [&](int r) { return (int)((uint32_t)r * prm.per_g >> 16); };
    const int tok = x * Tm + token_of(row);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!failed && !mbar_wait(bar, parity)) failed = true;
    };
    int seg = 0, i0 = 0;
    uint32_t ns = 0;  // S tiles (and last P V's) so far of this row tile
    // The slots of `seg` count the segments with key tiles.
    for (int now = 0;; now ^= 1) {
      named_bar_sync(3, 288);  // the segment is there (nothing of the one before it is still read)
      if (!ms.any_seg[now]) break;
      const PSeg& sg = ms.seg[now];
      const int sl = seg & (C::kSlots - 1), nt = sg.nt, kt0 = sg.kt0;
      const bool valid = row < Tm * G && tok < sg.toks;
      const int lim = valid ? sg.pos0 + tok + 1 : 0;      // keys the row sees
      const int lim_all = sg.pos0 + x * Tm + 1;           // keys every row of the tile sees
      if (nt > 0) {
        const int ahead = (sl + C::NV) & (C::kSlots - 1);
        if (tid < D) ms.nankey[ahead][tid] = INT32_MAX;
        if (tid == 0) ms.any_nan[ahead] = ms.bad[ahead] = 0;
      }
      // rows of q and out, a warp its own 32, D / 8 lanes a row
      constexpr int RW = 256 / D;  // rows of a step
      const int rr0 = (row & ~31) + lane / (D / 8), rr1 = (row & ~31) + 32, rch = lane % (D / 8);
      const int toks = sg.toks;
      const int64_t at0 = ((int64_t)(sg.q0 + x * Tm) * prm.Hq + sg.g * G) * D + rch * 8;
      auto row_ok = [&](int rr) { return rr < Tm * G && x * Tm + token_of(rr) < toks; };
      auto at_row = [&](int rr) {
        const int in = token_of(rr);
        return at0 + ((int64_t)in * (prm.Hq - G) + rr) * D;
      };
      float rs = 0.f;  // softmax scale (log2) x the row's power of two
      if (nt > 0) {
        // rows into their places, rounded to f16 there after the rotation
        const uint32_t tile = sbase + x * C::kTile;
        auto place = [&](int r, int ch) { return tile + (ch >> 3) * C::kPanel + swz128(r, ch & 7); };
#pragma unroll 1
        for (int rr = rr0; rr < rr1; rr += RW) {
          if (row_ok(rr)) cp_async16(place(rr, rch), prm.q + at_row(rr));
          else sts16(place(rr, rch), make_uint4(0, 0, 0, 0));
        }
        cp_async_wait_all();
        __syncwarp();
        // the largest magnitude bounds the rotated ones by sqrt 2, which the power of two
        // leaves room for
        uint32_t big = 0;
#pragma unroll 4
        for (int ch = 0; ch < D / 8; ++ch) {
          const uint4 v = lds16(place(row, ch));
          big = __vmaxu2(big, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
        const uint32_t tb = max(big & 0xffffu, big >> 16) << 16;
        const int ex = min(max((int)(tb >> 23) - 127, -119), 126);
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);  // largest to [1, 2)
        rs = tb >= 0x7f800000u ? __int_as_float(0x7fc00000)
                               : prm.scale_log2 * __uint_as_float((uint32_t)(ex + 127) << 23);
        const int pos = max(sg.pos0 + tok, 0);
        const uint64_t down2 = f2_make(down, down);
        uint64_t squares = f2_make(0.f, 0.f);
#pragma unroll 1
        for (int ch = 0; ch < D / 16; ++ch) {  // 8 pairs: elements 8 ch .. and D/2 + 8 ch ..
          const uint32_t pa = place(row, ch), pb = place(row, ch + D / 16);
          const uint4 va = lds16(pa), vb = lds16(pb);
          const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
          uint32_t a[4], b[4], al[4], bl[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float s0, c0, s1, c1;
            __sincosf(turn_angle(pos, prm.turn[ch * 8 + 2 * e]), &s0, &c0);
            __sincosf(turn_angle(pos, prm.turn[ch * 8 + 2 * e + 1]), &s1, &c1);
            const uint64_t u = f2_mul(bf16x2_to_f2(wa[e]), down2), y = f2_mul(bf16x2_to_f2(wb[e]), down2);
            squares = f2_fma(u, u, f2_fma(y, y, squares));
            const uint64_t cs = f2_make(c0, c1), sn = f2_make(s0, s1);
            float r0, r1;
            f2_split(f2_sub(f2_mul(u, cs), f2_mul(y, sn)), r0, r1);
            split2(r0, r1, a[e], al[e]);
            f2_split(f2_fma(y, cs, f2_mul(u, sn)), r0, r1);
            split2(r0, r1, b[e], bl[e]);
          }
          sts16(pa + C::offL, make_uint4(al[0], al[1], al[2], al[3]));
          sts16(pb + C::offL, make_uint4(bl[0], bl[1], bl[2], bl[3]));
          sts16(pa, make_uint4(a[0], a[1], a[2], a[3]));
          sts16(pb, make_uint4(b[0], b[1], b[2], b[3]));
        }
        float sq0, sq1;
        f2_split(squares, sq0, sq1);
        float bound = sqrtf(sq0 + sq1) * rs * prm.largest;
#pragma unroll
        for (int o = 16; o; o >>= 1) bound = fmaxf(bound, __shfl_xor_sync(0xffffffffu, bound, o));
        if (lane == 0) ms.qpart[warp] = bound;
        fence_proxy_async_smem();
        mbar_arrive(&ms.qready);
      }
      float m = kNone;
      bool far = false;  // some V scale of the segment is above 2^kPlain
      uint64_t acc = f2_make(0.f, 0.f);
      const bool live = x == 0 || sg.two;
      for (int e = 0; live && e < nt; ++e) {
        const int i = i0 + e, key0 = (kt0 + e) * kKT;
        const bool edge = key0 + kKT > lim_all;
        wait(&ms.sfull[x], ns++ & 1u);
        tc::fence_after_sync();
        const Scales* scales = ms.scales[i & (kRing - 1)];
        const uint32_t sca = smem_u32(scales);
        uint4 s0 = lds16(sca), s1;
        far |= s0.w == 2u;  // (the maximum is above all sums from here on)
        const bool own = far || s0.w != 0;
        // 16 scores v of a group with scales sw as weights exp2(f v + log2 scale - m), packed;
        // their sum without the scale into acc; returns their largest exponent
        auto weights = [&](auto own_sum, uint4 sw, const uint32_t (&v)[16], uint32_t* pk, int left) {
          const bool seen = left > 0;  // (a scale that the row does not see may be NaN)
          const float f = __uint_as_float(sw.x) * rs, lg = seen ? __uint_as_float(sw.y) : 0.f;
          const float w = decltype(own_sum)::value ? 1.f : seen ? fabsf(__uint_as_float(sw.z)) : 0.f;
          const uint64_t g2 = f2_make(f, f), nm2 = f2_make(lg - m, lg - m);
          uint64_t sum = 0;
          float top = kNone;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float a, b;
            f2_split(f2_fma(f2_make(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), g2, nm2), a, b);
            if (2 * k >= left) a = -INFINITY;
            if (2 * k + 1 >= left) b = -INFINITY;
            top = max3f(top, a, b);
            const float pa = ex2_approx(a), pb = ex2_approx(b);
            const uint64_t p = decltype(own_sum)::value ? f2_make(ex2_approx(a - lg), ex2_approx(b - lg)) : f2_make(pa, pb);
            sum = k == 0 ? p : f2_add(sum, p);
            pk[k] = to_f16x2(pa, pb);
          }
          acc = f2_fma(sum, f2_make(w, w), acc);
          return top;
        };
        // One pass with the maximum as it is; P stays in registers until it is known that
        // no row's scores passed it by too much.
        bool done = false;
        if (!edge && e > 0) {
          const uint64_t keep = acc;
          uint32_t va[16], vb[16], pk[64];
          float top = kNone;
          tc::ld16(ts, va);
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            tc::ld16(ts + c * 16 + 16, vb);
            s1 = lds16(sca + c * 16 + 16);
            top = fmaxf(top, weights(std::false_type{}, s0, va, pk + c * 8, 16));
            tc::wait_ld();
            if (c + 2 < 8) {
              tc::ld16(ts + c * 16 + 32, va);
              s0 = lds16(sca + c * 16 + 32);
            }
            top = fmaxf(top, weights(std::false_type{}, s1, vb, pk + c * 8 + 8, 16));
            tc::wait_ld();
          }
          done = !__any_sync(0xffffffffu, top > kSlack || own);
          if (done) {
#pragma unroll
            for (int c = 0; c < 4; ++c) st16(ts + c * 16, *reinterpret_cast<const uint32_t(*)[16]>(pk + c * 16));
          } else {
            acc = keep;
          }
        }
        if (!done) {
          // the tile's maximum first.  A row whose maximum jumps scales its O and sum down;
          // the TMEM load and store are warp-collective, so the warp does it for any of its
          // rows
          float mx = kNone;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t v[16];
            tc::ld16(ts + c * 16, v);
            tc::wait_ld();
            const int left = edge ? lim - key0 - c * 16 : 16;  // columns of these that the row sees
            const float f = scales[c].k * rs;
            float t = -INFINITY;
#pragma unroll
            for (int k = 0; k < 16; ++k) t = fmaxf(t, k < left ? __uint_as_float(v[k]) * f : -INFINITY);
            mx = fmaxf(mx, t + scales[c].vlog);
          }
          const bool move = mx - m > kSlack;
          if (__any_sync(0xffffffffu, move)) {
            // (in two steps: where the maximum moves by V scales the sum may be far from 1)
            const float half = move ? ex2_approx(0.5f * (m - mx)) : 1.f, fm = half * half;
            if (move) m = mx;
            const uint64_t half2 = f2_make(half, half);
            acc = f2_mul(f2_mul(acc, half2), half2);
            if (e > 0) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t ov[16];
                tc::ld16(to + c * 16, ov);
                tc::wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * fm);
                st16(to + c * 16, ov);
              }
            }
          }
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t v[16], pk[8];
            tc::ld16(ts + c * 16, v);
            tc::wait_ld();
            const int left = edge ? lim - key0 - c * 16 : 16;
            s0 = lds16(sca + c * 16);
            if (own) weights(std::true_type{}, s0, v, pk, left);
            else weights(std::false_type{}, s0, v, pk, left);
            tc::st8(ts + c * 8, pk);
          }
        }
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(&ms.pfull[x]);
      }
      if (live) {
        if (nt > 0) wait(&ms.sfull[x], ns++ & 1u);
        tc::fence_after_sync();
        float a0, a1;
        f2_split(acc, a0, a1);
        const float sum = a0 + a1;
        const bool bad = nt > 0 && ms.bad[sl], none = lim <= 0 || bad, whole = sg.whole, nan = nt > 0 && ms.any_nan[sl];
        if (valid && whole && !none && !(sum <= 3.0e38f)) report(prm.status, GIST_ATTN_STATUS_RANGE);
        const float inv = whole ? 1.f / sum : 1.f;
        float* part = prm.parts + (int64_t)(2 * me + sg.slot) * 256 * (D + 2);  // [256][D], then maxima, sums
        // through the row's place in q's room, so that a warp stores whole rows: all columns
        // as bf16, or one half after the other as fp32
        const uint32_t tile = sbase + x * C::kTile;
        auto place = [&](int r, int ch) { return tile + (ch >> 3) * C::kPanel + swz128(r, ch & 7); };
#pragma unroll 1
        for (int half = 0; half < (whole ? 1 : 2); ++half) {
#pragma unroll 1
          for (int c = 0; c < (whole ? D / 16 : D / 32); ++c) {
            const int col = half * (D / 2) + c * 16;
            float o[16];
            uint32_t ov[16];
            tc::ld16(to + col, ov);  // (without a tile: whatever is there, not used)
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = none || nt == 0 ? 0.f : __uint_as_float(ov[e]) * inv;
            if (nan && !none) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (ms.nankey[sl][col + e] < lim) o[e] = __int_as_float(0x7fc00000);
            }
            if (whole) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = float2_to_bf16x2(o[2 * e], o[2 * e + 1]);
              sts16(place(row, 2 * c), make_uint4(w[0], w[1], w[2], w[3]));
              sts16(place(row, 2 * c + 1), make_uint4(w[4], w[5], w[6], w[7]));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                sts16(place(row, 4 * c + e), make_uint4(__float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
                                                        __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3])));
            }
          }
          __syncwarp();
#pragma unroll 1
          for (int rr = rr0; rr < rr1; rr += RW) {
            const uint4 v = lds16(place(rr, rch));
            if (row_ok(rr)) {
              if (whole) stg16(prm.out + at_row(rr), v);
              else stg16(part + (x * 128 + rr) * D + half * (D / 2) + rch * 4, v);
            }
          }
          __syncwarp();
        }
        if (valid && !whole) {
          part[256 * D + tid] = m;
          part[256 * (D + 1) + tid] = bad ? -1.f : sum;
        }
        tc::fence_before_sync();
      }
      i0 += nt;
      seg += nt > 0;
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

// Adds up the parts of the units that cross CTAs, a warp four rows at a time: O, m and
// sum in key order.  Block y takes 32 rows of the unit that CTA blockIdx.x + 1 left a
// header for.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ PrefillParams prm, int W) {
  constexpr int R = 4, E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = blockIdx.x + 1;
  const int G = prm.rq.G, Tm = prm.Tm, row0 = blockIdx.y * 32 + warp * R, x = row0 >> 7;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinRun u = prm.join[w];
  if (u.cost == 0 || (row0 & 127) >= Tm * G) return;
  float m[R], sum[R], o[R][E];
  bool bad[R];  // (rows past the unit's hold anything: each by itself)
#pragma unroll
  for (int k = 0; k < R; ++k) {
    bad[k] = false;
    m[k] = kNone;
    sum[k] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[k][e] = 0.f;
  }
  auto first = [&](int v) { return u.share * v + min((int64_t)v, u.rest) - u.at; };  // CTA v's, from the unit's
  auto tile = [&](int64_t at) { return at >= u.cost ? u.tiles : (int)(u.tiles * max(at, (int64_t)0) / u.cost); };
  int k0 = 0;
  for (int v = w - 1; v < W && first(v) < u.cost; ++v) {
    const int k1 = tile(first(v + 1));
    if (k0 == 0 && k1 == u.tiles) return;  // one CTA had all of its tiles
    if (k0 < k1) {
      const float* p = prm.parts + (int64_t)(2 * v + (first(v) > 0 ? 0 : 1)) * 256 * (D + 2);
      float pm[R], ps[R], po[R][E];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        pm[k] = p[256 * D + row0 + k];
        ps[k] = p[256 * (D + 1) + row0 + k];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 y = *reinterpret_cast<const float2*>(p + (row0 + k) * D + lane * E + e);
          po[k][e] = y.x;
          po[k][e + 1] = y.y;
        }
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const float top = fmaxf(m[k], pm[k]), h0 = exp2f(0.5f * (m[k] - top)), h1 = exp2f(0.5f * (pm[k] - top));
        const float f0 = h0 * h0, f1 = h1 * h1;
        bad[k] |= ps[k] < 0.f;
        m[k] = top;
        sum[k] = sum[k] * h0 * h0 + ps[k] * h1 * h1;
#pragma unroll
        for (int e = 0; e < E; ++e) o[k][e] = o[k][e] * f0 + f1 * po[k][e];
      }
    }
    k0 = k1;
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int in = (row0 & 127) + k, tok = x * Tm + in / G;
    if (in >= Tm * G || tok >= u.toks) continue;
    const bool none = bad[k] || u.pos0 + tok < 0;
    if (lane == 0 && !none && !(sum[k] <= 3.0e38f)) report(prm.status, GIST_ATTN_STATUS_RANGE);
    const float inv = 1.f / sum[k];
    bf16* dst = prm.out + ((int64_t)(u.q0 + tok) * prm.Hq + u.g * G + in % G) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = none ? 0u : float2_to_bf16x2(o[k][e] * inv, o[k][e + 1] * inv);
  }
}

// CTAs: one an SM, fewer where the token rows and the table cannot hold that many key
// tiles (every request with min_new tokens or more may end in a pair that is not full).
int grid_of(const PagedProblem& pb, int min_new, int sms) {
  const int Tm = 128 / pb.G;
  const int64_t requests = pb.T / min_new < pb.B ? pb.T / min_new : pb.B;
  const double pairs = (double)pb.T / (2 * Tm) + requests;
  const double tiles = requests == 0 ? 0 : pairs * pb.Hkv * ((double)((int64_t)pb.W * pb.block_len + kKT - 1) / kKT);
  return tiles < sms ? (int)tiles : sms;
}

template <int D>
int launch(const PagedProblem& pb, void* workspace, int min_new, int sms, cudaStream_t stream) {
  const int grid = grid_of(pb, min_new, sms);
  if (grid == 0) return GIST_ATTN_OK;
  PrefillParams prm{};
  prm.q = static_cast<const bf16*>(pb.q);
  prm.out = static_cast<bf16*>(pb.out);
  prm.pool = pb.pool;
  prm.scale = pb.scale;
  prm.join = static_cast<JoinRun*>(workspace);
  prm.parts = reinterpret_cast<float*>(prm.join + grid);
  prm.status = pb.status;
  prm.rq = requests_of(pb);
  prm.Hq = pb.Hq;
  prm.L = pb.L;
  prm.layer = pb.layer;
  prm.num_blocks = pb.num_blocks;
  prm.min_new = min_new;
  prm.Tm = 128 / pb.G;
  prm.scale_log2 = pb.scale_log2;
  prm.per_g = (65536u + pb.G - 1) / pb.G;
  prm.largest = pb.flags & GIST_ATTN_FLAG_PREROTATED ? 0.f : 448.f * sqrtf((float)D);  // (bf16 fits f16)
  for (int j = 0; j < 64; ++j) prm.turn[j] = pb.turn[j];
  constexpr int smem = (int)(PCfg<D>::offMisc + sizeof(PMisc<D>));
  static_assert(smem <= 227 * 1024, "shared memory");
  if (cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  prefill_kernel<D><<<grid, kThreads, smem, stream>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return GIST_ATTN_ERR_LAUNCH;
  if (grid == 1) return GIST_ATTN_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid - 1, 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, prm, grid) == cudaSuccess ? GIST_ATTN_OK : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace

size_t paged_prefill_workspace(const PagedProblem& pb, int min_new, int sms) {
  return (size_t)grid_of(pb, min_new, sms) * (sizeof(JoinRun) + 2 * 256 * (pb.d + 2) * sizeof(float));
}

int launch_paged_prefill(const PagedProblem& pb, void* workspace, int min_new, int sms, cudaStream_t stream) {
  return pb.d == 64 ? launch<64>(pb, workspace, min_new, sms, stream) : launch<128>(pb, workspace, min_new, sms, stream);
}

}  // namespace gattn
