// paged_bf16.cu -- one new token a request over a bf16 paged cache, each request with
// a length of its own: the decode step of [KV page, "Reusable-state"] behind the
// block table of [Suffix page, §6 问题四], the cache's axis split over warps and CTAs.
//
//   o[h] = sum_j p_j V_j,  p = softmax_j(scale R(q[h]) . K_j),  j < kv_len
//
// Work: a unit is (request, KV head, up to 16 of its query heads), its keys in
// tiles of 16.  All units' tiles in a row are cut into equal runs, one a CTA, and each run
// into equal runs a warp, so that any mix of lengths keeps every SM busy.  A
// warp streams its tiles through a ring of its own (cp.async, no barrier with other
// warps) and keeps the softmax of the unit that it is in: a maximum m, the sum l of
// 2^(s - m) and O = sum 2^(s - m) V.  Parts of one unit join by
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  O = sum 2^(m_i - m) O_i
// first over the CTA's warps in shared memory, then, for units that cross CTAs, in a second
// kernel; the order of the sums is fixed.
//
// A tile: S^T = K q^T on mma.sync m16n8k16 (the keys are the 16 rows, the heads the N),
// then O^T += V^T P with V^T by ldmatrix.trans and P by movmatrix.  q (rotated in fp32) and P
// are sums of three bf16 terms, which hold all of fp32's bits: products are exact, sums fp32,
// and of the outputs 0.03 % are not the exact value's bf16 (0.1 % where scores pass a hundred); with
// two terms, 17 bits, 0.4 and 0.6 %, and large scores lost their last digits to q's.  The third
// term costs 1.5 % of the time of the 48 requests below, 1-3 % where HBM is the bound, and up to a
// fifth where the products are (128 heads on one KV head: 81 and 99 us).  Up to two heads have the terms side by
// side in the columns of one MMA, up to four in those of two, more take three MMAs.  The
// maximum moves only where a score is more than 8 (log2) above it, so that a tile needs one vote
// in place of a reduction.
//
// Warps an SM: twelve with rings of two tiles of 128-wide heads (192 KB) take the least time of
// 48 requests (123.1 us; 11: 124.0, 10: 124.4; with two terms eight with three tiles took 2 % more than
// twelve, six 8 %), but leave 168 registers a thread, which sixteen heads (255) do not fit.  Heads of
// 64 keep eight with six tiles: twelve cost six short conversations 0.7 us and gain nothing.
//
// Bound: HBM, up to 16 heads a KV head (every K/V byte is read once; at most 32 flops a byte).  48
// requests of 200-9000 keys, 32/8 heads of 128 (757 MB): 122 us, 0.92 of the copy rate; 32/32 heads 124 us,
// 0.94.  What is left there: SMs are not equally near to memory, with equal runs
// some take 1.13 times the mean.  One sequence of 180 k keys, 14/2 heads of 64 (92 MB):
// 26 us, 4.5 of them before the first keys and 5.6 in the two joins.  Six short
// conversations: 9.8 us.  More than 16 heads a KV head are units of 16, each of which reads the keys
// again, from L2 where it can: 16 requests of 4000 keys with 2 KV heads of 128 (66 MB) take 31.5 us with
// 32 heads, 39 with 64 and 58 with 128; 32 of them with one KV head and 128 heads 99 us.
//
// Pages: [KV page] "为什么自回归推理缓存 KV，而不缓存历史 Q？";
//        [Suffix page] icman.com.cn news 64898.
#include <math.h>

#include "common.cuh"
#include "follow.cuh"
#include "frag.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace gattn {
namespace {

constexpr int kKeys = 16;      // of a tile
constexpr int kWindow = 64;    // tiles of a warp's run that are resolved ahead
constexpr float kRise = 8.f;   // a maximum stays until a score is so much above it (log2)
constexpr float kBad = -1.f;   // as a sum: the unit met a bad block id

struct Bf16Params {
  const bf16* q;
  const bf16* pool;
  bf16* out;
  const int32_t* block_table;
  const int32_t* q_start;  // nullptr: request r's token is row r
  const int32_t* kv_len;
  int32_t* status;
  int4* head;    // [CTA] request and unit of its parts 0 and 1 (-1: none)
  float* parts;  // [CTA][2] of a unit that began in an earlier CTA; that begins here and goes on
  float* kept;   // [CTA][warp] of a unit that began in an earlier warp, while the warp goes on
  int B, T, Hq, Hkv, G, chunks, block_len, W, num_blocks, L, layer, least, ctas;
  float scale_log2;
  uint64_t turn[64];

  // Tiles of one unit of request r: 0 if it has no token, one where it sees no key.
  __device__ __forceinline__ int tiles(int r, bool* bad = nullptr) const {
    if (q_start) {
      const int a = q_start[r], b = q_start[r + 1];
      if (a < 0 || b > T || b < a || b - a > 1) {
        if (bad) *bad = true;
        return 0;
      }
      if (b == a) return 0;
    }
    return max(1, (length(r, bad) + kKeys - 1) / kKeys);
  }
  __device__ __forceinline__ int length(int r, bool* bad = nullptr) const {
    const int kv = kv_len[r];
    if (kv > W * block_len) {
      if (bad) *bad = true;
      return 0;
    }
    return max(kv, 0);
  }
  __device__ __forceinline__ int row(int r) const { return q_start ? q_start[r] : r; }
  __device__ __forceinline__ int units() const { return Hkv * chunks; }
};

// One tile of a run: where its keys are (elements into the pool; -1: a bad block id), its
// request, and keys (5 bits), first / last tile of the unit, unit in the request.
struct __align__(16) Tile {
  int64_t at;
  int32_t r;
  uint32_t info;
};
constexpr uint32_t kFirst = 32, kLast = 64;

// Heads a unit: 2, 4, 8 or 16.  q and P are sums of three bf16 terms; a step of 16 dimensions (keys) is one
// MMA with them side by side in the columns (up to two heads), one of two and one of the third (four), or
// three.
template <int H>
struct Terms {
  static constexpr int beside = H == 2 ? 3 : H == 4 ? 2 : 1, mmas = H == 2 ? 1 : H == 4 ? 2 : 3;
};
template <int D, int H>
struct Ring {
  static constexpr bool many = D == 128 && H < 16;
  static constexpr int warps = many ? 12 : 8, threads = warps * 32;
  static constexpr int stages = many ? 2 : D == 128 ? 3 : 6;
  static constexpr uint32_t tile = kKeys * D * 2, stage = 2 * tile;
  static constexpr uint32_t warp = stages * stage;
  static constexpr uint32_t windows = warps * warp;
  static constexpr uint32_t bytes = windows + warps * kWindow * sizeof(Tile);
};
// A part in shared memory or the workspace: O [H][D], m [H], l [H].
template <int D, int H>
constexpr int kPart = H * (D + 2);

// Byte offset of 16-byte chunk c of row r in a tile of rows of 2 D bytes.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return r * (2 * D) + ((c ^ (r & 7)) << 4);
}

// Two elements of head h of a finished unit, from the joined O, l.
template <int D>
__device__ __forceinline__ void write_pair(const Bf16Params& p, int r, int unit, int h, int e, float a, float b, float l) {
  const int g = unit / p.chunks, head = (unit - g * p.chunks) * 16 + h;
  if (head >= p.G) return;
  const bool none = l == kBad || p.length(r) == 0;
  if (e == 0 && !none && !(l > 0.f && l <= 3.0e38f)) report(p.status, GIST_ATTN_STATUS_RANGE);
  const float inv = 1.f / l;
  *reinterpret_cast<uint32_t*>(p.out + ((int64_t)p.row(r) * p.Hq + g * p.G + head) * D + e) =
      none ? 0u : float2_to_bf16x2(a * inv, b * inv);
}
// Two fp32 as sums of three bf16, each the rounded remainder of the ones before: all of their bits.
__device__ __forceinline__ void terms3(uint64_t v, uint32_t (&t)[3]) {
  t[0] = f2_to_bf16x2(v);
  v = f2_sub(v, bf16x2_to_f2(t[0]));
  t[1] = f2_to_bf16x2(v);
  t[2] = f2_to_bf16x2(f2_sub(v, bf16x2_to_f2(t[1])));
}
// The term that the `part`-th part of the columns has in MMA i of a step (none: zeros).
template <int H>
__device__ __forceinline__ uint32_t term_of(const uint32_t (&t)[3], int i, int part) {
  const int beside = Terms<H>::beside;
  if (beside == 1) return t[i];
  if (beside == 2) return i == 0 ? (part == 0 ? t[0] : t[1]) : part == 0 ? t[2] : 0u;
  return part == 0 ? t[0] : part == 1 ? t[1] : part == 2 ? t[2] : 0u;
}
// What a part with maximum m counts for beside a common maximum `top`.
__device__ __forceinline__ float weight(float m, float top) { return m == top ? 1.f : ex2_approx(m - top); }

template <int D, int H>
__global__ void __launch_bounds__(Ring<D, H>::threads, 1) decode_kernel(const __grid_constant__ Bf16Params p) {
  constexpr int NT = H == 16 ? 2 : 1, KS = D / 16, HK = KS / 2, BESIDE = Terms<H>::beside, MMAS = Terms<H>::mmas,
                COLS = H < 8 ? H : 8, SUMS = MMAS == 3 ? 3 : 2 * MMAS;
  using R = Ring<D, H>;
  constexpr int kWarps = R::warps, kThreads = R::threads, S = R::stages, PIECES = D / 8;  // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int warp_sum[kWarps], start_r, start_pre, total;
  __shared__ int4 piece[2 * kWarps];  // the warps' open parts: request, unit, whether it begins and ends there
  __shared__ int4 unit_of[2 * kWarps];  // units of those parts: first part, end, whether another CTA has parts too, slot
  __shared__ int units_here;
  __shared__ int tiles_before[kThreads];  // of the requests ahead of each thread's
  __shared__ float part_weight[2 * kWarps][H], unit_top[2 * kWarps][H], unit_sum[2 * kWarps][H];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  let_follow();
  // the frequencies are read here, while nothing else can be done: each line of them is a miss
  // of the constant cache, and a warp that waits for one issues nothing
  __shared__ uint64_t turn[D / 2];
  if (tid < D / 2) turn[tid] = p.turn[tid];
  wait_before();

  // ---- this CTA's run of tiles, and the request that it begins in
  bool bad = false;
  int lo = 0, hi = 0;
  scan_requests<kThreads>(p.B, [&](int r) { return p.tiles(r, blockIdx.x == 0 ? &bad : nullptr) * p.units(); }, warp_sum,
                          &start_r, &start_pre, &total, [&](int all) {
                            const int per = max((all + (int)gridDim.x - 1) / (int)gridDim.x, p.least);
                            lo = (int)min((int64_t)blockIdx.x * per, (int64_t)all);
                            hi = min(lo + per, all);
                            return lo < hi ? lo : -1;
                          },
                          tiles_before);
  if (bad) report(p.status, GIST_ATTN_STATUS_BAD_BLOCK);
  if (start_r < 0) {
    if (tid == 0) p.head[blockIdx.x] = make_int4(-1, -1, -1, -1);
    return;
  }
  const int share = (hi - lo + kWarps - 1) / kWarps;
  const int w0 = min(lo + warp * share, hi), w1 = min(w0 + share, hi);

  // ---- the run's tiles resolved, 32 at a time, a lane a tile
  Tile* window = reinterpret_cast<Tile*>(smem + R::windows) + warp * kWindow;
  const int per_block = p.block_len / kKeys;
  const int64_t plane = (int64_t)p.block_len * D, v_off = p.Hkv * plane;
  const int per_thread = (p.B + kThreads - 1) / kThreads;
  int walk_r = start_r, walk_pre = start_pre;  // first tile of request walk_r
  auto resolve = [&](int x0) {
    const int x = x0 + lane;
    if (x < w1) {
      int n = p.tiles(walk_r), r = walk_r, pre = walk_pre;
      bool jumped = false;
      while (x >= pre + n * p.units()) {
        pre += n * p.units();
        n = p.tiles(++r);
        // a request without a token: there may be thousands, so on to the thread's requests that hold
        // the tile, 43 of 16384 at most (two requests 16 k slots apart: 34 us, 1740 with a walk over
        // them all)
        if (n == 0 && !jumped) {
          jumped = true;
          int t = 0;
#pragma unroll 1
          for (int step = 256; step; step >>= 1)
            if (t + step < kThreads && tiles_before[t + step] <= x) t += step;
          if (t * per_thread > r) {
            r = t * per_thread;
            pre = tiles_before[t];
            n = p.tiles(r);
          }
        }
      }
      const int unit = (x - pre) / n, j = x - pre - unit * n, len = p.length(r);
      Tile t;
      t.r = r;
      t.at = 0;
      const int keys = min(max(len - j * kKeys, 0), kKeys);
      t.info = keys | (j == 0 ? kFirst : 0) | (j == n - 1 ? kLast : 0) | (uint32_t)unit << 8;
      if (keys > 0) {
        const int b = j / per_block, id = p.block_table[(int64_t)r * p.W + b];
        t.at = id >= 0 && id < p.num_blocks
                   ? (((int64_t)id * p.L + p.layer) * 2 * p.Hkv + unit / p.chunks) * plane + (int64_t)(j - b * per_block) * kKeys * D
                   : -1;
        if (t.at < 0) report(p.status, GIST_ATTN_STATUS_BAD_BLOCK);
      }
      window[(x - w0) % kWindow] = t;
      walk_r = r;
      walk_pre = pre;
    }
    // the last tile's request is the next ones' first
    const int last = min(w1 - x0, 32) - 1;
    walk_r = __shfl_sync(0xffffffffu, walk_r, last);
    walk_pre = __shfl_sync(0xffffffffu, walk_pre, last);
    __syncwarp();
  };
  const uint32_t ring = smem_u32(smem) + warp * R::warp;
  const int c16 = lane % PIECES, r16 = lane / PIECES;
  constexpr int kSpots = 8 / (32 / PIECES);  // copies after which the swizzle repeats: eight rows
  uint32_t spot[kSpots];
#pragma unroll
  for (int i = 0; i < kSpots; ++i) spot[i] = swz<D>(r16 + i * (32 / PIECES), c16);
  auto issue = [&](int x) {
    if (x < w1) {
      if (x > w0 && (x - w0) % 32 == 0) resolve(x);
      const Tile t = window[(x - w0) % kWindow];
      const int keys = t.at < 0 ? 0 : (int)(t.info & 31);
      const uint32_t st = ring + (x - w0) % S * R::stage;
      const bf16* k = p.pool + (t.at < 0 ? 0 : t.at) + c16 * 8;
      if (keys == kKeys) {  // nearly all of them: addresses but for constants
        const bf16* from = k + r16 * D;
#pragma unroll
        for (int i = 0; i < kKeys * PIECES / 32; ++i) {
          const uint32_t to = st + spot[i % kSpots] + i / kSpots * (kSpots * (32 / PIECES) * 2 * D);
          cp_async16(to, from + i * (32 / PIECES) * D);
          cp_async16(to + R::tile, from + i * (32 / PIECES) * D + v_off);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < kKeys * PIECES / 32; ++i) {
          const int r = r16 + i * (32 / PIECES);
          const int bytes = r < keys ? 16 : 0;  // rows that nothing sees are zeros
          const bf16* from = k + (r < keys ? r * D : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(st + swz<D>(r, c16)), "l"(from), "r"(bytes) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(st + R::tile + swz<D>(r, c16)), "l"(from + v_off), "r"(bytes)
                       : "memory");
        }
      }
    }
    cp_async_commit();
  };
  // ---- q of a unit: fetched ahead, then rotated at the token's position, hi and lo
  // (16 bytes a lane: a long sequence has every warp of the GPU read the same few rows at once)
  constexpr int CQ = D / 32;  // 16-byte chunks of a head's row a lane: chunks 4 i + t4
  uint4 raw[NT][CQ];
  auto fetch_q = [&](const Tile& t) {
    const int unit = t.info >> 8, g = unit / p.chunks, h0 = (unit - g * p.chunks) * 16;
    const bf16* rows = p.q + ((int64_t)p.row(t.r) * p.Hq + g * p.G + h0) * D + t4 * 8;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = n * 8 + (g8 & (COLS - 1));
#pragma unroll
      for (int i = 0; i < CQ; ++i)
        raw[n][i] = h0 + col < p.G ? *reinterpret_cast<const uint4*>(rows + col * D + i * 32) : make_uint4(0, 0, 0, 0);
    }
  };
  if (w0 < w1) {  // before the keys, which would be ahead of it in the memory's queues
    resolve(w0);
    fetch_q(window[0]);
  }
  for (int x = w0; x < w0 + S - 1; ++x) issue(x);

  uint32_t qt[NT][MMAS][KS][2];
  float m[NT][2], l[NT][2], o[KS][NT][4];
  auto turn_q = [&](const Tile& t) {
    const int pos = max(p.length(t.r) - 1, 0);
    // the four lanes of a head have four chunks of four words; each wants its word of every chunk
    uint32_t word[NT][KS][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < CQ; ++i) {
        const uint32_t v[4] = {raw[n][i].x, raw[n][i].y, raw[n][i].z, raw[n][i].w};
        uint32_t got[4];  // from lane t4 ^ s: its chunk's word t4
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int w = t4 ^ s;  // the word that the lane asking wants
          const uint32_t lo = w & 1 ? v[1] : v[0], hi = w & 1 ? v[3] : v[2];
          got[s] = __shfl_xor_sync(0xffffffffu, w & 2 ? hi : lo, s);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // chunk 4 i + c came from lane c, in step c ^ t4
          const uint32_t lo = t4 & 1 ? got[c ^ 1] : got[c], hi = t4 & 1 ? got[c ^ 3] : got[c ^ 2];
          word[n][2 * i + c / 2][c & 1] = t4 & 2 ? hi : lo;
        }
      }
#pragma unroll
    for (int ks = 0; ks < HK; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = ks * 16 + e * 8 + t4 * 2;
        uint64_t sn, cs;
        sincos_turns(turn_part(pos, turn[j]), turn_part(pos, turn[j + 1]), sn, cs);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint64_t x = bf16x2_to_f2(word[n][ks][e]), y = bf16x2_to_f2(word[n][ks + HK][e]);
          const uint64_t a = f2_sub(f2_mul(x, cs), f2_mul(y, sn)), b = f2_fma(x, sn, f2_mul(y, cs));
          uint32_t at[3], bt[3];
          terms3(a, at);
          terms3(b, bt);
#pragma unroll
          for (int i = 0; i < MMAS; ++i) {
            qt[n][i][ks][e] = term_of<H>(at, i, g8 / COLS);
            qt[n][i][ks + HK][e] = term_of<H>(bt, i, g8 / COLS);
          }
        }
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int d = 0; d < KS; ++d) o[d][n][0] = o[d][n][1] = o[d][n][2] = o[d][n][3] = 0.f;
    }
  };

  // ---- the tiles
  constexpr int P = kPart<D, H>;
  float* kept = p.kept + ((int64_t)blockIdx.x * kWarps + warp) * P;
  float* left = reinterpret_cast<float*>(smem + warp * R::warp);  // once the ring is done with
  bool wrong = false, begins = false;  // the unit met a bad block id; its first tile is in this run
  if (lane < 2) piece[2 * warp + lane] = make_int4(-1, -1, 0, 0);
  __syncwarp();
  for (int x = w0; x < w1; ++x) {
    issue(x + S - 1);
    cp_async_wait_group<S - 1>();
    __syncwarp();
    const Tile t = window[(x - w0) % kWindow];
    if (x == w0 || (t.info & kFirst)) {
      turn_q(t);
      wrong = false;
      begins = t.info & kFirst;
    }
    if (x + 1 < w1 && (window[(x + 1 - w0) % kWindow].info & kFirst)) fetch_q(window[(x + 1 - w0) % kWindow]);
    wrong |= t.at < 0;
    const int keys = t.info & 31;
    const uint32_t st = ring + (x - w0) % S * R::stage;
    float s[NT][4], sums[NT][SUMS][4] = {};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t a[4];
      ldsm_x4(st + swz<D>(lane & 15, 2 * ks + (lane >> 4)), a);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < MMAS; ++i) mma_16816(sums[n][(i + ks * MMAS) % SUMS], a, qt[n][i][ks][0], qt[n][i][ks][1]);
      }
    }
    bool rise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = sums[n][0][e];
#pragma unroll
        for (int i = 1; i < SUMS; ++i) v += sums[n][i][e];
#pragma unroll
        for (int sh = COLS / 2; sh < 4; sh <<= 1) v += __shfl_xor_sync(0xffffffffu, v, sh);
        v *= p.scale_log2;
        if (g8 + (e >> 1) * 8 >= keys) v = -INFINITY;
        s[n][e] = v;
        rise |= v > m[n][e & 1] + kRise;
      }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = fmaxf(s[n][c], s[n][c + 2]);
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
          top = fmaxf(top, m[n][c]);
          const float f = m[n][c] == top ? 1.f : ex2_approx(m[n][c] - top);
          m[n][c] = top;
          l[n][c] *= f;
#pragma unroll
          for (int d = 0; d < KS; ++d) {
            o[d][n][c] *= f;
            o[d][n][c + 2] *= f;
          }
        }
    }
    uint32_t pt[NT][MMAS][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = ex2_approx(s[n][2 * h] - m0), b = ex2_approx(s[n][2 * h + 1] - m1);
        l[n][0] += a;
        l[n][1] += b;
        uint32_t t3[3];
        terms3(f2_make(a, b), t3);
#pragma unroll
        for (int i = 0; i < MMAS; ++i) pt[n][i][h] = movmatrix_trans(term_of<H>(t3, i, 2 * t4 / COLS));
      }
    }
#pragma unroll
    for (int d = 0; d < KS; ++d) {
      uint32_t a[4];
      // matrices: (keys 0-7, dims 0-7), (keys 0-7, dims 8-15), (keys 8-15, dims 0-7), (8-15, 8-15)
      ldsm_x4_trans(st + R::tile + swz<D>((lane & 7) + ((lane >> 4) << 3), 2 * d + ((lane >> 3) & 1)), a);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < MMAS; ++i) mma_16816(o[d][n], a, pt[n][i][0], pt[n][i][1]);
      }
    }
    __syncwarp();
    const bool ends = t.info & kLast;
    if (!ends && x + 1 < w1) continue;

    // ---- a unit, or this warp's part of one, is done
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], sh);
        if (wrong) l[n][c] = kBad;
#pragma unroll
        for (int sh = COLS / 2; sh < 4; sh <<= 1)
#pragma unroll
          for (int d = 0; d < KS; ++d) {
            o[d][n][c] += __shfl_xor_sync(0xffffffffu, o[d][n][c], sh);
            o[d][n][c + 2] += __shfl_xor_sync(0xffffffffu, o[d][n][c + 2], sh);
          }
      }
    const int unit = t.info >> 8;
    if (begins && ends) {
      // rows of P^T's layout to a head a lane group: pairs of heads, transposed
      const bool none = wrong || p.length(t.r) == 0;
      const int g = unit / p.chunks, h0 = (unit - g * p.chunks) * 16;
      bf16* out = p.out + ((int64_t)p.row(t.r) * p.Hq + g * p.G + h0) * D;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int h = n * 8 + 2 * t4 % COLS + c;
          if (lane < 4 && h0 + h < p.G && !none && !(l[n][c] > 0.f && l[n][c] <= 3.0e38f)) report(p.status, GIST_ATTN_STATUS_RANGE);
        }
        const float i0 = 1.f / l[n][0], i1 = 1.f / l[n][1];
        const bool mine = h0 + n * 8 + g8 < p.G && g8 < H;
#pragma unroll
        for (int d = 0; d < KS; ++d)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t v = movmatrix_trans(float2_to_bf16x2(o[d][n][2 * e] * i0, o[d][n][2 * e + 1] * i1));
            if (mine) *reinterpret_cast<uint32_t*>(out + (n * 8 + g8) * D + d * 16 + e * 8 + t4 * 2) = none ? 0u : v;
          }
      }
      continue;
    }
    const bool last = x + 1 == w1;
    float* to = last ? left : kept;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = n * 8 + t4 * 2 + c;
        if (h >= H) continue;
#pragma unroll
        for (int d = 0; d < KS; ++d) {
          to[h * D + d * 16 + g8] = o[d][n][c];
          to[h * D + d * 16 + 8 + g8] = o[d][n][c + 2];
        }
        if (g8 == 0) {
          to[H * D + h] = m[n][c];
          to[H * D + H + h] = l[n][c];
        }
      }
    if (lane == 0) piece[2 * warp + last] = make_int4(t.r, unit, begins, ends);
  }
  __syncthreads();

  // ---- the warps' parts joined: whole units are written, the others left for the next kernel.
  // First the weights, a warp a head and a lane a part; parts of one unit follow one another.
  constexpr int kParts = 2 * kWarps;
  static_assert(kParts <= 32, "a lane a part");
  auto part = [&](int j) -> const float* {
    return j & 1 ? reinterpret_cast<const float*>(smem + (j >> 1) * R::warp) : p.kept + ((int64_t)blockIdx.x * kWarps + (j >> 1)) * P;
  };
  {
    const int4 id = lane < kParts ? piece[lane] : make_int4(-1, -1, 0, 0);
    const bool valid = id.x >= 0;
    const uint32_t upto = (2u << lane) - 1, valids = __ballot_sync(0xffffffffu, valid);
    const int before = 31 - __clz(valids & (upto >> 1));  // the part before (-1: none)
    const int px = __shfl_sync(0xffffffffu, id.x, max(before, 0)), py = __shfl_sync(0xffffffffu, id.y, max(before, 0));
    const bool first = valid && (before < 0 || px != id.x || py != id.y);
    const uint32_t firsts = __ballot_sync(0xffffffffu, first), later = firsts & ~upto;
    const int begin = 31 - __clz(firsts & upto), end = later ? __ffs(later) - 1 : 32;  // of this lane's unit
    const uint32_t members = valids & (upto | (end == 32 ? 0xffffffffu : (1u << end) - 1)) & (begin < 0 ? 0u : ~((1u << begin) - 1));
    for (int h = warp; h < H; h += kWarps) {
      const float mine = valid ? part(lane)[H * D + h] : -INFINITY, lj = valid ? part(lane)[H * D + H + h] : 0.f;
      float top = mine;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const float v = __shfl_up_sync(0xffffffffu, top, s);
        if (lane - s >= begin && lane >= s) top = fmaxf(top, v);
      }
      top = __shfl_sync(0xffffffffu, top, end - 1);
      const float f = valid ? weight(mine, top) : 0.f;
      float sum = valid ? f * lj : 0.f;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const float v = __shfl_up_sync(0xffffffffu, sum, s);
        if (lane - s >= begin && lane >= s) sum += v;
      }
      sum = __shfl_sync(0xffffffffu, sum, end - 1);
      if (__ballot_sync(0xffffffffu, valid && lj == kBad) & members) sum = kBad;
      if (lane < kParts) part_weight[lane][h] = f;
      if (first) {
        unit_top[lane][h] = top;
        unit_sum[lane][h] = sum;
      }
    }
    if (warp == 0) {
      const int ends = __shfl_sync(0xffffffffu, id.w, 31 - __clz(members | 1u));
      const int slot = id.z ? 1 : 0;
      const bool open = first && !(id.z && ends);
      if (first) unit_of[__popc(firsts & (upto >> 1))] = make_int4(lane, end, open, slot);
      if (lane == 0) units_here = __popc(firsts);
      // at most one unit began before this CTA, and at most one goes on behind it
      int4 head = make_int4(-1, -1, -1, -1);
      const uint32_t s0 = __ballot_sync(0xffffffffu, open && slot == 0), s1 = __ballot_sync(0xffffffffu, open && slot == 1);
      head.x = __shfl_sync(0xffffffffu, id.x, s0 ? __ffs(s0) - 1 : 0);
      head.y = __shfl_sync(0xffffffffu, id.y, s0 ? __ffs(s0) - 1 : 0);
      head.z = __shfl_sync(0xffffffffu, id.x, s1 ? __ffs(s1) - 1 : 0);
      head.w = __shfl_sync(0xffffffffu, id.y, s1 ? __ffs(s1) - 1 : 0);
      if (lane == 0) p.head[blockIdx.x] = make_int4(s0 ? head.x : -1, s0 ? head.y : -1, s1 ? head.z : -1, s1 ? head.w : -1);
    }
  }
  __syncthreads();
  constexpr int QUADS = H * D / 4;  // four elements of a head a thread
  for (int i = tid; i < units_here * QUADS; i += kThreads) {
    const int4 u = unit_of[i / QUADS];
    const int quad = i % QUADS, h = quad / (D / 4), e = quad % (D / 4) * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = u.x; j < min(u.y, kParts); ++j) {
      if (piece[j].x < 0) continue;
      const float f = part_weight[j][h];
      const float4 v = *reinterpret_cast<const float4*>(part(j) + quad * 4);
      a.x += f * v.x;
      a.y += f * v.y;
      a.z += f * v.z;
      a.w += f * v.w;
    }
    const int4 id = piece[u.x];
    if (!u.z) {
      write_pair<D>(p, id.x, id.y, h, e, a.x, a.y, unit_sum[u.x][h]);
      write_pair<D>(p, id.x, id.y, h, e + 2, a.z, a.w, unit_sum[u.x][h]);
      continue;
    }
    float* to = p.parts + ((int64_t)blockIdx.x * 2 + u.w) * P;
    *reinterpret_cast<float4*>(to + quad * 4) = a;
    if (e == 0) {
      to[H * D + h] = unit_top[u.x][h];
      to[H * D + H + h] = unit_sum[u.x][h];
    }
  }
}

// Joins the CTAs' parts of a unit: block c takes the one that begins in CTA c and goes on in the
// next ones.  Four elements of a head a thread; where threads are left, groups of them share out
// the parts, so that many parts are read at once.
constexpr int kJoinThreads = 1024, kMostCtas = 192;
template <int D, int H, int HB>  // HB < H: block (u, i) takes the u-th unit's i-th HB heads
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Bf16Params p) {
  constexpr int P = kPart<D, H>, QUADS = HB * D / 4, GROUPS = kJoinThreads / QUADS, AHEAD = 4;
  __shared__ float4 red[GROUPS > 1 ? kJoinThreads : 1];
  __shared__ float part_top[kMostCtas][HB], part_sum[kMostCtas][HB], unit_sum[HB];
  __shared__ int begins_in;
  const int tid = threadIdx.x, h0 = blockIdx.y * HB, lane = tid & 31, warp = tid >> 5;
  if (HB < H && tid == 0) begins_in = -1;
  if (HB < H) __syncthreads();
  let_follow();
  wait_before();
  const int4 other = tid < p.ctas ? p.head[tid] : make_int4(-1, -1, -1, -1);
  int4 id;
  if (HB < H) {
    id.z = blockIdx.x / p.units();
    id.w = blockIdx.x - id.z * p.units();
    if (other.z == id.z && other.w == id.w) begins_in = tid;
  } else {
    id = p.head[blockIdx.x];
    if (id.z < 0) return;
  }
  // the CTAs that go on with a unit follow one another
  const int parts = 1 + __syncthreads_count(other.x == id.z && other.y == id.w);
  const int c = HB < H ? begins_in : blockIdx.x;
  if (c < 0) return;
  auto part = [&](int j) { return p.parts + ((int64_t)(c + j) * 2 + (j == 0)) * P; };
  const int quad = tid % QUADS, group = tid / QUADS, h = quad / (D / 4), e = quad % (D / 4) * 4;
  float4 v[AHEAD];  // read beside the maxima, whose weights they wait for
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (group + k * GROUPS < parts) v[k] = *reinterpret_cast<const float4*>(part(group + k * GROUPS) + h0 * D + quad * 4);
  for (int i = tid; i < parts * HB; i += kJoinThreads) {
    part_top[i / HB][i % HB] = part(i / HB)[H * D + h0 + i % HB];
    part_sum[i / HB][i % HB] = part(i / HB)[H * D + H + h0 + i % HB];
  }
  __syncthreads();
  if (warp < HB) {  // a warp a head: the maximum, each part's weight, the sum
    float top = -INFINITY, sum = 0.f;
    bool none = false;
    for (int j = lane; j < parts; j += 32) top = fmaxf(top, part_top[j][warp]);
#pragma unroll
    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    for (int j = lane; j < parts; j += 32) {
      const float lj = part_sum[j][warp], f = weight(part_top[j][warp], top);
      none |= lj == kBad;
      sum += f * lj;
      part_top[j][warp] = f;
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    none = __any_sync(0xffffffffu, none);
    if (lane == 0) unit_sum[warp] = none ? kBad : sum;
  }
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = group; j0 < parts; j0 += AHEAD * GROUPS) {
    float4 next[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int j = j0 + (AHEAD + k) * GROUPS;
      if (j < parts) next[k] = *reinterpret_cast<const float4*>(part(j) + h0 * D + quad * 4);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (j0 + k * GROUPS < parts) {
        const float f = part_top[j0 + k * GROUPS][h];
        o.x += f * v[k].x;
        o.y += f * v[k].y;
        o.z += f * v[k].z;
        o.w += f * v[k].w;
      }
      v[k] = next[k];
    }
  }
  if constexpr (GROUPS > 1) {
    red[tid] = o;
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) {
      const float4 v = red[k * QUADS + quad];
      o.x += v.x;
      o.y += v.y;
      o.z += v.z;
      o.w += v.w;
    }
  }
  write_pair<D>(p, id.z, id.w, h0 + h, e, o.x, o.y, unit_sum[h]);
  write_pair<D>(p, id.z, id.w, h0 + h, e + 2, o.z, o.w, unit_sum[h]);
}

int heads_of(const PagedProblem& pb) { return pb.G <= 2 ? 2 : pb.G <= 4 ? 4 : pb.G <= 8 ? 8 : 16; }
size_t part_bytes(const PagedProblem& pb) { return (size_t)heads_of(pb) * (pb.d + 2) * sizeof(float); }

template <int D, int H>
int launch(const PagedProblem& pb, void* workspace, int sms, cudaStream_t stream) {
  const int ctas = sms < kMostCtas ? sms : kMostCtas;
  Bf16Params p{};
  p.q = static_cast<const bf16*>(pb.q);
  p.pool = reinterpret_cast<const bf16*>(pb.pool);
  p.out = static_cast<bf16*>(pb.out);
  p.block_table = pb.block_table;
  p.q_start = pb.q_start;
  p.kv_len = pb.kv_len;
  p.status = pb.status;
  p.head = static_cast<int4*>(workspace);
  p.parts = reinterpret_cast<float*>(p.head + ctas);
  p.kept = p.parts + (size_t)ctas * 2 * kPart<D, H>;
  p.B = pb.B;
  p.T = pb.T;
  p.Hq = pb.Hq;
  p.Hkv = pb.Hkv;
  p.G = pb.G;
  p.chunks = (pb.G + 15) / 16;
  p.block_len = pb.block_len;
  p.W = pb.W;
  p.num_blocks = pb.num_blocks;
  p.L = pb.L;
  p.layer = pb.layer;
  p.least = Ring<D, H>::warps;
  p.ctas = ctas;
  p.scale_log2 = pb.scale_log2;
  for (int j = 0; j < 64; ++j) p.turn[j] = pb.turn[j];
  constexpr int smem = Ring<D, H>::bytes;
  if (cudaFuncSetAttribute(decode_kernel<D, H>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  if (!launch_following(decode_kernel<D, H>, dim3(ctas), dim3(Ring<D, H>::threads), smem, stream, 0, p)) return GIST_ATTN_ERR_LAUNCH;
  // where units are few each has many parts: a block for two of its heads
  const bool few = H > 2 && (int64_t)pb.B * pb.Hkv * p.chunks * 4 < ctas;
  const dim3 grid = few ? dim3(pb.B * pb.Hkv * p.chunks, H / 2) : dim3(ctas);
  return launch_following(few ? join_kernel<D, H, 2> : join_kernel<D, H, H>, grid, dim3(kJoinThreads), 0, stream, 0, p)
             ? GIST_ATTN_OK
             : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace

size_t paged_bf16_workspace(const PagedProblem& pb, int sms) {
  const int warps = pb.d == 64 ? Ring<64, 8>::warps : pb.G <= 8 ? Ring<128, 8>::warps : Ring<128, 16>::warps;
  return (size_t)sms * (sizeof(int4) + (2 + warps) * part_bytes(pb));
}

int launch_paged_bf16(const PagedProblem& pb, void* workspace, int sms, cudaStream_t stream) {
  const int H = heads_of(pb);
  if (pb.d == 64)
    return H == 2   ? launch<64, 2>(pb, workspace, sms, stream)
           : H == 4 ? launch<64, 4>(pb, workspace, sms, stream)
           : H == 8 ? launch<64, 8>(pb, workspace, sms, stream)
                    : launch<64, 16>(pb, workspace, sms, stream);
  return H == 2   ? launch<128, 2>(pb, workspace, sms, stream)
         : H == 4 ? launch<128, 4>(pb, workspace, sms, stream)
         : H == 8 ? launch<128, 8>(pb, workspace, sms, stream)
                  : launch<128, 16>(pb, workspace, sms, stream);
}

}  // namespace gattn
