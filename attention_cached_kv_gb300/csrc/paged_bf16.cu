// paged_bf16.cu -- one new token a request over a bf16 paged cache, each request with
// a length of its own: the decode step of [KV page, "Reusable-state"] behind the
// block table of [Suffix page, §6 问题四], the cache's axis split over warps and CTAs.
//
//   o[h] = sum_j p_j V_j,  p = softmax_j(scale R(q[h]) . K_j),  j < kv_len
//
// Work: a unit is (request, KV head, up to 16 of its query heads), its keys in
// tiles of 16.  All units' tiles in a row are cut into equal runs, one a CTA, and each run
// into equal runs a warp, so that any mix of lengths keeps every SM equally busy.  A
// warp streams its tiles through a ring of its own (cp.async, no barrier with other
// warps) and keeps the softmax of the unit that it is in: a maximum m, the sum l of
// 2^(s - m) and O = sum 2^(s - m) V.  Parts of one unit join by
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  O = sum 2^(m_i - m) O_i
// first over the CTA's warps in shared memory, then, for units that cross CTAs, in a second
// kernel; the order of the sums is fixed.
//
// A tile: S^T = K q^T on mma.sync m16n8k16 (the keys are the 16 rows, the heads the N),
// then O^T += V^T P with V^T by ldmatrix.trans and P by movmatrix.  q (rotated in
// fp32) and P keep 16 bits as bf16 hi + lo; up to four heads take columns 0-3 for hi
// and 4-7 for lo of one MMA, more take two MMAs.  The maximum moves only where a score
// is more than 8 (log2) above it, so that a tile needs one vote in place of a reduction.
//
// Bound: HBM (every K/V byte is read once; at most 32 flops a byte).
//
// Pages: [KV page] "为什么自回归推理缓存 KV，而不缓存历史 Q？";
//        [Suffix page] icman.com.cn news 64898.
#include <math.h>

#include "common.cuh"
#include "frag.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace gattn {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
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
  int B, T, Hq, Hkv, G, chunks, block_len, W, num_blocks, L, layer, least;
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

template <int D>
struct Ring {
  static constexpr int stages = D == 128 ? 3 : 6;
  static constexpr uint32_t tile = kKeys * D * 2, stage = 2 * tile;
  static constexpr uint32_t warp = stages * stage;
  static constexpr uint32_t windows = kWarps * warp;
  static constexpr uint32_t bytes = windows + kWarps * kWindow * sizeof(Tile);
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
// What a part with maximum m counts for beside a common maximum `top`.
__device__ __forceinline__ float weight(float m, float top) { return m == top ? 1.f : ex2_approx(m - top); }

// MODE 0: up to four heads, hi and lo side by side; 1: up to eight; 2: up to sixteen.
template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ Bf16Params p) {
  constexpr int H = MODE == 0 ? 4 : MODE == 1 ? 8 : 16, NT = MODE == 2 ? 2 : 1, KS = D / 16, HK = KS / 2;
  constexpr int S = Ring<D>::stages, PIECES = D / 8;  // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int warp_sum[kWarps], start_r, start_pre, total;
  __shared__ int4 piece[2 * kWarps];  // the warps' open parts: request, unit, whether it begins and ends there
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's run of tiles, and the request that it begins in
  bool bad = false;
  int lo = 0, hi = 0;
  scan_requests<kThreads>(p.B, [&](int r) { return p.tiles(r, blockIdx.x == 0 ? &bad : nullptr) * p.units(); }, warp_sum,
                          &start_r, &start_pre, &total, [&](int all) {
                            const int per = max((all + (int)gridDim.x - 1) / (int)gridDim.x, p.least);
                            lo = (int)min((int64_t)blockIdx.x * per, (int64_t)all);
                            hi = min(lo + per, all);
                            return lo < hi ? lo : -1;
                          });
  if (bad) report(p.status, GIST_ATTN_STATUS_BAD_BLOCK);
  if (start_r < 0) {
    if (tid == 0) p.head[blockIdx.x] = make_int4(-1, -1, -1, -1);
    return;
  }
  const int share = (hi - lo + kWarps - 1) / kWarps;
  const int w0 = min(lo + warp * share, hi), w1 = min(w0 + share, hi);

  // ---- the run's tiles resolved, 32 at a time, a lane a tile
  Tile* window = reinterpret_cast<Tile*>(smem + Ring<D>::windows) + warp * kWindow;
  const int per_block = p.block_len / kKeys;
  const int64_t plane = (int64_t)p.block_len * D, v_off = p.Hkv * plane;
  int walk_r = start_r, walk_pre = start_pre;  // first tile of request walk_r
  auto resolve = [&](int x0) {
    const int x = x0 + lane;
    if (x < w1) {
      int n = p.tiles(walk_r), r = walk_r, pre = walk_pre;
      while (x >= pre + n * p.units()) {
        pre += n * p.units();
        n = p.tiles(++r);
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
  const uint32_t ring = smem_u32(smem) + warp * Ring<D>::warp;
  const int c16 = lane % PIECES, r16 = lane / PIECES;
  auto issue = [&](int x) {
    if (x < w1) {
      if ((x - w0) % 32 == 0) resolve(x);
      const Tile t = window[(x - w0) % kWindow];
      const int keys = t.at < 0 ? 0 : (int)(t.info & 31);
      const uint32_t st = ring + (x - w0) % S * Ring<D>::stage;
      const bf16* k = p.pool + (t.at < 0 ? 0 : t.at) + c16 * 8;
#pragma unroll
      for (int i = 0; i < kKeys * PIECES / 32; ++i) {
        const int r = r16 + i * (32 / PIECES);
        const int bytes = r < keys ? 16 : 0;  // rows that nothing sees are zeros
        const bf16* from = k + (r < keys ? r * D : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(st + swz<D>(r, c16)), "l"(from), "r"(bytes) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(st + Ring<D>::tile + swz<D>(r, c16)), "l"(from + v_off), "r"(bytes)
                     : "memory");
      }
    }
    cp_async_commit();
  };
  for (int x = w0; x < w0 + S - 1; ++x) issue(x);

  uint32_t qh[NT][KS][2], ql[NT][KS][2];
  float m[NT][2], l[NT][2], o[KS][NT][4];
  // ---- q of a unit: rotated at the token's position, hi and lo
  auto load_q = [&](const Tile& t) {
    const int unit = t.info >> 8, g = unit / p.chunks, h0 = (unit - g * p.chunks) * 16;
    const int pos = max(p.length(t.r) - 1, 0);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = MODE == 0 ? g8 & 3 : n * 8 + g8;
      const bool in = h0 + col < p.G;
      const bf16* row = p.q + ((int64_t)p.row(t.r) * p.Hq + g * p.G + (in ? h0 + col : 0)) * D;
#pragma unroll
      for (int ks = 0; ks < HK; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = ks * 16 + e * 8 + t4 * 2;
          uint64_t x = bf16x2_to_f2(*reinterpret_cast<const uint32_t*>(row + j));
          uint64_t y = bf16x2_to_f2(*reinterpret_cast<const uint32_t*>(row + j + D / 2));
          uint64_t sn, cs;
          sincos_turns(turn_part(pos, p.turn[j]), turn_part(pos, p.turn[j + 1]), sn, cs);
          const uint64_t a = f2_sub(f2_mul(x, cs), f2_mul(y, sn)), b = f2_fma(x, sn, f2_mul(y, cs));
          const uint32_t ah = f2_to_bf16x2(a), bh = f2_to_bf16x2(b);
          const uint32_t al = f2_to_bf16x2(f2_sub(a, bf16x2_to_f2(ah))), bl = f2_to_bf16x2(f2_sub(b, bf16x2_to_f2(bh)));
          const bool low = MODE == 0 && g8 >= 4;
          qh[n][ks][e] = !in ? 0u : low ? al : ah;
          qh[n][ks + HK][e] = !in ? 0u : low ? bl : bh;
          ql[n][ks][e] = in ? al : 0u;
          ql[n][ks + HK][e] = in ? bl : 0u;
        }
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int d = 0; d < KS; ++d) o[d][n][0] = o[d][n][1] = o[d][n][2] = o[d][n][3] = 0.f;
    }
  };

  // ---- the tiles
  constexpr int P = kPart<D, H>;
  float* kept = p.kept + ((int64_t)blockIdx.x * kWarps + warp) * P;
  float* left = reinterpret_cast<float*>(smem + warp * Ring<D>::warp);  // once the ring is done with
  bool wrong = false, begins = false;  // the unit met a bad block id; its first tile is in this run
  if (lane < 2) piece[2 * warp + lane] = make_int4(-1, -1, 0, 0);
  __syncwarp();
  for (int x = w0; x < w1; ++x) {
    issue(x + S - 1);
    cp_async_wait_group<S - 1>();
    __syncwarp();
    const Tile t = window[(x - w0) % kWindow];
    if (x == w0 || (t.info & kFirst)) {
      load_q(t);
      wrong = false;
      begins = t.info & kFirst;
    }
    wrong |= t.at < 0;
    const int keys = t.info & 31;
    const uint32_t st = ring + (x - w0) % S * Ring<D>::stage;
    float s[NT][4], s2[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t a[4];
      ldsm_x4(st + swz<D>(lane & 15, 2 * ks + (lane >> 4)), a);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (MODE == 0 && (ks & 1)) {
          mma_16816(s2[n], a, qh[n][ks][0], qh[n][ks][1]);
        } else {
          mma_16816(s[n], a, qh[n][ks][0], qh[n][ks][1]);
          if (MODE != 0) mma_16816(s2[n], a, ql[n][ks][0], ql[n][ks][1]);
        }
      }
    }
    bool rise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = s[n][e] + s2[n][e];
        if (MODE == 0) v += __shfl_xor_sync(0xffffffffu, v, 2);
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
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = ex2_approx(s[n][2 * h] - m0), b = ex2_approx(s[n][2 * h + 1] - m1);
        l[n][0] += a;
        l[n][1] += b;
        const uint32_t hi2 = float2_to_bf16x2(a, b);
        const uint32_t lo2 = f2_to_bf16x2(f2_sub(f2_make(a, b), bf16x2_to_f2(hi2)));
        ph[n][h] = movmatrix_trans(MODE == 0 && t4 >= 2 ? lo2 : hi2);
        if (MODE != 0) pl[n][h] = movmatrix_trans(lo2);
      }
    }
#pragma unroll
    for (int d = 0; d < KS; ++d) {
      uint32_t a[4];
      // matrices: (keys 0-7, dims 0-7), (keys 0-7, dims 8-15), (keys 8-15, dims 0-7), (8-15, 8-15)
      ldsm_x4_trans(st + Ring<D>::tile + swz<D>((lane & 7) + ((lane >> 4) << 3), 2 * d + ((lane >> 3) & 1)), a);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_16816(o[d][n], a, ph[n][0], ph[n][1]);
        if (MODE != 0) mma_16816(o[d][n], a, pl[n][0], pl[n][1]);
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
        if (MODE == 0) {
#pragma unroll
          for (int d = 0; d < KS; ++d) {
            o[d][n][c] += __shfl_xor_sync(0xffffffffu, o[d][n][c], 2);
            o[d][n][c + 2] += __shfl_xor_sync(0xffffffffu, o[d][n][c + 2], 2);
          }
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
          const int h = n * 8 + (MODE == 0 ? (t4 & 1) * 2 : t4 * 2) + c;
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

  // ---- the warps' parts joined: whole units are written, the others left for the next kernel
  int4 head = make_int4(-1, -1, -1, -1);
  for (int i = 0; i < 2 * kWarps;) {
    const int4 id = piece[i];
    if (id.x < 0) {
      ++i;
      continue;
    }
    int end = i, ends = 0;  // the unit's parts are i .. end - 1 (with gaps)
    for (int j = i; j < 2 * kWarps; ++j) {
      const int4 other = piece[j];
      if (other.x < 0) continue;
      if (other.x != id.x || other.y != id.y) break;
      end = j + 1;
      ends |= other.w;
    }
    auto part = [&](int j) -> const float* {
      return j & 1 ? reinterpret_cast<const float*>(smem + (j >> 1) * Ring<D>::warp)
                   : p.kept + ((int64_t)blockIdx.x * kWarps + (j >> 1)) * P;
    };
    const int slot = id.z ? 1 : 0;
    float* to = p.parts + ((int64_t)blockIdx.x * 2 + slot) * P;
    if (!(id.z && ends)) {
      if (slot == 0) head.x = id.x, head.y = id.y;
      else head.z = id.x, head.w = id.y;
    }
    for (int k = tid; k < H * D / 2; k += kThreads) {
      const int h = k / (D / 2), e = (k - h * (D / 2)) * 2;
      float top = -INFINITY, sum = 0.f, a = 0.f, b = 0.f;
      bool none = false;
      for (int j = i; j < end; ++j)
        if (piece[j].x >= 0) top = fmaxf(top, part(j)[H * D + h]);
      for (int j = i; j < end; ++j) {
        if (piece[j].x < 0) continue;
        const float* from = part(j);
        const float f = weight(from[H * D + h], top), lj = from[H * D + H + h];
        none |= lj == kBad;
        sum += f * lj;
        a += f * from[h * D + e];
        b += f * from[h * D + e + 1];
      }
      if (none) sum = kBad;
      if (id.z && ends) {
        write_pair<D>(p, id.x, id.y, h, e, a, b, sum);
      } else {
        *reinterpret_cast<float2*>(to + h * D + e) = make_float2(a, b);
        if (e == 0) {
          to[H * D + h] = top;
          to[H * D + H + h] = sum;
        }
      }
    }
    i = end;
  }
  if (tid == 0) p.head[blockIdx.x] = head;
}

// Joins the CTAs' parts of a unit: block (c, h) takes head h of the unit that begins in
// CTA c and goes on in the next ones.
template <int D, int H>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Bf16Params p) {
  constexpr int P = kPart<D, H>, LANES = D / 2, GROUPS = kThreads / LANES;
  __shared__ float2 red[GROUPS][LANES];
  __shared__ float red_m[kWarps], red_l[kWarps];
  const int tid = threadIdx.x, c = blockIdx.x, h = blockIdx.y, ctas = gridDim.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 id = p.head[c];
  if (id.z < 0) return;
  int parts = 1;  // the CTAs that go on with a unit follow one another
  for (int i = c + 1; i < ctas; i += kThreads) {
    const int o = i + tid;
    const int4 other = o < ctas ? p.head[o] : make_int4(-1, -1, -1, -1);
    parts += __syncthreads_count(other.x == id.z && other.y == id.w);
  }
  auto part = [&](int j) { return p.parts + ((int64_t)(c + j) * 2 + (j == 0)) * P; };
  float top = -INFINITY;
  for (int j = tid; j < parts; j += kThreads) top = fmaxf(top, part(j)[H * D + h]);
#pragma unroll
  for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  if (tid % 32 == 0) red_m[tid / 32] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red_m[w]);
  float sum = 0.f;
  bool none = false;
  for (int j = tid; j < parts; j += kThreads) {
    const float lj = part(j)[H * D + H + h];
    none |= lj == kBad;
    sum += weight(part(j)[H * D + h], top) * lj;
  }
  none = __syncthreads_or(none);
#pragma unroll
  for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  if (tid % 32 == 0) red_l[tid / 32] = sum;
  const int e = tid % LANES, group = tid / LANES;
  float2 o = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int j = group; j < parts; j += GROUPS) {
    const float f = weight(part(j)[H * D + h], top);
    const float2 v = *reinterpret_cast<const float2*>(part(j) + h * D + e * 2);
    o.x += f * v.x;
    o.y += f * v.y;
  }
  red[group][e] = o;
  __syncthreads();
  if (group != 0) return;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += red_l[w];
#pragma unroll
  for (int k = 1; k < GROUPS; ++k) {
    o.x += red[k][e].x;
    o.y += red[k][e].y;
  }
  write_pair<D>(p, id.z, id.w, h, e * 2, o.x, o.y, none ? kBad : sum);
}

int heads_of(const PagedProblem& pb) { return pb.G <= 4 ? 4 : pb.G <= 8 ? 8 : 16; }
size_t part_bytes(const PagedProblem& pb) { return (size_t)heads_of(pb) * (pb.d + 2) * sizeof(float); }

template <int D, int MODE>
int launch(const PagedProblem& pb, void* workspace, int sms, cudaStream_t stream) {
  constexpr int H = MODE == 0 ? 4 : MODE == 1 ? 8 : 16;
  Bf16Params p{};
  p.q = static_cast<const bf16*>(pb.q);
  p.pool = reinterpret_cast<const bf16*>(pb.pool);
  p.out = static_cast<bf16*>(pb.out);
  p.block_table = pb.block_table;
  p.q_start = pb.q_start;
  p.kv_len = pb.kv_len;
  p.status = pb.status;
  p.head = static_cast<int4*>(workspace);
  p.parts = reinterpret_cast<float*>(p.head + sms);
  p.kept = p.parts + (size_t)sms * 2 * kPart<D, H>;
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
  p.least = 2 * kWarps;
  p.scale_log2 = pb.scale_log2;
  for (int j = 0; j < 64; ++j) p.turn[j] = pb.turn[j];
  constexpr int smem = Ring<D>::bytes;
  if (cudaFuncSetAttribute(decode_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  decode_kernel<D, MODE><<<sms, kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return GIST_ATTN_ERR_LAUNCH;
  // the joins may start while the last tiles run (and then wait for them)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sms, H);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D, H>, p) == cudaSuccess ? GIST_ATTN_OK : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace

size_t paged_bf16_workspace(const PagedProblem& pb, int sms) {
  return (size_t)sms * (sizeof(int4) + (2 + kWarps) * part_bytes(pb));
}

int launch_paged_bf16(const PagedProblem& pb, void* workspace, int sms, cudaStream_t stream) {
  if (pb.d == 64)
    return pb.G <= 4   ? launch<64, 0>(pb, workspace, sms, stream)
           : pb.G <= 8 ? launch<64, 1>(pb, workspace, sms, stream)
                       : launch<64, 2>(pb, workspace, sms, stream);
  return pb.G <= 4   ? launch<128, 0>(pb, workspace, sms, stream)
         : pb.G <= 8 ? launch<128, 1>(pb, workspace, sms, stream)
                     : launch<128, 2>(pb, workspace, sms, stream);
}

}  // namespace gattn
