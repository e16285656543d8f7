// proj_w4.cu -- projections of a few tokens with 4-bit weights and a scale per group
// of inputs: the QKV projection with RoPE in its epilogue and the output
// projection around the attention of a decoding step ([Gist page, "在线的一次
// attention"]: per layer X is projected to Q, K, V, then attends; the projections
// of gemm.cu need at least 22 tokens a pair).
//
//   y[t][n] = sum over groups of  s[n][group] * sum_{k in group} (c[n][k] - 8) x[t][k]
//
// Few tokens here (one or two, more of small weights: few_tokens() below), more in proj_w4_tc.cu.
//
// Bound: latency.  Its floor is the weights' bytes, but a CTA asks for all of its part (32 KB of codes, then
// 8 KB of x at 4096 inputs) at once, and start, one round of loads and the sums of its warps follow
// one another: one token, 4096 -> 6144, 13 MB: 7.1 us, 8.0 with weights that L2 has not, for a floor of
// 1.9; 5 tokens, 896 -> 1152: 3.6 us.  The codes less 8 are
// exact in bf16, so the inner sums run on mma.sync m16n8k16 with the weights
// as the 16 rows and the tokens as the N (even one token is cheaper there than on
// the CUDA cores, which would spend an FMA and a conversion a weight); the scale
// is applied in fp32 to each group's sum.
//
// Eight codes of a word become four bf16 pairs (k, k + 4): bits 4 j of both halves,
// or'ed into 128.0, are 128 + c exactly; less 136.  x is staged in shared
// memory with its elements in the same order.  A tile's 16 rows are 8 neighbours
// and their 8 rotation partners (half a head on), so a thread holds both values
// of a rotated pair.
//
// Pages: [Gist page] "把 item 压成 KV：gist 能不能用在相关性任务上".
#include <cooperative_groups.h>

#include "follow.cuh"
#include "frag.cuh"
#include "proj_w4.cuh"

namespace cg = cooperative_groups;

namespace gattn {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kStep = 128;   // inputs of a ring stage
constexpr int kStages = 8;   // of a warp's ring, 1 KB a row tile each
constexpr int kMaxX = 72 * 1024;  // staged x of a CTA, at most

// First row of a tile, and its other eight rows' distance.
__device__ __forceinline__ int tile_row(const W4Params& p, int tile, int& apart) {
  if (!p.position) {
    apart = 8;
    return tile * 16;
  }
  const int per_head = p.d / 16, head = tile / per_head;
  apart = p.d / 2;
  return head * p.d + (tile - head * per_head) * 8;
}

// NT tiles of 8 tokens, MR row tiles a warp, WR warps along the rows (the others along K).
template <int NT, int MR, int WR>
__global__ void __launch_bounds__(kThreads) w4_kernel(const __grid_constant__ W4Params p) {
  constexpr int WK = kWarps / WR, TN = NT * 8;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int wr = warp % WR, wk = warp / WR;
  const int split = cluster.num_blocks(), part = cluster.block_rank();
  const int tile0 = (blockIdx.x / split) * (MR * WR) + wr * MR;
  const int k0 = part * p.slice, k1 = min(k0 + p.slice, p.K);
  const int t0 = blockIdx.y * TN;
  const int tokens = min(TN, p.T - t0);
  const uint32_t pitch = p.slice * 2 + 64;  // of a token's staged row: 64 modulo 128
  const uint32_t xs = smem_u32(smem);
  const int staged = min(TN, p.T);  // rows of x in shared memory; MMA columns behind them repeat the last
  const uint32_t ring = xs + staged * pitch + warp * (kStages * MR * 1024);

  let_follow();
  wait_before();
  // ---- weights: rows of 64 bytes, 16 a row tile; chunk c of row r at c ^ (r / 2 mod 4)
  int row[MR], apart = 8;
#pragma unroll
  for (int m = 0; m < MR; ++m) row[m] = tile0 + m < p.tiles ? tile_row(p, tile0 + m, apart) : -1;
  const int steps = k1 > k0 ? (k1 - k0 + kStep - 1) / kStep : 0;
  const int mine = (steps - wk + WK - 1) / WK;  // steps wk, wk + WK, ...
  auto issue = [&](int i) {
    if (i < mine) {
      const int k = k0 + (wk + i * WK) * kStep;
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = h * 8 + g8, kk = k + t4 * 32;
          const bool in = row[m] >= 0 && kk < k1;
          const int64_t at = in ? (int64_t)(row[m] + h * apart + g8) * (p.K / 2) + kk / 2 : 0;
          cp_async16_or_zero(ring + ((i % kStages) * MR + m) * 1024 + r * 64 + ((t4 ^ ((r >> 1) & 3)) << 4), p.w + at, in);
        }
    }
    cp_async_commit();
  };
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  // ---- scales of a step, a step ahead
  const int shift = 31 - __clz(p.group), per32 = p.group / 32;
  const uint16_t* scale[MR][2];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      scale[m][h] = reinterpret_cast<const uint16_t*>(p.scale) + (int64_t)(max(row[m], 0) + h * apart + g8) * (p.K >> shift);
  uint32_t next[MR][4][2] = {};
  auto load_scales = [&](int i) {
    const int k = k0 + (wk + i * WK) * kStep;
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int kk = k + 32 * q;
          if (q % per32 == per32 - 1) next[m][q][h] = row[m] >= 0 && i < mine && kk < k1 ? load2(scale[m][h] + (kk >> shift)) : 0;
        }
  };
  load_scales(0);

  // ---- x: eight inputs as the pairs (k, k + 4), zeros past the inputs
  const int pieces = p.slice / 8;
  for (int i = tid; i < staged * pieces; i += kThreads) {
    const int t = i / pieces, c = i - t * pieces, k = k0 + c * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t < tokens && k < k1) v = load16(p.x + (int64_t)(t0 + t) * p.K + k);
    sts16(xs + t * pitch + c * 16, make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                              __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)));
  }
  __syncthreads();

  float acc[MR][NT][4];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;

  for (int i = 0; i < mine; ++i) {
    const int k = k0 + (wk + i * WK) * kStep;
    uint32_t sc[MR][4][2];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[m][q][h] = next[m][q][h];
    load_scales(i + 1);
    cp_async_wait_group<kStages - 2>();
    __syncwarp();
    const uint32_t st = ring + (i % kStages) * MR * 1024;
    float sum[MR][NT][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q % per32 == 0) {
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n) sum[m][n][0] = sum[m][n][1] = sum[m][n][2] = sum[m][n][3] = 0.f;
      }
      uint32_t a[MR][2][4];
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = h * 8 + g8;
          const uint32_t u = lds32(st + m * 1024 + r * 64 + ((q ^ ((r >> 1) & 3)) << 4) + t4 * 4);
          a[m][0][h] = codes_to_bf16x2(u);
          a[m][0][2 + h] = codes_to_bf16x2(u >> 4);
          a[m][1][h] = codes_to_bf16x2(u >> 8);
          a[m][1][2 + h] = codes_to_bf16x2(u >> 12);
        }
      const uint32_t xa = xs + (k - k0 + 32 * q) * 2 + t4 * 16;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = lds16(xa + min(n * 8 + g8, staged - 1) * pitch);
#pragma unroll
        for (int m = 0; m < MR; ++m) {
          mma_16816(sum[m][n], a[m][0], b.x, b.y);
          mma_16816(sum[m][n], a[m][1], b.z, b.w);
        }
      }
      if (q % per32 == per32 - 1) {
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][n][e] = fmaf(sum[m][n][e], __uint_as_float(sc[m][q][e >> 1] << 16), acc[m][n][e]);
      }
    }
    __syncwarp();
    issue(i + kStages - 1);
  }

  // ---- the warps along K and the CTAs of the cluster added up: [wk][row][token]
  cp_async_wait_all();
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  constexpr int RT = 16 * MR * WR, RP = TN + 1;
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[(wk * RT + (wr * MR + m) * 16 + (e >> 1) * 8 + g8) * RP + n * 8 + t4 * 2 + (e & 1)] = acc[m][n][e];
  if (split > 1) cluster.sync();
  else __syncthreads();
  // pairs of rows; the cluster's CTAs share them out
  constexpr int pairs = RT / 2 * TN;
  for (int i = part * kThreads + tid; i < pairs; i += split * kThreads) {
    const int t = i / (RT / 2), j = i - t * (RT / 2), tile = (blockIdx.x / split) * (MR * WR) + j / 8;
    if (t >= tokens || tile >= p.tiles) continue;
    const int at = ((j / 8) * 16 + (j & 7)) * RP + t;
    float a = 0.f, b = 0.f;
    for (int c = 0; c < split; ++c) {
      const float* from = split > 1 ? cluster.map_shared_rank(red, c) : red;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        a += from[w * RT * RP + at];
        b += from[w * RT * RP + at + 8 * RP];
      }
    }
    int far;
    const int n = tile_row(p, tile, far) + (j & 7);
    finish_pair(p, t0 + t, n, far, a, b);
  }
  if (split > 1) cluster.sync();  // no CTA leaves while another reads its sums
}

template <int NT, int MR, int WR>
int launch_as(W4Params p, int sms, cudaStream_t stream) {
  constexpr int TN = NT * 8, RT = MR * WR;
  const int blocks = (p.tiles + RT - 1) / RT, token_blocks = (p.T + TN - 1) / TN;
  // K is split over the CTAs of a cluster until x fits and every SM has a CTA or two
  int split = 1;
  auto slice = [&](int s) { return ((p.K + s - 1) / s + kStep - 1) / kStep * kStep; };
  const int staged = p.T < TN ? p.T : TN;
  while (split < 8 && (staged * (slice(split) * 2 + 64) > kMaxX ||
                       ((int64_t)blocks * token_blocks * split < 2 * sms && slice(split) >= 2 * kStep * (kWarps / WR))))
    split *= 2;
  p.slice = slice(split);
  const int x_bytes = staged * (p.slice * 2 + 64), ring = kWarps * kStages * MR * 1024;
  const int red = (kWarps / WR) * 16 * RT * (TN + 1) * 4;
  const int smem = x_bytes + ring > red ? x_bytes + ring : red;
  constexpr int kMostSmem = 227 * 1024;
  if (smem > kMostSmem || token_blocks > 65535) return GIST_ATTN_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(w4_kernel<NT, MR, WR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  return launch_following(w4_kernel<NT, MR, WR>, dim3(blocks * split, token_blocks), dim3(kThreads), smem, stream, split, p)
             ? GIST_ATTN_OK
             : GIST_ATTN_ERR_LAUNCH;
}

// Which kernel: this one reads the weights again for each eight tokens, that of proj_w4_tc.cu once for up to
// 64, but it has to fill 128 rows a CTA, and its clusters to exchange sums.  With M = 2^20 weights this one
// takes about 2 us and 0.5 a M and eight tokens, that one 4.3 us and 0.35 a chunk of 128 inputs that a
// CTA has (us, this / that: 1 M, 32 tokens 3.3-3.5 / 5.0-7.2; 2 M, 16: 3.1 / 4.6, 24: 5.5 / 4.9; 4 M, 16: 8.6 / 5.7;
// 25 M, 16: 28.6 / 9.6; 64 M, 16: 86 / 14.0; 64 rows of 65536 inputs, 32: 20.8 / 26.8, 64: 31.3 / 29.1).
// (3 M, eight: 4.5 / 4.7; 5 M, eight: 6.7 / 6.1; 6 M, three and eight: 5.1, 9.4 / 5.6; 12 M, four and eight: 9.3, 11.0 /
// 6.9).  One or two tokens take this one, which is 3 us ahead (25 M, one: 7.1 / 9.6; 48 M: 13.7 / 16.5) or 2 behind
// (64 M: 15.8 / 13.4; where K is split over a cluster).  Past 64 tokens that one always.
bool few_tokens(const W4Params& p, int sms) {
  if (p.T <= 2 || p.T > 64) return p.T <= 2;
  const int64_t m = 1 << 20;
  return (int64_t)p.N * p.K * ((p.T + 7) / 8) <= 3 * m + w4_tc_chunks(p, sms) * (m / 2);
}

int launch(const W4Params& p, int sms, cudaStream_t stream) {
  return few_tokens(p, sms) ? launch_as<1, 1, 1>(p, sms, stream) : launch_w4_tc(p, sms, stream);
}

}  // namespace

int launch_qkv_rope_w4(const PagedProblem& pb, const void* x, const void* w, const void* scale, const int32_t* position,
                       void* q, void* k_new, void* v_new, int d_model, int group, int sms, cudaStream_t stream) {
  W4Params p = {};
  p.x = static_cast<const bf16*>(x);
  p.w = static_cast<const uint8_t*>(w);
  p.scale = static_cast<const bf16*>(scale);
  p.out[0] = static_cast<bf16*>(q);
  p.out[1] = static_cast<bf16*>(k_new);
  p.out[2] = static_cast<bf16*>(v_new);
  p.position = position;
  p.status = pb.status;
  p.T = pb.T;
  p.d = pb.d;
  p.shift = pb.d == 64 ? 6 : 7;
  p.Hq = pb.Hq;
  p.Hkv = pb.Hkv;
  p.N = (pb.Hq + 2 * pb.Hkv) * pb.d;
  p.K = d_model;
  p.group = group;
  p.tiles = p.N / 16;
  for (int j = 0; j < 64; ++j) p.turn[j] = pb.turn[j];
  return launch(p, sms, stream);
}

int launch_out_proj_w4(const PagedProblem& pb, const void* attn, const void* w, const void* scale, void* y, int d_model,
                       int group, int sms, cudaStream_t stream) {
  W4Params p = {};
  p.x = static_cast<const bf16*>(attn);
  p.w = static_cast<const uint8_t*>(w);
  p.scale = static_cast<const bf16*>(scale);
  p.out[0] = static_cast<bf16*>(y);
  p.status = pb.status;
  p.T = pb.T;
  p.N = d_model;
  p.K = pb.Hq * pb.d;
  p.group = group;
  p.tiles = d_model / 16;
  return launch(p, sms, stream);
}

}  // namespace gattn
