// proj_w4_tc.cu -- the 4-bit projections of more than a few tokens (few_tokens() of
// proj_w4.cu says which) on the 5th-generation tensor core: 128 rows of weights are M, up
// to 64 tokens are N, so that the weights are still read once.
//
//   D[n][t] = sum_{k in group} (c[n][k] - 8) x[t][k]     (tcgen05 kind::f16, A in TMEM)
//   acc[n][t] += s[n][group] D[n][t]                     (fp32 registers)
//
// The codes less 8 are exact in bf16; with the group's scale they would be the sum of two bf16 (the
// product has up to twelve bits) and take two MMAs, which has not been tried: here each group's
// sums are read out of TMEM and scaled.  The converted weights go through TMEM and not through
// shared memory: writing and reading them there would cost 32 bytes for each 4 of codes, more than its
// bandwidth.
//
// A CTA has a tile of 128 rows and a part of K; the CTAs of a cluster have the parts
// of one tile, send each other the rows that the other adds up (bulk copies between
// their shared memories) and write those.  Warps: 0-3 convert (a thread a row, codes
// into TMEM), 4-7 scale and add (a thread a row), one issues MMAs, one loads codes and x by TMA.
//
// 64 tokens, 8192 -> 8192 (36.7 MB): 17.3 us, 17.8 with weights that L2 has not, for a floor of 5.4; 32 tokens,
// 4096 -> 4096: 8.0 and 8.3.
// Bound: no one stage (a stage of 128 inputs takes 1300 cycles, two CTAs an SM; without the
// conversion 1.0 us less, without the sums 1.7, without x 0.6, without most MMAs 0.6): one chunk
// and the exchange take 7.4 us, the 15 further chunks 10, and 104 of 152 SMs have two CTAs.
// Two CTAs an SM: one, with half as many parts of K, takes 19.8 us, three spill (34 us).  Twice
// the converting and adding warps: 20.0; twice the adding ones: 17.0-17.5.  Sums stored straight
// into the other CTAs' memory: 19.0, but 7.6 with 32 tokens.
//
// Pages: [Gist page] "把 item 压成 KV：gist 能不能用在相关性任务上".
#include <cooperative_groups.h>

#include "follow.cuh"
#include "proj_w4.cuh"
#include "tcgen05.cuh"

namespace cg = cooperative_groups;

namespace gattn {
namespace {

constexpr int kRows = 128, kPairs = 64, kThreads = 320, kMma = 8;  // kMma: the warp that issues MMAs
constexpr int kChunk = 128;          // inputs of a stage of codes: 64 bytes a row
constexpr int kRaw = 5;              // stages of codes, 8 KB each
constexpr int kSA = 2, kSB = 3;      // stages of converted weights in TMEM, of x in shared memory
constexpr int kCols = 256;           // TMEM columns: kSA x 64, then two accumulators

struct Bars {
  uint64_t a_full[kSA], a_empty[kSA], b_full[kSB], b_empty[kSB], c_full[kRaw], c_empty[kRaw], d_full[2], d_empty[2], sums;
  uint32_t tmem;
};

template <int TN>
struct Layout {
  static constexpr uint32_t tile_b = 2 * TN * 128;  // two tiles of 64 inputs
  static constexpr uint32_t raw = kSB * tile_b;
  static constexpr uint32_t bars = raw + kRaw * (kRows * 64);
  static constexpr uint32_t bytes = bars + 256 + 1024;  // + alignment
  // over the rings: this CTA's sums [pair][2][TN], then the parts of the pairs that it adds up
  static constexpr uint32_t sums = kRows * TN * 4;
  static_assert(2 * sums <= bars, "sums");
};

__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// TN tokens, groups of 16 PG inputs (PG MMAs).
template <int TN, int PG>
__global__ void __launch_bounds__(kThreads, 2)
    w4_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                 const __grid_constant__ W4Params p) {
  using L = Layout<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  Bars& bars = *reinterpret_cast<Bars*>(smem + L::bars);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int split = cluster.num_blocks(), part = cluster.block_rank();
  const int n0 = (blockIdx.x / split) * kRows, t0 = blockIdx.y * TN;
  const int k0 = part * p.slice, k1 = max(min(k0 + p.slice, p.K), k0);
  const int chunks = (k1 - k0 + kChunk - 1) / kChunk;

  let_follow();
  wait_before();
  // ---- the loading warp asks for the first stages before anything else
  auto load_codes = [&](int i) {  // inputs past K and rows past N are zeros (and counted)
    const int s = i % kRaw;
    mbar_arrive_expect_tx(&bars.c_full[s], kRows * 64);
    tma_load_2d(base + L::raw + s * (kRows * 64), &tm_w, &bars.c_full[s], (k0 + i * kChunk) / 2, n0);
  };
  auto load_x = [&](int i) {  // inputs past K and tokens past T likewise
    const int s = i % kSB;
    mbar_arrive_expect_tx(&bars.b_full[s], L::tile_b);
    tma_load_2d(base + s * L::tile_b, &tm_x, &bars.b_full[s], k0 + i * kChunk, t0);
    tma_load_2d(base + s * L::tile_b + TN * 128, &tm_x, &bars.b_full[s], k0 + i * kChunk + 64, t0);
  };
  if (warp > kMma && tc::elect_one()) {
    for (int s = 0; s < kRaw; ++s) mbar_init(&bars.c_full[s], 1), mbar_init(&bars.c_empty[s], 4);
    for (int s = 0; s < kSB; ++s) mbar_init(&bars.b_full[s], 1), mbar_init(&bars.b_empty[s], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    for (int i = 0; i < min(chunks, max(kRaw, kSB)); ++i) {
      if (i < kRaw) load_codes(i);
      if (i < kSB) load_x(i);
    }
  }
  if (warp == kMma) {
    tc::tmem_alloc(smem_u32(&bars.tmem), kCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < kSA; ++s) mbar_init(&bars.a_full[s], 4), mbar_init(&bars.a_empty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&bars.d_full[s], 1), mbar_init(&bars.d_empty[s], 4);
    mbar_init(&bars.sums, 1);
    fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars.tmem, lanes = (uint32_t)((warp & 3) * 32) << 16;
  const int groups = (k1 - k0) / (16 * PG);
  bool failed = false;
  auto wait = [&](uint64_t* bar, int use) {  // the use-th completion of a barrier (0: the first)
    if (__any_sync(0xffffffffu, !mbar_wait(bar, (uint32_t)use & 1u))) failed = true;
    return !failed;
  };
  float acc[TN];

  if (warp < 4) {
    // ---------------------------------------------------------- codes to bf16
    const uint32_t row = base + L::raw + tid * 64, swap = (lane >> 1 & 3) << 4;
    for (int i = 0; i < chunks && !failed; ++i) {
      const int at = i % kRaw, s = i % kSA;
      if (!wait(&bars.c_full[at], i / kRaw)) break;
      uint32_t u[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 v = lds16(row + at * (kRows * 64) + ((c << 4) ^ swap));
        u[4 * c] = v.x, u[4 * c + 1] = v.y, u[4 * c + 2] = v.z, u[4 * c + 3] = v.w;
      }
      if (i >= kSA && !wait(&bars.a_empty[s], i / kSA - 1)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) word_to_bf16(u[8 * h + j], a + 4 * j);
        st32(tmem + lanes + s * 64 + h * 32, a);
      }
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.a_full[s]);
        mbar_arrive(&bars.c_empty[at]);
      }
    }
  } else if (warp < kMma) {
    // ------------------------------------------------- the groups' sums, scaled and added
#pragma unroll
    for (int e = 0; e < TN; ++e) acc[e] = 0.f;
    const int n = n0 + (warp & 3) * 32 + lane;
    const uint16_t* scale = reinterpret_cast<const uint16_t*>(p.scale) + (int64_t)min(n, p.N - 1) * (p.K / p.group) + k0 / p.group;
    constexpr int kAhead = 4;  // scales are read so many groups ahead (where load2 stands: it is volatile), converted when used
    uint32_t next[kAhead];
#pragma unroll
    for (int g = 0; g < kAhead; ++g) next[g] = g < groups ? load2(scale + g) : 0;
    for (int g0 = 0; g0 < groups && !failed; g0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int g = g0 + j;
        if (g >= groups) break;
        const float now = __uint_as_float(next[j] << 16);
        next[j] = g + kAhead < groups ? load2(scale + g + kAhead) : 0;
        if (!wait(&bars.d_full[g & 1], g >> 1)) break;
        tc::fence_after_sync();
        const uint32_t d = tmem + lanes + kSA * 64 + (g & 1) * TN;
#pragma unroll
        for (int h = 0; h < TN / 16; ++h) {
          uint32_t v[16];
          tc::ld16_wait(d + 16 * h, v);
          if (h == TN / 16 - 1) {
            tc::fence_before_sync();  // the accumulator is read: the next group but one may have it
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.d_empty[g & 1]);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[16 * h + e] = fmaf(__uint_as_float(v[e]), now, acc[16 * h + e]);
        }
      }
    }
  } else if (warp == kMma) {
    // ------------------------------------------ MMAs, by one thread and with few instructions
    if (tc::elect_one()) {
      constexpr uint32_t idesc = tc::idesc_bf16_f32(kRows, TN, 0);
      const uint64_t x0 = tc::smem_desc_sw128(base, 16, 1024);  // addresses in units of 16 bytes
      constexpr int kGroups = 8 / PG;  // of a chunk
      int g = 0;
      for (int i = 0; i < chunks && !failed; ++i) {
        const int s = i % kSA, sb = i % kSB;
        failed = !mbar_wait(&bars.a_full[s], i / kSA & 1) || !mbar_wait(&bars.b_full[sb], i / kSB & 1);
        const uint64_t bd = x0 + sb * (L::tile_b / 16);
        const uint32_t a = tmem + s * 64;
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          if (failed || g >= groups) break;  // past K's end there is nothing left to add
          if (g >= 2 && !mbar_wait(&bars.d_empty[g & 1], ((g >> 1) - 1) & 1)) failed = true;
          tc::fence_after_sync();
          const uint32_t d = tmem + kSA * 64 + (g & 1) * TN;
#pragma unroll
          for (int k = 0; k < PG; ++k) {
            const int ks = j * PG + k;  // 16 inputs: 8 columns of A, 32 bytes of a row of x's tile
            tc::mma_ts(d, a + ks * 8, bd + (ks >> 2) * (TN * 128 / 16) + (ks & 3) * 2, idesc, k == 0 ? 0u : 1u);
          }
          tc::commit(smem_u32(&bars.d_full[g & 1]));
          ++g;
        }
        tc::commit(smem_u32(&bars.a_empty[s]));
        tc::commit(smem_u32(&bars.b_empty[sb]));
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------- codes and x, further stages
    if (tc::elect_one()) {
      int xs = min(chunks, kSB), cs = min(chunks, kRaw);  // asked for so far
      while (cs < chunks || xs < chunks) {
        if (xs < chunks) {
          if (!mbar_wait(&bars.b_empty[xs % kSB], (xs / kSB - 1) & 1)) break;
          load_x(xs++);
        }
        if (cs < chunks) {
          if (!mbar_wait(&bars.c_empty[cs % kRaw], (cs / kRaw - 1) & 1)) break;
          load_codes(cs++);
        }
      }
      failed = xs < chunks || cs < chunks;
      // none of the copies is left in flight
      for (int i = max(xs - kSB, 0); i < xs; ++i) failed |= !mbar_wait(&bars.b_full[i % kSB], i / kSB & 1);
      for (int i = max(cs - kRaw, 0); i < cs; ++i) failed |= !mbar_wait(&bars.c_full[i % kRaw], i / kRaw & 1);
    }
    __syncwarp();
  }
  if (__any_sync(0xffffffffu, failed) && lane == 0) report(p.status, GIST_ATTN_STATUS_TIMEOUT);

  // ---- the cluster's CTAs added up.  Pairs of rows that are rotated together lie next to
  // each other; 16-byte chunk c of a row of sums at c ^ (pair mod 8)
  tc::fence_before_sync();
  __syncthreads();  // the rings are done with
  const int half = p.position ? p.shift - 1 : 6;  // rows of a pair are 1 << half apart
  const int own = kPairs / split, q0 = part * own;  // the pairs that this CTA adds up
  const int bytes = own * 2 * TN * 4;
  if (tid == 0) mbar_arrive_expect_tx(&bars.sums, split * bytes);
  __syncwarp();
  cluster_arrive();
  if (warp == kMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kCols);
  }
  if (warp >= 4 && warp < kMma) {
    const int r = (warp & 3) * 32 + lane, pair = r >> (half + 1) << half | (r & ((1 << half) - 1)), which = r >> half & 1;
    const uint32_t row = base + (2 * pair + which) * (TN * 4);
#pragma unroll
    for (int c = 0; c < TN / 4; ++c)
      sts16(row + ((c ^ (pair & 7)) << 4), make_uint4(__float_as_uint(acc[4 * c]), __float_as_uint(acc[4 * c + 1]),
                                                      __float_as_uint(acc[4 * c + 2]), __float_as_uint(acc[4 * c + 3])));
    fence_proxy_async_smem();
  }
  __syncthreads();
  cluster_wait();  // the others' rings are done with too
  if (tid < split) {
    uint32_t dst, bar;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(base + L::sums + part * bytes), "r"(tid));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_u32(&bars.sums)), "r"(tid));
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(base + tid * bytes), "r"(bytes), "r"(bar)
                 : "memory");
  }
  const bool arrived = mbar_wait(&bars.sums, 0);
  __syncwarp();
  cluster_arrive();
  if (!arrived) {
    if (lane == 0) report(p.status, GIST_ATTN_STATUS_TIMEOUT);
  } else {
    const int tokens = min(TN, p.T - t0), own_log2 = 31 - __clz(own);
#pragma unroll 1  // once through straight code costs more, in misses of instructions
    for (int i = tid; i < own * tokens; i += kThreads) {
      const int q = i & (own - 1), t = i >> own_log2, pair = q0 + q;  // a pair of rows, a token
      const int n = n0 + (pair >> half << (half + 1) | (pair & ((1 << half) - 1)));
      if (n >= p.N) continue;
      const float* from = reinterpret_cast<const float*>(smem + L::sums + q * 2 * (TN * 4) + (((t >> 2) ^ (pair & 7)) << 4)) + (t & 3);
      float a = 0.f, b = 0.f;
      for (int s = 0; s < split; ++s) {
        a += from[s * (bytes / 4)];
        b += from[s * (bytes / 4) + TN];
      }
      finish_pair(p, t0 + t, n, 1 << half, 64.f * a, 64.f * b);
    }
  }
  __syncwarp();
  cluster_wait();  // no CTA leaves while its sums are being sent
}

// Chunks of K for each of `split` CTAs.
int chunks_of(int K, int split) { return ((K + kChunk - 1) / kChunk + split - 1) / split; }
// Parts of K: two CTAs an SM, where K has a few chunks for each.
int parts_of(const W4Params& p, int token_blocks, int sms) {
  const int64_t tiles = (p.N + kRows - 1) / kRows;
  int split = 1;
  while (split < 8 && tiles * token_blocks * split * 2 <= 2 * sms && split * 4 <= chunks_of(p.K, 1)) split *= 2;
  return split;
}

template <int TN, int PG>
int launch_as(W4Params p, int sms, cudaStream_t stream) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return GIST_ATTN_ERR_LAUNCH;
  alignas(64) CUtensorMap tm_x, tm_w;
  const cuuint32_t each[2] = {1, 1};
  const cuuint64_t dims_x[2] = {(cuuint64_t)p.K, (cuuint64_t)p.T}, stride_x[1] = {(cuuint64_t)p.K * 2};
  const cuuint64_t dims_w[2] = {(cuuint64_t)p.K / 2, (cuuint64_t)p.N}, stride_w[1] = {(cuuint64_t)p.K / 2};
  const cuuint32_t box_x[2] = {64, TN}, box_w[2] = {kChunk / 2, kRows};
  if (enc(&tm_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<bf16*>(p.x), dims_x, stride_x, box_x, each,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      enc(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.w), dims_w, stride_w, box_w, each,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return GIST_ATTN_ERR_UNSUPPORTED;
  const int tiles = (p.N + kRows - 1) / kRows, token_blocks = (p.T + TN - 1) / TN, split = parts_of(p, token_blocks, sms);
  p.slice = chunks_of(p.K, split) * kChunk;
  constexpr int smem = Layout<TN>::bytes;
  if (token_blocks > 65535) return GIST_ATTN_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(w4_tc_kernel<TN, PG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  return launch_following(w4_tc_kernel<TN, PG>, dim3(tiles * split, token_blocks), dim3(kThreads), smem, stream, split, tm_x, tm_w, p)
             ? GIST_ATTN_OK
             : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace

int w4_tc_chunks(const W4Params& p, int sms) { return chunks_of(p.K, parts_of(p, 1, sms)); }

int launch_w4_tc(const W4Params& p, int sms, cudaStream_t stream) {
  if (p.T <= 32)
    return p.group == 32   ? launch_as<32, 2>(p, sms, stream)
           : p.group == 64 ? launch_as<32, 4>(p, sms, stream)
                           : launch_as<32, 8>(p, sms, stream);
  return p.group == 32   ? launch_as<64, 2>(p, sms, stream)
         : p.group == 64 ? launch_as<64, 4>(p, sms, stream)
                         : launch_as<64, 8>(p, sms, stream);
}

}  // namespace gattn
