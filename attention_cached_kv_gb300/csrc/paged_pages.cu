// paged_pages.cu -- the blocks ("pages") of a paged cache between steps: sharing
// them with forked requests, giving them back, moving them together, copying them
// ([Suffix page, §6 问题四]: a logical slot is found through the block table, so
// a block moves by rewriting entries).
//
// free      ref[b] = number of live entries naming b; the free list is the ids
//           with ref 0 in ascending order.  Nothing is counted up and down
//           between calls, so a lost count cannot leak a block.
// compact   n = blocks in use.  The k-th id in use from n on goes to the k-th unused
//           id below n; there are as many of one as of the other, and no source is a
//           destination, so the copies need no order.
// fork      a child's row is its parent's; where the parent's last block is
//           filled in part, the child gets a block of its own and a copy of it.
// copy      the data, from the lists that fork and compact leave on the device.
//
// Bound: the tables are latency (few hundred KB, dependent passes), the copy is HBM.
// Free list of 2048 requests over 131 k blocks 12.9 us, of 32 over 2240 5.2 us; their
// compaction 8 us and the copy of its 238 MB (476 moved) 68 us, 7.0 TB/s with what stays
// in L2; a fork of 48 samples (99 MB of rows) 32.6 us.
//
// Pages: [Suffix page] icman.com.cn news 64898.
#include <cooperative_groups.h>

#include "common.cuh"
#include "follow.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace gattn {
namespace {

// ------------------------------------------------------- free and compact ---
//
// One cluster does the whole of it, its barriers between the passes, so one launch
// is enough and no counter has to be zeroed before.
constexpr int kCtas = 8, kThreads = 1024, kWarps = kThreads / 32;
constexpr int kSeg = 128;  // entries of one row that a warp takes at a time
// Segments and ids that one cluster does alone: past them the passes over the table are bound by
// eight SMs' atomics (2048 rows of 126 entries: 19 us alone, 13 in three kernels).
constexpr int kAlone = 512, kAloneIds = 16384;
// That one CTA does, whose barriers cost next to nothing (4 rows 3.4 us for 5.7 in a cluster, 64 rows
// 5.9 for 6.7; 128 rows of 128 entries 11.1 for 8.3).
constexpr int kFew = 64, kFewIds = 4096;

// Blocks of a request: the live entries of its row.
__device__ __forceinline__ int blocks_of(int len, int block_len, int W, bool& bad) {
  if (len <= 0) return 0;
  const unsigned n = ((unsigned)len + block_len - 1) / block_len;
  if (n > (unsigned)W) bad = true;
  return min((int)n, W);
}

// Calls visit(r, j0, n) by whole warps for the segments [j0, j0 + kSeg) of every row of the
// table, n the row's live entries; kAtOnce segments a call (n < 0: none), so that their loads
// are in flight together.
constexpr int kAtOnce = 4;
template <class Visit>
__device__ __forceinline__ void each_segment(const PagesArgs& a, unsigned warp, unsigned warps, bool& bad, Visit visit) {
  const int lane = threadIdx.x & 31;
  // (counted in 31 bits; each warp does these divisions, so they are not of 64 bits)
  const unsigned per_row = ((unsigned)a.W + kSeg - 1) / kSeg, units = (unsigned)a.B * per_row;
  const unsigned share = (units + warps - 1) / warps;
  const unsigned u0 = min(warp * share, units), u1 = min(u0 + share, units);
  for (unsigned base = u0; base < u1; base += 32) {
    const unsigned mine = base + lane;  // each lane reads the length of one of 32 units
    int row = 0, seg = 0, n = -1;
    if (mine < u1) {
      row = (int)(per_row == 1 ? mine : mine / per_row);
      seg = (int)(mine - row * per_row);
      n = blocks_of(a.cached_len[row], a.block_len, a.W, bad);
    }
    const int m = (int)min(32u, u1 - base);
    for (int i = 0; i < m; i += kAtOnce) {
      int r[kAtOnce], j0[kAtOnce], live[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {  // lanes past m have n = -1
        r[k] = __shfl_sync(0xffffffffu, row, i + k);
        j0[k] = __shfl_sync(0xffffffffu, seg, i + k) * kSeg;
        live[k] = __shfl_sync(0xffffffffu, n, i + k);
      }
      visit(r, j0, live);
    }
  }
}

// A warp's slice [b0, b1) of the ids, 32 at a time: which of them are in use.  The masks of
// up to 1024 ids stay with the lanes after the first pass, longer slices are read again.
struct Slice {
  const int32_t* ids;
  int b0, b1;
  uint32_t kept;  // lane i: the i-th mask

  // Calls visit(first id, mask) in order.
  template <bool READ, class Visit>
  __device__ __forceinline__ void each(Visit visit) {
    const int lane = threadIdx.x & 31;
    const bool read = READ || b1 - b0 > 1024;
    for (int b = b0; b < b1; b += 8 * 32) {
      uint32_t m[8];
      if (read) {
        int v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = b + 32 * k + lane < b1 ? __ldcg(ids + b + 32 * k + lane) : 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m[k] = __ballot_sync(0xffffffffu, v[k] != 0);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) m[k] = __shfl_sync(0xffffffffu, kept, (b - b0) / 32 + k);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (b + 32 * k >= b1) break;
        if (READ && lane == (((b - b0) / 32 + k) & 31)) kept = m[k];
        visit(b + 32 * k, m[k]);
      }
    }
  }
};

// Counts (or marks) the ids that live entries name.
template <bool COMPACT>
__device__ __forceinline__ void mark(const PagesArgs& a, int gw, int warps) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  each_segment(a, gw, warps, bad, [&](const int (&r)[kAtOnce], const int (&j0)[kAtOnce], const int (&n)[kAtOnce]) {
    int id[kAtOnce][kSeg / 32];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int k = 0; k < kSeg / 32; ++k) {
        const int j = j0[u] + 32 * k + lane;
        id[u][k] = j < n[u] ? a.block_table[(int64_t)r[u] * a.W + j] : -1;
        bad |= j < n[u] && (id[u][k] < 0 || id[u][k] >= a.num_blocks);
      }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int k = 0; k < kSeg / 32; ++k) {
        if (id[u][k] < 0 || id[u][k] >= a.num_blocks) continue;
        if constexpr (COMPACT) a.ids[id[u][k]] = 1;
        else atomicAdd(&a.ids[id[u][k]], 1);
      }
  });
  if (bad) report(a.status, GIST_ATTN_STATUS_BAD_BLOCK);
}

// The table with the new ids.
__device__ __forceinline__ void rename(const PagesArgs& a, int gw, int warps) {
  const int lane = threadIdx.x & 31;
  bool bad = false;  // reported by mark
  each_segment(a, gw, warps, bad, [&](const int (&r)[kAtOnce], const int (&j0)[kAtOnce], const int (&live)[kAtOnce]) {
    int id[kAtOnce][kSeg / 32];
    auto inside = [&](int u, int k) { return live[u] >= 0 && j0[u] + 32 * k + lane < a.W; };
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int k = 0; k < kSeg / 32; ++k) id[u][k] = inside(u, k) ? a.block_table[(int64_t)r[u] * a.W + j0[u] + 32 * k + lane] : -1;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int k = 0; k < kSeg / 32; ++k)
        if (j0[u] + 32 * k + lane < live[u] && id[u][k] >= 0 && id[u][k] < a.num_blocks) id[u][k] = __ldcg(a.ids + id[u][k]);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int k = 0; k < kSeg / 32; ++k)
        if (inside(u, k)) a.table_out[(int64_t)r[u] * a.W + j0[u] + 32 * k + lane] = id[u][k];
  });
}

// ALONE: the whole of the work; otherwise the passes over the table, which are wide, have
// kernels of their own and this one has the passes over the ids, which depend on each other.
template <bool COMPACT, bool ALONE, int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kThreads) tables_kernel(const __grid_constant__ PagesArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  auto sync = [&]() {
    if (CTAS > 1) cluster.sync();
    else __syncthreads();
  };
  __shared__ int count[kWarps];                // ids in use in each warp's slice
  __shared__ int below[kWarps];                // COMPACT: those of them below n
  __shared__ int all[CTAS * kWarps], all_below;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, gw = cta * kWarps + warp;

  let_follow();
  wait_before();
  if constexpr (ALONE) {
    for (int b = cta * kThreads + tid; b < a.num_blocks; b += CTAS * kThreads) a.ids[b] = 0;
    sync();
    mark<COMPACT>(a, gw, CTAS * kWarps);
    sync();
  }

  // each warp's slice of the ids: how many are in use
  const int per = ((a.num_blocks + CTAS * kWarps - 1) / (CTAS * kWarps) + 31) & ~31;
  Slice s;
  s.ids = a.ids;
  s.b0 = min(gw * per, a.num_blocks);  // 2^30 ids at most, so this is below 2^31
  s.b1 = min(s.b0 + per, a.num_blocks);
  s.kept = 0;
  int used = 0;
  s.each<true>([&](int, uint32_t m) { used += __popc(m); });
  if (lane == 0) count[warp] = used;
  sync();
  if (tid < CTAS * kWarps) all[tid] = *cluster.map_shared_rank(&count[tid % kWarps], tid / kWarps);
  __syncthreads();
  int before = 0, n = 0;  // ids in use ahead of the slice, and in all
  for (int w = lane; w < CTAS * kWarps; w += 32) {
    n += all[w];
    before += w < gw ? all[w] : 0;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  before = __reduce_add_sync(0xffffffffu, before);
  const uint32_t ahead = (1u << lane) - 1;

  if constexpr (!COMPACT) {
    if (CTAS > 1) cluster.barrier_arrive();  // this CTA has read the others' counts
    const int free = a.num_blocks - n;
    s.each<false>([&](int b, uint32_t m) {
      const int id = b + lane;
      // the unused ids ahead of an id: the id itself less those in use ahead of it
      if (id < s.b1 && !(m >> lane & 1)) a.free_blocks[id - before - __popc(m & ahead)] = id;
      before += __popc(m);
    });
    for (int i = free + cta * kThreads + tid; i < a.num_blocks; i += CTAS * kThreads) a.free_blocks[i] = -1;
    if (cta == 0 && tid == 0) {
      a.free_range[0] = 0;
      a.free_range[1] = free;
    }
    if (CTAS > 1) cluster.barrier_wait();  // and they have read this one's
    return;
  }

  // ids in use below n, which say how many blocks move
  int low = 0;
  s.each<false>([&](int b, uint32_t m) { low += b + 32 <= n ? __popc(m) : b < n ? __popc(m & ((1u << (n - b)) - 1)) : 0; });
  if (lane == 0) below[warp] = low;
  sync();
  if (tid == 0) all_below = 0;
  __syncthreads();
  if (tid < CTAS * kWarps) atomicAdd(&all_below, *cluster.map_shared_rank(&below[tid % kWarps], tid / kWarps));
  __syncthreads();
  const int stay = all_below, moves = n - stay;
  s.each<false>([&](int b, uint32_t m) {
    const int id = b + lane;
    const bool use = m >> lane & 1;
    const int rank = before + __popc(m & ahead);  // ids in use ahead of this one
    if (use && id >= n) a.src[rank - stay] = id;
    if (id < s.b1 && !use && id < n) a.dst[id - rank] = id;
    if (id < s.b1) a.ids[id] = use && id < n ? id : -1;
    before += __popc(m);
  });
  for (int i = moves + cta * kThreads + tid; i < a.num_blocks / 2; i += CTAS * kThreads) a.src[i] = a.dst[i] = -1;
  for (int i = cta * kThreads + tid; i < a.num_blocks; i += CTAS * kThreads) a.free_blocks[i] = i < a.num_blocks - n ? n + i : -1;
  if (cta == 0 && tid == 0) {
    a.count[0] = moves;
    a.free_range[0] = 0;
    a.free_range[1] = a.num_blocks - n;
  }
  sync();
  for (int k = cta * kThreads + tid; k < moves; k += CTAS * kThreads) a.ids[__ldcg(a.src + k)] = __ldcg(a.dst + k);
  if constexpr (ALONE) {
    sync();
    rename(a, gw, CTAS * kWarps);
  }
}

__global__ void __launch_bounds__(kThreads) zero_kernel(const __grid_constant__ PagesArgs a) {
  let_follow();
  wait_before();
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.num_blocks; b += gridDim.x * kThreads) a.ids[b] = 0;
}
template <bool COMPACT>
__global__ void __launch_bounds__(kThreads) mark_kernel(const __grid_constant__ PagesArgs a) {
  let_follow();
  wait_before();
  mark<COMPACT>(a, blockIdx.x * kWarps + (threadIdx.x >> 5), gridDim.x * kWarps);
}
__global__ void __launch_bounds__(kThreads) rename_kernel(const __grid_constant__ PagesArgs a) {
  let_follow();
  wait_before();
  rename(a, blockIdx.x * kWarps + (threadIdx.x >> 5), gridDim.x * kWarps);
}

// ------------------------------------------------------------------- fork ---
//
// Every CTA sums over all requests by itself (as the plan does), then takes rows of its
// own; the rows read are those of requests that are not forked, so none is written.
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ int take[];  // [B] index among the blocks taken; -1: none needed, -2: not served, -3: not forked
  __shared__ int warp_sum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_follow();
  wait_before();
  const int per = (a.B + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, a.B), r1 = min(r0 + per, a.B);
  const int begin = max(a.free_range[0], 0), end = max(min(a.free_range[1], a.num_free), 0);
  const int avail = max(end - begin, 0);
  // 1: a block is needed, 0: none, -2: cannot be forked, -3: is not
  auto asked = [&](int r) {
    const int p = a.parent[r];
    if (p < 0 || p == r) return -3;
    if (p >= a.B) return -2;
    const int pp = a.parent[p];
    if (pp >= 0 && pp != p) return -2;
    const int c = a.cached_len[p];
    if (c < 0 || (int64_t)c > (int64_t)a.W * a.block_len) return -2;
    return c % a.block_len != 0 ? 1 : 0;
  };
  int own = 0;
  for (int r = r0; r < r1; ++r) own += asked(r) == 1;
  int inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int before = inc - own, needed = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    needed += warp_sum[w];
  }
  const int taken = min(needed, avail);
  for (int r = r0; r < r1; ++r) {
    const int n = asked(r);
    take[r] = n < 0 ? n : n == 0 ? -1 : before < avail ? before : -2;
    before += n == 1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.count[0] = taken;
    a.free_range_out[0] = max(a.free_range[0], 0) + taken;
    a.free_range_out[1] = a.free_range[1];
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = taken + tid; i < a.B; i += kThreads) a.src[i] = a.dst[i] = a.rows[i] = -1;

  int bits = 0;
  for (int r = blockIdx.x * kWarps + warp; r < a.B; r += gridDim.x * kWarps) {
    const int k = take[r];
    if (k == -3) {
      if (lane == 0) a.cached_len_out[r] = a.cached_len[r];
      continue;
    }
    if (k == -2) {
      bits |= GIST_ATTN_STATUS_NOT_SERVED;
      if (lane == 0) a.cached_len_out[r] = 0;
      continue;
    }
    const int p = a.parent[r], c = a.cached_len[p], full = c / a.block_len, part = c - full * a.block_len;
    const int32_t* from = a.block_table + (int64_t)p * a.W;
    int32_t* to = a.block_table + (int64_t)r * a.W;
    int src = -1, dst = -1;
    if (k >= 0) {
      src = from[full];
      dst = a.free_blocks[begin + k];
    }
    const bool ok = k < 0 || (src >= 0 && src < a.num_blocks && dst >= 0 && dst < a.num_blocks);
    if (lane == 0) {
      if (k >= 0) {
        a.src[k] = ok ? src : -1;
        a.dst[k] = ok ? dst : -1;
        a.rows[k] = ok ? part : -1;
      }
      a.cached_len_out[r] = ok ? c : 0;
      if (ok && k >= 0) to[full] = dst;
    }
    if (ok) {
      for (int j = lane; j < full; j += 32) to[j] = from[j];
    } else {
      bits |= GIST_ATTN_STATUS_BAD_BLOCK;
    }
  }
  if (bits && lane == 0) report(a.status, bits);
}

// ------------------------------------------------------------------- copy ---
//
// Chunks of kCopyThreads x V 16-byte pieces, a thread's V loads in flight together; a
// copy of `rows` rows of a block counts the pieces of those rows alone, plane after plane.
constexpr int kCopyThreads = 256;

template <int V>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
  let_follow();
  wait_before();
  const int n = a.count ? min(max(*a.count, 0), a.n) : a.n;
  const int row = a.plane / a.block_len;  // pieces of a row
  const int whole = a.planes * a.plane;
  const int chunks = (whole + kCopyThreads * V - 1) / (kCopyThreads * V);
  const int64_t total = (int64_t)n * chunks;
  bool bad = false;
  for (int64_t at = blockIdx.x; at < total; at += gridDim.x) {
    const int i = (int)(at / chunks), first = (int)(at - (int64_t)i * chunks) * (kCopyThreads * V);
    const int s = a.src[i], d = a.dst[i];
    if (s < 0 || d < 0) continue;
    const int rows = a.rows ? a.rows[i] : a.block_len;
    if (s >= a.num_blocks || d >= a.num_blocks || rows < 0 || rows > a.block_len) {
      bad = true;
      continue;
    }
    if (s == d) continue;
    const uint4* from = a.pool + (int64_t)s * whole;
    uint4* to = a.pool + (int64_t)d * whole;
    const int run = rows * row, pieces = run * a.planes;  // of the planes' parts that are copied
    const unsigned inverse = run > 1 ? 0xffffffffu / (unsigned)run : 0;  // x / run is umulhi(x, inverse) or one more
    if (a.scale && first == 0)
      for (int k = threadIdx.x; k < a.planes; k += kCopyThreads)
        a.scale[(int64_t)d * a.planes + k] = a.scale[(int64_t)s * a.planes + k];
    uint4 v[V];
    int off[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int x = first + k * kCopyThreads + threadIdx.x;
      off[k] = x < pieces ? x : -1;
      if (rows != a.block_len && x < pieces) {
        int pl = (int)__umulhi((unsigned)x, inverse), rest = x - pl * run;
        while (rest >= run) {
          ++pl;
          rest -= run;
        }
        off[k] = pl * a.plane + rest;
      }
      if (off[k] >= 0) v[k] = __ldcs(from + off[k]);
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (off[k] >= 0) __stcs(to + off[k], v[k]);
  }
  if (bad && threadIdx.x == 0) report(a.status, GIST_ATTN_STATUS_BAD_BLOCK);
}

}  // namespace

int launch_pages_tables(const PagesArgs& a, bool compact, int sms, cudaStream_t stream) {
  const int64_t segments = (int64_t)a.B * ((a.W + kSeg - 1) / kSeg);
  auto launch = [&](void (*kernel)(PagesArgs), int grid) { return launch_following(kernel, dim3(grid), dim3(kThreads), 0, stream, 0, a); };
  bool ok;
  if (segments <= kFew && a.num_blocks <= kFewIds) {
    ok = launch(compact ? tables_kernel<true, true, 1> : tables_kernel<false, true, 1>, 1);
  } else if (segments <= kAlone && a.num_blocks <= kAloneIds) {
    ok = launch(compact ? tables_kernel<true, true, kCtas> : tables_kernel<false, true, kCtas>, kCtas);
  } else {
    const int64_t want = (segments + kWarps * kAtOnce - 1) / (kWarps * kAtOnce);
    const int wide = want < 1 ? 1 : want > sms ? sms : (int)want;
    const int zeros = (a.num_blocks - 1) / (4 * kThreads) + 1;
    ok = launch(zero_kernel, zeros < sms ? zeros : sms) && launch(compact ? mark_kernel<true> : mark_kernel<false>, wide) &&
         launch(compact ? tables_kernel<true, false, kCtas> : tables_kernel<false, false, kCtas>, kCtas);
    if (compact) ok = ok && launch(rename_kernel, wide);
  }
  return ok ? GIST_ATTN_OK : GIST_ATTN_ERR_LAUNCH;
}

int launch_pages_fork(const ForkArgs& a, cudaStream_t stream) {
  const int smem = a.B * (int)sizeof(int);
  // always the largest limit, so that no thread's call lowers it between another's two lines here
  if (smem > 32 * 1024 &&
      cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanRequests * (int)sizeof(int)) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  const int want = (a.B + kWarps - 1) / kWarps, grid = want < 1 ? 1 : want > 64 ? 64 : want;
  return launch_following(fork_kernel, dim3(grid), dim3(kThreads), smem, stream, 0, a) ? GIST_ATTN_OK : GIST_ATTN_ERR_LAUNCH;
}

int launch_pages_copy(const CopyArgs& a, int sms, cudaStream_t stream) {
  const int64_t pieces = (int64_t)a.n * a.planes * a.plane;
  // small copies: less a thread, so that all SMs take part; large ones: several waves of CTAs, as
  // SMs are not equally near to memory (32 an SM 79.4, 8 an SM 84.6, 4 an SM 88.9 us a compaction
  // of 238 MB; a CTA a chunk of what the list can hold 105)
  const bool large = pieces >= (int64_t)sms * 8 * kCopyThreads * 8;
  const int V = large ? 8 : 2;
  const int64_t chunks = (int64_t)a.n * ((a.planes * (int64_t)a.plane + kCopyThreads * V - 1) / (kCopyThreads * V));
  const int grid = (int)(chunks < 32 * sms ? chunks : 32 * sms);
  return launch_following(large ? copy_kernel<8> : copy_kernel<2>, dim3(grid), dim3(kCopyThreads), 0, stream, 0, a)
             ? GIST_ATTN_OK
             : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace gattn
