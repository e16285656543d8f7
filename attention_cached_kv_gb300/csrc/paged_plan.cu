// paged_plan.cu -- block table, slots and positions of one ragged serving step,
// from the requests' lengths ([Suffix page, §6 问题四]: a logical slot is found
// through the block table).
//
// With c, n a request's cached and new tokens and b the block length it needs
// ceil((c + n) / b) - ceil(c / b) blocks.  Exclusive sums over the requests of n
// and of the needs give every request its first token row and its first free
// block; a token's request is then a search in the sums, and all it needs
// follows from its position pos = c + i: the block pos / b is an old entry of
// the table, or the (pos / b - ceil(c / b))-th block taken.  The token at a taken
// block's first row (there is always one) writes the table's entry.
//
// Bound: latency (loads, a scan, a search).  Every CTA scans all requests by
// itself, so CTAs never wait for one another and nothing has to be zeroed; the
// tokens are dealt out in runs of kThreads.  The sums stay in shared memory.  32
// requests: 3.7 us; 2048 with 262 k tokens: 9.1 us.
//
// Pages: [Suffix page] icman.com.cn news 64898.
#include "common.cuh"
#include "kernels.h"

namespace gattn {
namespace {

constexpr int kThreads = 1024;

struct Sums {
  long long tokens, blocks;
};

// A request's new tokens in the packing, and the blocks it asks for (-1: its
// lengths are invalid).
__device__ __forceinline__ void asked(const PlanArgs& a, int r, int& n, int& need) {
  const int c = a.cached_len[r], m = a.new_len[r];
  n = max(m, 0);
  if (c < 0 || m < 0 || (long long)c + m > (long long)a.W * a.block_len) {
    need = -1;
    return;
  }
  const int b = a.block_len;
  need = (int)(((unsigned)c + m + b - 1) / b - ((unsigned)c + b - 1) / b);
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int sm[];
  int* start = sm;            // [B + 1] first token row, at most T
  int* take = sm + a.B + 1;   // [B] index of the first taken block in free_blocks; -1: not served
  __shared__ Sums warp_sum[kThreads / 32];
  __shared__ long long taken_all;  // blocks taken in this step
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, a.B), r1 = min(r0 + per, a.B);
  const int begin = max(a.free_range[0], 0), end = max(min(a.free_range[1], a.num_free), 0);
  const long long avail = max(end - begin, 0);

  Sums own = {0, 0};
  for (int r = r0; r < r1; ++r) {
    int n, need;
    asked(a, r, n, need);
    own.tokens += n;
    own.blocks += max(need, 0);
  }
  Sums inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc.tokens, o);
    const long long k = __shfl_up_sync(0xffffffffu, inc.blocks, o);
    if (lane >= o) {
      inc.tokens += t;
      inc.blocks += k;
    }
  }
  if (lane == 31) warp_sum[warp] = inc;
  if (tid == 0) taken_all = 0;
  __syncthreads();
  if (warp == 0) {
    Sums w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, w.tokens, o);
      const long long k = __shfl_up_sync(0xffffffffu, w.blocks, o);
      if (lane >= o) {
        w.tokens += t;
        w.blocks += k;
      }
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  long long tok = inc.tokens - own.tokens, blk = inc.blocks - own.blocks;
  if (warp > 0) {
    tok += warp_sum[warp - 1].tokens;
    blk += warp_sum[warp - 1].blocks;
  }
  bool refused = false;
  long long last = 0;
  for (int r = r0; r < r1; ++r) {
    int n, need;
    asked(a, r, n, need);
    const bool served = need >= 0 && tok + n <= a.T && (need == 0 || blk + need <= avail);
    start[r] = (int)min(tok, (long long)a.T);
    take[r] = served ? begin + (int)min(blk, avail) : -1;
    if (served && need > 0) last = blk + need;
    refused |= !served;
    if (blockIdx.x == 0) {
      a.q_start[r] = start[r];
      a.kv_len[r] = served ? a.cached_len[r] + n : 0;
    }
    tok += n;
    blk += max(need, 0);
  }
  if (r1 == a.B && (r0 < r1 || tid == 0)) {  // the last request's thread (or any, without requests)
    start[a.B] = (int)min(tok, (long long)a.T);
    if (blockIdx.x == 0) a.q_start[a.B] = start[a.B];
  }
  // the requests that take blocks are the first of those that need some, so the
  // largest end is the number taken
  if (blockIdx.x == 0 && last > 0) atomicMax(reinterpret_cast<unsigned long long*>(&taken_all), (unsigned long long)last);
  if (blockIdx.x == 0 && refused) report(a.status, GIST_ATTN_STATUS_NOT_SERVED);
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    a.free_range_out[0] = max(a.free_range[0], 0) + (int)taken_all;
    a.free_range_out[1] = a.free_range[1];
  }

  bool bad = false;
  const int total = start[a.B];
  for (int64_t row = blockIdx.x * kThreads + tid; row < a.T; row += gridDim.x * kThreads) {
    const int t = (int)row;
    if (t >= total) {
      a.slot[t] = -1;
      a.position[t] = -1;
      continue;
    }
    int lo = 0, hi = a.B;  // start[lo] <= t < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int tk = take[lo];
    int slot = -1, pos = -1;
    if (tk >= 0) {
      const int c = a.cached_len[lo];
      pos = c + (t - start[lo]);
      const int b = pos / a.block_len, row = pos - b * a.block_len;
      const int have = (int)(((unsigned)c + a.block_len - 1) / a.block_len);
      int32_t* entry = a.block_table + (int64_t)lo * a.W + b;
      int id;
      if (b < have) {
        id = *entry;
      } else {
        id = a.free_blocks[tk + b - have];
        if (row == 0) *entry = id;
      }
      if (id >= 0 && id < a.num_blocks) slot = id * a.block_len + row;
      else bad = true;
    }
    a.slot[t] = slot;
    a.position[t] = pos;
  }
  if (bad) report(a.status, GIST_ATTN_STATUS_BAD_BLOCK);
}

}  // namespace

int launch_paged_plan(const PlanArgs& a, cudaStream_t stream) {
  const int smem = (2 * a.B + 1) * (int)sizeof(int);
  // the limit holds for all threads of the process: always the same one, so that no call
  // lowers it between another's two lines here
  constexpr int kMost = (2 * kPlanRequests + 1) * (int)sizeof(int);
  if (smem > 32 * 1024 &&
      cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  const int64_t want = ((int64_t)a.T + kThreads - 1) / kThreads;
  const int grid = want < 1 ? 1 : want > 128 ? 128 : (int)want;
  plan_kernel<<<grid, kThreads, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? GIST_ATTN_OK : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace gattn
