// paged_attn.cu -- causal attention of each request's new tokens over its E4M3
// paged cache ([KV page, "Reusable-state"]: o_t = softmax(q_t K_{<=t}^T / sqrt(d))
// V_{<=t}; [Suffix page, §2 and the end of §5]: one byte an element behind a block
// table).
//
// One CTA a (token row, query head): tiles of 128 keys, a thread a key for the
// scores, a running maximum and sum, then a thread an element of the output.
//
// Pages: [KV page] "为什么自回归推理缓存 KV，而不缓存历史 Q？";
//        [Suffix page] icman.com.cn news 64898.
#include "kernels.h"
#include "paged.cuh"

namespace gattn {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float e4m3_to_float(uint8_t c) {
  return f16x2_to_float2(e4m3x2_to_f16x2(c)).x;
}

template <int D>
__global__ void __launch_bounds__(kThreads) attn_kernel(const __grid_constant__ PagedProblem pb, int min_new) {
  __shared__ float q[D], w[kThreads], red[8];
  __shared__ int who, bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x, h = blockIdx.y, g = h / pb.G;
  if (tid == 0) who = -1, bad = 0;
  __syncthreads();
  for (int r = tid; r < pb.B; r += kThreads) {
    const int a = pb.q_start[r], b = pb.q_start[r + 1];
    if (a < 0 || b > pb.T || b < a || b - a > pb.max_new) {
      if (t == 0) report(pb.status, GIST_ATTN_STATUS_BAD_BLOCK);
    } else if (t >= a && t < b) {
      atomicMax(&who, r);
    }
  }
  __syncthreads();
  const int r = who;
  if (r < 0 || pb.q_start[r + 1] - pb.q_start[r] < min_new) return;
  const int kv_len = pb.kv_len[r];
  const int pos = kv_len - (pb.q_start[r + 1] - t);
  const bool fits = kv_len <= pb.W * pb.block_len;
  const bf16* src = static_cast<const bf16*>(pb.q) + ((int64_t)t * pb.Hq + h) * D;
  if (tid < D / 2) {
    float sn, cs;
    __sincosf(turn_angle(pos, pb.turn[tid]), &sn, &cs);
    const float x = __bfloat162float(src[tid]), y = __bfloat162float(src[tid + D / 2]);
    q[tid] = x * cs - y * sn;
    q[tid + D / 2] = y * cs + x * sn;
  }
  __syncthreads();
  float m = -INFINITY, sum = 0.f, acc = 0.f;
  for (int k0 = 0; k0 <= pos && fits; k0 += kThreads) {
    const int key = k0 + tid;
    float s = -INFINITY, vs = 0.f;
    int64_t row = 0;
    if (key <= pos) {
      const int blk = pb.block_table[(int64_t)r * pb.W + key / pb.block_len];
      if (blk < 0 || blk >= pb.num_blocks) {
        bad = 1;
      } else {
        const int64_t plane = ((int64_t)blk * pb.L + pb.layer) * 2 * pb.Hkv + g;
        row = (plane * pb.block_len + key % pb.block_len) * D;
        float dot = 0.f;
        for (int e = 0; e < D; e += 4) {
          const uint32_t c = *reinterpret_cast<const uint32_t*>(pb.pool + row + e);
          for (int i = 0; i < 4; ++i) dot += q[e + i] * e4m3_to_float((uint8_t)(c >> (8 * i)));
        }
        s = dot * (pb.scale[plane] * pb.scale_log2);
        vs = pb.scale[plane + pb.Hkv];
      }
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float used = mn == -INFINITY ? 0.f : mn;
    const float p = key <= pos ? exp2f(s - used) : 0.f;
    const float f = exp2f(m - used);
    m = mn;
    float ps = p;
    for (int o = 16; o; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
    if (lane == 0) red[4 + warp] = ps;
    w[tid] = p * vs;
    __syncthreads();
    sum = sum * f + ((red[4] + red[5]) + (red[6] + red[7]));
    acc *= f;
    if (tid < D && !bad) {
      for (int i = 0; i < min(kThreads, pos + 1 - k0); ++i) {
        const int kk = k0 + i, blk = pb.block_table[(int64_t)r * pb.W + kk / pb.block_len];
        const int64_t plane = ((int64_t)blk * pb.L + pb.layer) * 2 * pb.Hkv + pb.Hkv + g;
        acc += w[i] * e4m3_to_float(pb.pool[(plane * pb.block_len + kk % pb.block_len) * D + tid]);
      }
    }
    __syncthreads();
  }
  if (tid == 0 && (bad || !fits)) report(pb.status, GIST_ATTN_STATUS_BAD_BLOCK);
  const bool none = bad || !fits || pos < 0;
  if (tid == 0 && !none && !(sum <= 3.0e38f)) report(pb.status, GIST_ATTN_STATUS_RANGE);
  if (tid < D)
    static_cast<bf16*>(pb.out)[((int64_t)t * pb.Hq + h) * D + tid] = __float2bfloat16(none ? 0.f : acc / sum);
}

}  // namespace

size_t paged_attn_workspace(const PagedProblem& pb) { return paged_decode_workspace(pb); }

int launch_paged_attn(const PagedProblem& pb, void* workspace, cudaStream_t stream) {
  if (pb.Hq > 65535) return GIST_ATTN_ERR_UNSUPPORTED;
  const int few = paged_decode_rows(pb) / pb.G;  // new tokens that the decode kernel takes
  if (few > 0) {
    const int rc = launch_paged_decode(pb, workspace, stream);
    if (rc != GIST_ATTN_OK || pb.max_new <= few) return rc;
  }
  const dim3 grid((unsigned)pb.T, (unsigned)pb.Hq);
  if (pb.d == 64)
    attn_kernel<64><<<grid, kThreads, 0, stream>>>(pb, few + 1);
  else
    attn_kernel<128><<<grid, kThreads, 0, stream>>>(pb, few + 1);
  return cudaGetLastError() == cudaSuccess ? GIST_ATTN_OK : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace gattn
