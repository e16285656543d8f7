// paged_append.cu -- new tokens' K/V into the E4M3 paged pool
// ([KV page, "Reusable-state"]: the new K/V are appended to the cache;
// [Suffix page, §2 and the end of §5]: one byte an element).
//
// A block's scale is a power of two, so a code's precision does not depend on it
// (E4M3's four significant bits) and rescaling a block's earlier rows when its
// scale grows is exact but for subnormal codes.  It is chosen from the unrotated
// keys (|R(k)| <= sqrt 2 max |k|, hence 316 in 448's place): one pass finds it
// without a sine, and it does not hang on how a rotation rounds.
//
// A unit is the new tokens of one block (consecutive rows, some perhaps skipped), a
// KV head and K or V; one CTA takes the units whose first token lies in its `chunk`
// tokens (all of a prompt's block, a single token of a decoding step).  A thread holds
// elements j .. j + 3 and j + d/2 .. j + d/2 + 3 of a row, so it rotates its own pairs with
// four sines, and the rows stay in registers between the pass for the largest magnitude and
// the one that converts.
// Sine and cosine are carried to fp32's last place, though E4M3 keeps four bits: what
// they are off by moves values that lie next to the middle of two codes.  Of 1.8 million
// values 1.5 differ from the definition's (rotated in fp32 by torch: 0.8); by __sincosf,
// off by 2^-21, 7.5 did, in 26 us where this takes 29.
// Bound: a unit's chain of load, largest magnitude, sines, conversion and store, with
// barriers between and nothing of the next unit under way (issue is at 50 %, DRAM at 25 %;
// three bytes an element: bf16 in, E4M3 out): 14.2 k tokens of 8 heads of 128 in 29.5 us =
// 3.1 TB/s; few tokens: latency, 64 tokens in 6.7 us.
//
// Pages: [KV page] "为什么自回归推理缓存 KV，而不缓存历史 Q？";
//        [Suffix page] icman.com.cn news 64898.
#include "kernels.h"
#include "paged.cuh"

namespace gattn {
namespace {

constexpr int kThreads = 128;
constexpr int kHold = 8;  // rows a thread keeps in registers

struct PagedAppendParams {
  const bf16* x[2];  // k_new, v_new
  uint8_t* pool;
  float* scale;
  const int32_t* slot;
  const int32_t* position;
  int32_t* status;
  int T, Hkv, block_len, num_blocks, L, layer, chunk;
  uint64_t turn[64];
};

// Magnitude bits of a bf16 pair, and the larger of two pairs half by half.
__device__ __forceinline__ uint32_t abs2(uint32_t v) { return v & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t top2(uint32_t m, uint2 v) { return __vmaxu2(m, __vmaxu2(abs2(v.x), abs2(v.y))); }
constexpr uint32_t kInf = 0x7f80u;  // bf16 magnitudes from here on are not finite
// The same with 0 for what is not finite.
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
  const uint32_t lo = v & 0x7fffu, hi = (v >> 16) & 0x7fffu;
  return (lo < kInf ? lo : 0u) | (hi < kInf ? hi : 0u) << 16;
}

__device__ __forceinline__ uint32_t encode4(const float (&f)[4]) {
  return (uint32_t)e4m3x2(f[0], f[1]) | (uint32_t)e4m3x2(f[2], f[3]) << 16;
}
// As encode4 (which saturates infinities), with NaN codes for all that is not finite.
__device__ __forceinline__ uint32_t encode4_odd(const float (&f)[4]) {
  uint32_t r = encode4(f);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (!(fabsf(f[e]) <= 3.4e38f)) r = (r & ~(0xffu << (8 * e))) | 0x7fu << (8 * e);
  return r;
}
template <int D>
__global__ void __launch_bounds__(kThreads, 7)
    append_fp8_kernel(const __grid_constant__ PagedAppendParams prm) {
  constexpr int kLanes = D / 8;               // threads of a row
  constexpr int kRows = kThreads / kLanes;    // rows of a pass
  __shared__ uint32_t red[kThreads / 32], heads[kThreads / 32];
  __shared__ int run_len, pos_of[kThreads];  // positions of a unit's first kThreads tokens
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // heads vary fastest: CTAs that run together read whole token rows
  const int y = blockIdx.x % (2 * prm.Hkv), first = blockIdx.x / (2 * prm.Hkv);
  const int kv = y & 1, g = y >> 1;
  const int bl = prm.block_len, j = (tid % kLanes) * 4, row0 = tid / kLanes;
  const bf16* x = prm.x[kv];
  const int t0 = first * prm.chunk, t1 = min(t0 + prm.chunk, prm.T);
  const bool rotate = kv == 0 && prm.position != nullptr;
  // read once into registers: a constant read by 16 threads at 16 places is slow (and
  // read again and again, unless the compiler cannot know that it is one)
  uint64_t turn[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    turn[q] = rotate ? prm.turn[j + q] : 0;
    asm volatile("" : "+l"(turn[q]));
  }

  const unsigned rows_in_pool = (unsigned)prm.num_blocks * bl;
  auto skipped = [&](int s) { return (unsigned)s >= rows_in_pool; };  // negative or outside
  // Token t opens the block's unit unless an earlier token of the call lies in the
  // block: entry t - i of the slots is then s - i, with skipped ones between.
  {
    const int t = t0 + tid;
    bool head = false;
    if (t < t1) {
      const int s = prm.slot[t];
      head = !skipped(s);
      if (!head && s >= 0) report(prm.status, GIST_ATTN_STATUS_BAD_BLOCK);
      if (head && t > 0) {
        const int off = s % bl, before = prm.slot[t - 1];
        if (off > 0 && before == s - 1) head = false;
        if (off > 0 && skipped(before))
          for (int i = 2; i <= min(off, t) && head; ++i) head = prm.slot[t - i] != s - i;
      }
    }
    const uint32_t set = __ballot_sync(0xffffffffu, head);
    if (lane == 0) heads[warp] = set;
    __syncthreads();
  }
  uint32_t left = 0;
  for (int w = -1;;) {
    while (left == 0 && ++w < kThreads / 32) left = heads[w];
    if (w == kThreads / 32) break;
    const int h = w * 32 + __ffs(left) - 1;
    left &= left - 1;
    const int t = t0 + h, s = prm.slot[t], blk = s / bl, off = s - blk * bl;
    // its tokens: entries t + e that are s + e, up to one that is neither that nor skipped
    const int most = min(bl - off, prm.T - t);
    int len = most;
    bool holes = false;
    for (int i = 0; i < most; i += kThreads) {
      if (tid == 0) run_len = most;
      __syncthreads();
      const int e = i + tid, v = e < most ? prm.slot[t + e] : s + e;
      if (!skipped(v) && v != s + e) atomicMin(&run_len, e);
      if (i == 0 && rotate && e < most) pos_of[e] = prm.position[t + e];
      holes |= __syncthreads_or(skipped(v));
      len = run_len;
      __syncthreads();
      if (len < most) break;
    }
    if (holes) {  // up to the last token that is there
      if (tid == 0) run_len = 0;
      __syncthreads();
      for (int e = tid; e < len; e += kThreads)
        if (!skipped(prm.slot[t + e])) atomicMax(&run_len, e + 1);
      __syncthreads();
      len = run_len;
      __syncthreads();
    }
    auto live = [&](int i) { return i < len && (!holes || !skipped(prm.slot[t + i])); };

    const int64_t plane = (((int64_t)blk * prm.L + prm.layer) * 2 + kv) * prm.Hkv + g;
    const bf16* src = x + ((int64_t)t * prm.Hkv + g) * D + j;
    const int64_t pitch = (int64_t)prm.Hkv * D;
    uint2 lo[kHold], hi[kHold];
    uint32_t big = 0;
#pragma unroll
    for (int p = 0; p < kHold; ++p) {
      const int i = row0 + p * kRows;
      lo[p] = hi[p] = make_uint2(0, 0);
      if (live(i)) {
        lo[p] = *reinterpret_cast<const uint2*>(src + i * pitch);
        hi[p] = *reinterpret_cast<const uint2*>(src + i * pitch + D / 2);
      }
    }
#pragma unroll
    for (int p = 0; p < kHold; ++p) big = top2(top2(big, lo[p]), hi[p]);
    for (int i = row0 + kHold * kRows; i < len; i += kRows)
      if (live(i)) {
        big = top2(big, *reinterpret_cast<const uint2*>(src + i * pitch));
        big = top2(big, *reinterpret_cast<const uint2*>(src + i * pitch + D / 2));
      }
    auto over_cta = [&](uint32_t pair) {  // the largest half of all threads' pairs
      const uint32_t m = __reduce_max_sync(0xffffffffu, max(pair & 0xffffu, pair >> 16));
      if (lane == 0) red[warp] = m;
      __syncthreads();
      return max(max(red[0], red[1]), max(red[2], red[3]));
    };
    const float old = off > 0 ? prm.scale[plane] : 0.f;
    uint32_t top = over_cta(big);
    const bool odd = top >= kInf;  // something is not finite: the largest of the rest
    if (odd) {
      uint32_t m = 0;
      for (int i = row0; i < len; i += kRows)
        if (live(i))
          for (int e = 0; e < D; e += D / 2) {
            const uint2 x2 = *reinterpret_cast<const uint2*>(src + i * pitch + e);
            m = __vmaxu2(m, __vmaxu2(finite2(x2.x), finite2(x2.y)));
          }
      __syncthreads();
      top = over_cta(m);
    }
    // the smallest power of two >= top / limit (limit / 512 = 0.875 or 0.6171875)
    const uint32_t bits = top << 16;
    const int e2 = (int)(bits >> 23) - 126;  // top = m 2^e2, m in [0.5, 1)
    const float m = __uint_as_float((bits & 0x7fffffu) | 0x3f000000u);
    int e = m <= (rotate ? 0.6171875f : 0.875f) ? e2 - 9 : e2 - 8;
    e = top == 0 ? -100 : min(max(e, -100), 119);
    const float need = __uint_as_float((uint32_t)(e + 127) << 23);
    const float scale = fmaxf(old, need);
    uint8_t* dst = prm.pool + plane * bl * D + (int64_t)off * D + j;
    if (off > 0 && scale > old) {  // the earlier rows (skipped ones too) at the larger scale
      const float f = old / scale;
      uint4* rows = reinterpret_cast<uint4*>(prm.pool + plane * bl * D);
      auto turn4 = [&](uint32_t c) {
        const float2 a = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)c));
        const float2 b = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(c >> 16)));
        const float v[4] = {a.x * f, a.y * f, b.x * f, b.y * f};
        return encode4_odd(v);
      };
#pragma unroll 4
      for (int i = tid; i < (off + (holes ? len : 0)) * (D / 16); i += kThreads) {
        if (i >= off * (D / 16) && live(i / (D / 16) - off)) continue;
        const uint4 c = rows[i];
        rows[i] = make_uint4(turn4(c.x), turn4(c.y), turn4(c.z), turn4(c.w));
      }
    }
    if (tid == 0 && (off == 0 || scale > old)) prm.scale[plane] = scale;
    const float inv = 1.f / scale;
    const uint64_t inv2 = f2_make(inv, inv);
    auto put = [&](int i, uint2 a, uint2 b) {
      // divided by the scale before (or, as a factor of sine and cosine, in) the
      // rotation: the largest bf16 values cannot overflow
      uint64_t f0 = bf16x2_to_f2(a.x), f1 = bf16x2_to_f2(a.y), h0 = bf16x2_to_f2(b.x), h1 = bf16x2_to_f2(b.y);
      if (rotate) {
        const int pos = i < kThreads ? pos_of[i] : prm.position[t + i];
        uint64_t s0, s1, c0, c1;
        sincos_turns(turn_part(pos, turn[0]), turn_part(pos, turn[1]), s0, c0);
        sincos_turns(turn_part(pos, turn[2]), turn_part(pos, turn[3]), s1, c1);
        s0 = f2_mul(s0, inv2);
        s1 = f2_mul(s1, inv2);
        c0 = f2_mul(c0, inv2);
        c1 = f2_mul(c1, inv2);
        const uint64_t x0 = f0, x1 = f1;
        f0 = f2_sub(f2_mul(x0, c0), f2_mul(h0, s0));
        f1 = f2_sub(f2_mul(x1, c1), f2_mul(h1, s1));
        h0 = f2_fma(h0, c0, f2_mul(x0, s0));
        h1 = f2_fma(h1, c1, f2_mul(x1, s1));
      } else {
        f0 = f2_mul(f0, inv2);
        f1 = f2_mul(f1, inv2);
        h0 = f2_mul(h0, inv2);
        h1 = f2_mul(h1, inv2);
      }
      float f[4], h[4];
      f2_split(f0, f[0], f[1]);
      f2_split(f1, f[2], f[3]);
      f2_split(h0, h[0], h[1]);
      f2_split(h1, h[2], h[3]);
      uint32_t wf = encode4(f), wh = encode4(h);
      if (odd) {
        wf = encode4_odd(f);
        wh = encode4_odd(h);
      }
      uint8_t* row = dst + i * D;
      *reinterpret_cast<uint32_t*>(row) = wf;
      *reinterpret_cast<uint32_t*>(row + D / 2) = wh;
    };
#pragma unroll
    for (int p = 0; p < kHold; ++p) {
      const int i = row0 + p * kRows;
      if (live(i)) put(i, lo[p], hi[p]);
    }
    for (int i = row0 + kHold * kRows; i < len; i += kRows)
      if (live(i))
        put(i, *reinterpret_cast<const uint2*>(src + i * pitch),
            *reinterpret_cast<const uint2*>(src + i * pitch + D / 2));
    __syncthreads();  // the shared arrays are free again
  }
}

}  // namespace

int launch_paged_append(const PagedProblem& pb, const void* k_new, const void* v_new, void* pool,
                        float* scale, const int32_t* slot, const int32_t* position,
                        cudaStream_t stream) {
  PagedAppendParams prm{};
  prm.x[0] = static_cast<const bf16*>(k_new);
  prm.x[1] = static_cast<const bf16*>(v_new);
  prm.pool = static_cast<uint8_t*>(pool);
  prm.scale = scale;
  prm.slot = slot;
  prm.position = (pb.flags & GIST_ATTN_FLAG_PREROTATED) ? nullptr : position;
  prm.status = pb.status;
  prm.T = pb.T;
  prm.Hkv = pb.Hkv;
  prm.block_len = pb.block_len;
  prm.num_blocks = pb.num_blocks;
  prm.L = pb.L;
  prm.layer = pb.layer;
  for (int j = 0; j < 64; ++j) prm.turn[j] = pb.turn[j];
  // Tokens a CTA: one while there are few (each may be a unit of its own), up to a
  // block's worth where the tokens are many, so that no CTA is without a unit.
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  const int64_t share = (int64_t)pb.T * 2 * pb.Hkv / (8LL * sms);
  const int most = pb.block_len < 16 ? 16 : pb.block_len < kThreads ? pb.block_len : kThreads;
  prm.chunk = share < 1 ? 1 : share < most ? (int)share : most;
  const int64_t grid = ((int64_t)pb.T + prm.chunk - 1) / prm.chunk * 2 * pb.Hkv;
  if (grid > 0x7fffffff) return GIST_ATTN_ERR_UNSUPPORTED;
  if (pb.d == 64)
    append_fp8_kernel<64><<<(unsigned)grid, kThreads, 0, stream>>>(prm);
  else
    append_fp8_kernel<128><<<(unsigned)grid, kThreads, 0, stream>>>(prm);
  return cudaGetLastError() == cudaSuccess ? GIST_ATTN_OK : GIST_ATTN_ERR_LAUNCH;
}

}  // namespace gattn
