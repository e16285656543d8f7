// paged_api.cu -- the C ABI of the ragged serving step (plan, append, attention
// over the E4M3 paged cache): argument checks on the host, then one launch
// function each.  Nothing here allocates device memory or keeps state.
//
// Pages: [KV page] "为什么自回归推理缓存 KV，而不缓存历史 Q？";
//        [Suffix page] icman.com.cn news 64898.
#include <math.h>
#include <stdint.h>

#include "gist_attn.h"
#include "kernels.h"

namespace gattn {
namespace {

constexpr int kMaxAppendBlock = 1 << 20;  // a block's rows and bytes are counted in 32 bits

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The sizes every entry point reads.
int check_sizes(const gist_paged_dims& d) {
  if (d.num_requests < 0 || d.num_tokens < 0 || d.block_len < 1 || d.max_blocks < 1 ||
      d.num_blocks < 1)
    return GIST_ATTN_ERR_DIMS;
  if ((int64_t)d.num_blocks * d.block_len > INT32_MAX ||
      (int64_t)d.max_blocks * d.block_len > INT32_MAX)
    return GIST_ATTN_ERR_DIMS;
  return GIST_ATTN_OK;
}

// The model's dimensions as well (append and attention).
int check_dims(const gist_paged_dims* dm, PagedProblem* pb) {
  if (!dm) return GIST_ATTN_ERR_NULL;
  const gist_paged_dims& d = *dm;
  const int rc = check_sizes(d);
  if (rc != GIST_ATTN_OK) return rc;
  if (d.max_new < 1 || d.num_q_heads < 1 || d.num_kv_heads < 1 ||
      d.num_q_heads % d.num_kv_heads != 0 || d.num_layers < 1 || d.layer < 0 ||
      d.layer >= d.num_layers)
    return GIST_ATTN_ERR_DIMS;
  if (!(d.rope_theta > 0.f) || !isfinite(d.rope_theta) || !(d.softmax_scale >= 0.f) ||
      !isfinite(d.softmax_scale))
    return GIST_ATTN_ERR_DIMS;
  if (d.flags & ~GIST_ATTN_FLAG_PREROTATED) return GIST_ATTN_ERR_DIMS;
  if (d.head_dim != 64 && d.head_dim != 128) return GIST_ATTN_ERR_UNSUPPORTED;
  // planes of block_len rows are counted in 32 bits
  if ((double)d.num_blocks * d.num_layers * 2 * d.num_kv_heads > 2147483647.0)
    return GIST_ATTN_ERR_DIMS;
  pb->status = d.status;
  pb->B = d.num_requests;
  pb->T = d.num_tokens;
  pb->max_new = d.max_new;
  pb->Hq = d.num_q_heads;
  pb->Hkv = d.num_kv_heads;
  pb->G = d.num_q_heads / d.num_kv_heads;
  pb->d = d.head_dim;
  pb->block_len = d.block_len;
  pb->W = d.max_blocks;
  pb->num_blocks = d.num_blocks;
  pb->L = d.num_layers;
  pb->layer = d.layer;
  pb->flags = d.flags;
  const double scale = d.softmax_scale > 0.f ? (double)d.softmax_scale : 1.0 / sqrt((double)d.head_dim);
  pb->scale_log2 = (float)(scale * 1.4426950408889634);  // log2(e)
  const bool rotate = !(d.flags & GIST_ATTN_FLAG_PREROTATED);
  // theta^(-2j/d) as a product of two powers, of j's upper and lower three bits: 14 calls of
  // pow for 64 (0.8 us of these checks for 1.4), off by a unit or two of the last place more
  double low[8] = {1.0}, high[8] = {1.0};
  for (int k = 1; rotate && k < 8; ++k) {
    low[k] = pow((double)d.rope_theta, -2.0 * k / (double)d.head_dim);
    if (8 * k < d.head_dim / 2) high[k] = pow((double)d.rope_theta, -16.0 * k / (double)d.head_dim);
  }
  for (int j = 0; j < 64; ++j) {
    double turns = 0.0;  // theta_j / (2 pi) modulo 1
    if (rotate && j < d.head_dim / 2) {
      turns = high[j >> 3] * low[j & 7] * 0.15915494309189535;
      turns -= floor(turns);
    }
    const uint64_t turn = turns < 1.0 ? (uint64_t)ldexp(turns, 64) : 0;
    pb->turn[j] = turn + ((turn & 0x80000000u) << 1);  // the lower half as a signed number
  }
  return GIST_ATTN_OK;
}

}  // namespace
}  // namespace gattn

using gattn::aligned;
using gattn::PagedProblem;

extern "C" int gist_paged_plan(const int32_t* cached_len, const int32_t* new_len,
                               int32_t* block_table, const int32_t* free_blocks, int32_t num_free,
                               const int32_t* free_range, int32_t* q_start, int32_t* kv_len,
                               int32_t* slot, int32_t* position, int32_t* free_range_out,
                               const gist_paged_dims* dims, cudaStream_t stream) {
  if (!dims) return GIST_ATTN_ERR_NULL;
  const int rc = gattn::check_sizes(*dims);
  if (rc != GIST_ATTN_OK) return rc;
  if (num_free < 0) return GIST_ATTN_ERR_DIMS;
  if (dims->num_requests > gattn::kPlanRequests) return GIST_ATTN_ERR_UNSUPPORTED;
  const bool some = dims->num_requests > 0, tokens = dims->num_tokens > 0;
  if (!q_start || !free_range || !free_range_out ||
      (some && (!cached_len || !new_len || !block_table || !kv_len)) ||
      (num_free > 0 && !free_blocks) || (tokens && (!slot || !position)))
    return GIST_ATTN_ERR_NULL;
  if ((some && kv_len == cached_len) || free_range_out == free_range) return GIST_ATTN_ERR_DIMS;
  const void* ptrs[] = {cached_len, new_len, block_table, free_blocks, free_range, q_start,
                        kv_len,     slot,    position,    free_range_out, dims->status};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return GIST_ATTN_ERR_ALIGN;
  const gattn::PlanArgs a = {cached_len, new_len, block_table, free_blocks, free_range, q_start,
                             kv_len, slot, position, free_range_out, dims->status,
                             dims->num_requests, dims->num_tokens, dims->block_len,
                             dims->max_blocks, dims->num_blocks, num_free};
  return gattn::launch_paged_plan(a, stream);
}

extern "C" int gist_kv_append_fp8(const void* k_new, const void* v_new, void* kv_pool_e4m3,
                                  float* kv_scale, const int32_t* slot, const int32_t* position,
                                  const gist_paged_dims* dims, cudaStream_t stream) {
  PagedProblem pb{};
  const int rc = gattn::check_dims(dims, &pb);
  if (rc != GIST_ATTN_OK) return rc;
  if (pb.block_len > gattn::kMaxAppendBlock) return GIST_ATTN_ERR_UNSUPPORTED;
  if (pb.T == 0) return GIST_ATTN_OK;
  if (!k_new || !v_new || !kv_pool_e4m3 || !kv_scale || !slot ||
      (!position && !(pb.flags & GIST_ATTN_FLAG_PREROTATED)))
    return GIST_ATTN_ERR_NULL;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(kv_pool_e4m3, 16) ||
      !aligned(kv_scale, 4) || !aligned(slot, 4) || !aligned(position, 4) || !aligned(pb.status, 4))
    return GIST_ATTN_ERR_ALIGN;
  return gattn::launch_paged_append(pb, k_new, v_new, kv_pool_e4m3, kv_scale, slot, position, stream);
}

namespace gattn {
namespace {
int check_attn(const gist_paged_dims* dims, PagedProblem* pb) {
  const int rc = check_dims(dims, pb);
  if (rc != GIST_ATTN_OK) return rc;
  if (pb->block_len % 16 != 0 || pb->G > 128 || (int64_t)pb->W * pb->block_len > 1 << 30) return GIST_ATTN_ERR_UNSUPPORTED;
  // key tiles over all requests and heads are counted in 32 bits
  const double tiles = (double)pb->B * pb->Hkv * ((double)pb->W * pb->block_len / 128 + 1);
  if (tiles > 2147483647.0) return GIST_ATTN_ERR_UNSUPPORTED;
  return GIST_ATTN_OK;
}

int device_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return GIST_ATTN_ERR_LAUNCH;
  return GIST_ATTN_OK;
}

// New tokens of a request that paged_decode takes, at most (0: none of them).
int few_tokens(const PagedProblem& pb) { return paged_decode_rows(pb) / pb.G; }

// The two kernels run one after the other and share the workspace.
size_t attn_workspace(const PagedProblem& pb, int sms) {
  const int few = few_tokens(pb);
  const size_t a = few > 0 ? paged_decode_workspace(pb, sms) : 0;
  const size_t b = pb.max_new > few ? paged_prefill_workspace(pb, few + 1, sms) : 0;
  return a > b ? a : b;
}
}  // namespace
}  // namespace gattn

extern "C" size_t gist_attn_paged_workspace_bytes(const gist_paged_dims* dims) {
  PagedProblem pb{};
  int sms = 0;
  if (gattn::check_attn(dims, &pb) != GIST_ATTN_OK || pb.B == 0 || pb.T == 0 ||
      gattn::device_sms(&sms) != GIST_ATTN_OK)
    return 0;
  return gattn::attn_workspace(pb, sms);
}

extern "C" int gist_attn_paged_fp8kv(const void* q, const void* kv_pool_e4m3,
                                     const float* kv_scale, const int32_t* block_table,
                                     const int32_t* q_start, const int32_t* kv_len, void* out,
                                     void* workspace, size_t workspace_bytes,
                                     const gist_paged_dims* dims, cudaStream_t stream) {
  PagedProblem pb{};
  int rc = gattn::check_attn(dims, &pb);
  if (rc != GIST_ATTN_OK) return rc;
  if (pb.B == 0 || pb.T == 0) return GIST_ATTN_OK;
  if (!q || !kv_pool_e4m3 || !kv_scale || !block_table || !q_start || !kv_len || !out)
    return GIST_ATTN_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv_pool_e4m3, 16) || !aligned(out, 16) || !aligned(kv_scale, 4) ||
      !aligned(block_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
      !aligned(pb.status, 4))
    return GIST_ATTN_ERR_ALIGN;
  int sms = 0;
  rc = gattn::device_sms(&sms);
  if (rc != GIST_ATTN_OK) return rc;
  const size_t need = gattn::attn_workspace(pb, sms);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return GIST_ATTN_ERR_SCRATCH;
  pb.q = q;
  pb.out = out;
  pb.pool = static_cast<const uint8_t*>(kv_pool_e4m3);
  pb.scale = kv_scale;
  pb.block_table = block_table;
  pb.q_start = q_start;
  pb.kv_len = kv_len;
  const int few = gattn::few_tokens(pb);
  if (few > 0) {
    rc = gattn::launch_paged_decode(pb, workspace, sms, stream);
    if (rc != GIST_ATTN_OK) return rc;
  }
  return pb.max_new > few ? gattn::launch_paged_prefill(pb, workspace, few + 1, sms, stream) : GIST_ATTN_OK;
}
