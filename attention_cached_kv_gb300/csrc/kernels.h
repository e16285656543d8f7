// kernels.h -- host-side launch interface between the C-ABI layer and the
// kernel translation units.  Host code only; no device code here.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gist_attn.h"

namespace gattn {

// Everything a kernel needs, already validated by the C-ABI layer.
struct Problem {
  const void* q;
  const void* k_new;
  const void* v_new;
  const void* kv_pool;
  const int32_t* item_ids;
  const int32_t* block_table;
  const int32_t* pos_offset;
  void* out;
  int32_t* status;
  int P, l, Hq, Hkv, G, d, block_len, blocks_per_pair, num_blocks, L, layer;
  int C;             // cached keys per pair
  const int32_t* gist_start;  // [P] or nullptr: the gist mask (streaming prefill only)
  int gist_len;
  int flags;                  // GIST_ATTN_FLAG_* (pre-rotated inputs: inv_freq is all 0)
  float scale_log2;  // softmax scale * log2(e)
  float inv_freq[64];  // rope_theta^(-2j/d), j < d/2
  double inv_freq_d[64];  // the same in double (the pool writers rotate in double)
};

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// The driver's tensor-map encoder, fetched once through the runtime (no libcuda link).
EncodeTiledFn encode_tiled_fn();

// Each returns GIST_ATTN_OK or a negative GIST_ATTN_ERR_* code.
int launch_prefill(const Problem& pb, cudaStream_t stream);
int launch_prefill_tc(const Problem& pb, cudaStream_t stream);
int launch_prefill_tc_fp8(const Problem& pb, const float* kv_scale, cudaStream_t stream);
int launch_prefill_long(const Problem& pb, cudaStream_t stream);
int launch_prefill_long_on(const Problem& pb, const void* q, const void* k, const void* v, int C,
                           bool f16, const float2* q_base, const float2* q_rel, cudaStream_t stream);
// The staged path (stage.cu): workspace layout, fit and launch (pre-pass + long kernel).
struct StageLayout {
  size_t base_off, rel_off, k_off, v_off, bytes;
};
StageLayout stage_layout(const Problem& pb);
int launch_staged(const Problem& pb, void* workspace, cudaStream_t stream);
int launch_decode(const Problem& pb, cudaStream_t stream);
int launch_decode_long(const Problem& pb, cudaStream_t stream);
int launch_decode_long_fp8(const Problem& pb, const float* kv_scale, cudaStream_t stream);
int launch_decode_short(const Problem& pb, cudaStream_t stream);
int launch_decode_short_fp8(const Problem& pb, const float* kv_scale, cudaStream_t stream);
int launch_gather(const Problem& pb, void* dst, cudaStream_t stream);
int launch_decode_long_stats(const Problem& pb, float* block_mass, cudaStream_t stream);
int launch_decode_gqa(const Problem& pb, cudaStream_t stream);
int launch_decode_gqa_fp8(const Problem& pb, const float* kv_scale, cudaStream_t stream);
int launch_decode_gqa_stats(const Problem& pb, float* block_mass, cudaStream_t stream);
int launch_append(const Problem& pb, void* pool, const int32_t* slot, cudaStream_t stream);
int launch_store(const Problem& pb, void* pool, const int32_t* first_row, const int32_t* store_pos,
                 cudaStream_t stream);
// The projections either side of the attention (gemm.cu).
int launch_qkv_rope(const Problem& pb, const void* x, const void* w, int d_model, void* q,
                    void* kn, void* vn, cudaStream_t stream);
int launch_out_proj(const Problem& pb, const void* attn, const void* w, int d_model, void* y,
                    cudaStream_t stream);

// ---- the ragged serving step (paged_*.cu) ----
struct PagedProblem {
  const void* q;
  void* out;
  const uint8_t* pool;  // E4M3
  const float* scale;
  const int32_t* block_table;
  const int32_t* q_start;
  const int32_t* kv_len;
  int32_t* status;
  int B, T, max_new, Hq, Hkv, G, d, block_len, W, num_blocks, L, layer, flags;
  float scale_log2;      // softmax scale * log2(e)
  uint64_t turn[64];     // RoPE: theta_j / 2 pi modulo 1, in units of 2^-64, the lower half
                         // signed (0: no rotation)
};
struct PlanArgs {
  const int32_t* cached_len;
  const int32_t* new_len;
  int32_t* block_table;
  const int32_t* free_blocks;
  const int32_t* free_range;
  int32_t* q_start;
  int32_t* kv_len;
  int32_t* slot;
  int32_t* position;
  int32_t* free_range_out;
  int32_t* status;
  int B, T, block_len, W, num_blocks, num_free;
};
constexpr int kPlanRequests = 16384;  // at most: the plan keeps 8 bytes a request in shared memory
int launch_paged_plan(const PlanArgs& a, cudaStream_t stream);
int launch_paged_append(const PagedProblem& pb, const void* k_new, const void* v_new, void* pool,
                        float* scale, const int32_t* slot, const int32_t* position,
                        cudaStream_t stream);
// Requests of at most paged_decode_rows query rows (new tokens x group): a run of
// key tiles a CTA (paged_decode.cu); the others: row tiles (paged_prefill.cu),
// which take the requests of min_new new tokens or more.
int launch_paged_decode(const PagedProblem& pb, void* workspace, int sms, cudaStream_t stream);
size_t paged_decode_workspace(const PagedProblem& pb, int sms);
int paged_decode_rows(const PagedProblem& pb);
int launch_paged_prefill(const PagedProblem& pb, void* workspace, int min_new, int sms,
                         cudaStream_t stream);
size_t paged_prefill_workspace(const PagedProblem& pb, int min_new, int sms);

// One token a request over a bf16 pool (paged_bf16.cu); pb.pool is the bf16 pool, pb.q_start may be null.
int launch_paged_bf16(const PagedProblem& pb, void* workspace, int sms, cudaStream_t stream);
size_t paged_bf16_workspace(const PagedProblem& pb, int sms);

// The blocks of a paged cache between steps (paged_pages.cu).
struct PagesArgs {
  const int32_t* cached_len;
  const int32_t* block_table;
  int32_t* table_out;  // compact: may be block_table
  int32_t* ids;        // [num_blocks]: reference counts, or new ids
  int32_t* src;        // compact: [num_blocks / 2]
  int32_t* dst;
  int32_t* count;
  int32_t* free_blocks;  // [num_blocks]
  int32_t* free_range;
  int32_t* status;
  int B, W, block_len, num_blocks;
};
struct ForkArgs {
  const int32_t* cached_len;
  const int32_t* parent;
  int32_t* block_table;
  const int32_t* free_blocks;
  const int32_t* free_range;
  int32_t* cached_len_out;
  int32_t* src;  // [B]
  int32_t* dst;
  int32_t* rows;
  int32_t* count;
  int32_t* free_range_out;
  int32_t* status;
  int B, W, block_len, num_blocks, num_free;
};
struct CopyArgs {
  uint4* pool;
  float* scale;  // or nullptr
  const int32_t* src;
  const int32_t* dst;
  const int32_t* rows;   // or nullptr: whole blocks
  const int32_t* count;  // device; or nullptr: n
  int32_t* status;
  int n, num_blocks, block_len;
  int planes, plane;  // of a block, and 16-byte pieces of a plane
};
int launch_pages_tables(const PagesArgs& a, bool compact, int sms, cudaStream_t stream);
int launch_pages_fork(const ForkArgs& a, cudaStream_t stream);
int launch_pages_copy(const CopyArgs& a, int sms, cudaStream_t stream);

// Projections of a few tokens with 4-bit weights (proj_w4.cu).
int launch_qkv_rope_w4(const PagedProblem& pb, const void* x, const void* w, const void* scale, const int32_t* position,
                       void* q, void* k_new, void* v_new, int d_model, int group, int sms, cudaStream_t stream);
int launch_out_proj_w4(const PagedProblem& pb, const void* attn, const void* w, const void* scale, void* y, int d_model,
                       int group, int sms, cudaStream_t stream);

// Whether the prefill kernel can hold this problem's tiles in shared memory.
bool prefill_fits(const Problem& pb);
bool prefill_tc_fits(const Problem& pb);
bool prefill_long_fits(const Problem& pb);
bool prefill_long_grid_ok(const Problem& pb, int rows);
bool staged_fits(const Problem& pb);
bool decode_fits(const Problem& pb);
bool decode_long_fits(const Problem& pb);
bool decode_short_fits(const Problem& pb);
bool decode_long_stats_fits(const Problem& pb);
bool decode_gqa_fits(const Problem& pb);
bool decode_gqa_stats_fits(const Problem& pb);

}  // namespace gattn
