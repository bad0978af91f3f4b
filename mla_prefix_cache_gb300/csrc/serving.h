// Parameters and launchers of the serving operators over the paged latent
// cache: appending new rows (append.cu) and decode attention (decode.cu).
#pragma once

#include "internal.h"

namespace mla {

// Rows of a batch of requests, described on the device: rows [first, last) of
// request r are cu_q[r] .. cu_q[r + 1], or, without cu_q, rows per_req of each.
// Values are clamped to [0, rows], so a bad cu_q cannot lead outside the rows.
struct BatchRows {
  const int32_t* cu_q;      // optional [num_reqs + 1]
  const int32_t* seq_lens;  // [num_reqs]: tokens of each request, the batch's rows included
  int num_reqs;
  int rows;
  int per_req;              // rows of each request when cu_q is null
};

struct AppendParams {
  const uint16_t* kv;            // [rows] rows of 576 bf16, row_stride elements apart
  int64_t row_stride;
  const int32_t* pos;            // [rows]
  const uint16_t* norm_weight;   // optional [512] bf16
  float norm_eps;
  BatchRows batch;
  const int32_t* block_table;    // [num_reqs][max_blocks]
  int max_blocks;
  uint8_t* cache;
  int num_blocks;
  float kv_scale;
  uint32_t* err;                 // optional
  uint64_t rope_frac[kDr / 2];
};
cudaError_t launch_cache_append(const AppendParams& p, bool fp8, cudaStream_t s);

struct DecodeParams {
  const uint16_t* q;             // [rows][H][192], q_rope not rotated
  const int32_t* q_pos;          // [rows]
  BatchRows batch;
  const int32_t* block_table;    // [num_reqs][max_blocks]
  int max_blocks;
  const uint8_t* cache;
  int num_blocks;
  float kv_scale;
  const int64_t* segments;       // optional [..][3]: start, length, rope offset
  const int32_t* seg_ptr;        // [num_reqs + 1]
  int num_segments;
  const uint16_t* kv_b_proj;     // [512][H * 256]
  int num_heads;
  float scale;
  void* out;                     // [rows][H][128]
  int out_bf16;
  float* lse;                    // optional [rows][H]
  uint32_t* err;
  uint64_t rope_frac[kDr / 2];
};
cudaError_t launch_decode(const DecodeParams& p, bool fp8, cudaStream_t s);

}  // namespace mla
