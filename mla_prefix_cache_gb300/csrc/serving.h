// Parameters and launchers of the serving operators over the paged latent
// cache: appending new rows (append.cu) and decode attention (decode.cu).
#pragma once

#include "absorb.h"
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
  float inv_scale;               // 1 / kv_scale
  uint32_t* err;                 // optional
  int per_warp;                  // consecutive rows of a warp (set by the launcher)
  uint64_t rope_frac[kDr / 2];
};
cudaError_t launch_cache_append(AppendParams p, bool fp8, cudaStream_t s);

// The decode attention's clusters (two CTAs each): the persistent grid of a
// GB300's 152 SMs.  Each has two slots for the states of pieces that it shares
// with its neighbours.
constexpr int kDecodeClusters = 76;
constexpr int kDecodeSlots = 2 * kDecodeClusters;
constexpr int kItemRows = 128;   // (token, head) rows of a work item
constexpr int kWalkBytes = 128;  // a walk's share of the workspace

// What both kernels know of the batch's work.
struct DecodeBatch {
  BatchRows rows;
  const int64_t* segments;   // optional [..][3]: start, length, rope offset
  const int32_t* seg_ptr;    // [num_reqs + 1]
  int num_segments;
  int max_blocks;
  int num_heads;
};

// Latent attention (decode.cu).  Workspace arrays:
struct DecodeSpace {
  uint32_t* err;
  int32_t* first;        // [num_reqs + 2]: the requests' first work units, all units, clusters in use
  uint32_t* walks;       // [kDecodeClusters][kWalkBytes]: each cluster's walk over its work, at its first range
  uint8_t* qlat;         // bf16 [rows * H][512], or E4M3 [2][rows * H][512]
  float* qscale;         // [rows * H]: the E4M3 rows' scales
  float* lat;            // [rows * H][512]: states of rows whose keys one cluster had
  float* lat_lse;        // [rows * H]
  float* part;           // [kDecodeSlots][128][512]: states of shared rows
  float* part_lse;       // [kDecodeSlots][128]
};

// Query absorption and plan (headproj.cu).  As QAbsorbParams, but the E4M3 form
// has also the codes of what the first ones leave, e4m3(qlat / s - qlat8) (the two
// together hold qlat to about 2^-8 of itself), and the launch, a dependent one,
// sets the error word and leaves the attention's plan: `first` and `walks`.
struct DecodeQParams : QAbsorbParams {
  CUtensorMap tm_out2;     // the second codes, as tm_out
  DecodeBatch batch;
  int clusters;            // of the attention's grid
  int32_t* first;
  uint32_t* walks;
};
cudaError_t launch_decode_qabsorb(const DecodeQParams& p, cudaStream_t s);
// The attention's clusters on the current device: as many as are resident at once.
cudaError_t decode_clusters(int* clusters);

struct DecodeParams {
  CUtensorMap tm_q;      // qlat as [rows * H][512] bf16, or [2 * rows * H][512] bytes, box 128 B x 128
  CUtensorMap tm_s;      // the cache's rows in blocks of 128 B, box 128 B x 64 rows x 1
  CUtensorMap tm_o;      // the same, box 128 B x 32 rows x 4 (bf16) or 128 B x 64 rows x 2 (FP8)
  CUtensorMap tm_lat;    // lat as [rows * H][512], box 32 x 32
  CUtensorMap tm_part;   // part as [kDecodeSlots * 128][512], box 32 x 32
  DecodeBatch batch;
  DecodeSpace ws;
  const uint16_t* q;             // [rows][H][192], q_rope not rotated
  const int32_t* q_pos;          // [rows]
  const int32_t* block_table;    // [num_reqs][max_blocks]
  int num_blocks;
  float kv_scale;                // 1 for bf16 rows
  float scale_log2;
  uint64_t wait_limit_ns;        // bound of every wait (a timeout sets kErrTimeout)
  int withhold;                  // test hook: this cluster's loads of Q and scores' keys are not made, so the waits for them run out (-1: none)
  uint64_t rope_frac[kDr / 2];
};
cudaError_t launch_decode_attn(const DecodeParams& p, bool fp8, int clusters, cudaStream_t s);

// Joining of the pieces' states and the output projection (decode_out.cu):
// out[t][h] = out_scale sum_pieces w o W_UV,h, lse[t][h].
struct DecodeOutParams {
  CUtensorMap tm_w;      // kv_b_proj as [512][H * 256], box 64 x 128
  DecodeBatch batch;
  DecodeSpace ws;
  int tile;              // tokens of a CTA (at most 64)
  void* out;             // [rows][H][128]
  int out_bf16;
  float* lse;            // optional [rows][H]
  float out_scale;
};
cudaError_t launch_decode_out(const DecodeOutParams& p, cudaStream_t s);

}  // namespace mla
