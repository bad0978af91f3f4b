// Parameters and launchers of the operators of a sparse decoding step: block
// tables (assign.cu), means of cache blocks (means.cu), scores of blocks
// (scores.cu) and the choice of blocks (select.cu).
#pragma once

#include "serving.h"

namespace mla {

// Error word, beside internal.h's bits: a request was left without blocks.
constexpr uint32_t kErrNoBlocks = 4u;

constexpr int kMaxAssignReqs = 8192;   // 24 B of shared memory each
struct AssignParams {
  int32_t* table;            // [num_reqs][max_blocks]
  int max_blocks;
  int32_t* held;             // [num_reqs]
  int32_t* shared;           // optional [num_reqs]
  int32_t* free_blocks;      // [capacity]
  int capacity;
  int32_t* free_count;
  BatchRows batch;           // rows: of slots (0: none wanted); per_req as everywhere
  int64_t* slots;            // optional [rows]
  uint32_t* err;             // optional
};
cudaError_t launch_assign_blocks(const AssignParams& p, cudaStream_t s);

struct MeansParams {
  const uint8_t* cache;
  int num_blocks;
  float kv_scale;
  BatchRows batch;
  const int32_t* block_table;    // [num_reqs][max_blocks]
  int max_blocks;
  uint16_t* means;               // [num_blocks][576] bf16
  uint32_t* err;                 // optional
  uint64_t wait_limit_ns;        // bound of every wait (a timeout sets kErrTimeout)
  int withhold;                  // test hook: this CTA of the ring kernel adds nothing up, so its loads' wait for room runs out (-1: none)
};
cudaError_t launch_block_means(const MeansParams& p, bool fp8, cudaStream_t s);

// Query absorption, launched dependently, into rows [qlat 512 | q_rope turned by
// its position 64] of 576 bf16; clears the error word.
struct ScoreQParams : QAbsorbParams {
  const uint16_t* q;       // [tokens][H][192], q_rope not rotated
  const int32_t* q_pos;    // [tokens]
  uint16_t* rows;          // [tokens * H][576]
  uint64_t rope_frac[kDr / 2];
};
cudaError_t launch_score_qabsorb(const ScoreQParams& p, cudaStream_t s);
// The same with the two E4M3 terms of qlat that decode attention over an FP8 cache
// takes (see DecodeQParams): tm_out and tm_out2 are theirs, qscale is set.
struct SparseQParams : ScoreQParams {
  CUtensorMap tm_out2;
  CUtensorMap tm_rows;     // the rows' bf16 qlat as (column, head, token), box 64 x 1 x 128
};
cudaError_t launch_sparse_qabsorb(const SparseQParams& p, cudaStream_t s);

constexpr int kScoreTile = 64;   // blocks of a tile
struct ScoreParams {
  CUtensorMap tm_q;              // the queries' rows as [rows * H][576], box 64 x 128
  BatchRows batch;
  const int32_t* block_table;    // [num_reqs][max_blocks]
  int max_blocks;
  int num_blocks;
  int num_heads;
  int per_item;                  // queries of an item: as many as have 128 rows at most
  const uint16_t* means;         // [num_blocks][576] bf16
  float scale_log2;
  uint64_t wait_limit_ns;        // bound of every wait (a timeout sets kErrTimeout)
  int withhold;                  // test hook: this CTA's mean rows are not loaded, so the waits for them run out (-1: none)
  void* out;                     // [rows][max_blocks]
  int out_bf16;
  // workspace
  uint32_t* err;
  int32_t* state;                // 0: a batch to be scored, else a cu_q that does not ascend
  uint4* s;                      // [max_blocks / 8][rows * H]: f16 scores in log2 units, less ml's maximum, 8 blocks a word
  float2* ml;                    // [max_blocks / 32][rows * H]: the maximum of 32 blocks and their sum of 2^(s - maximum)
  // for the attention over the chosen blocks, optional: the queries as requests of one row
  int keep;
  int32_t* lens;                 // [rows]: their lengths
  int32_t* cu;                   // [rows + 1]: their rows, where some of the batch's have no request
};
cudaError_t launch_block_scores(const ScoreParams& p, cudaStream_t s);

struct SelectParams {
  const void* scores;            // [rows][max_blocks] fp32 or bf16
  int scores_bf16;
  BatchRows batch;
  const int32_t* block_table;    // [num_reqs][max_blocks]
  int max_blocks;
  int keep, sinks, recent;
  int32_t* table;                // [rows][keep]
  int32_t* lens;                 // [rows]; with a plan they are there already
  uint32_t* err;                 // optional
  // a CTA more plans the attention over the chosen blocks (first: null for none)
  DecodeBatch decode;
  int clusters;
  int32_t* first;
  uint32_t* walks;
};
cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t s);

}  // namespace mla
