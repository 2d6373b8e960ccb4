// Kernel launches of a ragged serving step: planning, append, read-back and
// chunk attention (declared for the host entry points in api_serve.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"

namespace kvq {

// Rows one planning call takes (their prefix sums live in shared memory).
constexpr int kPlanRows = 8192;

struct PlanArgs {
  const int32_t* old_lens;
  const int32_t* new_lens;
  int batch, capacity, num_tokens, num_entries;
  int32_t* users;  // pages' user counts (NULL: slot layout)
  int32_t* table;  // block table (NULL: slot layout)
  int page_shift, pages_per_seq, num_pages;
  int32_t* lens;
  int32_t* cu;
  int4* map;
  uint32_t* err;
};

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream);

// One layer's packed cache as a number of equal blocks: the pages of the
// pool, or the batch rows' slots.
struct BlockCache {
  uint8_t* k_codes;
  uint8_t* v_codes;
  uint32_t* k_params;
  uint32_t* v_params;
  int kv_heads, head_dim, bits_k, bits_v, group, group_v;
  int gshift_k, gshift_v;  // log2 of the group sizes
  int blocks;        // pages, or batch rows
  int block_tokens;  // positions of a block
  bool rotate_keys;
};

struct RaggedArgs {
  BlockCache c;
  const void* k;  // append: inputs; read-back: outputs (written through)
  const void* v;
  int64_t k_stride, v_stride;  // elements from one token to the next
  int dtype, num_tokens, num_entries;
  const int4* map;
  uint32_t* err;
};

cudaError_t launch_append_ragged(const RaggedArgs& a, cudaStream_t stream);
cudaError_t launch_dequantize_ragged(const RaggedArgs& a, cudaStream_t stream);

// Chunk attention: binary16 pieces of an operand (1 to 3, see chunk.cuh), and
// what follows from it: rows of a unit of work and positions of a tile.
constexpr int unit_rows(int pieces) { return pieces == 3 ? 128 : 256; }
// (8-bit keys and values of head_dim 128 leave no room for a ring of four
// blocks beside tiles of 128)
constexpr int tile_tokens(int pieces, int head_dim, int bits_kv) {
  return pieces == 1 && !(head_dim == 128 && bits_kv == 16) ? 128 : 64;
}
// Steps that a unit's queries and output are worth in the division of work (20
// thousand cycles on B200 for bf16 and head_dim 128, a step about 5).  One value
// for all instances: measured with 1, 2, 3, 5 and 8, us on B200,
//   prefill of 4 rows of 2000-4000 tokens  bf16 569 534 510 489 526, head_dim 64
//     455 424 407 430 466, K8V8 726 704 676 637 641, f16 862 841 814 799 818,
//     f32 1470 1405 1425 1483 1575, head_dim 64 1146 1140 1158 1193 1248;
//   6 rows of 100-700 tokens  bf16 121 105 97 97 103, f16 150 131 120 116 125,
//     f32 252 225 226 237 244;
//   16 rows of 4 tokens  bf16 86 86 89 93 101, f16 135 136 140 144 152,
//     f32 158 155 158 164 172.
// (3 is within 6 % of the best of each.)
constexpr int kUnitCost = 3;
// Batch rows one call takes (their prefix sums lie in the tiles' memory).
constexpr int kChunkRows = 16384;

struct ChunkArgs {
  BlockCache c;
  const int32_t* table;  // block table (NULL: slot layout)
  int page_shift, pages_per_seq;
  int batch, capacity;
  const void* q;
  int64_t q_stride;
  int q_dtype, q_heads, gq, num_tokens;
  const int32_t* cu;
  const int32_t* seq_lens;
  int max_q_len, max_seq_len;
  bool causal;
  float sm_scale_log2;  // softmax scale times log2(e)
  void* out;
  int out_dtype;
  uint32_t* err;
  // division of work: a CTA takes at least min_share steps, or whole units
  bool whole_units;
  int min_share;
  int max_units;  // units of a batch row, at most
  // partial results of units cut by a share's border, two places per CTA
  // (0: a piece that continues a unit, 1: one that begins it)
  int part_rows;  // rows of a place
  int* ws_head;   // [grid][2][8]: valid, first token, kv head, first row, rows, last piece
  float2* ws_ml;  // [grid][2][part_rows]: (reference exponent, sum; -1: the row sees nothing)
  float* ws_o;    // [grid][2][part_rows][D]
  // Failure-detection test knob (kvq_debug_inject_wait_timeout): when
  // fault_stage is 0 or 1, that block of the first CTA's ring expects one
  // arrival more than its copies bring, so that the wait on it runs out; every
  // bounded wait of the launch gives up after wait_limit_ns.
  int fault_stage;
  uint32_t wait_limit_ns;
};

cudaError_t launch_chunk(const ChunkArgs& a, int pieces, int grid, cudaStream_t stream);

}  // namespace kvq
