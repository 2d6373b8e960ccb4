// Host helpers shared by the files of entry points (defined in api.cu):
// argument checks, page mapping and the per-device error word.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"

namespace kvq {

int to_status(cudaError_t e);
bool aligned(const void* p, size_t a);
bool valid_dtype(int t);

// Checks a descriptor (no CUDA call); a kvq_status.
int check_cache(const kvq_cache_desc* c);

// Values' group size (group_v = 0 means the keys' group).
int group_v_of(const kvq_cache_desc* c);

// Page mapping of a cache (block_table NULL: slot layout).
void page_args(const kvq_cache_desc* c, const int32_t** table, int* shift, int* per_seq,
               int* num_pages);

// Device address of the error word on the current device; a kvq_status.
int error_word(uint32_t** out);

// One-shot test knob: the stage that the launch being prepared drops (-1:
// none), and the limit of its bounded waits.
int take_fault(unsigned long long* wait_limit_ns);

// Decode attention of batch rows that bring one token each at most: row b's is
// row cu_tokens[b] of q and out ([num_tokens][Hq][D]).
int decode_single_tokens(const kvq_cache_desc* cache, const void* q, int32_t q_dtype,
                         int32_t num_q_heads, int32_t num_tokens, const int32_t* cu_tokens,
                         const int32_t* seq_lens, int32_t max_seq_len, float sm_scale, void* out,
                         int32_t out_dtype, void* workspace, size_t workspace_bytes,
                         kvq_stream_t stream);

}  // namespace kvq
