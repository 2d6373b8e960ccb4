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

}  // namespace kvq
