// Rows of a ragged step that bring one token each at most (decode and combine
// kernels).
#pragma once

#include <stdint.h>

namespace kvq {

// Row of q and out that is batch row b's one token, from the offsets of a
// ragged step (which the kernel before may have written: coherent loads); -1:
// it has none, -2: its offsets are not usable.
__device__ __forceinline__ int single_token_row(const int32_t* cu, int num_tokens, int b) {
  const int start = cu[b], end = cu[b + 1];
  if (start < 0 || end < start || end > num_tokens || end - start > 1) return -2;
  return end > start ? start : -1;
}

}  // namespace kvq
