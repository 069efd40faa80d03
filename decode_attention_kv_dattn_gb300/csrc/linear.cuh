// What the step and the prompt form of linear attention share.
#pragma once

#include "common.cuh"

namespace dattn {

// Cache row of call row b, or -1 (reported): the step then takes a state of
// zeros and the prompt form skips the row; neither writes a state.
__device__ __forceinline__ int state_row(const LinearArgs& a, int b, bool report) {
  const int row = a.stream_rows ? a.stream_rows[b] : b;
  if (row >= 0 && row < a.n_rows) return row;
  if (report) raise_error(a.err, ERR_INDEX);
  return -1;
}

}  // namespace dattn
