// Launchers of the row-moving kernels (permute.cu).
#pragma once

#include "rows.cuh"

namespace moe {

struct PermuteArgs {
  int T, d, R, N, dtype;
  RowsIn tok;                // spread: x [T, d]; collect: rows [N, d]
  const float* w;            // [T, R] or null (1)
  const int32_t* row_slot;   // [N] (spread)
  const int32_t* slot_row;   // [T, R]
  RowsIn other;              // with dw: spread: rows [N, d]; collect: x [T, d]
  RowsOut out;               // spread: rows [N, d]; collect: y [T, d]
  float* dw;                 // [T, R] or null
};
cudaError_t launch_spread(const PermuteArgs& a, cudaStream_t s);
cudaError_t launch_collect(const PermuteArgs& a, cudaStream_t s);

}  // namespace moe
