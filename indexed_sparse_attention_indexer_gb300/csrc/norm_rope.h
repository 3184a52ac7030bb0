// Internal launcher of the head norm + rotation kernel.  Argument validation
// happens in dsi_abi.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dsi.h"

namespace dsi {

// What both sides of a call share.
struct RopeArgs {
  const float* table;        // [table_rows, rope_dim]: cosines, then sines
  const int64_t* positions;  // [n_rows]
  int64_t table_rows, n_rows;
  float eps;
  int d, rope_offset, rope_dim, interleaved;
};

// q / k: n_heads == 0 for a side that the call does not have.
cudaError_t launch_norm_rope(const dsi_heads& q, const dsi_heads& k, const RopeArgs& a, int* err,
                             cudaStream_t st);

}  // namespace dsi
