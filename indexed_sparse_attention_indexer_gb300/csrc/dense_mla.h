// Internal launcher of attention over the whole latent cache or a window of
// it.  Argument validation happens in dsi_abi.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dsi {

struct DenseArgs {
  const bf16* q;               // [rows, H, 576]
  CacheView c;                 // decode: tokens_per_seq query rows to a sequence
  const float* latent_scale;   // FP8 rows: [positions, 5], else null
  int rows, T, H, decode;      // T: query rows to a sequence (a prefill: all rows)
  int64_t q_offset, window, n_sink;
  float scale;
  bf16* out;                   // [rows, H, 512]
  float* lse;                  // [rows, H] or null
  void* ws;                    // dense_mla_workspace() bytes, or null: no split
  int* err;
};

size_t dense_mla_workspace();
cudaError_t launch_dense_mla(const DenseArgs& a, cudaStream_t st);

}  // namespace dsi
