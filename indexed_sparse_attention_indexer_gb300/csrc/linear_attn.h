// Internal launchers of linear attention with a decay for each head.  Argument
// validation happens in dsi_abi.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dsi {

struct LinearArgs {
  dsi_linear a;
  const int32_t* starts;     // prefill: [batch + 1], else null
  int64_t n_tokens;
  int batch, T;              // T: decode, tokens of every sequence
  int group;                 // heads to a key and value head
  int few;                   // prefill: sequences of so many tokens at most go token by token (-1: none)
  int* err;
};

// Slot that sequence b starts from / leaves its state in; -1: none.
__device__ __forceinline__ int64_t checked_slot(const LinearArgs& p, int s) {
  if (s < 0) return -1;
  if (s >= p.a.n_slots) { report(p.err, kErrBounds); return -1; }
  return s;
}
__device__ __forceinline__ int64_t in_slot(const LinearArgs& p, int b) {
  if (!p.a.state) return -1;
  return checked_slot(p, p.a.in_slots ? __ldg(p.a.in_slots + b) : b);
}
__device__ __forceinline__ int64_t out_slot(const LinearArgs& p, int b) {
  if (!p.a.state) return -1;
  const int32_t* s = p.a.out_slots ? p.a.out_slots : p.a.in_slots;
  return checked_slot(p, s ? __ldg(s + b) : b);
}

// Start of sequence b, held in 0 .. n_tokens.
__device__ __forceinline__ int held_start(const LinearArgs& p, int b) {
  const int s = __ldg(p.starts + b);
  return s < 0 ? 0 : s > p.n_tokens ? (int)p.n_tokens : s;
}
// First token and number of tokens of sequence b.
__device__ __forceinline__ void tokens_of(const LinearArgs& p, int b, int64_t& first, int& n) {
  if (!p.starts) {
    first = (int64_t)b * p.T;
    n = p.T;
    return;
  }
  const int s0 = held_start(p, b), s1 = held_start(p, b + 1);
  if (s0 != __ldg(p.starts + b) || s1 != __ldg(p.starts + b + 1) || s1 < s0) report(p.err, kErrBounds);
  first = s0;
  n = s1 > s0 ? s1 - s0 : 0;
}

// SMs of the current device.
inline int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    cudaGetLastError();
    return 152;                                // no device: a GB300's
  }
  return sms;
}

// Token by token: every sequence, or a prefill's of p.few tokens at most.
cudaError_t launch_linear_recurrent(const LinearArgs& p, cudaStream_t st);
size_t linear_prefill_workspace(int64_t n_tokens, int batch, int H, int dk, int dv);
cudaError_t launch_linear_prefill(const LinearArgs& p, void* ws, cudaStream_t st);

}  // namespace dsi
