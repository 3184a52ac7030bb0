// Attention over the whole latent cache, or over a sliding window of it with
// the first positions visible.
//
// One warp takes one head of one query row: 18 query dims and 16 output dims
// a lane, the visible positions one after the other (a coalesced 1152-byte
// row, a shuffle sum for the logit, an online softmax step).  The eight heads
// of a block read the same rows through L1.  Bound by instruction issue.
#include "dense_mla.h"

#include "kernels.h"

namespace dsi {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Physical row of position p of sequence b; -1 (reported) for a bad page id.
__device__ __forceinline__ int64_t row_of(const CacheView& c, int b, int64_t p, int* err) {
  if (!c.block_table) return (int64_t)b * c.s_max + p;
  const int64_t pg = p / c.page_size;
  const int page = __ldg(c.block_table + (int64_t)b * c.max_pages + pg);
  if (page < 0 || page >= c.num_pages) { report(err, kErrBounds); return -1; }
  return (int64_t)page * c.page_size + (p - pg * c.page_size);
}

__global__ void __launch_bounds__(256)
dense_mla_simt(DenseArgs a) {
  const int r = blockIdx.x, h = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (h >= a.H) return;
  const int b = seq_of_row(a.c, r, a.decode);
  const int64_t n = visible_len(a.c, r, a.decode, a.q_offset);
  const int64_t lo = n > a.window ? n - a.window : 0;
  const int64_t sinks = a.n_sink < lo ? a.n_sink : lo;
  float q[18], o[16];
  const bf16* qrow = a.q + ((int64_t)r * a.H + h) * DSI_D_QK;
#pragma unroll
  for (int i = 0; i < 18; ++i) q[i] = __bfloat162float(qrow[i * 32 + lane]);
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int64_t j = 0; j < sinks + (n - lo); ++j) {
    const int64_t p = j < sinks ? j : lo + (j - sinks);
    const int64_t row = row_of(a.c, b, p, a.err);
    float c[18], dot = 0.f;
#pragma unroll
    for (int i = 0; i < 18; ++i) {
      const int d = i * 32 + lane;
      if (row < 0) {
        c[i] = 0.f;
      } else if (a.latent_scale) {
        __nv_fp8_e4m3 v;
        v.__x = reinterpret_cast<const uint8_t*>(a.c.latent)[row * DSI_D_QK + d];
        c[i] = __bfloat162float(__float2bfloat16(static_cast<float>(v) * a.latent_scale[row * 5 + d / 128]));
      } else {
        c[i] = __bfloat162float(a.c.latent[row * DSI_D_QK + d]);
      }
      dot = fmaf(q[i], c[i], dot);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
    const float v = dot * a.scale * kLog2e;
    const float m_new = fmaxf(m, v);
    const float f = m == -INFINITY ? 0.f : exp2f(m - m_new), pr = exp2f(v - m_new);
    m = m_new;
    l = l * f + pr;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = fmaf(pr, c[i], o[i] * f);
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  bf16* out = a.out + ((int64_t)r * a.H + h) * DSI_D_LATENT;
#pragma unroll
  for (int i = 0; i < 16; ++i) out[i * 32 + lane] = __float2bfloat16(o[i] * inv);
  if (a.lse && lane == 0) a.lse[(int64_t)r * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) / kLog2e;
}

}  // namespace

size_t dense_mla_workspace() { return 256; }

cudaError_t launch_dense_mla(const DenseArgs& a, cudaStream_t st) {
  dense_mla_simt<<<dim3((unsigned)a.rows, (unsigned)((a.H + 7) / 8)), 256, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dsi
