// Attention over a prefix that the whole batch shares and over every sequence's
// own rows: one warp a head and query row.
#include "dense_mla.h"
#include "kernels.h"

namespace dsi {
namespace {

constexpr int kPer = DSI_D_QK / 32;              // dims of a lane: 2 * lane, 2 * lane + 1 of every 64

// Cache row of position p of sequence b; -1 (reported) for a bad page id.
__device__ __forceinline__ int64_t row_of(const CacheView& c, int b, int p, int* err) {
  if (!c.block_table) return (int64_t)b * c.s_max + p;
  const int page = __ldg(c.block_table + (int64_t)b * c.max_pages + p / c.page_size);
  if (page < 0 || page >= c.num_pages) { report(err, kErrBounds); return -1; }
  return (int64_t)page * c.page_size + p % c.page_size;
}

__global__ void __launch_bounds__(256)
prefix_mla_simt(DenseArgs a, CacheView prefix, const float* prefix_scale) {
  const int lane = threadIdx.x & 31;
  const int64_t at = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;   // (row, head)
  if (at >= (int64_t)a.rows * a.H) return;
  const int r = (int)(at / a.H);
  const int n_prefix = (int)visible_len(prefix, 0, 1, 0), n_own = (int)visible_len(a.c, r, 1, 0);
  float q[kPer], o[kPer - 2];
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) {
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(a.q + at * DSI_D_QK + i * 64 + lane * 2));
    q[2 * i] = x.x;
    q[2 * i + 1] = x.y;
  }
#pragma unroll
  for (int i = 0; i < kPer - 2; ++i) o[i] = 0.f;
  float top = -INFINITY, sum = 0.f;
  for (int s = 0; s < n_prefix + n_own; ++s) {
    const bool shared = s < n_prefix;
    const CacheView& c = shared ? prefix : a.c;
    const float* scale = shared ? prefix_scale : a.latent_scale;
    const int64_t row = row_of(c, shared ? 0 : r / a.T, shared ? s : s - n_prefix, a.err);
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      float2 x = make_float2(0.f, 0.f);
      if (row >= 0 && scale) {
        const uint8_t* code = reinterpret_cast<const uint8_t*>(c.latent) + row * DSI_D_QK + i * 64 + lane * 2;
        const __nv_fp8x2_e4m3 two = *reinterpret_cast<const __nv_fp8x2_e4m3*>(code);
        const float2 y = static_cast<float2>(two);
        const float f = __ldg(scale + row * 5 + i / 2);
        x = __bfloat1622float2(__floats2bfloat162_rn(y.x * f, y.y * f));
      } else if (row >= 0) {
        x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(c.latent + row * DSI_D_QK + i * 64 + lane * 2));
      }
      v[2 * i] = x.x;
      v[2 * i + 1] = x.y;
    }
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) l = fmaf(q[i], v[i], l);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) l += __shfl_xor_sync(0xffffffffu, l, m);
    l *= a.scale;
    const float next = fmaxf(top, l), keep = top == -INFINITY ? 0.f : expf(top - next);
    const float w = l == -INFINITY ? 0.f : expf(l - next);
    sum = sum * keep + w;
#pragma unroll
    for (int i = 0; i < kPer - 2; ++i) o[i] = fmaf(w, v[i], o[i] * keep);
    top = next;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < kPer / 2 - 1; ++i)
    *reinterpret_cast<__nv_bfloat162*>(a.out + at * DSI_D_LATENT + i * 64 + lane * 2) =
        __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
  if (a.lse && lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

size_t prefix_mla_workspace(int, int) { return 256; }

cudaError_t launch_prefix_mla(const DenseArgs& a, const CacheView& prefix, const float* prefix_scale,
                              cudaStream_t st) {
  const int64_t blocks = ((int64_t)a.rows * a.H + 7) / 8;
  prefix_mla_simt<<<(unsigned)blocks, 256, 0, st>>>(a, prefix, prefix_scale);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dsi
