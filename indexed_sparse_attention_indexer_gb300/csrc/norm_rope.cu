// Head norms and position rotation in one pass, keys straight into the cache.
//
// One vector is one head of one token.  It is read once into registers, its
// norm statistics are a shuffle reduction in fp32, the rotation and the
// optional quantisation happen on the registers, and it is written once.
//
// Layout of a vector over lanes: the two halves of a half-split rotation are
// rope_dim / 2 dims apart, so the vector is cut into units of two 16-byte
// chunks that belong together (the chunk and its partner; dims outside the
// rotation two chunks in a row), and a lane owns whole units: no exchange
// between lanes for the rotation, and a lane writes only chunks that it alone
// has read, which makes x == out safe.
#include "kernels.h"
#include "norm_rope.h"

namespace dsi {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// scale groups of a block's vectors: a group is two units or more, and a lane
// holds at most four units
constexpr int kGroupSlots = kThreads * 2;
// below this a tile's reciprocal scale could overflow: divide instead
constexpr float kTinyScale = 1e-35f;

// How one side's vectors are dealt out: a warp takes `steps` times 32 / lanes
// vectors in a row; with steps > 1 they all are heads of one token.
struct Deal {
  int64_t blocks;
  int steps;
};

// First dim of chunk (8 dims) `half` of unit u, or -1 past the end.  hc: chunks
// in half the rotation, which starts at chunk r0; the other chunks follow in order.
__device__ __forceinline__ int dim_of(int u, int half, int hc, int r0, int chunks) {
  if (u < hc) return (r0 + u + half * hc) * 8;
  const int v = 2 * (u - hc) + half;
  const int c = v < r0 ? v : v + 2 * hc;
  return c < chunks ? c * 8 : -1;
}

__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// U: units a lane holds; `lanes` (a power of two) lanes share a vector.
// QUANT: either side has a quantised out.
template <int U, bool QUANT>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(const __grid_constant__ dsi_heads q, const __grid_constant__ dsi_heads k,
                 const __grid_constant__ RopeArgs a, int lanes, Deal dq, Deal dk, int* err) {
  __shared__ unsigned int s_max[QUANT ? kGroupSlots : 1];   // quantised out: group maxima
  const bool is_q = blockIdx.x < dq.blocks;
  const dsi_heads& s = is_q ? q : k;
  const int steps = is_q ? dq.steps : dk.steps;
  const int64_t block = is_q ? blockIdx.x : blockIdx.x - dq.blocks;
  const int lane = threadIdx.x & 31, per_warp = 32 / lanes;
  const int sub = lane & (lanes - 1), slot = lane / lanes;
  const int chunks = a.d >> 3, hc = a.rope_dim >> 4, r0 = a.rope_offset >> 3;
  const int normed = s.norm == DSI_NORM_NONE ? 0 : s.norm_dim;   // dims below it are normed
  const int64_t vectors = a.n_rows * s.n_heads;
  const bool quant = QUANT && s.out_dtype != DSI_BF16;
  const int group = s.out_dtype == DSI_MXFP8_E4M3 ? s.out_group : 128;      // dims of a scale
  const int groups = (a.d + group - 1) / group;
  const int gshift = 31 - __clz(group);
  // group maxima of this vector (a vector's lanes sit in one warp)
  unsigned int* gmax = s_max + (QUANT ? (threadIdx.x / lanes) * groups : 0);

  int off[U][2];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) off[i][h] = dim_of(sub + i * lanes, h, hc, r0, chunks);

  const int64_t first = ((block * kWarps + (threadIdx.x >> 5)) * steps) * per_warp + slot;
  bool live = first < vectors;
  // (counts below 2^31 divide in 32 bits)
  const int64_t row = !live ? 0 : vectors <= 0x7fffffff ? (int64_t)((unsigned)first / (unsigned)s.n_heads)
                                                       : first / s.n_heads;
  int head = live ? (int)(first - row * s.n_heads) : 0;
  int64_t pos = 0, dst = row;
  if (live) {
    pos = __ldg(a.positions + row);
    if (s.dst_rows) dst = __ldg(s.dst_rows + row);
    if (dst < 0) {
      live = false;
    } else if (pos < 0 || pos >= a.table_rows || dst >= s.out_rows) {
      if (sub == 0) report(err, kErrBounds);
      live = false;
    }
  }
  const float* cs = a.table + (live ? pos : 0) * a.rope_dim;
  const int half = a.rope_dim >> 1;
  const bf16* x = static_cast<const bf16*>(s.x) + row * s.ld_row + head * s.ld_head;

  for (int step = 0; step < steps; ++step, head += per_warp, x += per_warp * s.ld_head) {
    float y[U][2][8];
    uint4 raw[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        raw[i][h] = make_uint4(0, 0, 0, 0);
        if (live && off[i][h] >= 0) raw[i][h] = *reinterpret_cast<const uint4*>(x + off[i][h]);
      }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) bf16x8_to_f32(raw[i][h], y[i][h]);
    if (normed) {
      const bool layer = s.norm == DSI_NORM_LAYER;
      const float inv_n = 1.f / (float)normed;
      float mean = 0.f;
      if (layer) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if ((unsigned)off[i][h] < (unsigned)normed)
#pragma unroll
              for (int e = 0; e < 8; ++e) sum += y[i][h][e];
        mean = lanes_sum(sum, lanes) * inv_n;
        sum = 0.f;
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((unsigned)off[i][h] < (unsigned)normed)
#pragma unroll
            for (int e = 0; e < 8; ++e) { const float t = y[i][h][e] - mean; sum = fmaf(t, t, sum); }
      const float r = rsqrtf(lanes_sum(sum, lanes) * inv_n + a.eps);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((unsigned)off[i][h] < (unsigned)normed) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][h][e] = (y[i][h][e] - mean) * r;
            if (s.weight) {
              load8(s.weight + off[i][h], w);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[i][h][e] *= w[e];
            }
            if (s.bias) {
              load8(s.bias + off[i][h], w);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[i][h][e] += w[e];
            }
          }
    }
    // rotation
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = sub + i * lanes;
      if (u >= hc) continue;
      float c[8], sn[8];
      if (!a.interleaved) {
        load8(cs + u * 8, c);
        load8(cs + half + u * 8, sn);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float ya = y[i][0][e], yb = y[i][1][e];
          y[i][0][e] = ya * c[e] - yb * sn[e];
          y[i][1][e] = ya * sn[e] + yb * c[e];
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {      // chunk u + h * hc of the rotation: four pairs
          const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + (u + h * hc) * 4));
          const float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + half + (u + h * hc) * 4));
          c[0] = c4.x; c[1] = c4.y; c[2] = c4.z; c[3] = c4.w;
          sn[0] = s4.x; sn[1] = s4.y; sn[2] = s4.z; sn[3] = s4.w;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ya = y[i][h][2 * e], yb = y[i][h][2 * e + 1];
            y[i][h][2 * e] = ya * c[e] - yb * sn[e];
            y[i][h][2 * e + 1] = ya * sn[e] + yb * c[e];
          }
        }
      }
    }
    if (!quant) {
      if (live) {
        bf16* out = static_cast<bf16*>(s.out) + dst * s.ld_out_row + head * s.ld_out_head;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (off[i][h] < 0) continue;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(y[i][h][2 * e], y[i][h][2 * e + 1]);
              w[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(out + off[i][h]) = make_uint4(w[0], w[1], w[2], w[3]);
          }
      }
      continue;
    }
    if constexpr (QUANT) {
      // largest magnitude of every scale group (order does not matter to a maximum)
      for (int g = sub; g < groups; g += lanes) gmax[g] = 0u;
      __syncwarp();
      if (live) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float m[2] = {0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) m[h] = fmaxf(m[h], fabsf(y[i][h][e]));
          const int g0 = off[i][0] >> gshift, g1 = off[i][1] >> gshift;    // (-1 past the end)
          if (g0 >= 0) atomicMax(gmax + g0, __float_as_uint(g0 == g1 ? fmaxf(m[0], m[1]) : m[0]));
          if (g1 >= 0 && g1 != g0) atomicMax(gmax + g1, __float_as_uint(m[1]));
        }
      }
      __syncwarp();
      if (live) {
        const int64_t vec = dst * s.n_heads + head;
        uint8_t* out = static_cast<uint8_t*>(s.out) + vec * a.d;
        const bool mx = s.out_dtype == DSI_MXFP8_E4M3;
        for (int g = sub; g < groups; g += lanes) {
          const float m = __uint_as_float(gmax[g]);
          if (mx) static_cast<uint8_t*>(s.out_scale)[vec * groups + g] = (uint8_t)(mx_exponent(m) + 127);
          else static_cast<float*>(s.out_scale)[vec * groups + g] = __fdiv_rn(m, 448.f);
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (off[i][h] < 0) continue;
            const float m = __uint_as_float(gmax[off[i][h] >> gshift]);
            float inv, sc = 1.f;
            if (mx) {
              inv = __uint_as_float((uint32_t)(127 - mx_exponent(m)) << 23);   // 2^-X: exact
            } else {
              sc = __fdiv_rn(m, 448.f);
              inv = sc >= kTinyScale ? __frcp_rn(sc) : 0.f;
            }
            if (inv == 0.f && sc > 0.f) {        // a tiny tile: no reciprocal
#pragma unroll
              for (int e = 0; e < 8; ++e) y[i][h][e] = __fdiv_rn(y[i][h][e], sc);
              inv = 1.f;
            }
            uint32_t w2[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const float* z = y[i][h] + 4 * p;
              const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
                  make_float2(z[0] * inv, z[1] * inv), __NV_SATFINITE, __NV_E4M3);
              const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
                  make_float2(z[2] * inv, z[3] * inv), __NV_SATFINITE, __NV_E4M3);
              w2[p] = (uint32_t)lo | ((uint32_t)hi << 16);
            }
            *reinterpret_cast<uint2*>(out + off[i][h]) = make_uint2(w2[0], w2[1]);
          }
      }
      __syncwarp();   // the maxima are read before the next vector clears them
    }
  }
}

// A warp's heads of one token: more of them (up to kMostSteps warpfuls) reuse the
// token's positions and weights, fewer spread a small call over the device.
constexpr int kMostSteps = 8;
Deal deal(int64_t rows, int heads, int lanes, int sms) {
  const int per_warp = 32 / lanes;
  Deal d = {0, 1};
  if (rows == 0 || heads == 0) return d;
  const int64_t vectors = rows * heads;
  // at least eight warps an SM sub-partition
  while (d.steps < kMostSteps && heads % (per_warp * d.steps * 2) == 0 &&
         vectors / ((int64_t)per_warp * d.steps * 2) >= (int64_t)sms * 32)
    d.steps *= 2;
  const int64_t per_block = (int64_t)kWarps * per_warp * d.steps;
  d.blocks = (vectors + per_block - 1) / per_block;
  return d;
}

}  // namespace

cudaError_t launch_norm_rope(const dsi_heads& q, const dsi_heads& k, const RopeArgs& a, int* err,
                             cudaStream_t st) {
  const int chunks = a.d / 8, hc = a.rope_dim / 16;
  const int units = hc + (chunks - 2 * hc + 1) / 2;
  // lanes a vector: as many as leave at most four units a lane, and further
  // up only while no lane idles
  int lanes = 1;
  while (lanes < 32 && (units + lanes - 1) / lanes > 4) lanes *= 2;
  while (lanes < 32 && units % (lanes * 2) == 0) lanes *= 2;
  const int u = (units + lanes - 1) / lanes;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const Deal dq = deal(a.n_rows, q.n_heads, lanes, sms), dk = deal(a.n_rows, k.n_heads, lanes, sms);
  if (dq.blocks + dk.blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const bool quant = (q.n_heads && q.out_dtype != DSI_BF16) || (k.n_heads && k.out_dtype != DSI_BF16);
  auto kern = quant ? (u == 1   ? norm_rope_kernel<1, true>
                       : u == 2 ? norm_rope_kernel<2, true>
                       : u == 3 ? norm_rope_kernel<3, true>
                                : norm_rope_kernel<4, true>)
                    : (u == 1   ? norm_rope_kernel<1, false>
                       : u == 2 ? norm_rope_kernel<2, false>
                       : u == 3 ? norm_rope_kernel<3, false>
                                : norm_rope_kernel<4, false>);
  kern<<<(unsigned)(dq.blocks + dk.blocks), kThreads, 0, st>>>(q, k, a, lanes, dq, dk, err);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dsi
