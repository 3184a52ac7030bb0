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
// scale groups of a block's vectors: a group is two units or more, and a lane
// holds at most four units
constexpr int kGroupSlots = kThreads * 2;

// Chunk (8 dims) `half` of unit u, or -1 past the end.  hc: chunks in half
// the rotation, starting at chunk r0; the other chunks follow in order.
__device__ __forceinline__ int chunk_of(int u, int half, int hc, int r0, int chunks) {
  if (u < hc) return r0 + u + half * hc;
  const int v = 2 * (u - hc) + half;
  const int c = v < r0 ? v : v + 2 * hc;
  return c < chunks ? c : -1;
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
template <int U>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(dsi_heads q, dsi_heads k, RopeArgs a, int lanes, int64_t q_blocks, int* err) {
  __shared__ unsigned int s_max[kGroupSlots];   // quantised out: group maxima
  const bool is_q = blockIdx.x < q_blocks;
  const dsi_heads& s = is_q ? q : k;
  const int64_t block = is_q ? blockIdx.x : blockIdx.x - q_blocks;
  const int64_t blocks = is_q ? q_blocks : gridDim.x - q_blocks;
  const int per_block = kThreads / lanes;
  const int sub = threadIdx.x & (lanes - 1), slot = threadIdx.x / lanes;
  const int chunks = a.d >> 3, hc = a.rope_dim >> 4, r0 = a.rope_offset >> 3;
  const int normed = s.norm == DSI_NORM_NONE ? 0 : s.norm_dim >> 3;
  const int64_t vectors = a.n_rows * s.n_heads;
  const bool quant = s.out_dtype != DSI_BF16;
  const int gchunks = s.out_dtype == DSI_MXFP8_E4M3 ? s.out_group >> 3 : 16;   // chunks of a scale
  const int groups = (chunks + gchunks - 1) / gchunks;
  // group maxima of this vector (a vector's lanes sit in one warp)
  unsigned int* gmax = s_max + slot * groups;

  // whole warps step together: the shuffles need every lane
  for (int64_t base = block * per_block; base < vectors; base += blocks * per_block) {
    const int64_t v = base + slot;
    bool live = v < vectors;
    const int64_t row = live ? v / s.n_heads : 0;
    const int head = live ? (int)(v - row * s.n_heads) : 0;
    int64_t pos = 0, dst = row;
    if (live) {
      pos = __ldg(a.positions + row);
      if (s.dst_rows) dst = __ldg(s.dst_rows + row);
      if (pos < 0 || pos >= a.table_rows || dst >= s.out_rows) {
        if (dst >= 0 && sub == 0) report(err, kErrBounds);
        live = false;
      }
      if (dst < 0) live = false;
    }
    const bf16* x = static_cast<const bf16*>(s.x) + row * s.ld_row + head * s.ld_head;
    float y[U][2][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = chunk_of(sub + i * lanes, h, hc, r0, chunks);
        if (live && c >= 0) {
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(x + c * 8), y[i][h]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][h][e] = 0.f;
        }
        if (c >= 0 && c < normed) {
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += s.norm == DSI_NORM_LAYER ? y[i][h][e] : y[i][h][e] * y[i][h][e];
        }
      }
    if (s.norm != DSI_NORM_NONE) {
      const float inv_n = 1.f / (float)s.norm_dim;
      float mean = 0.f, power = lanes_sum(sum, lanes) * inv_n;
      if (s.norm == DSI_NORM_LAYER) {
        mean = power;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = chunk_of(sub + i * lanes, h, hc, r0, chunks);
            if (c >= 0 && c < normed) {
#pragma unroll
              for (int e = 0; e < 8; ++e) { const float t = y[i][h][e] - mean; sum += t * t; }
            }
          }
        power = lanes_sum(sum, lanes) * inv_n;
      }
      const float r = rsqrtf(power + a.eps);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = chunk_of(sub + i * lanes, h, hc, r0, chunks);
          if (c >= 0 && c < normed) {
            float w[8];
            if (s.weight) load8(s.weight + c * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              y[i][h][e] = (y[i][h][e] - mean) * r;
              if (s.weight) y[i][h][e] *= w[e];
            }
            if (s.bias) {
              load8(s.bias + c * 8, w);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[i][h][e] += w[e];
            }
          }
        }
    }
    // rotation
    if (live) {
      const float* cs = a.table + pos * a.rope_dim;
      const int half = a.rope_dim >> 1;
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
    }
    if (!quant) {
      if (!live) continue;
      bf16* out = static_cast<bf16*>(s.out) + dst * s.ld_out_row + head * s.ld_out_head;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = chunk_of(sub + i * lanes, h, hc, r0, chunks);
          if (c < 0) continue;
          __align__(16) bf16 o8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o8[e] = __float2bfloat16(y[i][h][e]);
          *reinterpret_cast<uint4*>(out + c * 8) = *reinterpret_cast<const uint4*>(o8);
        }
      continue;
    }
    // largest magnitude of every scale group (order does not matter to a maximum)
    for (int g = sub; g < groups; g += lanes) gmax[g] = 0u;
    __syncwarp();
    if (live) {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = chunk_of(sub + i * lanes, h, hc, r0, chunks);
          if (c < 0) continue;
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[i][h][e]));
          atomicMax(gmax + c / gchunks, __float_as_uint(m));
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
          const int c = chunk_of(sub + i * lanes, h, hc, r0, chunks);
          if (c < 0) continue;
          const float m = __uint_as_float(gmax[c / gchunks]);
          float z[8];
          if (mx) {
            const float inv = __uint_as_float((uint32_t)(127 - mx_exponent(m)) << 23);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = y[i][h][e] * inv;
          } else {
            const float sc = __fdiv_rn(m, 448.f);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = sc > 0.f ? __fdiv_rn(y[i][h][e], sc) : 0.f;
          }
          uint32_t w2[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
                make_float2(z[4 * p], z[4 * p + 1]), __NV_SATFINITE, __NV_E4M3);
            const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(z[4 * p + 2], z[4 * p + 3]), __NV_SATFINITE, __NV_E4M3);
            w2[p] = (uint32_t)lo | ((uint32_t)hi << 16);
          }
          *reinterpret_cast<uint2*>(out + c * 8) = make_uint2(w2[0], w2[1]);
        }
    }
    __syncwarp();   // the maxima are read before the next vector clears them
  }
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
  const int per_block = kThreads / lanes, u = (units + lanes - 1) / lanes;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t cap = (int64_t)sms * 8;   // resident blocks of 256 threads
  int64_t qb = (a.n_rows * q.n_heads + per_block - 1) / per_block;
  int64_t kb = (a.n_rows * k.n_heads + per_block - 1) / per_block;
  if (qb + kb > cap) {                    // in proportion, one block at least for a side with work
    const int64_t all = qb + kb;
    qb = qb ? qb * cap / all + 1 : 0;
    kb = kb ? kb * cap / all + 1 : 0;
  }
  auto kern = u == 1 ? norm_rope_kernel<1>
              : u == 2 ? norm_rope_kernel<2>
              : u == 3 ? norm_rope_kernel<3>
                       : norm_rope_kernel<4>;
  kern<<<(unsigned)(qb + kb), kThreads, 0, st>>>(q, k, a, lanes, qb, err);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dsi
