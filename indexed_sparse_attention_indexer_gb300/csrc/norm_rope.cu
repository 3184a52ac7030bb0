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
// has read, which makes x == out safe.  Vectors arrive through a ring of cp.async
// copies, each thread's own: no thread waits for another.
//
// What bounds it.  Issue slots: ~200 instructions a unit of 16 dims (conversions,
// statistics, rotation, codes), 53-58 % of them used at the two resident blocks that
// 115-128 registers a thread leave.  8192 tokens of 64 + 1 heads of 128: 55.5 us, 5.0
// TB/s, 73 % of the measured copy rate.  65537 latent rows to FP8: 62.6 us, 2.1 TB/s (31
// %); there a quarter of the lanes' units lie past the vector (36 units on 16 lanes of three),
// and every chunk of 8 dims computes its scale and reciprocal anew.  One token with 65 heads:
// 6.8 us, a launch.
#include "kernels.h"
#include "norm_rope.h"
#include "tc_common.cuh"

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
// vectors in a row.
struct Deal {
  int64_t blocks;
  int steps;
};
// steps whose vectors are on their way into shared memory (each thread's own
// slots: no thread waits for another)
template <int U>
constexpr int kDepth = U <= 2 ? 4 : 2;
template <int U>
constexpr int kRingBytes = kDepth<U> * U * 2 * kThreads * 16;

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

// What a unit's eight pairs are turned by, weights included:
//   z_a = t_a a - t_b b + ea,  z_b = t_a c + t_b d + eb   (t: the normed vector
// before weight and bias; dims outside the rotation: t_a a + ea and t_b d + eb alone).
// (b is kept negated.)  Half-split: pair p is dim p of the unit's first and of its second chunk;
// interleaved: dims 2 (p % 4) and 2 (p % 4) + 1 of chunk p / 4.
template <bool LAYER>
struct Turn {
  float a[8], b[8], c[8], d[8], ea[LAYER ? 8 : 1], eb[LAYER ? 8 : 1];
};
template <bool IL>
__device__ __forceinline__ int chunk_a(int p) { return IL ? p >> 2 : 0; }
template <bool IL>
__device__ __forceinline__ int chunk_b(int p) { return IL ? p >> 2 : 1; }
template <bool IL>
__device__ __forceinline__ int dim_a(int p) { return IL ? 2 * (p & 3) : p; }
template <bool IL>
__device__ __forceinline__ int dim_b(int p) { return IL ? 2 * (p & 3) + 1 : p; }

// One side of a call.  U: units a lane holds; `lanes` (a power of two) lanes
// share a vector; NORM: dsi_norm; IL: interleaved pairs; QUANT: quantised out.
template <int U, int NORM, bool IL, bool QUANT>
__device__ __forceinline__ void side(const dsi_heads& s, const RopeArgs& a, int64_t block, const Deal& deal,
                                     int lanes, uint4* ring, unsigned int* s_max, int* err) {
  constexpr bool LAYER = NORM == DSI_NORM_LAYER;
  const int lane = threadIdx.x & 31, per_warp = 32 / lanes;
  const int sub = lane & (lanes - 1), slot = lane / lanes;
  const int chunks = a.d >> 3, hc = a.rope_dim >> 4, r0 = a.rope_offset >> 3;
  const int64_t vectors = a.n_rows * s.n_heads;

  int off[U][2];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) off[i][h] = dim_of(sub + i * lanes, h, hc, r0, chunks);
  auto normed = [&](int i, int h) { return NORM != DSI_NORM_NONE && (unsigned)off[i][h] < (unsigned)s.norm_dim; };

  const int64_t first = ((block * kWarps + (threadIdx.x >> 5)) * deal.steps) * per_warp + slot;
  // Token and head of this lane's vector, and where it is; moved on by per_warp
  // vectors a step (counts below 2^31 divide in 32 bits).
  struct Cursor {
    int64_t row;
    int head, left;            // steps that have a vector, from here on
    const bf16* x;
  };
  Cursor at;
  at.row = s.n_heads == 1 ? first : vectors <= 0x7fffffff ? (int64_t)((unsigned)first / (unsigned)s.n_heads)
                                                         : first / s.n_heads;
  at.head = (int)(first - at.row * s.n_heads);
  at.left = first >= vectors ? 0 : (int)min((int64_t)deal.steps, (vectors - first + per_warp - 1) / per_warp);
  at.x = static_cast<const bf16*>(s.x) + at.row * s.ld_row + at.head * s.ld_head;
  const int64_t dx = s.n_heads == 1 ? per_warp * s.ld_row : per_warp * s.ld_head;
  auto advance = [&](Cursor& c) {
    --c.left;
    if (s.n_heads == 1) {
      c.row += per_warp;
    } else {
      c.head += per_warp;
      if (c.head >= s.n_heads) {
        const int q = c.head / s.n_heads;
        c.row += q;
        c.head -= q * s.n_heads;
        c.x = static_cast<const bf16*>(s.x) + c.row * s.ld_row + c.head * s.ld_head;
        return;
      }
    }
    c.x += dx;
  };
  // A vector's copies begin up to kDepth steps before it is used, whether or not it
  // will be skipped.
  Cursor ahead = at;
  uint32_t put = tc::smem_u32(ring + threadIdx.x);
  const uint32_t ring0 = put;
  constexpr uint32_t kSlot = U * 2 * kThreads * 16, kEnd = kDepth<U> * kSlot;
  auto issue = [&]() {
    if (ahead.left > 0) {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (off[i][h] >= 0) tc::cp_async_16(put + (i * 2 + h) * kThreads * 16, ahead.x + off[i][h]);
      advance(ahead);
    }
    put = put + kSlot == ring0 + kEnd ? ring0 : put + kSlot;
    tc::cp_async_commit();
  };
  auto token_of = [&](const Cursor& c, int64_t& pos, int64_t& dst) {
    pos = 0;
    dst = -1;                  // (no vector any more: not live)
    if (c.left > 0) {
      pos = __ldg(a.positions + c.row);
      dst = s.dst_rows ? __ldg(s.dst_rows + c.row) : c.row;
    }
  };
  int64_t pos, dst;
  token_of(at, pos, dst);
#pragma unroll
  for (int i = 0; i < kDepth<U>; ++i) issue();

  const float* cs = a.table;
  const int half = a.rope_dim >> 1;
  auto angles = [&](int u, float (&c)[8], float (&sn)[8]) {
    if (!IL) {
      load8(cs + u * 8, c);
      load8(cs + half + u * 8, sn);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + (u + h * hc) * 4));
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + half + (u + h * hc) * 4));
        c[4 * h] = c4.x; c[4 * h + 1] = c4.y; c[4 * h + 2] = c4.z; c[4 * h + 3] = c4.w;
        sn[4 * h] = s4.x; sn[4 * h + 1] = s4.y; sn[4 * h + 2] = s4.z; sn[4 * h + 3] = s4.w;
      }
    }
  };
  const bool turns = sub < hc;                  // the lane's only unit is rotated
  auto turn_of = [&](Turn<LAYER>& t) {          // of the lane's only unit
    float c[8], sn[8], w[2][8], b[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int e = 0; e < 8; ++e) { w[h][e] = 1.f; b[h][e] = -0.f; }   // (-0 added keeps every value)
      if (normed(0, h) && s.weight) load8(s.weight + off[0][h], w[h]);
      if (LAYER && normed(0, h) && s.bias) load8(s.bias + off[0][h], b[h]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) { c[e] = 1.f; sn[e] = 0.f; }
    if (turns) angles(sub, c, sn);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float wa = w[chunk_a<IL>(p)][dim_a<IL>(p)], wb = w[chunk_b<IL>(p)][dim_b<IL>(p)];
      t.a[p] = wa * c[p];
      t.d[p] = wb * c[p];
      t.b[p] = turns ? -(wb * sn[p]) : -0.f;
      t.c[p] = turns ? wa * sn[p] : -0.f;
      if (LAYER) {
        const float ba = b[chunk_a<IL>(p)][dim_a<IL>(p)], bb = b[chunk_b<IL>(p)][dim_b<IL>(p)];
        t.ea[p] = turns ? ba * c[p] - bb * sn[p] : ba;
        t.eb[p] = turns ? ba * sn[p] + bb * c[p] : bb;
      }
    }
  };
  // one unit a lane: what a token's heads share stays in registers
  constexpr bool kKeep = U == 1;
  [[maybe_unused]] Turn<LAYER> kept;
  bool live = false;

  const uint4* get = ring + threadIdx.x;
  int64_t token = -1;

#pragma unroll 1
  for (int step = 0; step < deal.steps; ++step) {
    // (a new token for any of the warp's vectors: the whole warp looks again)
    if (__any_sync(0xffffffffu, at.row != token)) {
      token = at.row;
      live = dst >= 0;
      if (live && (pos < 0 || pos >= a.table_rows || dst >= s.out_rows)) {
        if (sub == 0) report(err, kErrBounds);
        live = false;
      }
      cs = a.table + (live ? pos : 0) * a.rope_dim;
      if constexpr (kKeep) turn_of(kept);
    }
    const int head = at.head;
    const int64_t dst_now = dst;
    const bool here = at.left > 0;
    advance(at);
    if (at.row != token) token_of(at, pos, dst);     // the next step's, on their way meanwhile
    tc::cp_async_wait<kDepth<U> - 1>();
    float y[U][2][8];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (here && off[i][h] >= 0) raw = get[(i * 2 + h) * kThreads];
        bf16x8_to_f32(raw, y[i][h]);
      }
    get = get + U * 2 * kThreads == ring + threadIdx.x + kDepth<U> * U * 2 * kThreads ? ring + threadIdx.x
                                                                                      : get + U * 2 * kThreads;
    if (NORM != DSI_NORM_NONE) {
      const float inv_n = 1.f / (float)s.norm_dim;
      float sum = 0.f;
      if (LAYER) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (normed(i, h))
#pragma unroll
              for (int e = 0; e < 8; ++e) sum += y[i][h][e];
        const float mean = lanes_sum(sum, lanes) * inv_n;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (normed(i, h))
#pragma unroll
              for (int e = 0; e < 8; ++e) y[i][h][e] -= mean;
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (normed(i, h))
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(y[i][h][e], y[i][h][e], sum);
      const float r = rsqrtf(lanes_sum(sum, lanes) * inv_n + a.eps);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float rr = normed(i, h) ? r : 1.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][h][e] *= rr;
        }
    }
    if constexpr (kKeep) {
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        float& za = y[0][chunk_a<IL>(p)][dim_a<IL>(p)];
        float& zb = y[0][chunk_b<IL>(p)][dim_b<IL>(p)];
        // (a dim outside the rotation never meets its neighbour, which may be infinite)
        const float ta = za, tb = zb, oa = turns ? ta : 0.f, ob = turns ? tb : 0.f;
        za = fmaf(ta, kept.a[p], LAYER ? fmaf(ob, kept.b[p], kept.ea[p]) : ob * kept.b[p]);
        zb = fmaf(tb, kept.d[p], LAYER ? fmaf(oa, kept.c[p], kept.eb[p]) : oa * kept.c[p]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (normed(i, h)) {
            float w[8];
            if (s.weight) {
              load8(s.weight + off[i][h], w);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[i][h][e] *= w[e];
            }
            if (LAYER && s.bias) {
              load8(s.bias + off[i][h], w);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[i][h][e] += w[e];
            }
          }
        if (sub + i * lanes < hc) {
          float c[8], sn[8];
          angles(sub + i * lanes, c, sn);
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            float& za = y[i][chunk_a<IL>(p)][dim_a<IL>(p)];
            float& zb = y[i][chunk_b<IL>(p)][dim_b<IL>(p)];
            const float ta = za, tb = zb;
            za = fmaf(ta, c[p], -tb * sn[p]);
            zb = fmaf(tb, c[p], ta * sn[p]);
          }
        }
      }
    }
    if constexpr (!QUANT) {
      if (live) {
        bf16* out = static_cast<bf16*>(s.out) + dst_now * s.ld_out_row + head * s.ld_out_head;
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
    } else {
      const bool mx = s.out_dtype == DSI_MXFP8_E4M3;
      const int group = mx ? s.out_group : 128;        // dims of a scale
      const int groups = (a.d + group - 1) / group, gshift = 31 - __clz(group);
      // group maxima of this vector (a vector's lanes sit in one warp)
      unsigned int* gmax = s_max + (threadIdx.x / lanes) * groups;
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
        const int64_t vec = dst_now * s.n_heads + head;
        uint8_t* out = static_cast<uint8_t*>(s.out) + vec * a.d;
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
    issue();                    // into the slots just read
  }
  tc::cp_async_wait<0>();
}

template <int U, bool IL, bool QUANT>
__device__ __forceinline__ void side_of(const dsi_heads& s, const RopeArgs& a, int64_t block, const Deal& d,
                                        int lanes, uint4* ring, unsigned int* s_max, int* err) {
  if (s.norm == DSI_NORM_RMS) side<U, DSI_NORM_RMS, IL, QUANT>(s, a, block, d, lanes, ring, s_max, err);
  else if (s.norm == DSI_NORM_LAYER) side<U, DSI_NORM_LAYER, IL, QUANT>(s, a, block, d, lanes, ring, s_max, err);
  else side<U, DSI_NORM_NONE, IL, QUANT>(s, a, block, d, lanes, ring, s_max, err);
}

template <int U, bool IL, bool QUANT>
__global__ void __launch_bounds__(kThreads, 2)
norm_rope_kernel(const __grid_constant__ dsi_heads q, const __grid_constant__ dsi_heads k,
                 const __grid_constant__ RopeArgs a, int lanes, const __grid_constant__ Deal dq,
                 const __grid_constant__ Deal dk, int* err) {
  extern __shared__ uint4 ring[];
  __shared__ unsigned int s_max[QUANT ? kGroupSlots : 1];   // quantised out: group maxima
  const bool is_q = blockIdx.x < dq.blocks;
  const dsi_heads& s = is_q ? q : k;
  const Deal& d = is_q ? dq : dk;
  const int64_t block = is_q ? blockIdx.x : blockIdx.x - dq.blocks;
  if (QUANT && s.out_dtype != DSI_BF16) side_of<U, IL, true>(s, a, block, d, lanes, ring, s_max, err);
  else side_of<U, IL, false>(s, a, block, d, lanes, ring, s_max, err);
}

// One wave of resident blocks (two an SM) where the call is large enough: more
// steps a warp overlap more loads and reuse a token's angles.  (48 heads of 96, 1537
// tokens: 11.4 us so, 14.3 us with a quarter of the steps and four waves.)
constexpr int kMostSteps = 16;
Deal deal_out(int64_t rows, int heads, int lanes, int sms) {
  Deal d = {0, 1};
  if (rows == 0 || heads == 0) return d;
  const int64_t warp_steps = (rows * heads + 32 / lanes - 1) / (32 / lanes);
  const int64_t resident = (int64_t)sms * 2 * kWarps;
  const int64_t steps = (warp_steps + resident - 1) / resident;
  d.steps = (int)(steps < kMostSteps ? steps : kMostSteps);
  d.blocks = (warp_steps + (int64_t)kWarps * d.steps - 1) / ((int64_t)kWarps * d.steps);
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
  const Deal dq = deal_out(a.n_rows, q.n_heads, lanes, sms), dk = deal_out(a.n_rows, k.n_heads, lanes, sms);
  if (dq.blocks + dk.blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const bool quant = (q.n_heads && q.out_dtype != DSI_BF16) || (k.n_heads && k.out_dtype != DSI_BF16);
  using Kernel = void (*)(const dsi_heads, const dsi_heads, const RopeArgs, int, Deal, Deal, int*);
  static const Kernel kernels[4][2][2] = {
      {{norm_rope_kernel<1, false, false>, norm_rope_kernel<1, false, true>},
       {norm_rope_kernel<1, true, false>, norm_rope_kernel<1, true, true>}},
      {{norm_rope_kernel<2, false, false>, norm_rope_kernel<2, false, true>},
       {norm_rope_kernel<2, true, false>, norm_rope_kernel<2, true, true>}},
      {{norm_rope_kernel<3, false, false>, norm_rope_kernel<3, false, true>},
       {norm_rope_kernel<3, true, false>, norm_rope_kernel<3, true, true>}},
      {{norm_rope_kernel<4, false, false>, norm_rope_kernel<4, false, true>},
       {norm_rope_kernel<4, true, false>, norm_rope_kernel<4, true, true>}}};
  const Kernel kern = kernels[u - 1][a.interleaved ? 1 : 0][quant ? 1 : 0];
  const int ring = u == 1 ? kRingBytes<1> : u == 2 ? kRingBytes<2> : u == 3 ? kRingBytes<3> : kRingBytes<4>;
  if (ring > 40 * 1024) {      // with the group maxima, past what needs no asking
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (e != cudaSuccess) return e;
  }
  kern<<<(unsigned)(dq.blocks + dk.blocks), kThreads, ring, st>>>(q, k, a, lanes, dq, dk, err);
  note_launch();
  return cudaGetLastError();
}

}  // namespace dsi
