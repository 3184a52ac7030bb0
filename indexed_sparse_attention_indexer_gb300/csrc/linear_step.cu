// Linear attention with a decay for each head, token by token (the form of a
// decode step, and of a prefill's sequences of a few tokens): S = exp(g) S + k v^T, out = scale S^T q.
//
// A CTA takes one head of one sequence, or some columns of its state: 4 COLS of
// the dv columns, all dk rows, held in registers (a float4 of columns for every
// 8th group of rows a thread) from the load of the state to its store.  q and k of up to
// four tokens wait in shared memory; every thread sums its rows' share of q^T S,
// and the shares meet in shared memory once for those tokens.
//
// Bound by the state's bytes, each way once: 64 x 64 heads of 128 x 128, 537 MB, 88.8 us, 6.1 TB/s (91 %
// of the measured copy rate); in registers of 64-column halves 106 us, with four CTAs an SM (64
// registers a thread, some spilled) 126.  24 sequences x 4 tokens x 32 heads of 64 x 64, 26 MB: 7.4 us.
#include "kernels.h"
#include "linear_attn.h"

namespace dsi {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 4;                       // tokens between two meetings of the CTA

// DIMS: 64 or 128, what dk is at most.
template <int COLS, int DIMS>
__global__ void __launch_bounds__(kThreads)
linear_recurrent(const __grid_constant__ LinearArgs p, int parts) {
  constexpr int kRows = 32 / COLS;               // rows of a warp at a time
  constexpr int kSteps = DIMS / (kRows * kWarps);
  __shared__ __align__(16) float q_s[kTokens][DIMS], k_s[kTokens][DIMS];
  __shared__ float4 sum_s[kTokens][kWarps][32];
  const dsi_linear& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x % parts, bh = blockIdx.x / parts;
  const int b = bh / a.n_heads, h = bh - b * a.n_heads, hk = h / p.group;
  const int c = (part * COLS + lane % COLS) * 4;  // first of this thread's columns
  const bool col = c < a.dv;
  const int row0 = warp * kRows + lane / COLS;
  grid_dep_wait();
  int64_t first;
  int n;
  tokens_of(p, b, first, n);
  if (p.starts && n > p.few) return;             // the chunked kernel's
  const int64_t src = in_slot(p, b), dst = out_slot(p, b);
  const int64_t head = (int64_t)h * a.dk * a.dv, slot = (int64_t)a.n_heads * a.dk * a.dv;

  float4 s[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = row0 + i * kRows * kWarps;
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (src >= 0 && col && r < a.dk)
      s[i] = *reinterpret_cast<const float4*>(a.state + src * slot + head + (int64_t)r * a.dv + c);
  }
  const float d1 = expm1f(__ldg(a.log_decay + h));   // decay - 1

  for (int t0 = 0; t0 < n; t0 += kTokens) {
    const int nt = min(kTokens, n - t0);
    if (t0 > 0) __syncthreads();                 // the tokens before are done with
    for (int i = tid; i < nt * 2 * (DIMS / 8); i += kThreads) {
      const int u = i % (DIMS / 8), t = (i / (DIMS / 8)) >> 1;
      const bool key = (i / (DIMS / 8)) & 1;
      const bf16* x = key ? reinterpret_cast<const bf16*>(a.k) + (first + t0 + t) * a.ld_k_row + hk * a.ld_k_head
                          : reinterpret_cast<const bf16*>(a.q) + (first + t0 + t) * a.ld_q_row + h * a.ld_q_head;
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (u * 8 < a.dk) bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(x) + u), f);
      float4* to = reinterpret_cast<float4*>((key ? k_s : q_s)[t] + u * 8);
      to[0] = make_float4(f[0], f[1], f[2], f[3]);
      to[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
    uint2 v[kTokens];
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
      v[t] = t < nt && col ? __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const bf16*>(a.v) +
                                                                  (first + t0 + t) * a.ld_v_row + hk * a.ld_v_head + c))
                           : make_uint2(0u, 0u);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      if (t >= nt) break;
      const float2 v0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v[t].x));
      const float2 v1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v[t].y));
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = row0 + i * kRows * kWarps;
        const float kk = k_s[t][r], qq = q_s[t][r];
        s[i].x = fmaf(kk, v0.x, fmaf(s[i].x, d1, s[i].x));
        s[i].y = fmaf(kk, v0.y, fmaf(s[i].y, d1, s[i].y));
        s[i].z = fmaf(kk, v1.x, fmaf(s[i].z, d1, s[i].z));
        s[i].w = fmaf(kk, v1.y, fmaf(s[i].w, d1, s[i].w));
        o.x = fmaf(qq, s[i].x, o.x);
        o.y = fmaf(qq, s[i].y, o.y);
        o.z = fmaf(qq, s[i].z, o.z);
        o.w = fmaf(qq, s[i].w, o.w);
      }
      sum_s[t][warp][lane] = o;
    }
    __syncthreads();
    const int t = tid / COLS, cc = tid % COLS, at = (part * COLS + cc) * 4;
    if (t < nt && at < a.dv) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int y = 0; y < kRows; ++y) {
          const float4 x = sum_s[t][w][y * COLS + cc];
          o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
        }
      __nv_bfloat162 w2[2] = {__floats2bfloat162_rn(o.x * a.scale, o.y * a.scale),
                              __floats2bfloat162_rn(o.z * a.scale, o.w * a.scale)};
      *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(a.out) + (first + t0 + t) * a.ld_out_row +
                                h * a.ld_out_head + at) = *reinterpret_cast<const uint2*>(w2);
    }
  }
  if (dst >= 0 && (dst != src || n > 0)) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = row0 + i * kRows * kWarps;
      if (col && r < a.dk)
        *reinterpret_cast<float4*>(a.state + dst * slot + head + (int64_t)r * a.dv + c) = s[i];
    }
  }
}

template <int COLS, int DIMS>
cudaError_t launch_for(const LinearArgs& p, cudaStream_t st) {
  const int parts = (p.a.dv + 4 * COLS - 1) / (4 * COLS);
  // Where registers keep it to two CTAs an SM (41 KB of shared memory) the rest is to be L1, through which the states
  // come: behind a kernel of 226 KB it would find that kernel's split.  256 sequences x 32 heads of 128 x 128: a
  // prefill of one token each 212 -> 178 us, a step behind a prompt's chunk 171 -> 168, behind itself 167 as before.
  // The narrower ones hold more CTAs, which a quarter has no room for: 11.7 -> 13.1 us.
  if (DIMS * COLS == 128 * 32) {
    const cudaError_t c = cudaFuncSetAttribute(linear_recurrent<COLS, DIMS>, cudaFuncAttributePreferredSharedMemoryCarveout, 25);
    if (c != cudaSuccess) return c;
  }
  const cudaError_t e = launch_overlapped(linear_recurrent<COLS, DIMS>, dim3((unsigned)(p.batch * p.a.n_heads * parts)),
                                          dim3(kThreads), 0, st, p, parts);
  note_launch();
  return e;
}

template <int COLS>
cudaError_t launch(const LinearArgs& p, cudaStream_t st) {
  return p.a.dk > 64 ? launch_for<COLS, 128>(p, st) : launch_for<COLS, 64>(p, st);
}

}  // namespace

cudaError_t launch_linear_recurrent(const LinearArgs& p, cudaStream_t st) {
  // A wide head is one CTA, or four where they fill the device at most three times.  us for 16 / 64 /
  // 100 / 128 / 256 heads of 128 x 128: one 3.70 / 3.81 / 3.91 / 3.90 / 5.55, two 2.98 / 3.18 / 3.90 / 3.87 / 6.55,
  // four 2.47 / 2.98 / 3.70 / 4.21 / 6.67.
  if (p.a.dv > 64 && (int64_t)p.batch * p.a.n_heads * 4 > 3 * sm_count()) return launch<32>(p, st);
  return p.a.dv > 32 && p.a.dv <= 64 ? launch<16>(p, st) : launch<8>(p, st);
}

}  // namespace dsi
