// Linear attention with a decay for each head over prompts, on the tcgen05 tensor
// cores: 128 tokens of a sequence (a chunk) at a time.  With lam = exp(g), the
// state S that the chunk finds and its tokens i, j = 0 .. r-1 (r = 128 but for the last):
//   out_i = scale (sum_{j <= i} lam^(i-j) (q_i . k_j) v_j + lam^(i+1) S^T q_i)
//   S    <- S + expm1(g r) S + sum_j k_j (lam^(r-1-j) v_j)^T
//
// A CTA takes 64 of the dv columns of one head: they do not meet the other columns but
// in q . k, which is computed again.  Per chunk four products, all 128 rows high:
//   P  = Q K^T                [tokens x tokens]   decayed, masked, to bf16 in place (TMEM)
//   OI = P V                  [tokens x 64]
//   OX = Q S                  [tokens x 64]       S rounded to bf16
//   ST += K^T V'              [dk x 64]           V' = decayed V in two bf16 parts: the state
//                                                 stays exact to 2^-16 of what enters it
// and ST, the state, stays in fp32 in TMEM from a sequence's first chunk to its last.
//
// Roles (20 warps), each walking the same list of (sequence, head, columns):
//   0 copies (TMA), 1 MMAs, 4-7 P, 8-11 V', 12-15 the state, 16-19 outputs.
// A chunk's rows behind the sequence's end (other sequences') are cleared or never
// stored.  A v that is not finite is taken out of V before P V (its weight
// of 0 for earlier tokens would give NaN) and the column's later outputs become
// NaN; in V' it stays, and makes the state's column NaN.
#include "kernels.h"
#include "linear_attn.h"
#include "tc_waits.cuh"
#include "tma_host.h"

namespace dsi {
using namespace tc;

namespace {

constexpr int kC = 128;                        // tokens of a chunk
constexpr int kCols = 64;                      // columns of the state that a CTA takes
constexpr int kTile = kC * 128;                // 64 dims of a chunk, 16 KB
constexpr int kStages = 2;
constexpr int kStageBytes = 5 * kTile;         // Q (two tiles), K (two), V
constexpr int kThreads = 640;

constexpr int oVh = kStages * kStageBytes;     // V', high and low parts
constexpr int oVl = oVh + kTile;
constexpr int oS = oVl + kTile;                // the state in bf16: [dk][64]
constexpr int oPow = oS + kTile;               // P's warps: powers of lam, [4][128]
constexpr int oRev = oPow + 4 * 128 * 4;       // ... lam^31 .. lam^0, [4][32]
constexpr int kMarks = 3;                      // (V' is up to two chunks before the outputs)
constexpr int oBad = oRev + 4 * 32 * 4;        // [kMarks][4] a warp's rows of V hold something not finite
constexpr int oFirst = oBad + kMarks * 4 * 4;  // [kMarks][4][64] the first such row of a column
constexpr int oBar = oFirst + kMarks * 4 * 64;
constexpr int kBars = 3 * kStages + 2 + 2 + 2 + 5;
constexpr int oSlot = oBar + kBars * 8;
constexpr int kSmem = oSlot + 16 + 1024;
static_assert(kSmem <= 227 * 1024 && oBar % 8 == 0, "shared memory");

constexpr uint32_t TM_P = 0;                   // two tiles of 128 columns
constexpr uint32_t TM_OI = 256;
constexpr uint32_t TM_ST = 320;
constexpr uint32_t TM_OX = 384;                // two tiles of 64 columns
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t IDESC_P = idesc_f32(1, kC, kC);
constexpr uint32_t IDESC_O = idesc_f32_bmn(1, kC, kCols);
constexpr uint32_t IDESC_ST = IDESC_O | (1u << 15);   // A, too, is MN-major (K^T)

struct Plan {
  int parts;                                   // 64-column parts of dv
  int items;                                   // (sequence, head, part)
};

struct Item {
  int b, h, part, n;                           // n: the sequence's tokens
  int chunks;
  int64_t first;                               // its first token
};
__device__ __forceinline__ bool next_item(const LinearArgs& p, const Plan& plan, int& walk, Item& it) {
  if (walk >= plan.items) return false;
  it.part = walk % plan.parts;
  const int bh = walk / plan.parts;
  it.b = bh / p.a.n_heads;
  it.h = bh - it.b * p.a.n_heads;
  tokens_of(p, it.b, it.first, it.n);
  it.chunks = (it.n + kC - 1) / kC;
  walk += gridDim.x;
  return true;
}

// lam^n: 1 for n = 0, whatever lam is.
__device__ __forceinline__ float power(float g, int n) { return n == 0 ? 1.f : expf(g * (float)n); }

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_st16w(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ bool bf16x2_finite(uint32_t w) {
  return (w & 0x7F80u) != 0x7F80u && (w & 0x7F800000u) != 0x7F800000u;
}

__global__ void __launch_bounds__(kThreads, 1)
linear_chunk(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
             const __grid_constant__ CUtensorMap vmap, const __grid_constant__ LinearArgs p,
             const __grid_constant__ Plan plan) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* qk_full = reinterpret_cast<uint64_t*>(smem + oBar);   // [kStages] Q and K landed
  uint64_t* v_full = qk_full + kStages;        // [kStages] V landed
  uint64_t* empty = v_full + kStages;          // [kStages] a chunk's MMAs done
  uint64_t* s_full = empty + kStages;          // [2] q . k in TMEM
  uint64_t* p_full = s_full + 2;               // [2] P in TMEM
  uint64_t* p_empty = p_full + 2;              // [2] P V done
  uint64_t* v_ready = p_empty + 2;             // V cleaned, V' written
  uint64_t* st_ready = v_ready + 1;            // state decayed, its bf16 form written
  uint64_t* st_done = v_ready + 2;             // K^T V' (and Q S) done
  uint64_t* o_full = v_ready + 3;              // OI and OX done
  uint64_t* o_empty = v_ready + 4;             // ... read out
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + oSlot);
  const dsi_linear& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&qk_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_empty[i], 1);
    }
    mbar_init(v_ready, 4);
    mbar_init(st_ready, 4);
    mbar_init(st_done, 1);
    mbar_init(o_full, 1);
    mbar_init(o_empty, 4);
    s_abort = 0;
    s_err = p.err;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, TMEM_COLS);
  if (tid == 0) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  grid_dep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = *tmem_slot;
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  const int row = (warp & 3) * 32 + lane;      // of a chunk, or of the state
  int walk = blockIdx.x;
  Item it;
  int t = 0;                                   // chunks so far
  bool ok = true;

  if (warp == 0) {
    // ======================= copies ==============================================
    if (lane == 0) {
      const bool wide = a.dk > 64;             // (else the second tiles are not read, but for
                                               // rows of ST that nobody reads)
#pragma unroll 1
      while (ok && next_item(p, plan, walk, it)) {
        const int hk = it.h / p.group;
#pragma unroll 1
        for (int c = 0; c < it.chunks; ++c, ++t) {
          const int s = t % kStages;
          if (!(ok = wait1(&empty[s], ((uint32_t)(t / kStages) & 1u) ^ 1u))) break;
          uint8_t* st = smem + s * kStageBytes;
          const int at = (int)it.first + c * kC;
          mbar_arrive_expect_tx(&qk_full[s], (wide ? 4 : 2) * kTile);
          tma_load_3d(st, &qmap, 0, it.h, at, &qk_full[s]);
          tma_load_3d(st + 2 * kTile, &kmap, 0, hk, at, &qk_full[s]);
          if (wide) {
            tma_load_3d(st + kTile, &qmap, 64, it.h, at, &qk_full[s]);
            tma_load_3d(st + 3 * kTile, &kmap, 64, hk, at, &qk_full[s]);
          }
          mbar_arrive_expect_tx(&v_full[s], kTile);
          tma_load_3d(st + 4 * kTile, &vmap, it.part * kCols, hk, at, &v_full[s]);
        }
      }
      // never leave the CTA with a copy still landing in shared memory
      if (s_abort) {
        volatile int no_abort = 0;
        for (int i = max(0, t - kStages); i < t; ++i) {
          mbar_wait(&qk_full[i % kStages], (uint32_t)(i / kStages) & 1u, &no_abort, p.err, 100000000ull);
          mbar_wait(&v_full[i % kStages], (uint32_t)(i / kStages) & 1u, &no_abort, p.err, 100000000ull);
        }
      }
    }
  } else if (warp == 1) {
    // ======================= MMAs ================================================
    if (lane == 0) {
      const int steps = (a.dk + 15) / 16;
      const uint64_t d_vh = desc_sw128_mn(smem_u32(smem + oVh), kTile), d_vl = desc_sw128_mn(smem_u32(smem + oVl), kTile);
      const uint64_t d_s = desc_sw128_mn(smem_u32(smem + oS), kTile);
      auto qk = [&](int i) {                   // chunk i's q . k
        const int s = i % kStages;
        if (!wait1(&qk_full[s], (uint32_t)(i / kStages) & 1u)) return false;
        if (!wait1(&p_empty[i & 1], ((uint32_t)(i >> 1) & 1u) ^ 1u)) return false;
        tc_fence_after();
        const uint32_t base = smem_u32(smem + s * kStageBytes);
        const uint64_t q = desc_sw128(base), k = desc_sw128(base + 2 * kTile);
#pragma unroll 1
        for (int x = 0; x < steps; ++x) {
          const uint64_t off = (uint64_t)(((x >> 2) * kTile + (x & 3) * 32) >> 4);
          mma_bf16(tmem + TM_P + (i & 1) * kC, q + off, k + off, IDESC_P, x > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[i & 1]);
        return true;
      };
      // one chunk ahead: whether there is one
      int c = -1;
      it.chunks = 0;
      auto advance = [&]() {
        if (++c < it.chunks) return true;
        c = 0;
        do {
          if (!next_item(p, plan, walk, it)) return false;
        } while (it.chunks == 0);
        return true;
      };
      bool more = advance();
      if (more) ok = qk(0);
#pragma unroll 1
      while (ok && more) {
        more = advance();
        const int s = t % kStages;
        const uint32_t base = smem_u32(smem + s * kStageBytes);
        if (!(ok = wait1(st_ready, (uint32_t)t & 1u))) break;
        tc_fence_after();
        const uint64_t q = desc_sw128(base);
#pragma unroll 1
        for (int x = 0; x < steps; ++x)
          mma_bf16(tmem + TM_OX + (t & 1) * kCols, q + (uint64_t)(((x >> 2) * kTile + (x & 3) * 32) >> 4),
                   d_s + (uint64_t)((x * 2048) >> 4), IDESC_O, x > 0 ? 1u : 0u);
        if (!(ok = wait1(v_ready, (uint32_t)t & 1u))) break;
        tc_fence_after();
        const uint64_t k = desc_sw128_mn(base + 2 * kTile, kTile);
#pragma unroll
        for (int x = 0; x < 2 * (kC / 16); ++x)
          mma_bf16(tmem + TM_ST, k + (uint64_t)(((x & 7) * 2048) >> 4),
                   (x < 8 ? d_vh : d_vl) + (uint64_t)(((x & 7) * 2048) >> 4), IDESC_ST, 1u);
        mma_commit(st_done);
        // the next chunk's q . k before this one's P V, if it is there already
        bool ahead = false;
        if (more && mbar_test_wait(&qk_full[(t + 1) % kStages], (uint32_t)((t + 1) / kStages) & 1u)) {
          if (!(ok = qk(t + 1))) break;
          ahead = true;
        }
        if (!(ok = wait1(&p_full[t & 1], (uint32_t)(t >> 1) & 1u) && wait1(o_empty, ((uint32_t)t & 1u) ^ 1u))) break;
        tc_fence_after();
        const uint64_t v = desc_sw128_mn(base + 4 * kTile, kTile);
#pragma unroll
        for (int x = 0; x < kC / 16; ++x)
          mma_bf16_tmem_a(tmem + TM_OI, tmem + TM_P + (t & 1) * kC + x * 8, v + (uint64_t)((x * 2048) >> 4), IDESC_O,
                          x > 0 ? 1u : 0u);
        mma_commit(o_full);
        mma_commit(&p_empty[t & 1]);
        mma_commit(&empty[s]);
        ++t;
        if (more && !ahead && !(ok = qk(t))) break;
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ======================= P ===================================================
    // Thread = token i, blocks of 32 tokens j: whole ones before the warp's own rows take
    // lam^(i-j) as lam^(i-j31) lam^(j31-j) (j31 the block's last token: both
    // exponents are positive), the warp's own block by table; the rest is 0.
    const int w = warp & 3;
    float* pow_s = reinterpret_cast<float*>(smem + oPow) + w * 128;
    float* rev_s = reinterpret_cast<float*>(smem + oRev) + w * 32;
    int h = -1;
#pragma unroll 1
    while (ok && next_item(p, plan, walk, it)) {
      if (it.h != h) {
        h = it.h;
        const float g = __ldg(a.log_decay + h);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) pow_s[i * 32 + lane] = power(g, i * 32 + lane);
        rev_s[lane] = power(g, 31 - lane);
        __syncwarp();
      }
#pragma unroll 1
      for (int c = 0; c < it.chunks; ++c, ++t) {
        if (!(ok = wait32(&s_full[t & 1], (uint32_t)(t >> 1) & 1u))) break;
        tc_fence_after();
        const uint32_t t_p = tmem + lane_base + TM_P + (t & 1) * kC;
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t out[16];
          if (blk <= w) {
            float v[32];
            tmem_ld32(t_p + blk * 32, v);
            tmem_ld_wait();
            if (blk < w) {
              const float far = pow_s[row - blk * 32 - 31];
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(rev_s + j);
                out[j / 2] = pack_bf16(v[j] * (far * f.x), v[j + 1] * (far * f.y));
                out[j / 2 + 1] = pack_bf16(v[j + 2] * (far * f.z), v[j + 3] * (far * f.w));
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const float f0 = pow_s[max(0, lane - j)], f1 = pow_s[max(0, lane - j - 1)];
                out[j / 2] = pack_bf16(j <= lane ? v[j] * f0 : 0.f, j + 1 <= lane ? v[j + 1] * f1 : 0.f);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) out[j] = 0u;
          }
          tmem_st16w(t_p + blk * 16, out);     // (over logits that this thread has read)
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t & 1]);
      }
    }
  } else if (warp >= 8 && warp < 12) {
    // ======================= V' ==================================================
    const int w = warp & 3;
#pragma unroll 1
    while (ok && next_item(p, plan, walk, it)) {
      const float g = __ldg(a.log_decay + it.h);
#pragma unroll 1
      for (int c = 0; c < it.chunks; ++c, ++t) {
        const int s = t % kStages, r = min(kC, it.n - c * kC);
        uint8_t* st = smem + s * kStageBytes;
        const float f = row < r ? power(g, r - 1 - row) : 0.f;
        if (!(ok = wait32(&v_full[s], (uint32_t)(t / kStages) & 1u))) break;
        if (t > 0 && !(ok = wait32(st_done, (uint32_t)(t - 1) & 1u))) break;
        bool bad = false;
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {
          const uint32_t off = sw128_offset((uint32_t)row, (uint32_t)u);
          const uint4 v4 = *reinterpret_cast<const uint4*>(st + 4 * kTile + off);
          const uint32_t x[4] = {v4.x, v4.y, v4.z, v4.w};
          uint32_t hi[4], lo[4];
          bool fine = true;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            fine = fine && bf16x2_finite(x[e]);
            const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[e]));
            const float y0 = y.x * f, y1 = y.y * f;
            hi[e] = pack_bf16(y0, y1);
            const float2 z = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi[e]));
            lo[e] = pack_bf16(y0 - z.x, y1 - z.y);
          }
          if (row >= r) {
#pragma unroll
            for (int e = 0; e < 4; ++e) hi[e] = lo[e] = 0u;
            *reinterpret_cast<uint4*>(st + 4 * kTile + off) = make_uint4(0, 0, 0, 0);
          } else {
            bad = bad || !fine;
          }
          *reinterpret_cast<uint4*>(smem + oVh + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(smem + oVl + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (row >= r) {                        // K's, too: what they hold must not meet V' of 0
#pragma unroll
          for (int u = 0; u < 16; ++u)
            *reinterpret_cast<uint4*>(st + 2 * kTile + (u >> 3) * kTile + sw128_offset((uint32_t)row, (uint32_t)(u & 7))) =
                make_uint4(0, 0, 0, 0);
        }
        const bool any = __any_sync(0xffffffffu, bad);
        if (lane == 0) reinterpret_cast<volatile int*>(smem + oBad)[t % kMarks * 4 + w] = any;
        if (__builtin_expect(any, 0)) {
          uint8_t* first = smem + oFirst + (t % kMarks * 4 + w) * kCols;
#pragma unroll 1
          for (int x = 0; x < kCols; ++x) {
            uint16_t* e = reinterpret_cast<uint16_t*>(st + 4 * kTile + sw128_offset((uint32_t)row, (uint32_t)(x >> 3))) + (x & 7);
            const bool out = row < r && (*e & 0x7F80u) == 0x7F80u;
            const uint32_t who = __ballot_sync(0xffffffffu, out);
            if (out) *e = 0;
            if (lane == 0) first[x] = who ? (uint8_t)(w * 32 + __ffs(who) - 1) : (uint8_t)kC;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_ready);
      }
    }
  } else if (warp >= 12 && warp < 16) {
    // ======================= the state ===========================================
    // Thread = row of the state; rows that the head does not have are left alone.
    const bool rows = (warp & 3) * 32 < a.dk, live = row < a.dk;
#pragma unroll 1
    while (ok && next_item(p, plan, walk, it)) {
      const float g = __ldg(a.log_decay + it.h);
      const int64_t src = in_slot(p, it.b), dst = out_slot(p, it.b);
      const int cols = min(kCols, a.dv - it.part * kCols);          // a multiple of 8
      const int64_t head = ((int64_t)it.h * a.dk + row) * a.dv + it.part * kCols;
      const int64_t slot = (int64_t)a.n_heads * a.dk * a.dv;
      if (it.chunks == 0) {
        if (dst >= 0 && dst != src && live)
          for (int x = 0; x < cols; x += 4)
            *reinterpret_cast<float4*>(a.state + dst * slot + head + x) =
                src >= 0 ? *reinterpret_cast<const float4*>(a.state + src * slot + head + x) : make_float4(0.f, 0.f, 0.f, 0.f);
        continue;
      }
#pragma unroll 1
      for (int c = 0; c < it.chunks; ++c, ++t) {
        const float d1 = expm1f(g * (float)min(kC, it.n - c * kC));
        if (c > 0 && !(ok = wait32(st_done, (uint32_t)(t - 1) & 1u))) break;
        tc_fence_after();
        if (rows) {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            float s[32];
            if (c == 0) {
#pragma unroll
              for (int x = 0; x < 32; x += 4) {
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                if (src >= 0 && live && half * 32 + x < cols)
                  y = *reinterpret_cast<const float4*>(a.state + src * slot + head + half * 32 + x);
                s[x] = y.x; s[x + 1] = y.y; s[x + 2] = y.z; s[x + 3] = y.w;
              }
              __syncwarp();
            } else {
              tmem_ld32(tmem + lane_base + TM_ST + half * 32, s);
              tmem_ld_wait();
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
              *reinterpret_cast<uint4*>(smem + oS + sw128_offset((uint32_t)row, (uint32_t)(half * 4 + u))) =
                  make_uint4(pack_bf16(s[8 * u], s[8 * u + 1]), pack_bf16(s[8 * u + 2], s[8 * u + 3]),
                             pack_bf16(s[8 * u + 4], s[8 * u + 5]), pack_bf16(s[8 * u + 6], s[8 * u + 7]));
            uint32_t y[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) y[x] = __float_as_uint(fmaf(s[x], d1, s[x]));
            tmem_st32(tmem + lane_base + TM_ST + half * 32, y);
          }
          tmem_st_wait();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(st_ready);
      }
      if (!ok) break;
      if (!(ok = wait32(st_done, (uint32_t)(t - 1) & 1u))) break;
      tc_fence_after();
      if (rows && dst >= 0) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float s[32];
          tmem_ld32(tmem + lane_base + TM_ST + half * 32, s);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            if (live && half * 32 + x < cols)
              *reinterpret_cast<float4*>(a.state + dst * slot + head + half * 32 + x) =
                  make_float4(s[x], s[x + 1], s[x + 2], s[x + 3]);
          __syncwarp();
        }
      }
    }
  } else if (warp >= 16) {
    // ======================= outputs =============================================
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && a.ld_out_row % 16 == 0 && a.ld_out_head % 16 == 0;
#pragma unroll 1
    while (ok && next_item(p, plan, walk, it)) {
      const float since = a.scale * power(__ldg(a.log_decay + it.h), row + 1);
      const int cols = min(kCols, a.dv - it.part * kCols);
#pragma unroll 1
      for (int c = 0; c < it.chunks; ++c, ++t) {
        if (!(ok = wait32(o_full, (uint32_t)t & 1u))) break;
        tc_fence_after();
        const int4 bad = *reinterpret_cast<const int4*>(smem + oBad + t % kMarks * 16);
        const bool live = row < it.n - c * kC;
        bf16* to = reinterpret_cast<bf16*>(a.out) + (it.first + c * kC + row) * a.ld_out_row +
                   (int64_t)it.h * a.ld_out_head + it.part * kCols;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float x[32], y[32];
          tmem_ld32(tmem + lane_base + TM_OI + half * 32, x);
          tmem_ld32(tmem + lane_base + TM_OX + (t & 1) * kCols + half * 32, y);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = fmaf(y[i], since, x[i] * a.scale);
          if (__builtin_expect(bad.x | bad.y | bad.z | bad.w, 0)) {
            const uint8_t* first = smem + oFirst + t % kMarks * 4 * kCols + half * 32;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              int from = kC;
              if (bad.x) from = min(from, (int)first[i]);
              if (bad.y) from = min(from, (int)first[kCols + i]);
              if (bad.z) from = min(from, (int)first[2 * kCols + i]);
              if (bad.w) from = min(from, (int)first[3 * kCols + i]);
              if (row >= from) x[i] = __int_as_float(0x7fc00000);
            }
          }
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty);
          }
          uint32_t o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
          if (live) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              bf16* at = to + half * 32 + i * 16;
              const int left = cols - half * 32 - i * 16;
              if (wide && left >= 16) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(at), "r"(o[8 * i]),
                             "r"(o[8 * i + 1]), "r"(o[8 * i + 2]), "r"(o[8 * i + 3]), "r"(o[8 * i + 4]),
                             "r"(o[8 * i + 5]), "r"(o[8 * i + 6]), "r"(o[8 * i + 7])
                             : "memory");
              } else {
                if (left >= 8) reinterpret_cast<uint4*>(at)[0] = make_uint4(o[8 * i], o[8 * i + 1], o[8 * i + 2], o[8 * i + 3]);
                if (left >= 16) reinterpret_cast<uint4*>(at)[1] = make_uint4(o[8 * i + 4], o[8 * i + 5], o[8 * i + 6], o[8 * i + 7]);
              }
            }
          }
          __syncwarp();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
}

// Map of [tokens, heads, dims] with any pitches, boxes of 128 tokens by 64 dims.
bool map_heads(CUtensorMap* m, const void* base, int64_t tokens, int heads, int dims, int64_t ld_row, int64_t ld_head) {
  auto enc = tma_encode_fn();
  if (!enc) return false;
  cuuint64_t size[3] = {(cuuint64_t)dims, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)ld_head * 2, (cuuint64_t)ld_row * 2};
  cuuint32_t box[3] = {64, 1, kC}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), size, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t linear_prefill_workspace(int64_t, int, int, int, int) { return 256; }

cudaError_t launch_linear_prefill(const LinearArgs& p, void*, cudaStream_t st) {
  int dev = 0, sms = 152;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(linear_chunk, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  if (p.n_tokens == 0) return launch_linear_recurrent(p, st);   // (nothing but states to pass on)
  Plan plan;
  plan.parts = (p.a.dv + kCols - 1) / kCols;
  plan.items = p.batch * p.a.n_heads * plan.parts;
  CUtensorMap qmap, kmap, vmap;
  if (!map_heads(&qmap, p.a.q, p.n_tokens, p.a.n_heads, p.a.dk, p.a.ld_q_row, p.a.ld_q_head) ||
      !map_heads(&kmap, p.a.k, p.n_tokens, p.a.n_kv_heads, p.a.dk, p.a.ld_k_row, p.a.ld_k_head) ||
      !map_heads(&vmap, p.a.v, p.n_tokens, p.a.n_kv_heads, p.a.dv, p.a.ld_v_row, p.a.ld_v_head))
    return cudaErrorInvalidValue;
  e = launch_overlapped(linear_chunk, dim3((unsigned)(plan.items < sms ? plan.items : sms)), dim3(kThreads), kSmem, st,
                        qmap, kmap, vmap, p, plan);
  note_launch();
  return e;
}

}  // namespace dsi
