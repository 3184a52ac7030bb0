// Linear attention with a decay for each head over prompts, on the tcgen05 tensor
// cores: 128 tokens of a sequence (a chunk) at a time.  With lam = exp(g), the
// state S that the chunk finds and its tokens i, j = 0 .. r-1 (r = 128 but for the last):
//   out_i = scale (sum_{j <= i} lam^(i-j) (q_i . k_j) v_j + lam^(i+1) S^T q_i)
//   S    <- S + expm1(g r) S + sum_j k_j (lam^(r-1-j) v_j)^T
//
// A CTA takes 64 of the dv columns of one head: they do not meet the other columns but
// in q . k, which is computed again.  Per chunk four products, all 128 rows high:
//   P  = Q K^T     [tokens x tokens]   decayed, masked, to bf16 in place (TMEM)
//   OI = P V       [tokens x 64]
//   OX = Q S       [tokens x 64]       S rounded to bf16
//   D  = K^T V'    [dk x 64]           V' = decayed V in three bf16 parts, which hold it to its last bit;
//                                      K^T is turned into TMEM (as an MN-major operand in shared
//                                      memory a product of 16 tokens takes 130 cycles, not 46)
// and the state, S <- S + expm1(g r) S + D, stays in the registers of its warps, in fp32, from a
// sequence's first chunk to its last.  Its error against 64 bits is 6.5e-7 of its norm (two parts of V'
// made it 2.5e-6 and calls 1 to 7 % shorter).
//
// Roles (28 warps), each walking the same list of (sequence, head, columns):
//   0 products Q S and P V, 1 K^T V', 2 Q K^T, 3 copies (TMA) and the list, 4-7 P,
//   8-15 V' and K^T, 16-23 the state, 24-27 outputs.
//
// A chunk's rows behind the sequence's end (other sequences') are cleared or never
// stored.  A v that is not finite is taken out of V before P V (its weight
// of 0 for earlier tokens would give NaN) and the column's later outputs become
// NaN; in V' it stays, and makes the state's column NaN.
//
// What bounds it.  8192 tokens, 64 heads of 128 x 128: 147 us, 3.7 TB/s (55 % of the measured copy
// rate): 64 chunks in a row on each of 128 CTAs, about 4500 cycles a chunk, 2.3 us; its bytes at the copy rate
// would take 2450.  Counted over 32 chunks (4800 cycles each with start and end): 2580 cycles of the warps' loads
// and stores to shared memory (logits, P, outputs, V', S, K^T), 1790 of the tensor pipe for 48 products, issue
// slots half full.  So no pipe is full; the products' operands and the copies, which the first count leaves
// out, are about 1400 and 640 cycles of that memory by their bytes, and whether they or the roles' waits for one another
// set the pace has not been told apart.  A sequence's start and end cost about 3 us on top (76 heads: one
// sequence of 32 chunks 79 us, four of 8 90, 32 of one 166).
// More warps for P or the outputs, three tiles of P, both terms of an output in one
// accumulator took 3 to 20 % longer; one issuer of products for all four 25 %, its lane in a branch of
// its own another 15 %; much larger loops (110 KB of code) twice the time.
#include "kernels.h"
#include "linear_attn.h"
#include "tc_waits.cuh"
#include "tc_warp.cuh"
#include "tma_host.h"

namespace dsi {
using namespace tc;

namespace {

constexpr int kC = 128;                        // tokens of a chunk
constexpr int kCols = 64;                      // columns of the state that a CTA takes
constexpr int kTile = kC * 128;                // 64 dims of a chunk, 16 KB
constexpr int kQk = 2;                         // chunks of Q and of K in shared memory
constexpr int kV = 2;                          // of V (a third, without a part of V', gains 1 to 2 %)
constexpr int kSplit = 3;                      // bf16 parts of V': 8 bits each of an fp32's 24
constexpr int kThreads = 896;

constexpr int oQ = 0;                          // [kQk][2] tiles
constexpr int oK = oQ + kQk * 2 * kTile;       // [kQk][2]
constexpr int oV = oK + kQk * 2 * kTile;       // [kV]
constexpr int oVp = oV + kV * kTile;           // V', its parts
constexpr int oS = oVp + kSplit * kTile;       // the state in bf16: [dk][64]
constexpr int kMarks = 4;                      // (the place of V t + 4 is free once P V of t + 2 is done, whose
                                               // P's tile was free once the outputs of t were read)
constexpr int oBad = oS + kTile;               // [kMarks][8] a warp's part of V holds something not finite
constexpr int oFirst = oBad + kMarks * 8 * 4;  // [kMarks][8][32] the first such row of a column
constexpr int oRing = oFirst + kMarks * 8 * 32;   // pieces of work
constexpr int oBar = oRing + 4 * 48;
constexpr int kBars = 4 * kQk + 3 * kV + 4 * 2 + 4 + 4 + 2 * 4;
constexpr int oSlot = oBar + kBars * 8;
constexpr int kSmem = oSlot + 8;
// (static variables take a kilobyte of their own, aligned like the rest)
static_assert(kSmem <= 226 * 1024 && oBad % 16 == 0 && oBar % 8 == 0 && oRing % 16 == 0, "shared memory");

constexpr uint32_t TM_P = 0;                   // two tiles of 128 columns: q . k, then P in the first half
constexpr uint32_t TM_OI = 64;                 // ... and OI in the second
constexpr uint32_t TM_OX = 256;                // two tiles of 64 columns
constexpr uint32_t TM_D = 384;
constexpr uint32_t TM_KT = 448;                // K^T in bf16: [dk][128 tokens]
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t IDESC_P = idesc_f32(1, kC, kC);
constexpr uint32_t IDESC_O = idesc_f32_bmn(1, kC, kCols);

struct Plan {
  int parts;                                   // 64-column parts of dv
  int items;                                   // (sequence, head, part); with a split an upper bound
  int split;                                   // chunks of a segment, or 0: sequences stay whole
  int segments;                                // that there is room for (starts that go back may ask for more: whole, too)
  float* seg;                                  // split: [segments][heads][dk][dv] states
};

// Long sequences of few heads are cut into segments of plan.split chunks.  A first pass
// (LOCAL) leaves what each but a sequence's last one adds to a state of zeros, linear_carry turns
// that into the state that each segment finds, and then all of them run side by side.
struct Item {
  int h, part, n;                              // n: the sequence's tokens; h -1: the list's end
  int c0, c1;                                  // chunks of the sequence
  int seg;                                     // segment's place in plan.seg, or -1
  int last;                                    // of the sequence
  int first;                                   // the sequence's first token
  int64_t src, dst;                            // slots, or -1
  float g;                                     // log decay
};
// Segments of sequence b where the call is split.
__device__ __forceinline__ int segments_of(const LinearArgs& p, const Plan& plan, int b) {
  int64_t first;
  int n;
  tokens_of(p, b, first, n);
  return max(1, ((n + kC - 1) / kC + plan.split - 1) / plan.split);
}

constexpr int kMaxSplit = 64;                  // sequences of a call that is split
constexpr int kMaxOrder = 256;                 // ... whose sequences are taken in order of length
constexpr int kBits = 2048;                    // more: a bit for every so many sequences, whether one is long

// Sequences to a bit, as a power of two.
__device__ __forceinline__ int bit_shift(const LinearArgs& p) { return max(0, 21 - __clz(p.batch - 1)); }

// First sequence from g on of more than p.few tokens, or p.batch.  (Batches of thousands of decoding rows
// are walked by the bit, a block that has one eight sequences at a time.)
__device__ __forceinline__ int next_long(const LinearArgs& p, const uint32_t* bits, int g) {
  const int shift = bit_shift(p);
  while (g < p.batch) {
    int w = g >> shift >> 5;
    uint32_t word = bits[w] & (0xffffffffu << ((g >> shift) & 31));
    while (word == 0u && ++w < kBits / 32) word = bits[w];
    if (word == 0u) return p.batch;
    const int block = w * 32 + __ffs(word) - 1;
    g = max(g, block << shift);
    if (shift == 0) return g;
    for (const int end = min(p.batch, (block + 1) << shift); g < end; g += 8) {
      int start[9], at = 8;
#pragma unroll
      for (int i = 0; i < 9; ++i) start[i] = held_start(p, min(end, g + i));
#pragma unroll
      for (int i = 7; i >= 0; --i)
        if (start[i + 1] - start[i] > p.few) at = i;
      if (at < 8) return g + at;
    }
    g = (block + 1) << shift;
  }
  return p.batch;
}

// The CTA's next piece of work; `round` counts them.  Rounds go back and forth over the CTAs,
// whole sequences from the longest to the shortest (table: their order).  Split: table[b] is the
// first segment of sequence b.  More than kMaxOrder sequences are taken as they come, the short ones left
// out by the bits in the table.  A search that takes long gives kNothingYet: no wait runs out over it.
// (Every CTA gets as many pieces as the others, not as much work: of a ragged batch the CTAs with the longest
// sequences end last.)
constexpr int kNothingYet = -2, kSteps = 1024;
template <bool LOCAL>
__device__ __forceinline__ void look_up(const LinearArgs& p, const Plan& plan, const uint8_t* table_s, int& round, Item& it) {
  for (int step = 0;; ++step) {
    it.h = -1;
    const int G = gridDim.x, at = (round & 1) ? G - 1 - (int)blockIdx.x : (int)blockIdx.x;
    const int64_t i64 = (int64_t)round * G + at;
    if (i64 >= plan.items) return;
    const int i = (int)i64, g = i / (plan.parts * p.a.n_heads), hp = i - g * plan.parts * p.a.n_heads;
    const int h = hp / plan.parts;
    ++round;
    it.part = hp - h * plan.parts;
    it.seg = -1;
    it.last = 1;
    it.c0 = 0;
    int b = plan.split == 0 && p.batch <= kMaxOrder ? table_s[g] : g;
    const int* first = reinterpret_cast<const int*>(table_s);
    if (plan.split) {
      if (g >= first[p.batch]) return;
      for (b = 0; first[b + 1] <= g;) ++b;
      it.last = g + 1 == first[b + 1];
      if (LOCAL && it.last) continue;
      it.c0 = (g - first[b]) * plan.split;
      if (first[b + 1] - first[b] > 1) it.seg = g;
    }
    if (!LOCAL && p.batch > kMaxOrder) {
      const int next = next_long(p, reinterpret_cast<const uint32_t*>(table_s), b);
      if (next == p.batch) return;
      if (next > b) {                          // on to the round that it begins in
        const unsigned lo = (unsigned)(next * plan.parts * p.a.n_heads), r0 = lo / (unsigned)G;
        round = max(round, (int)r0);
        // (its first pieces may be this round's behind the CTA's)
        if (round == (int)r0 && r0 * G + ((r0 & 1) ? G - 1 - blockIdx.x : blockIdx.x) < lo) ++round;
        if (step < kSteps) continue;
        it.h = kNothingYet;
        return;
      }
    }
    int64_t tok;
    tokens_of(p, b, tok, it.n);
    if (it.n <= p.few) {                       // and, in their order, all behind it
      if (plan.split == 0 && p.batch <= kMaxOrder) return;
      continue;
    }
    it.first = (int)tok;
    it.c1 = (it.n + kC - 1) / kC;
    if (it.seg >= 0) it.c1 = min(it.c1, it.c0 + plan.split);
    it.src = in_slot(p, b);
    it.dst = out_slot(p, b);
    it.g = __ldg(p.a.log_decay + h);
    it.h = h;
    return;
  }
}

// The list passes from the warp that copies to the others through a ring in shared memory: a look-up is several
// trips to memory, and a copy of it for each role would crowd the instruction cache.
constexpr int kRing = 4;
struct Ring {
  int4 a[kRing], b[kRing], c[kRing];
};
__device__ __forceinline__ void publish(Ring* r, int i, const Item& it) {
  const int s = i % kRing;
  r->a[s] = make_int4(it.h, it.part | (it.last << 1), it.n, it.first);
  r->b[s] = make_int4(it.c0, it.c1, it.seg, (int)it.src);
  r->c[s] = make_int4((int)it.dst, __float_as_int(it.g), 0, 0);
}
__device__ __forceinline__ void peek(const Ring* r, int i, Item& it) {
  const int s = i % kRing;
  const int4 a = r->a[s], b = r->b[s], c = r->c[s];
  it.h = a.x; it.part = a.y & 1; it.last = a.y >> 1; it.n = a.z; it.first = a.w;
  it.c0 = b.x; it.c1 = b.y; it.seg = b.z; it.src = b.w;
  it.dst = c.x;
  it.g = __int_as_float(c.y);
}

// lam^n: 1 for n = 0, whatever lam is.
__device__ __noinline__ float power(float g, int n) { return n == 0 ? 1.f : expf(g * (float)n); }

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Four 8 x 8 blocks of 16-bit values, transposed: thread i gets values 2 (i % 4) and + 1 of
// column i / 4 of each block, whose rows' addresses lanes 8 b .. 8 b + 7 give for block b.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t saddr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr) : "memory");
}
// 16 lanes x 32 columns: registers 2 c and 2 c + 1 hold column 4 c + i % 4 of lanes i / 4 and i / 4 + 8.
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Eight floats, a sector: one access where the address allows, else two.
__device__ __forceinline__ void load8(const float* p, bool wide, float* f) {
  if (wide) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "l"(p) : "memory");
  } else {
    const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
  }
}
__device__ __forceinline__ void store8(float* p, bool wide, const float* f) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                 "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// KB: blocks of 64 dims that dk takes.  LOCAL: the first pass over segments.
template <int KB, bool LOCAL>
__global__ void __launch_bounds__(kThreads, 1)
linear_chunk(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
             const __grid_constant__ CUtensorMap vmap, const __grid_constant__ LinearArgs p,
             const __grid_constant__ Plan plan) {
  __shared__ __align__(16) float pow_table[5][32];   // P's warps, from 1 on: scale lam^0 .. scale lam^31
  __shared__ __align__(8) uint8_t table_s[264];       // look_up's
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const smem = smem_raw;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + oBar);   // [kQk] Q landed
  uint64_t* k_full = q_full + kQk;             // [kQk] K landed
  uint64_t* q_empty = k_full + kQk;            // [kQk] Q done with
  uint64_t* k_empty = q_empty + kQk;           // [kQk] K done with: turned, and q . k done
  uint64_t* v_full = k_empty + kQk;            // [kV]
  uint64_t* v_empty = v_full + kV;             // [kV]
  uint64_t* v_clean = v_empty + kV;            // [kV] V without what is not finite or not the sequence's
  uint64_t* s_full = v_clean + kV;             // [2] q . k in TMEM
  uint64_t* p_full = s_full + 2;               // [2] P in TMEM
  uint64_t* o_full = p_full + 2;               // [2] OI and OX done
  uint64_t* o_empty = o_full + 2;              // [2] ... read out: P's tile and OX's are free
  uint64_t* v_ready = o_empty + 2;             // [2] V' and K^T of half the tokens written
  uint64_t* v_taken = v_ready + 2;             // [2] ... multiplied
  uint64_t* st_ready = v_taken + 2;            // the state's bf16 form written
  uint64_t* st_taken = st_ready + 1;           // Q S done
  uint64_t* d_full = st_ready + 2;             // K^T V' done
  uint64_t* d_empty = st_ready + 3;            // ... added to the state
  uint64_t* i_full = d_empty + 1;              // [kRing] a piece of work is there
  uint64_t* i_empty = i_full + kRing;          // [kRing] ... taken by all
  Ring* const ring = reinterpret_cast<Ring*>(smem + oRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + oSlot);
  const dsi_linear& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kQk; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&k_full[i], 1);
      mbar_init(&q_empty[i], 2);
      mbar_init(&k_empty[i], LOCAL ? 8 : 1 + 8);
    }
    for (int i = 0; i < kV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], LOCAL ? 8 : 1);
      mbar_init(&v_clean[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 2);
      mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_ready[i], 4);
      mbar_init(&v_taken[i], 1);
    }
    mbar_init(st_ready, 8);
    mbar_init(st_taken, 1);
    mbar_init(d_full, 1);
    mbar_init(d_empty, 8);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&i_full[i], 1);
      mbar_init(&i_empty[i], LOCAL ? 17 : 27);   // the warps that take pieces
    }
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
  if (plan.split) {                            // the sequences' first segments
    int total;
    const int n = tid < p.batch ? segments_of(p, plan, tid) : 0;
    const int before = block_exclusive_scan(n, reinterpret_cast<int*>(smem), total);
    if (tid <= p.batch) reinterpret_cast<int*>(table_s)[tid] = total > plan.segments ? tid : before;
    __syncthreads();
  } else if (p.batch <= kMaxOrder) {           // the sequences, longest first
    int* len = reinterpret_cast<int*>(smem);
    int64_t first;
    int n = 0;
    if (tid < p.batch) tokens_of(p, tid, first, n);
    if (tid < p.batch) len[tid] = n;
    __syncthreads();
    if (tid < p.batch) {
      int rank = 0;
      for (int b = 0; b < p.batch; ++b) rank += len[b] > n || (len[b] == n && b < tid);
      table_s[rank] = (uint8_t)tid;
    }
    __syncthreads();
  } else {                                     // which of them are long
    uint32_t* bits = reinterpret_cast<uint32_t*>(table_s);
    const int shift = bit_shift(p);
    if (tid < kBits / 32) bits[tid] = 0u;
    __syncthreads();
    for (int b0 = tid; b0 < p.batch; b0 += 4 * kThreads) {
      int n[4] = {};
      int64_t first;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (b0 + i * kThreads < p.batch) tokens_of(p, b0 + i * kThreads, first, n[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = (b0 + i * kThreads) >> shift;
        if (n[i] > p.few && !(reinterpret_cast<volatile uint32_t*>(bits)[at >> 5] >> (at & 31) & 1u))
          atomicOr(bits + (at >> 5), 1u << (at & 31));
      }
    }
    __syncthreads();
  }
  fence_proxy_async_smem();                    // copies land where the lengths were
  __syncthreads();
  grid_dep_launch();
  const uint32_t tmem = *tmem_slot;
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  const int row = (warp & 3) * 32 + lane;      // of a chunk, or of the state
  Item it;
  int items = 0;                               // taken so far
  int t = 0;                                   // chunks so far
  bool ok = true;
  // the role's next piece of work; false at the list's end
  auto next_item = [&]() {
    do {
      if (!(ok = wait32(&i_full[items % kRing], (uint32_t)(items / kRing) & 1u))) return false;
      peek(ring, items, it);
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[items % kRing]);
      ++items;
    } while (it.h == kNothingYet);
    return it.h >= 0;
  };

  if (warp == 3) {
    // ======================= copies ==============================================
    if (lane == 0) {
      int round = 0;
#pragma unroll 1
      while (ok) {
        look_up<LOCAL>(p, plan, table_s, round, it);
        if (!(ok = wait1(&i_empty[items % kRing], ((uint32_t)(items / kRing) & 1u) ^ 1u))) break;
        publish(ring, items, it);
        mbar_arrive(&i_full[items % kRing]);
        ++items;
        if (it.h == kNothingYet) continue;
        if (it.h < 0) break;
        const int hk = it.h / p.group;
#pragma unroll 1
        for (int c = it.c0; c < it.c1; ++c, ++t) {
          const int s = t % kQk, sv = t % kV, at = it.first + c * kC;
          const uint32_t ph = ((uint32_t)(t / kQk) & 1u) ^ 1u;
          if (!(ok = wait1(&k_empty[s], ph))) break;
          mbar_arrive_expect_tx(&k_full[s], KB * kTile);
#pragma unroll
          for (int x = 0; x < KB; ++x)
            tma_load_3d(smem + oK + (s * 2 + x) * kTile, &kmap, x * 64, hk, at, &k_full[s]);
          if (!(ok = wait1(&v_empty[sv], ((uint32_t)(t / kV) & 1u) ^ 1u))) break;
          mbar_arrive_expect_tx(&v_full[sv], kTile);
          tma_load_3d(smem + oV + sv * kTile, &vmap, it.part * kCols, hk, at, &v_full[sv]);
          if constexpr (!LOCAL) {
            if (!(ok = wait1(&q_empty[s], ph))) break;
            mbar_arrive_expect_tx(&q_full[s], KB * kTile);
#pragma unroll
            for (int x = 0; x < KB; ++x)
              tma_load_3d(smem + oQ + (s * 2 + x) * kTile, &qmap, x * 64, it.h, at, &q_full[s]);
          }
        }
      }
      // never leave the CTA with a copy still landing in shared memory (of chunk t some may be
      // under way: a wait that nothing ends is bounded)
      if (s_abort) {
        volatile int no_abort = 0;
        for (int i = max(0, t - max(kQk, kV)); i <= t; ++i) {
          if (!LOCAL) mbar_wait(&q_full[i % kQk], (uint32_t)(i / kQk) & 1u, &no_abort, p.err, 1000000ull);
          mbar_wait(&k_full[i % kQk], (uint32_t)(i / kQk) & 1u, &no_abort, p.err, 1000000ull);
          mbar_wait(&v_full[i % kV], (uint32_t)(i / kV) & 1u, &no_abort, p.err, 1000000ull);
        }
      }
    }
  } else if (warp == 1) {
    // ======================= D = K^T V' ==========================================
    const uint64_t d_vp = desc_sw128_mn(smem_u32(smem + oVp), kTile);
#pragma unroll 1
    while (ok && next_item()) {
#pragma unroll 1
      for (int c = it.c0; c < it.c1; ++c, ++t) {
        const uint32_t ph = (uint32_t)t & 1u;
        if (!(ok = wait32(d_empty, ph ^ 1u))) break;
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {     // 64 tokens at a time: the next chunk's go where they were
          if (!(ok = wait32(&v_ready[hf], ph))) break;
          tc_fence_after();
#pragma unroll 4
          for (int x = 0; x < kSplit * 4; ++x) {
            const int step = hf * 4 + (x & 3);
            mma_bf16_tmem_a_elect(tmem + TM_D, tmem + TM_KT + step * 8, d_vp + (uint64_t)(((x >> 2) * kTile + step * 2048) >> 4), IDESC_O,
                     hf + x > 0 ? 1u : 0u);
          }
          mma_commit_elect(&v_taken[hf]);
        }
        if (!ok) break;
        mma_commit_elect(d_full);
      }
    }
    __syncwarp();
  } else if (!LOCAL && warp == 2) {
    // ======================= Q K^T ===============================================
#pragma unroll 1
    while (ok && next_item()) {
#pragma unroll 1
      for (int c = it.c0; c < it.c1; ++c, ++t) {
        const int s = t % kQk;
        const uint32_t ph = (uint32_t)(t / kQk) & 1u;
        if (!(ok = wait32(&k_full[s], ph) && wait32(&q_full[s], ph) &&
                   wait32(&o_empty[t & 1], ((uint32_t)(t >> 1) & 1u) ^ 1u)))
          break;
        tc_fence_after();
        const uint64_t q = desc_sw128(smem_u32(smem + oQ + s * 2 * kTile)), k = desc_sw128(smem_u32(smem + oK + s * 2 * kTile));
#pragma unroll 4
        for (int x = 0; x < 4 * KB; ++x) {
          const uint64_t off = (uint64_t)(((x >> 2) * kTile + (x & 3) * 32) >> 4);
          mma_bf16_elect(tmem + TM_P + (t & 1) * kC, q + off, k + off, IDESC_P, x > 0 ? 1u : 0u);
        }
        mma_commit_elect(&s_full[t & 1]);
        mma_commit_elect(&k_empty[s]);
        mma_commit_elect(&q_empty[s]);
      }
    }
    __syncwarp();
  } else if (!LOCAL && warp == 0) {
    // ======================= Q S, P V ============================================
    const uint64_t d_s = desc_sw128_mn(smem_u32(smem + oS), kTile);
#pragma unroll 1
    while (ok && next_item()) {
#pragma unroll 1
      for (int c = it.c0; c < it.c1; ++c, ++t) {
        const int s = t % kQk;
        const uint32_t ph = (uint32_t)t & 1u;
        if (!(ok = wait32(st_ready, ph) && wait32(&q_full[s], (uint32_t)(t / kQk) & 1u) &&
                   wait32(&o_empty[t & 1], ((uint32_t)(t >> 1) & 1u) ^ 1u)))
          break;
        tc_fence_after();
        const uint64_t q = desc_sw128(smem_u32(smem + oQ + s * 2 * kTile));
#pragma unroll 4
        for (int x = 0; x < 4 * KB; ++x)
          mma_bf16_elect(tmem + TM_OX + (t & 1) * kCols, q + (uint64_t)(((x >> 2) * kTile + (x & 3) * 32) >> 4), d_s + (uint64_t)((x * 2048) >> 4),
                   IDESC_O, x > 0 ? 1u : 0u);
        mma_commit_elect(st_taken);
        mma_commit_elect(&q_empty[s]);
        mma_commit_elect(&o_full[t & 1]);
        if (!(ok = wait32(&v_clean[t % kV], (uint32_t)(t / kV) & 1u) && wait32(&p_full[t & 1], (uint32_t)(t >> 1) & 1u))) break;
        tc_fence_after();
        const uint64_t v = desc_sw128_mn(smem_u32(smem + oV + (t % kV) * kTile), kTile);
#pragma unroll 4
        for (int x = 0; x < kC / 16; ++x)
          mma_bf16_tmem_a_elect(tmem + TM_OI + (t & 1) * kC, tmem + TM_P + (t & 1) * kC + x * 8, v + (uint64_t)((x * 2048) >> 4), IDESC_O,
                          x > 0 ? 1u : 0u);
        mma_commit_elect(&o_full[t & 1]);
        mma_commit_elect(&v_empty[t % kV]);
      }
    }
    __syncwarp();
  } else if (!LOCAL && warp >= 4 && warp < 8) {
    // ======================= P ===================================================
    // Thread = token i, blocks of 32 tokens j: whole ones before the warp's own rows take
    // lam^(i-j) as lam^(i-j31) lam^(j31-j) (j31 the block's last token: both
    // exponents are positive), the warp's own block by table; the rest is 0.
    const int w = warp & 3;
    float* const pow_s = pow_table[w + 1];
    float far_of[3] = {0.f, 0.f, 0.f};         // lam^(i-j31) of the blocks before the warp's own
    int h = -1;
#pragma unroll 1
    while (ok && next_item()) {
      if (it.h != h) {
        h = it.h;
        const float g = it.g;
        __syncwarp();
        pow_s[lane] = a.scale * power(g, lane);
#pragma unroll
        for (int i = 0; i < 3; ++i) far_of[i] = power(g, max(0, row - i * 32 - 31));
        __syncwarp();
      }
#pragma unroll 1
      for (int c = it.c0; c < it.c1; ++c, ++t) {
        if (!(ok = wait32(&s_full[t & 1], (uint32_t)(t >> 1) & 1u))) break;
        tc_fence_after();
        const uint32_t t_p = tmem + lane_base + TM_P + (t & 1) * kC;
#pragma unroll 1
        for (int b = 0; b < 8; ++b) {          // 16 tokens
          uint32_t out[8];
          if (b <= 2 * w + 1) {
            float v[16];
            tmem_ld16(t_p + b * 16, v);
            const float* f_s = pow_s - (b & 1) * 16;
            float far = b < 2 ? far_of[0] : b < 4 ? far_of[1] : far_of[2];
            tmem_ld_wait();
            if (b < 2 * w) {
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(f_s + 28 - j);
                const float2 y0 = mul2(make_float2(v[j], v[j + 1]), mul2(make_float2(far, far), make_float2(f.w, f.z)));
                const float2 y1 = mul2(make_float2(v[j + 2], v[j + 3]), mul2(make_float2(far, far), make_float2(f.y, f.x)));
                out[j / 2] = pack_bf16(y0.x, y0.y);
                out[j / 2 + 1] = pack_bf16(y1.x, y1.y);
              }
            } else {
              const int own = lane - (b & 1) * 16;   // (what is read in front of the table is masked)
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float2 f = make_float2(f_s[lane - j], f_s[lane - j - 1]);
                const float2 y = mul2(make_float2(v[j], v[j + 1]), f);
                out[j / 2] = pack_bf16(j <= own ? y.x : 0.f, j + 1 <= own ? y.y : 0.f);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = 0u;
          }
          tmem_st_words<8>(t_p + b * 8, out);  // (over logits that this thread has read)
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t & 1]);
      }
    }
  } else if (warp >= 8 && warp < 16) {
    // ======================= V' and K^T ==========================================
    // Four warps to half the tokens.  V': thread = half a row of V, decayed and cut into parts once
    // the products with the V' before are done.  K^T: a warp turns 32 dims, 8 x 8 at a time.
    const int w = warp - 8, hf = w >> 2, u0 = (w & 1) * 4, quarter = w & 3;
    const int v_row0 = hf * 64 + ((w >> 1) & 1) * 32, v_row = v_row0 + lane;
    const uint32_t k_lane = (uint32_t)(hf * 64 + ((lane >> 4) & 1) * 8 + (lane & 7));        // token whose address this lane gives
    const uint32_t k_u = (uint32_t)((quarter & 1) * 4 + ((lane >> 3) & 1));                  // ... and 8 dims
#pragma unroll 1
    while (ok && next_item()) {
      const float g = it.g;
      float f = 0.f;
#pragma unroll 1
      for (int c = it.c0; c < it.c1; ++c, ++t) {
        const int s = t % kQk, sv = t % kV, r = min(kC, it.n - c * kC);
        uint8_t* st = smem + oV + sv * kTile;
        if (c == it.c0 || r < kC) f = v_row < r ? power(g, r - 1 - v_row) : 0.f;
        if (!(ok = wait32(&v_full[sv], (uint32_t)(t / kV) & 1u))) break;
        uint4 v[4];                              // (as they are: three parts of each would be 48 registers)
        float2 all = make_float2(0.f, 0.f);    // not finite if one of the values is not
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[u] = *reinterpret_cast<const uint4*>(st + sw128_offset((uint32_t)v_row, (uint32_t)(u0 + u)));
          const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) all = add2(all, __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[e])));
        }
        const bool bad = v_row < r && !(fabsf(all.x) + fabsf(all.y) < INFINITY);   // (or their sum)
        if (v_row >= r) {                        // behind the sequence: what K and V hold must not meet weights of 0
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t off = sw128_offset((uint32_t)v_row, (uint32_t)(u0 + u));
            *reinterpret_cast<uint4*>(st + off) = v[u] = make_uint4(0, 0, 0, 0);
          }
        }
        const bool any = __any_sync(0xffffffffu, bad);
        if (lane == 0) reinterpret_cast<volatile int*>(smem + oBad)[t % kMarks * 8 + w] = any;
        if (__builtin_expect(any, 0)) {
          uint8_t* first = smem + oFirst + (t % kMarks * 8 + w) * 32;
#pragma unroll 1
          for (int x = 0; x < 32; ++x) {
            uint16_t* e = reinterpret_cast<uint16_t*>(st + sw128_offset((uint32_t)v_row, (uint32_t)(u0 + (x >> 3)))) + (x & 7);
            const bool out = v_row < r && (*e & 0x7F80u) == 0x7F80u;
            const uint32_t who = __ballot_sync(0xffffffffu, out);
            if (out) *e = 0;
            if (lane == 0) first[x] = who ? (uint8_t)(v_row0 + __ffs(who) - 1) : (uint8_t)kC;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(LOCAL ? &v_empty[sv] : &v_clean[sv]);   // (nobody else reads it, or P V does)
        if (t > 0 && !(ok = wait32(&v_taken[hf], (uint32_t)(t - 1) & 1u))) break;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          uint32_t part[kSplit][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 y = mul2(__bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[e])), make_float2(f, f));
#pragma unroll
            for (int i = 0; i < kSplit; ++i) {   // the upper 16 bits (8 of the value), and what they leave
              const uint32_t lo = __float_as_uint(y.x), hi = __float_as_uint(y.y);
              part[i][e] = __byte_perm(lo, hi, 0x7632);
              y = add2(y, make_float2(-__uint_as_float(lo & 0xFFFF0000u), -__uint_as_float(hi & 0xFFFF0000u)));
            }
          }
#pragma unroll
          for (int i = 0; i < kSplit; ++i)
            *reinterpret_cast<uint4*>(smem + oVp + i * kTile + sw128_offset((uint32_t)v_row, (uint32_t)(u0 + u))) =
                make_uint4(part[i][0], part[i][1], part[i][2], part[i][3]);
        }
        fence_proxy_async_smem();
        if (!(ok = wait32(&k_full[s], (uint32_t)(t / kQk) & 1u))) break;
        tc_fence_after();
        if (quarter < 2 * KB) {
          const uint32_t kt = smem_u32(smem + oK + (s * 2 + (quarter >> 1)) * kTile);
#pragma unroll 1
          for (int m = 0; m < 2; ++m) {        // 16 dims
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 4; ++i)        // 16 tokens
              ldmatrix4_trans(kt + sw128_offset(k_lane + i * 16, k_u + m * 2), x + 4 * i);
            if (r < kC) {                      // behind the sequence: zeros
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int j = hf * 64 + (i >> 1) * 8 + (lane & 3) * 2;
                x[i] &= (j < r ? 0xFFFFu : 0u) | (j + 1 < r ? 0xFFFF0000u : 0u);
              }
            }
            tmem_st_16x128b_x8(tmem + ((uint32_t)(quarter * 32 + m * 16) << 16) + TM_KT + hf * 32, x);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&k_empty[s]);
          mbar_arrive(&v_ready[hf]);
        }
      }
    }
  } else if (warp >= 16 && warp < 24) {
    // ======================= the state ===========================================
    // Thread = 32 columns of a row of the state; rows from dk on are zeros, and none behind the
    // last block of 64.
    const bool rows = (warp & 3) < 2 * KB, live = row < a.dk;
    const bool wide = (reinterpret_cast<uintptr_t>(a.state) & 31) == 0;
    const int half = (warp - 16) >> 2;
#pragma unroll 1
    while (ok && next_item()) {
      const float g = it.g;
      const int64_t src = it.src, dst = it.dst;
      const int cols = live ? min(32, a.dv - it.part * kCols - half * 32) : 0;   // a multiple of 8, or none
      const int64_t head = ((int64_t)it.h * a.dk + row) * a.dv + it.part * kCols + half * 32;
      const int64_t slot = (int64_t)a.n_heads * a.dk * a.dv;
      float s[32], d1 = 0.f;
      const float* from = it.seg >= 0 ? plan.seg + it.seg * slot + head : src >= 0 ? a.state + src * slot + head : nullptr;
      float* to = it.last && dst >= 0 && (dst != src || it.n > 0) ? a.state + dst * slot + head : nullptr;
      if (LOCAL) {
        from = nullptr;
        to = plan.seg + it.seg * slot + head;
      }
#pragma unroll
      for (int x = 0; x < 32; x += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[x + i] = 0.f;
        if (from && x < cols) load8(from + x, wide, s + x);
      }
#pragma unroll 1
      for (int c = it.c0; c < it.c1; ++c, ++t) {
        if (c == it.c0 || it.n - c * kC < kC) d1 = expm1f(g * (float)min(kC, it.n - c * kC));
        if constexpr (!LOCAL) {
          if (t > 0 && !(ok = wait32(st_taken, (uint32_t)(t - 1) & 1u))) break;
          if (rows) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              *reinterpret_cast<uint4*>(smem + oS + sw128_offset((uint32_t)row, (uint32_t)(half * 4 + u))) =
                  make_uint4(pack_bf16(s[8 * u], s[8 * u + 1]), pack_bf16(s[8 * u + 2], s[8 * u + 3]),
                             pack_bf16(s[8 * u + 4], s[8 * u + 5]), pack_bf16(s[8 * u + 6], s[8 * u + 7]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(st_ready);
        }
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          const float2 y = make_float2(s[x], s[x + 1]), z = fma2(y, make_float2(d1, d1), y);
          s[x] = z.x; s[x + 1] = z.y;
        }
        if (!(ok = wait32(d_full, (uint32_t)t & 1u))) break;
        tc_fence_after();
        if (rows) {
#pragma unroll
          for (int x = 0; x < 32; x += 16) {
            float d[16];
            tmem_ld16(tmem + lane_base + TM_D + half * 32 + x, d);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 z = add2(make_float2(s[x + i], s[x + i + 1]), make_float2(d[i], d[i + 1]));
              s[x + i] = z.x; s[x + i + 1] = z.y;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty);
      }
      if (ok && to) {
#pragma unroll
        for (int x = 0; x < 32; x += 8)
          if (x < cols) store8(to + x, wide, s + x);
      }
      __syncwarp();
    }
  } else if (!LOCAL && warp >= 24) {
    // ======================= outputs =============================================
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && a.ld_out_row % 16 == 0 && a.ld_out_head % 16 == 0;
#pragma unroll 1
    while (ok && next_item()) {
      const float since = a.scale * power(it.g, row + 1);
      const int cols = min(kCols, a.dv - it.part * kCols);
#pragma unroll 1
      for (int c = it.c0; c < it.c1; ++c, ++t) {
        if (!(ok = wait32(&o_full[t & 1], (uint32_t)(t >> 1) & 1u))) break;
        tc_fence_after();
        const bool live = row < it.n - c * kC;
        bf16* to = reinterpret_cast<bf16*>(a.out) + ((int64_t)it.first + c * kC + row) * a.ld_out_row +
                   (int64_t)it.h * a.ld_out_head + it.part * kCols;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {          // 16 columns at a time
          float x[16], y[16];
          tmem_ld16(tmem + lane_base + TM_OI + (t & 1) * kC + q * 16, x);
          tmem_ld16(tmem + lane_base + TM_OX + (t & 1) * kCols + q * 16, y);
          tmem_ld_wait();
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 z = fma2(make_float2(y[2 * i], y[2 * i + 1]), make_float2(since, since), make_float2(x[2 * i], x[2 * i + 1]));
            o[i] = pack_bf16(z.x, z.y);
          }
          const int left = cols - q * 16;
          if (live) {
            if (wide && left >= 16) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(to + q * 16), "r"(o[0]),
                           "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                           : "memory");
            } else {
              if (left >= 8) reinterpret_cast<uint4*>(to + q * 16)[0] = make_uint4(o[0], o[1], o[2], o[3]);
              if (left >= 16) reinterpret_cast<uint4*>(to + q * 16)[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
          __syncwarp();
        }
        const uint4 bad0 = *reinterpret_cast<const uint4*>(smem + oBad + t % kMarks * 32);
        const uint4 bad1 = *reinterpret_cast<const uint4*>(smem + oBad + t % kMarks * 32 + 16);
        if (__builtin_expect(bad0.x | bad0.y | bad0.z | bad0.w | bad1.x | bad1.y | bad1.z | bad1.w, 0u)) {
          const uint8_t* first = smem + oFirst + t % kMarks * 8 * 32;
#pragma unroll 1
          for (int x = 0; x < (live ? cols : 0); ++x) {
            int from = kC;
#pragma unroll 1
            for (int i = x >> 5; i < 8; i += 2)          // the warps that had this column
              if (reinterpret_cast<const int*>(smem + oBad)[t % kMarks * 8 + i]) from = min(from, (int)first[i * 32 + (x & 31)]);
            if (row >= from) to[x] = __float2bfloat16(__int_as_float(0x7fc00000));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_empty[t & 1]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
}

// Split: what the segments of a sequence add, one after another, becomes what each of them finds.  A
// thread takes four columns of a row; eight segments' loads are under way together.
constexpr int kCarryThreads = 256;
__global__ void __launch_bounds__(kCarryThreads)
linear_carry(const __grid_constant__ LinearArgs p, const __grid_constant__ Plan plan) {
  __shared__ int first_s, total_s;
  const int per = p.a.dk * p.a.dv / 4, heads = p.a.n_heads;     // float4s of a head's state
  const int blocks = (heads * per + kCarryThreads - 1) / kCarryThreads;
  const int b = blockIdx.x / blocks, e = (blockIdx.x - b * blocks) * kCarryThreads + threadIdx.x;
  grid_dep_wait();
  grid_dep_launch();
  if (threadIdx.x == 0) first_s = total_s = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.batch; i += kCarryThreads) {
    const int m = segments_of(p, plan, i);
    if (i < b) atomicAdd(&first_s, m);         // those of the sequences before
    atomicAdd(&total_s, m);
  }
  __syncthreads();
  const int segs = segments_of(p, plan, b);
  if (segs <= 1 || total_s > plan.segments || e >= heads * per) return;
  const int64_t slot = (int64_t)heads * per, src = in_slot(p, b);
  float4* at = reinterpret_cast<float4*>(plan.seg) + first_s * slot + e;
  const float d1 = expm1f(__ldg(p.a.log_decay + e / per) * (float)(plan.split * kC));
  float4 s = src >= 0 ? reinterpret_cast<const float4*>(p.a.state)[src * slot + e] : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < segs; i0 += 8) {
    float4 add[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      add[i] = i0 + i + 1 < segs ? at[(i0 + i) * slot] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i0 + i >= segs) break;
      at[(i0 + i) * slot] = s;
      s.x = fmaf(s.x, d1, s.x) + add[i].x;
      s.y = fmaf(s.y, d1, s.y) + add[i].y;
      s.z = fmaf(s.z, d1, s.z) + add[i].z;
      s.w = fmaf(s.w, d1, s.w) + add[i].w;
    }
  }
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

namespace {

// Chunks of a segment, or 0 where sequences stay whole.  Times in chunks of one CTA: whole
// sequences take their length; a split takes its share of all chunks 1.6 times (the first
// pass reads K and V again) and three launches, about kSplitCost.  The host knows no length but the mean.
// A segment is then no shorter than sequences of that length allow in one round of CTAs: with the bare
// share a few segments more than there are CTAs doubled the last two launches (4 x 4096 tokens of 8 heads 114 us, so 77).
// us of heads of 128 x 128, whole and split (those that the rule takes marked *):
//   tokens x heads  1024 x 1 *23 / 21, 1536 x 1 31 / *22, 4096 x 1 72 / *23, 1536 x 8 32 / *24, 8192 x 8 137 / *46,
//     1024 x 16 *24 / 26, 1536 x 16 *32 / 29, 2048 x 16 40 / *33, 16384 x 16 265 / *132, 2048 x 32 *40 / 47,
//     3584 x 32 65 / *69, 8192 x 32 138 / *132, 4096 x 45 *74 / 82, 8192 x 60 *142 / 152
//   sequences       4 x 1024 x 2 *25 / 25, 4 x 2048 x 2 41 / *28, 4 x 2048 x 8 *42 / 48, 4 x 4096 x 8 75 / *77,
//     4 x 8192 x 8 139 / *132, 8 x 8192 x 2 138 / *77, 8 x 4096 x 8 *78 / 87
//   mixed           16000 and 3 of 4000, 8 heads 261 / *214; 6000, 5000, 4000, 3000 105 / *85; where the mean
//     misleads: 8192 and 7 of 40 *138 / 56
constexpr int kSplitCost = 8;
int segment_chunks(int64_t n_tokens, int batch, int H, int dv, int sms) {
  const int64_t chunks = (n_tokens + kC - 1) / kC, columns = (int64_t)H * ((dv + kCols - 1) / kCols);
  if (batch > kMaxSplit || batch * columns >= sms) return 0;
  const int64_t share = ((chunks + batch - 1) * columns + sms - 1) / sms;
  if (10 * (chunks / batch) <= 16 * share + 10 * kSplitCost) return 0;
  const int64_t mean = (chunks + batch - 1) / batch, pieces = sms / (batch * columns), even = (mean + pieces - 1) / pieces;
  const int64_t n = share > even ? share : even;
  return (int)(n < 2 ? 2 : n);
}
// At most so many segments (a sequence has one more than it has whole ones).
int64_t segments(int64_t n_tokens, int batch, int split) {
  return ((n_tokens + kC - 1) / kC + batch) / split + batch;
}

template <int KB, bool LOCAL>
cudaError_t launch(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, const LinearArgs& p,
                   const Plan& plan, int sms, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(linear_chunk<KB, LOCAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_overlapped(linear_chunk<KB, LOCAL>, dim3((unsigned)(plan.items < sms ? plan.items : sms)), dim3(kThreads),
                        kSmem, st, qmap, kmap, vmap, p, plan);
  note_launch();
  return e;
}

}  // namespace

size_t linear_prefill_workspace(int64_t n_tokens, int batch, int H, int dk, int dv) {
  const int split = segment_chunks(n_tokens, batch, H, dv, sm_count());
  return split ? (size_t)segments(n_tokens, batch, split) * H * dk * dv * sizeof(float) : 256;
}

// Sequences of at most so many tokens go token by token, in a launch of their own: decoding rows of a mixed
// batch, say.  us for 64 sequences x 32 heads of 128 x 128, so and by chunks: 1 token 48 / 133, 4 62 / 134, 8
// 85 / 135, 16 129 / 135; one sequence 3.6 / 9.3, 8 tokens 5.2 / 9.3, 16 7.3 / 9.3.  The launch costs 1 to 2 %
// where no sequence is short: 4 x 2048 tokens 82.7 -> 83.3 us, 64 x 200 192 -> 195.
constexpr int kFew = 8;

cudaError_t launch_linear_prefill(const LinearArgs& given, void* ws, cudaStream_t st) {
  LinearArgs p = given;
  p.few = -1;
  // (whatever can be refused is refused before the first launch)
  CUtensorMap qmap, kmap, vmap;
  if (p.n_tokens > kFew &&
      (!map_heads(&qmap, p.a.q, p.n_tokens, p.a.n_heads, p.a.dk, p.a.ld_q_row, p.a.ld_q_head) ||
       !map_heads(&kmap, p.a.k, p.n_tokens, p.a.n_kv_heads, p.a.dk, p.a.ld_k_row, p.a.ld_k_head) ||
       !map_heads(&vmap, p.a.v, p.n_tokens, p.a.n_kv_heads, p.a.dv, p.a.ld_v_row, p.a.ld_v_head)))
    return cudaErrorInvalidValue;
  if (p.batch > 1 || p.n_tokens <= kFew) {       // (one sequence among more rows than that is hardly as short)
    p.few = kFew;
    const cudaError_t e = launch_linear_recurrent(p, st);
    if (e != cudaSuccess || p.n_tokens <= kFew) return e;
  }
  const int sms = sm_count();
  Plan plan;
  plan.parts = (p.a.dv + kCols - 1) / kCols;
  plan.split = ws ? segment_chunks(p.n_tokens, p.batch, p.a.n_heads, p.a.dv, sms) : 0;
  plan.segments = plan.split ? (int)segments(p.n_tokens, p.batch, plan.split) : 0;
  plan.items = (plan.split ? plan.segments : p.batch) * p.a.n_heads * plan.parts;
  plan.seg = static_cast<float*>(ws);
  const bool wide = p.a.dk > 64;
  cudaError_t e;
  if (plan.split) {
    e = wide ? launch<2, true>(qmap, kmap, vmap, p, plan, sms, st) : launch<1, true>(qmap, kmap, vmap, p, plan, sms, st);
    if (e != cudaSuccess) return e;
    const int blocks = (p.a.n_heads * p.a.dk * p.a.dv / 4 + kCarryThreads - 1) / kCarryThreads;
    e = launch_overlapped(linear_carry, dim3((unsigned)(p.batch * blocks)), dim3(kCarryThreads), 0, st, p, plan);
    note_launch();
    if (e != cudaSuccess) return e;
  }
  return wide ? launch<2, false>(qmap, kmap, vmap, p, plan, sms, st) : launch<1, false>(qmap, kmap, vmap, p, plan, sms, st);
}

}  // namespace dsi
