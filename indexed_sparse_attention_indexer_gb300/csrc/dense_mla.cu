// Attention over the whole latent cache, or over a sliding window of it with
// the first positions visible, on the tcgen05 tensor cores.
//
// The rows of the MMA's M dimension are 128 (query token, head) pairs: as many
// consecutive tokens of one sequence as fit (a group; 128 heads: one token).
// One group's fp32 output (128 x 512) alone would fill a CTA's tensor memory,
// so a cluster of two CTAs shares a group by dimension:
//   CTA 0: logits over key dims   0..255 and 512..543, output dims   0..255
//   CTA 1: logits over key dims 256..511 and 544..575, output dims 256..511
// and the two partial logit tiles (128 x 64 positions, fp32) are swapped
// through distributed shared memory, so that both take the same softmax
// decisions.  Every cache row is read once from HBM for a group.
//
// A group's positions are cut into tiles of 64 aligned positions: those that
// hold sinks, then those from the window's start to the end of the history.
// The groups' tiles (and kGroupCost tiles' worth for each group's start and end),
// laid end to end, are dealt out in equal contiguous runs to the clusters (one
// resident per SM pair): a run may end inside a group, whose pieces are then
// joined by a second kernel from their running maxima and sums.  Where dealing
// out whole groups costs at most kWholeSlack tiles more, groups stay whole and
// nothing is joined.
//
// Roles in a CTA (16 warps; FP8 rows: 24), each walking the same list of pieces; the
// tile pipeline runs on across pieces:
//   producers (warps 0-1): a tile's rows into a 128-byte-swizzled stage (ring of 4)
//     by TMA boxes (warp 0; FP8 rows: into raw tiles), a group's queries (warp 1);
//     in tiles at an edge (not wholly visible to every token of the group) warp 1
//     turns rows that nobody sees into zeros, so that what they hold never meets the
//     tensor core (FP8 rows: the converting warps do);
//   logit issuer (warp 3): S = Qslice . C^T into one of two TMEM tiles;
//   exchange (warps 4-7): the group's query slice into TMEM (rope half: shared
//     memory); this CTA's partial logits out of TMEM into the peer's buffer;
//   softmax (warps 8-15, one row per thread, two sets of four warps, a half of each
//     tile's positions a set): own partial plus the peer's, mask, online softmax in
//     log2 units with a lazily moved reference max (the accumulator is rescaled only
//     when the max grows by more than 2^8), P in bf16 to shared memory, and the epilogue;
//   value issuer (warp 2): O += P . V from the same stage, a half tile at a time;
//   conversion (FP8 rows, warps 16-23): codes times scales, rounded to bf16, out of
//     the raw tiles into the stages.
// Exchange and softmax warps of lane quarters without rows (few heads) leave at
// once: what the tensor core computes there is never read.
// Every wait is bounded; the cluster syncs after set-up and before exit.
//
// What bounds it.  64 sequences of 32768 positions, 128 heads, bf16 rows: 580 us at 2070
// MHz, 4.2 TB/s (62 % of the measured copy rate) and 1007 TFLOP/s (53 % of the library
// GEMM's); 605 to 622 us where the power cap holds the clock near 1950 MHz.  A tile takes
// a cluster about 2750 cycles (the time's cycles over its 431 tiles).  Its bytes take
// 1700, its MMAs 1340 (64 columns
// take 46 cycles, not 32; P.V is at its rate), the exchange 1600 (distributed shared
// memory carries 20 bytes a cycle and SM each way): each is idle for a third to a half of
// the time, because a stage is held for ~10,000 cycles, from its copy to the end of its
// P.V, and there is room for four.  4096 tokens of 128 heads over windows of 1024: 1349
// us, 768 TFLOP/s: the same, and the softmax warps' 2.5 us for each group's output.
// Three softmax sets (640 threads) took 650 us, 64 positions of a tile in each of two
// sets in turn 812.
#include "dense_mla.h"

#include <atomic>

#include "kernels.h"
#include "tc_common.cuh"
#include "tma_host.h"

namespace dsi {
using namespace tc;

namespace {

constexpr int kM = 128;                        // rows of a group: (token, head) pairs
constexpr int kNp = 64;                        // positions per tile
constexpr int kBlockBytes = kNp * 128;         // 64 dims of a tile
constexpr int kRopeHalf = 32;                  // rope dims of each CTA
constexpr int kRopeOff = 4 * kBlockBytes;      // stage: four 64-dim blocks, then 64 rows of rope dims
constexpr int kRowBytes = 4 * 128 + kRopeHalf * 2;
constexpr int kStageBytes = kNp * kRowBytes;   // 36 KB
// 16 warps (four per SM sub-partition), at most 128 registers a thread; FP8 rows: 24, 80
constexpr int kProducers = 2;                  // warps 0-1
constexpr int kPvWarp = 2;
constexpr int kQkWarp = 3;                     // then exchange: warps 4-7
constexpr int kConvWarp0 = 16;                 // FP8 rows: conversion, warps 16-23
constexpr int kSmWarp0 = 8;                    // softmax: warps 8-11 first halves, 12-15 second ones
constexpr int kMaxClusters = 128;
// In tiles.  us at 4 / 8 / 16 / 32: 777 tokens of 32 heads over windows of 511 79.5 / 67.3 /
// 67.3 / 67.3 (FP8 rows 107.6 / 95.8 / 95.9 / 95.9), 100 x 512 x 128 heads 44.5 / 39.8 / 39.8 /
// 37.0, 48 x 2 tokens x 700 x 64 heads 45.1 / 27.6 / 25.3 / 25.3, 1000 tokens of 64 heads over
// windows of 200 103.3 / 103.5 / 90.1 / 90.1, 90 x 2000 x 128 heads 90.5 / 90.2 / 90.1 / 99.2.
constexpr int kWholeSlack = 8;
// What a piece costs beside its tiles, in tiles.  us at 2 / 4 / 6 / 8: 17 x 3000 x 128 heads 41.6 /
// 39.8 / 39.5 / 40.4, 90 x 2000 92.2 / 90.2 / 90.1 / 86.6, 100 x 512 39.8 / 39.8 / 49.1 / 46.4, 120
// of up to 1500 41.1 / 40.7 / 41.3 / 43.6.
constexpr int kGroupCost = 4;
// tiles between L2 prefetch and copy (64 x 32768 x 128 heads: 2 661 us, 4 635, 8 645, 16 714)
constexpr int kAhead = 4;
// partial logits travel in quarters of a tile (16 positions): three in flight for
// each half of a tile hide the round trip of a buffer (credit, stores, landing)
constexpr int kQuarter = 16;
constexpr int kHalf = 32;                      // positions of a softmax step
constexpr int kXRing = 3;
constexpr int kXBytes = kM * kQuarter * 4;

// FP8 rows: raw tiles of codes land beside the ring and are converted into it by eight
// warps (with four 308 us against 289 for 64 x 8192 x 128 heads, now 265).  A stage is
// held from the start of its conversion to the end of its P.V, 14,000 cycles over the
// three stages that there is room for (conversion 3500, logits 2400, exchange 3300,
// softmax and P.V 3400): that bounds them, not the bytes, of which bf16 rows have twice
// as many and take 175 us.
constexpr int kRawStages = 2;
constexpr int kRawRope = 2 * kNp * 128;        // two blocks of 128 dims, then 64 rows of 32 rope dims
constexpr int kRawBytes = kNp * (256 + kRopeHalf);

template <bool F8>
struct Layout {                                // shared memory, bytes
  static constexpr int stages = F8 ? 3 : 4;
  static constexpr int threads = F8 ? 768 : 512;
  static constexpr int fill_warps = F8 ? 9 : 2;   // warps that pass a slot of the ring on
  static constexpr int c = 0;
  static constexpr int raw = c + stages * kStageBytes;
  static constexpr int p = raw + (F8 ? kRawStages * kRawBytes : 0);   // P [128 x 64] bf16
  static constexpr int x = p + kM * kNp * 2;   // [2 halves][kXRing] the peer's partial logits
  static constexpr int qr = x + 2 * kXRing * kXBytes;                 // query rope half
  static constexpr int ref = qr + kM * kRopeHalf * 2;                 // reference maxima of the rows
  static constexpr int sums = ref + kM * 4;    // [2][2][128] (reference, sum) of both sets
  static constexpr int bar = sums + 4 * kM * 8;
  static constexpr int bars = 3 * stages + 16 + 4 * kXRing + 2 * kRawStages;
  static constexpr int misc = bar + bars * 8;
  static constexpr int scan = misc + 64;       // 40 ints
  static constexpr int bytes = scan + 160 + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory");
  static_assert(raw % 1024 == 0 && p % 1024 == 0 && qr % 512 == 0 && misc % 8 == 0, "alignment");
};

constexpr uint32_t TM_S = 0;      // two logit tiles of 64 columns
constexpr uint32_t TM_Q = 128;    // query slice: four 64-dim blocks, 128 columns
constexpr uint32_t TM_O = 256;    // output half, 256 columns
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t IDESC_S = idesc_f32(1, kM, kNp);
constexpr uint32_t IDESC_O = idesc_f32_bmn(1, kM, 256);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.f;

// What a cluster leaves for the join: the group that its last piece starts and
// does not finish (or -1), the group that its first piece continues (or -1),
// and whether it finishes it.
struct Record { int starts, continues, finishes, pad; };
struct Workspace {
  float* o;        // [2 * clusters][128][512] unnormalised outputs
  float2* ml;      // [2 * clusters][128] reference max, sum of weights
  Record* rec;     // [clusters]
};

struct Plan {
  int tokens;      // tokens of a group
  int per_seq;     // groups of a sequence
  int groups;
  int split;       // a workspace is there
  int live;        // lane quarters (32 rows) that a full group has rows in
};

struct Group {
  int b, row0, nt;             // sequence, first query row, tokens
  int n_first, n_last;         // visible lengths of the first and last token
  int lo, main0, sink_tiles, tiles;
};

__device__ __forceinline__ Group group_of(const DenseArgs& a, const Plan& p, int g) {
  Group r;
  r.b = p.per_seq == 1 ? g : g / p.per_seq;
  const int t0 = (g - r.b * p.per_seq) * p.tokens;
  r.nt = min(p.tokens, a.T - t0);
  r.row0 = r.b * a.T + t0;
  r.n_first = (int)visible_len(a.c, r.row0, a.decode, a.q_offset);
  r.n_last = r.nt == 1 ? r.n_first
                       : (int)visible_len(a.c, r.row0 + r.nt - 1, a.decode, a.q_offset);
  r.lo = max(0, r.n_first - (int)a.window);
  r.main0 = r.lo / kNp;
  r.sink_tiles = min((min((int)a.n_sink, r.lo) + kNp - 1) / kNp, r.main0);
  // a group that sees nothing still has a (wholly masked) tile: its output is written
  r.tiles = max(1, r.sink_tiles + max(0, (r.n_last + kNp - 1) / kNp - r.main0));
  return r;
}
__device__ __forceinline__ int tile_pos(const Group& g, int t) {
  return (t < g.sink_tiles ? t : g.main0 + t - g.sink_tiles) * kNp;
}
// Every token of the group sees all positions p0 .. p0 + len - 1.
__device__ __forceinline__ bool all_see(const DenseArgs& a, const Group& g, int p0, int len) {
  return p0 + len <= g.n_first && (p0 >= g.n_last - (int)a.window || p0 + len <= (int)a.n_sink);
}
__device__ __forceinline__ bool any_sees(const DenseArgs& a, const Group& g, int p) {
  return p < g.n_last && (p >= g.lo || p < (int)a.n_sink);
}

// A cluster's pieces: whole groups g, g + stride, ..., or what lies in a run of
// `left` units of the groups' costs laid end to end, from unit u of group g.  A
// group costs kGroupCost units (its queries, its output), then one a tile; a run
// that ends inside the former leaves the group to the next.
struct Walk {
  int g, u, left, stride;      // stride > 0: whole groups
};
struct Piece {
  Group grp;
  int g, t0, t1;
};
__device__ __forceinline__ bool next_piece(const DenseArgs& a, const Plan& p, Walk& w, Piece& x) {
  if (w.g >= p.groups || w.left <= 0) return false;
  x.g = w.g;
  x.grp = group_of(a, p, w.g);
  if (w.stride > 0) {
    x.t0 = 0;
    x.t1 = x.grp.tiles;
    w.g += w.stride;
    return true;
  }
  const int end = min(x.grp.tiles + kGroupCost, w.u + w.left);
  x.t0 = max(0, w.u - kGroupCost);
  x.t1 = max(0, end - kGroupCost);
  w.left -= end - w.u;
  w.u = 0;
  ++w.g;                       // (a run that ends inside the group has nothing left)
  return x.t1 > x.t0;
}

// Cache row of position p of sequence b; -1 (reported) for a bad page id.
__device__ __forceinline__ int row_of(const CacheView& c, int b, int p, int* err) {
  if (!c.block_table) return (int)((int64_t)b * c.s_max + p);
  const int pg = p / c.page_size;
  const int page = __ldg(c.block_table + (int64_t)b * c.max_pages + pg);
  if (page < 0 || page >= c.num_pages) { report(err, kErrBounds); return -1; }
  return page * c.page_size + (p - pg * c.page_size);
}

// Asks for `bytes` contiguous bytes (16-byte aligned, a multiple of 16) to be
// brought into L2.
__device__ __forceinline__ void bulk_prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Shared-memory descriptor of a K-major operand with rows of 64 bytes and 64-byte
// swizzle (atoms of 512 bytes).
__device__ __forceinline__ uint64_t desc_sw64(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(16u >> 4) << 16;                  // leading byte offset (unused here)
  d |= (uint64_t)(512u >> 4) << 32;                 // stride byte offset: next 8-row atom
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)4 << 61;                           // 64-byte swizzle
  return d;
}

// 16-byte chunk u of row r of such a tile (byte offset).
__host__ __device__ __forceinline__ uint32_t sw64_offset(uint32_t r, uint32_t u) {
  return r * 64u + ((u ^ ((r >> 1) & 3u)) << 4);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16 E4M3 codes times their tile scale, the fp32 product rounded to bf16 (lo =
// codes 0..7).
__device__ __forceinline__ void e4m3x16_scaled(const uint4& v, float sc, uint4& lo, uint4& hi) {
  float f[16];
  fp8x16_to_f32(v, f);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 p = unpack2(mul2(pack2(f[2 * i], f[2 * i + 1]), pack2(sc, sc)));
    const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  lo = make_uint4(w[0], w[1], w[2], w[3]);
  hi = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ bool bf16x8_finite(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    ok = ok && (w[i] & 0x7F80u) != 0x7F80u && (w[i] & 0x7F800000u) != 0x7F800000u;
  return ok;
}

// The rows of a stage whose bits are set become zeros, by a warp: a store of the warp
// covers four rows of a block, or eight rows of rope dims.  (One lane a row took 2500 to
// 9500 cycles for a tile at an edge.)
__device__ __forceinline__ void clear_rows(uint8_t* st, uint64_t rows, int lane) {
  const uint64_t four = rows >> (lane >> 3), eight = rows >> (lane >> 2);
  uint8_t* at = st + lane * 16;
#pragma unroll 1
  for (int blk = 0; blk < 4; ++blk, at += kBlockBytes)
#pragma unroll
    for (int i = 0; i < kNp / 4; ++i)
      if ((four >> (4 * i)) & 1u) *reinterpret_cast<uint4*>(at + i * 512) = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kNp / 8; ++i)
    if ((eight >> (8 * i)) & 1u) *reinterpret_cast<uint4*>(at + i * 512) = make_uint4(0, 0, 0, 0);
}

// Bounded waits whose slow path is out of line and takes few arguments: the
// roles' loops together have to stay small enough for the instruction cache.
__shared__ volatile int s_abort;               // a role has given up: the others follow
__shared__ int* s_err;                         // device status word

__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    if (ok) return true;
    if ((i & 255u) == 0) {
      if (s_abort) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        s_abort = 1;
        report(s_err, kErrTimeout);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || wait_on(smem_u32(bar), parity);
}
// Whole warps: all lanes proceed or none.
__device__ __forceinline__ bool wait32(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait1(bar, parity));
}
// ... for phases that the other CTA's arrivals and stores complete
__device__ __forceinline__ bool wait32_cluster(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity) || wait_on(smem_u32(bar), parity));
}

// A wait in two parts, for roles whose time is latency: ask early, work on, and
// wait only where the answer was no (a ready wait alone costs ~150 cycles).
__device__ __forceinline__ bool ask_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool settle(bool asked, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, asked || wait_on(smem_u32(bar), parity));
}

// Bits 0 .. k-1 of 64.
__device__ __forceinline__ uint64_t low_bits(int k) {
  return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1ull;
}

// 32 bytes, a whole sector: one store where the address allows, else two.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <bool F8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Layout<F8>::threads, 1)
dense_mla_tc(const __grid_constant__ CUtensorMap lmap, const __grid_constant__ CUtensorMap rmap,
             const __grid_constant__ CUtensorMap qmap, const __grid_constant__ DenseArgs a,
             const __grid_constant__ Plan plan, Workspace ws, int box) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  using Y = Layout<F8>;
  constexpr int kStages = Y::stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Y::bar);   // [kStages] tile in place
  uint64_t* empty = full + kStages;            // [kStages] stage free (value MMAs done)
  uint64_t* landed = empty + kStages;          // [kStages] an edge tile's copies landed
  uint64_t* s_full = landed + kStages;         // [2] logits in TMEM
  uint64_t* s_empty = s_full + 2;              // [2] logits read out (exchange and softmax)
  uint64_t* p_empty = s_full + 4;              // [2 halves] P.V done
  uint64_t* p_full = s_full + 6;               // [2 halves] P written
  uint64_t* q_ready = s_full + 8;              // query slice in place
  uint64_t* o_done = s_full + 9;               // a piece's last P.V done
  uint64_t* ref_set = s_full + 10;             // [4] a half tile's reference maxima (per lane quarter)
  uint64_t* sums_set = s_full + 14;            // both softmax sets' sums of a piece
  uint64_t* o_free = s_full + 15;              // a piece's output read out
  uint64_t* x_full = s_full + 16;              // [2 halves][kXRing] the peer's partial logits landed
  uint64_t* x_empty = x_full + 2 * kXRing;     // [2][kXRing] the peer has read what we sent
  uint64_t* raw_full = x_empty + 2 * kXRing;   // [kRawStages] FP8: codes landed
  uint64_t* raw_empty = raw_full + kRawStages; // [kRawStages] FP8: codes converted
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Y::misc);
  int* start_s = reinterpret_cast<int*>(smem + Y::misc + 8);                   // group, unit
  int* widest_s = reinterpret_cast<int*>(smem + Y::misc + 16);
  unsigned long long* total_s = reinterpret_cast<unsigned long long*>(smem + Y::misc + 24);
  unsigned int* taken_s = reinterpret_cast<unsigned int*>(smem + Y::misc + 32);
  int* scan_s = reinterpret_cast<int*>(smem + Y::scan);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rho = cluster_ctarank();
  const uint32_t peer = rho ^ 1u;
  const int k = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  int* err = a.err;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], Y::fill_warps);
      mbar_init(&empty[s], 1);
      mbar_init(&landed[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 3 * plan.live);
      mbar_init(&p_empty[i], 1);
      mbar_init(&p_full[i], plan.live);
    }
    mbar_init(q_ready, 32 * plan.live);
    mbar_init(o_done, 1);
    for (int i = 0; i < 2 * kXRing; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_empty[i], plan.live);
    }
    for (int i = 0; i < kRawStages; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 8);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&ref_set[i], 1);
    mbar_init(sums_set, plan.live * 2);
    mbar_init(o_free, plan.live * 2);
    taken_s[0] = taken_s[1] = 0u;
    s_abort = 0;
    s_err = err;
    start_s[0] = plan.groups;
    start_s[1] = 0;
    *widest_s = 0;
    *total_s = 0ull;
    fence_barrier_init();
  }
  if (warp == kQkWarp) tmem_alloc(tmem_slot, TMEM_COLS);
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&lmap);
    prefetch_tmap(&rmap);
    prefetch_tmap(&qmap);
  }
  grid_dep_wait();     // lengths, queries and cache rows may come from the kernel before
  __syncthreads();

  // ---- the cluster's share of the tiles (every CTA computes the same split) ----
  if (plan.split) {
    unsigned long long sum = 0;
    int widest = 0;
    for (int g = tid; g < plan.groups; g += Y::threads) {
      const int n = group_of(a, plan, g).tiles + kGroupCost;
      sum += (unsigned)n;
      widest = max(widest, n);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      widest = max(widest, __shfl_xor_sync(0xffffffffu, widest, o));
    }
    if (lane == 0) {
      atomicAdd(total_s, sum);
      atomicMax(widest_s, widest);
    }
  }
  __syncthreads();
  const unsigned long long total = *total_s;
  const unsigned long long even = (total + clusters - 1) / clusters;
  const unsigned long long whole =
      (unsigned long long)((plan.groups + clusters - 1) / clusters) * (unsigned)*widest_s;
  Walk walk;
  if (!plan.split || total >= (1ull << 30) || whole <= even + kWholeSlack) {
    walk.g = k;
    walk.u = 0;
    walk.left = 1;
    walk.stride = clusters;
  } else {
    const int share = (int)even;
    const long long start = (long long)share * k;
    long long before = 0;
    for (int g0 = 0; g0 < plan.groups && start < (long long)total; g0 += Y::threads) {
      const int g = g0 + tid;
      const int n = g < plan.groups ? group_of(a, plan, g).tiles + kGroupCost : 0;
      int chunk;
      const int at = block_exclusive_scan(n, scan_s, chunk);
      if (n > 0 && start >= before + at && start < before + at + n) {
        start_s[0] = g;
        start_s[1] = (int)(start - before - at);
      }
      before += chunk;
      if (start < before) break;               // uniform: found in this chunk
    }
    __syncthreads();
    walk.g = start_s[0];
    walk.u = start_s[1];
    walk.left = share;
    walk.stride = 0;
  }
  const uint32_t x_bytes = (uint32_t)plan.live * (kXBytes / 4);
  if (tid == 0)                                // the peer's first quarters
    for (int i = 0; i < 2 * kXRing; ++i) mbar_arrive_expect_tx(&x_full[i], x_bytes);
  tc_fence_before();
  cluster_sync();      // the peer's barriers exist (and are armed) before anyone uses them
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = *tmem_slot;

  if (warp < kProducers) {
    // ======================= producers ==========================================
    // A piece takes two ring slots for its query slice, then one a tile.
    Piece x;
    int slot = 0, tg = 0;                      // ring slots; tiles
    uint32_t edge_ph = 0;                      // parities of landed[]
    uint32_t issued = 0, issued_edge = 0;      // stages with a copy in flight; into an edge tile
    const int64_t cache_rows = a.c.block_table ? a.c.num_pages * a.c.page_size : a.c.batch * a.c.s_max;
    bool ok = true;
    // Every warp that waits for the ring's slots waits for each of them and arrives on
    // each of their full barriers, whoever fills it: a phase that it has not seen cannot
    // pass.  (A warp that left slots out could not tell by a parity which release it saw.)
    // FP8 rows: the ring is filled by the converting warps and, with queries, warp 1;
    // warp 0's copies go to the raw stages.
#pragma unroll 1
    while (ok && next_piece(a, plan, walk, x)) {
#pragma unroll 1
      for (int i = 0; i < 2 && (!F8 || warp == 1); ++i, ++slot) {
        const int stage = slot % kStages;
        if (!(ok = wait32(&empty[stage], ((uint32_t)(slot / kStages) & 1u) ^ 1u))) break;
        if (lane == 0) {
          // (by warp 1, while warp 0 goes on to the tiles)
          if (warp == 1) {
            uint8_t* st = smem + Y::c + stage * kStageBytes;
            mbar_arrive_expect_tx(&full[stage], 2 * kM * 128);
            issued |= 1u << stage;
            issued_edge &= ~(1u << stage);
            for (int bx = 0; bx < 2; ++bx)
              tma_load_2d(st + bx * kM * 128, &qmap, (int)rho * 256 + (2 * i + bx) * 64,
                          x.grp.row0 * a.H, &full[stage]);
          } else {
            mbar_arrive(&full[stage]);
          }
        }
      }
      if (!ok) break;
      int asked = x.t0;
#pragma unroll 1
      for (int t = x.t0; t < x.t1; ++t, ++tg, ++slot) {
        const bool raw = F8 && warp == 0;
        const int stage = raw ? tg % kRawStages : slot % kStages;
        const uint32_t ph = (uint32_t)(raw ? tg / kRawStages : slot / kStages) & 1u;
        const int p0 = tile_pos(x.grp, t);
        uint8_t* st = smem + (F8 ? Y::raw + stage * kRawBytes : Y::c + stage * kStageBytes);
        const bool whole = F8 || all_see(a, x.grp, p0, kNp);
        if (warp == 0) {
          // the tile by TMA, boxes of `box` rows (a page or a part of one) by 128 bytes of
          // dims; boxes that no token sees are left out
          uint64_t* bar = F8 ? &raw_full[stage] : whole ? &full[stage] : &landed[stage];
          if (!(ok = wait32(F8 ? &raw_empty[stage] : &empty[stage], ph ^ 1))) break;
          constexpr int kBlks = F8 ? 3 : 5;      // blocks of 128 bytes a row, the last the rope half
          const int boxes = kNp / box;
          const int pb = p0 + lane * box;        // lane's box, if it has one
          const bool seen = lane < boxes && pb < x.grp.n_last && (pb + box > x.grp.lo || pb < (int)a.n_sink);
          const int n = __popc(__ballot_sync(0xffffffffu, seen));
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, (uint32_t)(n * box * (F8 ? kRawBytes / kNp : kRowBytes)));
            if (!whole) mbar_arrive(&full[stage]);
            if (!F8) {
              issued |= 1u << stage;
              issued_edge = whole ? issued_edge & ~(1u << stage) : issued_edge | (1u << stage);
              edge_ph ^= whole ? 0u : 1u << stage;
            }
          }
          __syncwarp();
#pragma unroll 1
          for (int i = lane; i < boxes * kBlks; i += 32) {
            const int bx = i / kBlks, blk = i - bx * kBlks, p = p0 + bx * box;
            if (!(p < x.grp.n_last && (p + box > x.grp.lo || p < (int)a.n_sink))) continue;
            const int row = row_of(a.c, x.grp.b, p, err);
            // a bad page id: the box past the tensor's last row, which reads as zeros
            const int y = row < 0 ? (int)a.c.num_pages * a.c.page_size : row;
            if (blk < kBlks - 1)
              tma_load_2d(st + blk * kBlockBytes + bx * box * 128, &lmap,
                          (int)rho * 256 + blk * (256 / (kBlks - 1)), y, bar);
            else
              tma_load_2d(st + (F8 ? kRawRope + bx * box * kRopeHalf : kRopeOff + bx * box * kRopeHalf * 2),
                          &rmap, DSI_D_LATENT + (int)rho * kRopeHalf, y, bar);
          }
          // decode: the caches come from HBM; tiles are asked for into L2 kAhead tiles
          // before their copies (two a step until that far ahead, each CTA every other
          // tile, whole rows), so that a copy holds its stage only as long as L2 takes
          if (a.decode) {
            asked = max(asked, t + 2);
            for (int n2 = 0; n2 < 2 && asked < min(x.t1, t + kAhead); ++n2, ++asked) {
              const int p = tile_pos(x.grp, asked) + lane * box;
              if ((asked & 1) == (int)rho && lane < boxes && p < x.grp.n_last &&
                  (p + box > x.grp.lo || p < (int)a.n_sink)) {
                const int row = row_of(a.c, x.grp.b, p, err);
                constexpr int kPitch = F8 ? DSI_D_QK : 2 * DSI_D_QK;
                if (row >= 0 && (int64_t)row + box <= cache_rows)
                  bulk_prefetch_l2(reinterpret_cast<const uint8_t*>(a.c.latent) + (int64_t)row * kPitch,
                                   (uint32_t)(box * kPitch));
              }
            }
          }
          __syncwarp();
        } else {
          // warp 1 passes a whole tile on and cleans one at an edge first (FP8 rows: passes
          // on the slot, which holds no copy of its own any more)
          if (!whole) {
            // rows that no token sees become zeros (weight 0 times what they hold must
            // be 0); a row that only some tokens see and that holds NaN or an infinity
            // becomes zeros as a value and NaN in its rope dims: its logits are NaN, for
            // those that see it
            uint64_t none = 0, some = 0;         // rows that no token sees; that only some see
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int p = p0 + h * 32 + lane;
              const bool seen = any_sees(a, x.grp, p);
              none |= (uint64_t)__ballot_sync(0xffffffffu, !seen) << (32 * h);
              some |= (uint64_t)__ballot_sync(0xffffffffu, seen && !all_see(a, x.grp, p, 1)) << (32 * h);
            }
            if (!(ok = wait32(&landed[stage], (edge_ph >> stage) & 1u))) break;
            edge_ph ^= 1u << stage;
            clear_rows(st, none, lane);
            for (; some != 0ull; some &= some - 1ull) {      // (the warp looks at a row together)
              const int rr = __ffsll((long long)some) - 1;
              uint4* const c = reinterpret_cast<uint4*>(st + (lane >> 3) * kBlockBytes + sw128_offset(rr, lane & 7));
              uint4* const e = reinterpret_cast<uint4*>(st + kRopeOff + sw64_offset(rr, lane & 3));
              if (__any_sync(0xffffffffu, !bf16x8_finite(*c) || !bf16x8_finite(*e))) {
                *c = make_uint4(0, 0, 0, 0);
                if (lane < 4) *e = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
              }
            }
            fence_proxy_async_smem();   // the tensor core reads the stage through the async proxy
            __syncwarp();
          } else if (!(ok = wait32(&empty[stage], ph ^ 1))) {
            break;
          }
          if (F8) issued &= ~(1u << stage);
          if (lane == 0) mbar_arrive(&full[stage]);
        }
      }
    }
    // never leave the CTA with a copy still landing in shared memory
    if (lane == 0 && s_abort) {
      volatile int no_abort = 0;    // the drain is bounded by time only
#pragma unroll 1
      for (int s = 0; s < kStages; ++s) {
        if (!((issued >> s) & 1u)) continue;
        int last = slot;            // the last slot that used stage s
        while (last > 0 && last % kStages != s) --last;
        if ((issued_edge >> s) & 1u) mbar_wait(&landed[s], ((edge_ph >> s) & 1u) ^ 1u, &no_abort, err, 100000000ull);
        else mbar_wait(&full[s], (uint32_t)(last / kStages) & 1u, &no_abort, err, 100000000ull);
      }
      if (F8 && warp == 0)
        for (int i = max(0, tg - kRawStages); i < tg; ++i)
          mbar_wait(&raw_full[i % kRawStages], (uint32_t)(i / kRawStages) & 1u, &no_abort, err, 100000000ull);
    }
  } else if (F8 && warp >= kConvWarp0) {
    // ======================= FP8: conversion ======================================
    // Two threads for each half of a row: four pieces of 16 codes and half of the rope
    // piece for each: code * tile scale, rounded to bf16, into the ring stage.  The page is looked up two tiles ahead and the scales
    // are loaded one ahead, within a piece.
    const int c_thread = tid - kConvWarp0 * 32, rr = c_thread & 63, hh = c_thread >> 7, part = (c_thread >> 6) & 1;
    const int s0 = (int)rho * 2 + hh;            // tile of this thread's 128 latent dims
    Piece x = {};
    int slot = 0, tg = 0;
    bool ok = true;
    auto lookup = [&](int t) {                    // cache row of this thread's row of tile t
      const int p = t < x.t1 ? tile_pos(x.grp, t) + rr : -1;
      return p >= 0 && any_sees(a, x.grp, p) ? row_of(a.c, x.grp.b, p, err) : -1;
    };
    auto scales = [&](int row) {                  // of the latent dims and of the rope dims
      return row < 0 ? make_float2(0.f, 0.f)
                     : make_float2(__ldg(a.latent_scale + (int64_t)row * 5 + s0),
                                   __ldg(a.latent_scale + (int64_t)row * 5 + 4));
    };
#pragma unroll 1
    while (ok && next_piece(a, plan, walk, x)) {
      // (the query slots are waited for and passed on)
      for (int i = 0; i < 2 && ok; ++i, ++slot) {
        ok = wait32(&empty[slot % kStages], ((uint32_t)(slot / kStages) & 1u) ^ 1u);
        if (ok && lane == 0) mbar_arrive(&full[slot % kStages]);
      }
      if (!ok) break;
      int row_next = lookup(x.t0);
      float2 sc = scales(row_next);
      row_next = lookup(x.t0 + 1);
#pragma unroll 1
      for (int t = x.t0; t < x.t1; ++t, ++tg, ++slot) {
        const int stage = slot % kStages, rs = tg % kRawStages, p = tile_pos(x.grp, t) + rr;
        const float2 sc_next = scales(row_next);
        row_next = lookup(t + 2);
        const bool whole = all_see(a, x.grp, p - rr, kNp);       // the tile
        const bool seen = whole || any_sees(a, x.grp, p), partly = seen && !whole && !all_see(a, x.grp, p, 1);
        const uint8_t* raw = smem + Y::raw + rs * kRawBytes;
        uint8_t* st = smem + Y::c + stage * kStageBytes;
        if (!(ok = wait32(&raw_full[rs], (uint32_t)(tg / kRawStages) & 1u))) break;
        if (!(ok = wait32(&empty[stage], ((uint32_t)(slot / kStages) & 1u) ^ 1u))) break;
        bool bad = false;
#pragma unroll 1
        for (int i = 0; i < 5; ++i) {
          const bool rope = i == 4;              // (last: it takes the pieces' NaN)
          const int u = part * 4 + i;
          uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
          if (seen) {
            const uint4 v = *reinterpret_cast<const uint4*>(
                rope ? raw + kRawRope + rr * kRopeHalf + hh * 16 : raw + hh * kBlockBytes + sw128_offset(rr, u));
            e4m3x16_scaled(v, rope ? sc.y : sc.x, lo, hi);
          }
          // (edges: as for bf16 rows)
          if (__builtin_expect(!whole, 0)) {
            if (partly && !(bf16x8_finite(lo) && bf16x8_finite(hi))) {
              bad = true;
              lo = hi = make_uint4(0, 0, 0, 0);
            }
            if (rope && bad) lo = hi = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
          }
          uint8_t* blk = st + (hh * 2 + part) * kBlockBytes;
          if (rope)
            *reinterpret_cast<uint4*>(st + kRopeOff + sw64_offset(rr, hh * 2 + part)) = part ? hi : lo;
          else
            *reinterpret_cast<uint4*>(blk + sw128_offset(rr, 2 * i)) = lo,
            *reinterpret_cast<uint4*>(blk + sw128_offset(rr, 2 * i + 1)) = hi;
        }
        sc = sc_next;
        fence_proxy_async_smem();   // the tensor core reads the stage through the async proxy
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[rs]);
          mbar_arrive(&full[stage]);
        }
      }
    }
  } else if (warp == kQkWarp) {
    // ======================= logit issuer =======================================
    if (lane == 0) {
      Piece x;
      int slot = 0, tg = 0, pieces = 0;
      bool ok = true;
      const uint64_t qr = desc_sw64(smem_u32(smem + Y::qr));
#pragma unroll 1
      while (ok && next_piece(a, plan, walk, x)) {
        if (!(ok = wait1(q_ready, (uint32_t)pieces & 1u))) break;
        ++pieces;
        slot += 2;                               // the query slice
#pragma unroll 1
        for (int t = x.t0; t < x.t1; ++t, ++tg, ++slot) {
          const int stage = slot % kStages, sb = tg & 1;
          if (!(ok = wait1(&full[stage], (uint32_t)(slot / kStages) & 1u))) break;
          if (!(ok = wait1(&s_empty[sb], ((uint32_t)(tg >> 1) & 1u) ^ 1u))) break;
          tc_fence_after();
          const uint32_t t_s = tmem + TM_S + sb * kNp;
          const uint32_t base = smem_u32(smem + Y::c + stage * kStageBytes);
          const uint64_t d0 = desc_sw128(base);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            mma_bf16_tmem_a(t_s, tmem + TM_Q + i * 8,
                            d0 + (uint64_t)(((i >> 2) * kBlockBytes + (i & 3) * 32) >> 4), IDESC_S,
                            i > 0 ? 1u : 0u);
          const uint64_t dr = desc_sw64(base + kRopeOff);
#pragma unroll
          for (int i = 0; i < kRopeHalf / 16; ++i)
            mma_bf16(t_s, qr + (uint64_t)((i * 32) >> 4), dr + (uint64_t)((i * 32) >> 4), IDESC_S, 1u);
          mma_commit(&s_full[sb]);
        }
      }
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ======================= value issuer =======================================
    if (lane == 0) {
      Piece x;
      int slot = 0, tg = 0;
      bool ok = true;
      const uint64_t pd = desc_sw128(smem_u32(smem + Y::p));
#pragma unroll 1
      while (ok && next_piece(a, plan, walk, x)) {
        slot += 2;                               // the query slice
#pragma unroll 1
        for (int t = x.t0; t < x.t1; ++t, ++tg, ++slot) {
          const int stage = slot % kStages;
          const uint64_t vd = desc_sw128_mn(smem_u32(smem + Y::c + stage * kStageBytes), kBlockBytes);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            if (!(ok = wait1(&p_full[hf], (uint32_t)tg & 1u))) break;
            tc_fence_after();
#pragma unroll
            for (int i = 2 * hf; i < 2 * hf + 2; ++i)
              mma_bf16(tmem + TM_O, pd + (uint64_t)((i * 32) >> 4), vd + (uint64_t)((i * 2048) >> 4),
                       IDESC_O, (t > x.t0 || i > 0) ? 1u : 0u);
            mma_commit(&p_empty[hf]);
          }
          if (!ok) break;
          mma_commit(&empty[stage]);
          if (t + 1 == x.t1) mma_commit(o_done);
        }
      }
    }
    __syncwarp();
  } else if (warp < kSmWarp0) {
    // ======================= exchange ===========================================
    const int m = (warp & 3) * 32 + lane;              // row = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // exchange buffers [4-position group][row] x float4: a warp's stores of one
    // group are 512 contiguous bytes
    const uint32_t x_remote = map_to_rank(smem_u32(smem + Y::x), peer) + m * 16;
    const uint32_t xfull_remote = map_to_rank(smem_u32(x_full), peer);
    const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;   // a negative scale turns the queries' signs
    Piece x;
    int slot = 0, tg = 0;
    bool ok = true;
#pragma unroll 1
    while (ok && (warp & 3) < plan.live && next_piece(a, plan, walk, x)) {
      // The query slice: the rope half by plain loads (begun first), the four 64-dim
      // blocks out of the two ring slots that the producers filled ahead.  The
      // logit MMAs of the piece before are done: this warp has seen all its tiles.
      const bool live = m < x.grp.nt * a.H;
      uint4 rope[kRopeHalf / 8];
#pragma unroll
      for (int i = 0; i < kRopeHalf / 8; ++i)
        rope[i] = live ? __ldg(reinterpret_cast<const uint4*>(
                             a.q + ((int64_t)x.grp.row0 * a.H + m) * DSI_D_QK + DSI_D_LATENT + rho * kRopeHalf) + i)
                       : make_uint4(0, 0, 0, 0);
#pragma unroll 1
      for (int half = 0; half < 2; ++half, ++slot) {
        const int stage = slot % kStages;
        if (!(ok = wait32(&full[stage], (uint32_t)(slot / kStages) & 1u))) break;
#pragma unroll
        for (int bx = 0; bx < 2; ++bx) {
          const uint8_t* src = smem + Y::c + stage * kStageBytes + bx * kM * 128;
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 y = *reinterpret_cast<const uint4*>(src + sw128_offset(m, i));
            w[4 * i] = y.x ^ sign; w[4 * i + 1] = y.y ^ sign;
            w[4 * i + 2] = y.z ^ sign; w[4 * i + 3] = y.w ^ sign;
          }
          tmem_st32(tmem + lane_base + TM_Q + (half * 2 + bx) * 32, w);
        }
        tmem_st_wait();
        // the last of the live warps returns the slot (no barrier between them: a
        // warp that has given up must not leave the others waiting); a warp can be a
        // slot ahead of another but not a piece, so each half has its own count
        __syncwarp();
        if (lane == 0) {
          __threadfence_block();
          if ((atomicAdd(taken_s + half, 1u) + 1u) % (unsigned)plan.live == 0u) mbar_arrive(&empty[stage]);
        }
      }
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kRopeHalf / 8; ++i)
        *reinterpret_cast<uint4*>(smem + Y::qr + sw64_offset(m, i)) =
            make_uint4(rope[i].x ^ sign, rope[i].y ^ sign, rope[i].z ^ sign, rope[i].w ^ sign);
      slot += x.t1 - x.t0;
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(q_ready);
#pragma unroll 1
      for (int t = x.t0; t < x.t1; ++t, ++tg) {
        const int sb = tg & 1;
        if (!(ok = wait32(&s_full[sb], (uint32_t)(tg >> 1) & 1u))) break;
        tc_fence_after();
        // (a short loop and few registers at a time, here and in the softmax: the roles
        // share an instruction cache and, FP8 rows, 80 registers; with 64 logits at
        // once 4 % more time, FP8 8 %)
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          float v[kQuarter];
          tmem_ld16(tmem + lane_base + TM_S + sb * kNp + i * kQuarter, v);
          // once the peer has read what was in its buffer
          const int n = tg * 2 + (i & 1), buf = (i >> 1) * kXRing + n % kXRing;   // n: of this half so far
          if (!(ok = wait32_cluster(&x_empty[buf], ((uint32_t)(n / kXRing) & 1u) ^ 1u))) break;
          tmem_ld_wait();
          if (i == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[sb]);
          }
#pragma unroll
          for (int j = 0; j < kQuarter; j += 4)
            st_async_v4(x_remote + buf * kXBytes + j * (kM * 4),
                        make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]), xfull_remote + buf * 8);
        }
        if (!ok) break;
      }
    }
  } else {
    // ======================= softmax + epilogue ==================================
    // Two sets of four warps take a half each of every tile.  The reference maximum passes from half to half as soon as a half's
    // maximum is known, and each half has its own P.V; each set sums its own weights.
    const int set = (warp - kSmWarp0) >> 2, hf = set;        // the half of a tile
    const int quarter = warp & 3, m = quarter * 32 + lane;   // row = TMEM lane
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    uint8_t* const pbuf = smem + Y::p;
    const uint8_t* xrow = smem + Y::x + m * 16;
    volatile float* const ref_s = reinterpret_cast<float*>(smem + Y::ref) + m;
    const uint32_t xempty_remote = map_to_rank(smem_u32(x_empty), peer);
    // a scale of 0 becomes the smallest normal one: logits of 0, and "masked" times it stays -inf
    const float sl2 = a.scale == 0.f ? 1.17549435e-38f : fabsf(a.scale) * kLog2e;
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    Record rec = {-1, -1, 0, 0};
    Piece x;
    int tg = 0, pieces = 0;
    bool ok = true;
#pragma unroll 1
    while (ok && quarter < plan.live && next_piece(a, plan, walk, x)) {
      const int tok = min(m / a.H, x.grp.nt - 1);
      const int n_row = tok == 0 ? x.grp.n_first
                                 : (int)visible_len(a.c, x.grp.row0 + tok, a.decode, a.q_offset);
      const int lo_row = n_row - (int)a.window;
      float m_mine = -INFINITY, l_mine = 0.f;
#pragma unroll 1
      for (int t = x.t0; t < x.t1; ++t, ++tg) {
        const int sb = tg & 1;
        if (!(ok = wait32(&s_full[sb], (uint32_t)(tg >> 1) & 1u))) break;
        tc_fence_after();
        const int p0 = tile_pos(x.grp, t) + hf * kHalf;
        // this CTA's partial logits and the peer's
        float v[kHalf];
        tmem_ld32(tmem + lane_base + TM_S + sb * kNp + hf * kHalf, v);
        const int n0 = tg * 2, b0 = hf * kXRing + n0 % kXRing, b1 = hf * kXRing + (n0 + 1) % kXRing;
        const uint32_t ph0 = (uint32_t)(n0 / kXRing) & 1u, ph1 = (uint32_t)((n0 + 1) / kXRing) & 1u;
        const bool here0 = ask_cluster(&x_full[b0], ph0), here1 = ask_cluster(&x_full[b1], ph1);
        if (!(ok = settle(here0 && here1, &x_full[b0], ph0) && settle(here1, &x_full[b1], ph1))) break;
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[sb]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* xb = xrow + (i ? b1 : b0) * kXBytes;
          float4 y[kQuarter / 4];
          asm volatile("" ::: "memory");         // (the loads stay in their batch)
#pragma unroll
          for (int g4 = 0; g4 < kQuarter / 4; ++g4) y[g4] = *reinterpret_cast<const float4*>(xb + g4 * (kM * 16));
#pragma unroll
          for (int g4 = 0; g4 < kQuarter / 4; ++g4) {
            const int j = i * kQuarter + 4 * g4;
            const float2 s0 = unpack2(add2(pack2(v[j], v[j + 1]), pack2(y[g4].x, y[g4].y)));
            const float2 s1 = unpack2(add2(pack2(v[j + 2], v[j + 3]), pack2(y[g4].z, y[g4].w)));
            v[j] = s0.x; v[j + 1] = s0.y; v[j + 2] = s1.x; v[j + 3] = s1.y;
          }
        }
        // masked positions: -inf
        if (__builtin_expect(!all_see(a, x.grp, p0, kHalf), 0)) {
          const uint32_t see = (uint32_t)(low_bits(n_row - p0) &
                                          (~low_bits(lo_row - p0) | low_bits((int)a.n_sink - p0)));
#pragma unroll
          for (int j = 0; j < kHalf; ++j) v[j] = (see >> j) & 1u ? v[j] : -INFINITY;
        }
        const bool ref_here = (tg == 0 && hf == 0) || mbar_test_wait(&ref_set[quarter], (uint32_t)(hf ^ 1));
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(v[j], v[j + 4]);
#pragma unroll
        for (int j = 8; j < kHalf; j += 8)     // (three-operand maxima)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmaxf(fmaxf(mx[e], v[j + e]), v[j + 4 + e]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // What was read is free; lane quarter 0 re-arms first.  The credits are relaxed arrivals: one that
        // releases at cluster scope takes ~1000 cycles (64 x 32768 x 128 heads 580 -> 943 us, one fence
        // for both 797, by a warp of its own 757).  What they protect are this warp's loads, whose values
        // the peer's next stores can no longer change once they have arrived in registers, and an
        // arrival is not issued before they have: it waits for a vote on a maximum over all of them
        // (which is never the signalling NaN that the vote asks for: no arithmetic gives one).
        const bool arrived = !__any_sync(0xffffffffu, __float_as_uint(top) == 0x7F800001u);
        if (lane == 0 && arrived) {
          if (quarter == 0) {
            mbar_arrive_expect_tx_relaxed(&x_full[b0], x_bytes);
            mbar_arrive_expect_tx_relaxed(&x_full[b1], x_bytes);
          }
          mbar_arrive_remote_relaxed(xempty_remote + b0 * 8);
          mbar_arrive_remote_relaxed(xempty_remote + b1 * 8);
        }
        // (an infinite sum is a masked or an overflowed one: not scaled, 0 * inf is no logit)
        const float tmax = top == -INFINITY ? -INFINITY : top * sl2;
        // the reference after the half before (the other set's), moved when this
        // half's maximum exceeds it by far; what is in the accumulator moves with it
        if (!(ok = settle(ref_here, &ref_set[quarter], (uint32_t)(hf ^ 1)))) break;
        const float m_prev = t == x.t0 && hf == 0 ? -INFINITY : ref_s[0];
        float m_ref = m_prev, alpha = 1.f;
        bool rescale = false;
        if (m_prev == -INFINITY) {
          m_ref = tmax;                        // nothing in the accumulator yet
        } else if (tmax > m_prev + kRescaleLog2) {
          alpha = ex2_approx(m_prev - tmax);
          m_ref = tmax;
          rescale = true;
        }
        ref_s[0] = m_ref;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ref_set[quarter]);
        // This half of the P tile is free once its last P.V is done; a piece's first P
        // also waits until the output before is read out.
        if (!(ok = (tg == 0 || wait32(&p_empty[hf], (uint32_t)(tg - 1) & 1u)))) break;
        if (t == x.t0 && hf == 0 && pieces > 0 &&
            !(ok = wait32(o_free, (uint32_t)(pieces - 1) & 1u))) break;
        tc_fence_after();
        // weights 2^(logit * sl2 - reference), rounded to bf16 for P.V (half a step, to
        // nearest: the errors of a row's weights average out) and summed in fp32
        // before the rounding, which keeps the lse exact to fp32
        uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
        const float nmr = (m_ref == -INFINITY) ? 0.f : -m_ref;
        const uint64_t scale2 = pack2(sl2, sl2), nmr2 = pack2(nmr, nmr);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 4 * u + i;
            const float2 x2 = unpack2(fma2(pack2(v[2 * j], v[2 * j + 1]), scale2, nmr2));
            const float e0 = ex2_approx(x2.x), e1 = ex2_approx(x2.y);
            sum2[j & 3] = add2(sum2[j & 3], pack2(e0, e1));
            const __nv_bfloat162 p2 = __floats2bfloat162_rn(e0, e1);
            pk[i] = *reinterpret_cast<const uint32_t*>(&p2);
          }
          *reinterpret_cast<uint4*>(pbuf + sw128_offset(m, hf * 4 + u)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        const float2 tot = unpack2(add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3])));
        if (m_mine != m_ref) l_mine *= m_mine == -INFINITY ? 0.f : ex2_approx(m_mine - m_ref);
        m_mine = m_ref;
        l_mine += tot.x + tot.y;
        // TMEM loads and stores are warp-collective: rescale when any row of the
        // warp needs it (the others multiply by 1)
        if (__builtin_expect(__any_sync(0xffffffffu, rescale), 0)) {
          // Nothing may be under way into the accumulator: the other half's P.V just
          // before this one is done too.  (Its phase before that one is over, so the
          // parity tells: that P.V was committed before this half's last one.)
          if (!(ok = wait32(&p_empty[hf ^ 1], (uint32_t)(hf == 0 ? tg - 1 : tg) & 1u))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < 256; c0 += 16) {
            float o[16];
            tmem_ld16(tmem + lane_base + TM_O + c0, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_st16(tmem + lane_base + TM_O + c0, o);
          }
          tmem_st_wait();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[hf]);
      }
      if (!ok) break;
      // ---- the piece's sum over both sets (a set without tiles has none) --------
      volatile float2* const sums = reinterpret_cast<float2*>(smem + Y::sums) + (pieces & 1) * 2 * kM + m;
      sums[set * kM].x = m_mine;
      sums[set * kM].y = l_mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(sums_set);
      if (!(ok = wait32(sums_set, (uint32_t)pieces & 1u))) break;
      const float2 other = make_float2(sums[(set ^ 1) * kM].x, sums[(set ^ 1) * kM].y);
      const float m_ref = fmaxf(m_mine, other.x);
      // (a sum without a maximum is 0, or NaN: every logit was)
      float l_sum = l_mine * (m_mine == -INFINITY ? 1.f : exp2f(m_mine - m_ref));
      l_sum += other.y * (other.x == -INFINITY ? 1.f : exp2f(other.x - m_ref));
      if (!(ok = wait32(o_done, (uint32_t)pieces & 1u))) break;
      ++pieces;
      tc_fence_after();
      // ---- the piece's output: this CTA's 256 dims, 128 of them by each set ------
      const bool entire = x.t0 == 0 && x.t1 == x.grp.tiles;
      const int slot = 2 * k + (x.t0 == 0 ? 1 : 0);
      if (!entire) {
        if (x.t0 == 0) {
          rec.starts = x.g;
        } else {
          rec.continues = x.g;
          rec.finishes = x.t1 == x.grp.tiles;
        }
      }
      const bool live = m < x.grp.nt * a.H;
      const int64_t orow = (int64_t)x.grp.row0 * a.H + m;
      // nothing visible: 0; NaN stays NaN
      const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
      uint8_t* const dst0 = reinterpret_cast<uint8_t*>(
          entire ? (void*)(a.out + orow * DSI_D_LATENT + rho * 256)
                 : (void*)(ws.o + ((int64_t)slot * kM + m) * DSI_D_LATENT + rho * 256));
#pragma unroll 1
      for (int c0 = set * 128; c0 < set * 128 + 128; c0 += 32) {
        float o[32];
        __syncwarp();        // rows without an output skip the stores of the round before
        tmem_ld32(tmem + lane_base + TM_O + c0, o);
        tmem_ld_wait();
        if (!live) {
        } else if (entire) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
            w[i] = *reinterpret_cast<const uint32_t*>(&y);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) st_global_32(dst0 + c0 * 2 + i * 32, w + 8 * i, wide);
        } else {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) st_global_32(dst0 + c0 * 4 + i * 32, w + 8 * i, true);
        }
      }
      if (live && rho == 0 && set == 0) {
        if (!entire) ws.ml[slot * kM + m] = make_float2(m_ref, l_sum);
        else if (a.lse) a.lse[orow] = l_sum == 0.f ? -INFINITY : (m_ref + log2f(l_sum)) / kLog2e;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
    if (plan.split && rho == 0 && set == 0 && m == 0) ws.rec[k] = rec;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQkWarp) tmem_dealloc(tmem, TMEM_COLS);
  cluster_sync();      // the peer may still arrive on / write into this CTA until here
}

// Joins the pieces of split groups.  A group is split when a cluster starts it
// and does not finish it; its other pieces are the first ones of the next
// clusters, up to the first that finishes one.  Every block finds the split
// groups in the clusters' records (none: it leaves at once) and takes every
// gridDim.x-th of their rows.
constexpr int kJoinThreads = 128;
static_assert(kMaxClusters <= kJoinThreads && kJoinThreads * 4 == DSI_D_LATENT, "a thread a record, four dims a thread");
__global__ void __launch_bounds__(kJoinThreads)
dense_mla_join(DenseArgs a, Plan plan, Workspace ws, int clusters, int rows) {
  __shared__ float weight[kMaxClusters];
  __shared__ float red[2][4];
  __shared__ unsigned int starts_s[4], ends_s[4];
  __shared__ int owner_s[kMaxClusters], group_s[kMaxClusters];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();     // the pieces come from the kernel launched just before
  grid_dep_launch();
  Record rec = {-1, -1, 0, 0};
  if (tid < clusters) rec = ws.rec[tid];
  const unsigned int starts = __ballot_sync(0xffffffffu, rec.starts >= 0);
  const unsigned int ends = __ballot_sync(0xffffffffu, rec.finishes != 0);
  if (lane == 0) { starts_s[warp] = starts; ends_s[warp] = ends; }
  __syncthreads();
  int at = __popc(starts & ((1u << lane) - 1u)), owners = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < warp) at += __popc(starts_s[w]);
    owners += __popc(starts_s[w]);
  }
  if (owners == 0) return;
  if (rec.starts >= 0) { owner_s[at] = tid; group_s[at] = rec.starts; }
  for (int i = blockIdx.x; i < owners * rows; i += gridDim.x) {
    __syncthreads();   // the lists are complete; the row before is done with the weights
    const int oi = i / rows, m = i - oi * rows, k = owner_s[oi], g = group_s[oi];
    const int b = g / plan.per_seq, t0 = (g - b * plan.per_seq) * plan.tokens;
    if (m >= min(plan.tokens, a.T - t0) * a.H) continue;
    int end = clusters - 1;                      // the cluster that finishes the group
    for (int w = 3; w >= 0; --w) {
      const unsigned int later = w * 32 > k ? ends_s[w] : w * 32 + 31 <= k ? 0u : ends_s[w] & ~((2u << (k & 31)) - 1u);
      if (later) end = w * 32 + __ffs(later) - 1;
    }
    const int pieces = end - k + 1;              // <= kMaxClusters
    // piece 0: the last of cluster k; piece i: the first of cluster k + i
    float2 ml = make_float2(-INFINITY, 0.f);
    if (tid < pieces) ml = ws.ml[(2 * (k + tid) + (tid == 0 ? 1 : 0)) * kM + m];
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) red[0][warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
    weight[tid] = f;
    float sum = f * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int j = 0; j < pieces; ++j) {
      const int64_t slot = 2 * (k + j) + (j == 0 ? 1 : 0);
      const float4 v = reinterpret_cast<const float4*>(ws.o + (slot * kM + m) * DSI_D_LATENT)[tid];
      const float w = weight[j];
      o.x += w * v.x; o.y += w * v.y; o.z += w * v.z; o.w += w * v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t row = ((int64_t)b * a.T + t0) * a.H + m;
    __align__(8) bf16 o4[4] = {__float2bfloat16(o.x * inv), __float2bfloat16(o.y * inv),
                               __float2bfloat16(o.z * inv), __float2bfloat16(o.w * inv)};
    *reinterpret_cast<uint2*>(a.out + row * DSI_D_LATENT + tid * 4) = *reinterpret_cast<const uint2*>(o4);
    if (a.lse && tid == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) / kLog2e;
  }
}

// Two-CTA clusters that fit on the current device at once, queried once per
// device and form, after the kernel has been given its shared memory there; 0
// without a device.
template <bool F8>
int cluster_slots() {
  static std::atomic<int> cached[64];
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) { cudaGetLastError(); return 0; }
  v = cached[dev].load(std::memory_order_relaxed);
  if (v) return v;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(Layout<F8>::threads);
  cfg.dynamicSmemBytes = Layout<F8>::bytes;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(dense_mla_tc<F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Layout<F8>::bytes) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&v, dense_mla_tc<F8>, &cfg) != cudaSuccess || v < 1) {
    cudaGetLastError();
    return 0;
  }
  v = v < kMaxClusters ? v : kMaxClusters;
  cached[dev].store(v, std::memory_order_relaxed);
  return v;
}

constexpr size_t kSlotBytes = (size_t)kM * (DSI_D_LATENT * sizeof(float) + sizeof(float2));

template <bool F8>
cudaError_t launch(const CUtensorMap& map, const CUtensorMap& rmap, const CUtensorMap& qmap,
                   const DenseArgs& a, const Plan& plan, const Workspace& ws, int box, int clusters,
                   cudaStream_t st) {
  const cudaError_t e =
      launch_overlapped(dense_mla_tc<F8>, dim3(2u * (unsigned)clusters), dim3(Layout<F8>::threads),
                        Layout<F8>::bytes, st, map, rmap, qmap, a, plan, ws, box);
  note_launch();
  return e;
}

}  // namespace

size_t dense_mla_workspace() {
  int n = cluster_slots<false>() > cluster_slots<true>() ? cluster_slots<false>() : cluster_slots<true>();
  if (n == 0) n = 76;                            // no device: what a GB300 takes
  return (size_t)n * (2 * kSlotBytes + sizeof(Record));
}

cudaError_t launch_dense_mla(const DenseArgs& a, cudaStream_t st) {
  const bool f8 = a.latent_scale != nullptr;
  Plan plan;
  plan.tokens = kM / a.H < a.T ? kM / a.H : a.T;
  plan.per_seq = (a.T + plan.tokens - 1) / plan.tokens;
  const int64_t groups = (int64_t)plan.per_seq * (a.rows / a.T);
  plan.groups = (int)groups;                     // <= rows
  const int slots = f8 ? cluster_slots<true>() : cluster_slots<false>();
  if (slots == 0) return cudaErrorInvalidConfiguration;
  // at most a cluster a tile
  const int64_t span = a.window + a.n_sink < a.c.s_max ? a.window + a.n_sink + plan.tokens + 2 * kNp : a.c.s_max;
  const int64_t tiles = groups * ((span + kNp - 1) / kNp + 1);
  const int clusters = (int)(tiles < slots ? tiles : slots);
  // Groups that cannot be long enough for a split to pay, whatever the lengths are, stay
  // whole: no sums of tiles, no second kernel (24 x 4 tokens with windows of 129: 25.7 us
  // with them, 23.2 without; 17.4 now).
  const int64_t all = (a.c.s_max + kNp - 1) / kNp;
  const int64_t seen = (a.window + plan.tokens - 1 + kNp - 1) / kNp + 1 + (a.n_sink + kNp - 1) / kNp;
  const int64_t most = (all < seen ? all : seen) + kGroupCost;
  const int64_t least = (groups * (1 + kGroupCost) + clusters - 1) / clusters;
  plan.split = a.ws != nullptr && clusters > 1 &&
               (groups + clusters - 1) / clusters * most > least + kWholeSlack;
  plan.live = (plan.tokens * a.H + 31) / 32;
  Workspace ws = {nullptr, nullptr, nullptr};
  if (plan.split) {
    ws.o = static_cast<float*>(a.ws);
    ws.ml = reinterpret_cast<float2*>(ws.o + (size_t)2 * clusters * kM * DSI_D_LATENT);
    ws.rec = reinterpret_cast<Record*>(ws.ml + (size_t)2 * clusters * kM);
  }
  // TMA boxes: the largest part of 64 rows that pages are made of
  int box = kNp;
  if (a.c.block_table)
    while (a.c.page_size % box != 0) box /= 2;   // page sizes are multiples of 8
  CUtensorMap map, rmap;
  const uint64_t rows = a.c.block_table ? (uint64_t)a.c.num_pages * a.c.page_size
                                        : (uint64_t)a.c.batch * a.c.s_max;
  const bool mapped =
      f8 ? tma_map_2d(&map, a.c.latent, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, DSI_D_QK, 128, (uint32_t)box) &&
               tma_map_2d(&rmap, a.c.latent, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, DSI_D_QK, kRopeHalf,
                          (uint32_t)box, CU_TENSOR_MAP_SWIZZLE_NONE)
         : tma_map_2d(&map, a.c.latent, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, rows, DSI_D_QK, 64,
                      (uint32_t)box) &&
               tma_map_2d(&rmap, a.c.latent, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, rows, DSI_D_QK,
                          kRopeHalf, (uint32_t)box, CU_TENSOR_MAP_SWIZZLE_64B);
  if (!mapped) return cudaErrorInvalidValue;
  CUtensorMap qmap;
  if (!tma_map_2d(&qmap, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)a.rows * a.H, DSI_D_QK, 64, kM))
    return cudaErrorInvalidValue;
  cudaError_t e = f8 ? launch<true>(map, rmap, qmap, a, plan, ws, box, clusters, st)
                     : launch<false>(map, rmap, qmap, a, plan, ws, box, clusters, st);
  if (e != cudaSuccess || !plan.split) return e;
  // enough blocks for one resident wave: a call without split groups pays little
  const int64_t rows_at_most = (int64_t)clusters * plan.tokens * a.H;
  const int64_t wave = 16 * clusters;
  e = launch_overlapped(dense_mla_join, dim3((unsigned)(rows_at_most < wave ? rows_at_most : wave)),
                        dim3(kJoinThreads), 0, st, a, plan, ws, clusters, plan.tokens * a.H);
  note_launch();
  return e;
}

}  // namespace dsi
