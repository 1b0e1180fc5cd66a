// product_sm100.cuh -- the tcgen05 kernel of the grouped products (grouped_product.cu) and of the
// Newton-Schulz iteration (orthogonalize.cu).  For every group g it computes
//
//     out_g[r][c] = sum_k B_g[r][k] * A_g[c][k]        rows r, contiguous columns c
//
// with 16-bit operands (both bf16 or both fp16) and fp32 accumulators in tensor memory.  The
// contiguous output dimension is the MMA's M side (operand A), the rows are its N side (operand B),
// so a tile of few rows costs its own rows rounded up to 16 in the MMA instead of a whole tile, and a TMEM
// lane is an output column.
// Each operand is K-major (stored [index][k]) or MN-major (stored [k][index]); both come in by TMA
// with the 128-byte swizzle and only the descriptors differ, so no operand is ever transposed in
// memory.
//
// One tile is 256 columns x up to 256 rows on a cluster of two CTAs (tcgen05.mma.cta_group::2, M = 256):
// each CTA loads its own 128 columns and its half of the rows, 32 KB per 64-wide K block for a
// 128 x 256 x 64 product -- 64 bytes per cycle and SM at the tensor pipe's rate, where a one-CTA tile
// would need 96.  No load is multicast.  Tiles of 512 columns, with both accumulators of the tensor memory in
// one tile and 48 bytes per cycle, were measured and dropped: the accumulators are then not free while the
// epilogue reads them, and only a contraction of 7000 and more made up for it (K = 8192: 1326 -> 1385
// TFLOP/s sustained; K = 2880: 1210 -> 1190).
//
// Kernel layout (persistent clusters of two, 352 threads per CTA):
//   warp 0     TMA producer: 6 stages of 32 KB.
//   warp 1     TMEM allocation; in the even CTA one thread issues the pair's MMAs.
//   warps 2-9  epilogue: four TMEM lane quarters x two halves of the rows.
//   warp 10    ragged K: clears the rows behind a segment in its last K block.
// Tiles are dealt round-robin.  The tiles of the last, partly filled round are split along K when
// that shortens the round (few rows, one token: cost_of); each part stores its fp32 accumulators and
// the last part to arrive (an atomic counter per warp's share, no waiting) adds them in the order of
// the parts, so results do not depend on timing.
//
// Rounding.  The tensor core truncates when it aligns an addend to its accumulator, which biases a long sum
// towards zero.  Measured on this GPU through a library product with fp32 results, of the norm: terms of random
// signs 1.0e-6 (bf16) and 1.3e-6 (fp16) at k = 1024, 4.4e-6 and 4.9e-6 at 4096, 1.9e-5 at 16384, about 1.1e-9 per
// k; all-positive terms 2.2e-6 and 6.1e-6, 1.4e-5 and 2.6e-5, 8.3e-5 and 1.1e-4, about 5e-9 per k.  Where the
// result stays fp32 (kPromote), the accumulator is therefore drained every 512 k into registers and added there,
// rounded to nearest: 4.8e-7 and 6.5e-7, all-positive 9e-7 and 2.8e-6, at any k.  Of a 16-bit result, half a step of bf16 is
// 3.9e-3 and of fp16 4.9e-4 of it: only all-positive terms of fp16 at k beyond 16384 come near that.
//
// Every wait is bounded (kWaitLimitNs); on expiry the kernel sets kErrTimeout and returns.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>
#include <mutex>

#include "moe_common.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace product {

enum Ragged { kDense = 0, kRaggedRows = 1, kRaggedK = 2 };
enum Epilogue {
  kOut16 = 0,     // out = bf16 or fp16
  kOut32 = 1,     // out = fp32, promoted accumulation
  kGram = 2,      // symmetric: out = fp16(acc * c1), and its mirror image
  kPoly = 3,      // symmetric: out = fp16(c0 * src + acc * c1), and its mirror image; the diagonal goes to diag as
                  // c2 + diagonal / 4096, and out has zeros there
  kApply = 4,     // x = acc * c1 + diag * src + c2 * src_lo; out = fp16(x), out_lo = fp16(2048 (x - out)):
                  // out[column][row]
  kApplyLast = 5, // out = bf16(the same x * c0), rows of cols_out elements: out[column][row]
  kGrad = 6       // as kOut32, of groups of equal rows: leaves by TMA
};

constexpr int kTile = 256;               // rows (N) and columns (M) of a pair's tile
constexpr int kBK = 64;                  // K per stage
constexpr int kStages = 6;               // 5 beside kGrad's staging (stages_of)
constexpr int kThreads = 352;
constexpr int kEpiWarps = 8;
constexpr int kTileA = 128 * kBK * 2;    // 16 KB: this CTA's columns
constexpr int kTileB = 128 * kBK * 2;    // 16 KB: this CTA's rows, at most
constexpr int kStageBytes = kTileA + kTileB;
constexpr int kPromoteBlocks = 8;        // K blocks per accumulator drain (512 k)
constexpr int kMaxGroups = 1024;
constexpr int kBarBytes = 256;  // 3 per stage, 4 of the accumulators, the tensor memory's address
constexpr int kChunkBytes = 32 * 32 * 2;  // 32 rows x 32 columns of 16 bits: what a warp's epilogue handles at a time
// shared memory of an epilogue warp: a chunk of 16 bits turned from columns to rows; kGrad: two chunks of fp32
// on their way out
constexpr int staging_of(int epi) { return epi == kGrad ? 4 * kChunkBytes : epi == kOut32 || epi == kApply ? 0 : kChunkBytes; }
constexpr bool applies(int epi) { return epi == kApply || epi == kApplyLast; }
constexpr int stages_of(int epi) { return epi == kGrad ? kStages - 1 : kStages; }
// groups whose segments' bounds are held in shared memory (kGrad: what the staging leaves room for)
constexpr int table_groups(int epi) { return epi == kGrad ? 190 : kMaxGroups; }
constexpr size_t smem_bytes(int epi) {
  return 1024 + (size_t)stages_of(epi) * kStageBytes + kBarBytes + kEpiWarps * staging_of(epi) +
         16 + 4 * (epi == kGrad ? 2 * table_groups(epi) : epi <= kOut32 ? 3 * kMaxGroups : 0);
}
static_assert(smem_bytes(kOut16) <= 232448 && smem_bytes(kApply) <= 232448 && smem_bytes(kGrad) <= 232448, "shared memory budget");

// workspace of a launch: error word, counters (zero between launches), split-K partial sums
constexpr int kMaxParts = 148;           // split tiles x parts
constexpr int kMaxSplit = 16;
constexpr size_t kCounterBytes = 8192;   // 16 per split tile; fewer split tiles than clusters (<= 74)
constexpr size_t kPartialOffset = kWsHeader + kCounterBytes;
static_assert(kPartialOffset == MOE_PRODUCT_WS_ZEROED, "what has to be zero before the first launch");
inline int partial_rows(long long rows) { return rows >= kTile ? kTile : (int)((rows + 31) / 32 * 32); }
inline size_t partial_bytes(int prows) { return (size_t)kMaxParts * 2 * 128 * 4 * (size_t)prows; }

// Boxes of a K-major B: a tile's rows come in one request of the smallest box that holds half of them.
// The rows behind them are loaded for nothing, which costs less than exact boxes: four requests of
// 32 + 32 + 32 + 8 rows took a product of 1040 rows per segment from 923 to 1246 us.
constexpr int kBoxes = 5;
__host__ __device__ constexpr int box_rows(int i) { return i == 0 ? 128 : i == 1 ? 96 : i == 2 ? 64 : i == 3 ? 32 : 8; }
__device__ __forceinline__ int box_of(int half) { return half > 96 ? 0 : half > 64 ? 1 : half > 32 ? 2 : half > 8 ? 3 : 4; }

struct alignas(64) Params {
  CUtensorMap a;          // K-major: box 64 k x 128 columns; MN-major: box 64 columns x 64 k
  CUtensorMap b[kBoxes];  // K-major: boxes of 64 k x box_rows(i) rows; MN-major (the first): 64 rows x 64 k
  const int32_t* offsets;  // kRaggedRows / kRaggedK: segment bounds [G + 1]
  CUtensorMap out_map;     // kGrad: out in boxes of 32 columns x 32 and x 16 rows
  CUtensorMap out16_map;
  int G;                   // groups
  int M_total;             // rows of the ragged tensor
  int ct, lr;              // column tiles; a tile has at most 2^lr rows
  int tiles, split;        // not kRaggedRows: tiles, parts of each tile of the last round
  int rows, cols, K;       // rows (not kRaggedRows), columns and K (not kRaggedK) of a group
  uint32_t idesc;          // instruction descriptor without M and N
  int out_bf16;            // kOut16: bf16 instead of fp16
  int ld;                  // row pitch of src and out of the Newton-Schulz epilogues (multiples of 16)
  int cols_out;            // kApply, kApplyLast: columns of a row of X that exist; the latter: row pitch of out
  void* out;
  uint16_t* out_lo;        // kApply: in low_index's order
  const uint16_t* src;     // kPoly: symmetric; kApply, kApplyLast: X's high-order part
  const uint16_t* src_lo;  // kApply, kApplyLast: its low-order part, may be out_lo
  float* diag;             // kPoly: written, kApply and kApplyLast: read; a group's stands at its number x diag_ld
  int diag_ld;
  float c0, c1, c2;
  float* partial;
  int* counters;
  int prows;               // rows per partial tile
  int kb_typ;              // K blocks of a typical tile (the split's cost model)
  int rows_typ;            // kRaggedRows: rows of the mean segment (the same)
  int withhold_first_load; // test only: the even CTA never issues its first stage's copies
  int* err;
};

// ------------------------------------------------------------------------------ PTX of this kernel
__device__ __forceinline__ void tma_3d(const CUtensorMap* map, uint64_t* bar, void* dst, int32_t x, int32_t y,
                                       int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// completion counted on an mbarrier of either CTA of the pair (shared::cluster address); no multicast
__device__ __forceinline__ void tma_3d_pair(const CUtensorMap* map, uint32_t bar_cluster, void* dst, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// As mbar_wait, but a failed try sleeps until the phase completes (10 ms at most) instead of asking again:
// the polling of twenty waiting warps cost issue slots and power, 1150 -> 1195 TFLOP/s at the power limit
// for 32 experts of 1024 rows, [5760, 2880].  kCluster: sees what the other CTA's threads wrote before
// their arrival.
template <bool kCluster = false>
__device__ __forceinline__ bool sleep_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kCluster)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 10000000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 10000000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}
template <bool kCluster = false>
__device__ __forceinline__ bool sleep_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  if (sleep_try<kCluster>(a, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!sleep_try<kCluster>(a, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
  return true;
}
// Arrive on an mbarrier of the pair's even CTA, ordering nothing beyond this CTA: the reads of tensor memory
// that it reports have completed (tcgen05.wait::ld).  A release at cluster scope first waits for the
// thread's global stores, 3500 cycles a tile here.
__device__ __forceinline__ void mbar_arrive_even(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), 0)) : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read_but_one() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// generic accesses of shared memory before -> the TMA's or the tensor core's after
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// UMMA descriptor of an MN-major operand: 64-element chunks 8 KB apart, 8-k groups 1 KB apart
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// ------------------------------------------------------------------------------ schedule
constexpr int kBand = 8;  // row tiles of a band (item_of)

struct Sched {
  int full;   // tiles dealt whole
  int split;  // parts of each later tile
  int items;
  int per;    // not kRaggedRows: tiles of a group, rows of a tile
  int step;
  float inv_split, inv_band, inv_per;
};

// The size of the tiles and the parts into which those of the last, partly filled round are split along K.
// Cost in K blocks of a full tile (some 550 cycles): a block of a tile of few rows costs half as much, as
// the columns' operand comes in whole; a tile has a fixed share for filling the pipeline, the last one its
// epilogue; parts travel through memory, 8 rows x 8 parts at a time and a memory latency each.  Without the
// split a one-token product of 4 experts x [5760, 2880] leaves 3/4 of the clusters idle in its second round;
// with tiles of 256 rows only, one of 8 experts x 194 rows, [1000, 520], leaves 42 of 74 idle.  The host
// chooses both (choose); where segments decide how many tiles there are it takes the mean segment's size for
// the tiles, and the parts are chosen on the device.
__host__ __device__ inline float cost_of(int tiles, int clusters, int kb, int rows, int s) {
  const int full = tiles / clusters, r = tiles - full * clusters;
  const float block = 0.5f + (float)rows * (1.0f / 512.0f);
  float cost = (float)full * ((float)kb * block + 3.0f) + (float)rows * (1.0f / 64.0f);
  if (r > 0) {
    const int rounds = (r * s + clusters - 1) / clusters;
    cost += (float)rounds * ((float)kb / (float)s * block + 4.0f);
    if (s > 1) cost += 8.0f + 2.5f * (float)((rows + 15) / 16 * ((s + 7) / 8));
  }
  return cost;
}
__host__ __device__ inline int most_parts(int r, int kb) {
  const int a = kb / 2 < kMaxSplit ? kb / 2 : kMaxSplit, b = r > 0 ? kMaxParts / r : 1;
  return a < b ? a : b;
}
// parts of each of the r tiles of the last round; a whole warp
__device__ __forceinline__ int split_of(int r, int clusters, int kb, int rows, int lane) {
  const int s = lane + 1;
  const float cost = s <= most_parts(r, kb) || s == 1 ? cost_of(r, clusters, kb, rows, s) : 1e30f;
  const uint32_t least = __reduce_min_sync(0xffffffffu, __float_as_uint(cost));  // of positive numbers
  return __ffs(__ballot_sync(0xffffffffu, __float_as_uint(cost) == least));
}

struct Item {
  int g;
  int rt, ct;        // row tile, column tile
  int r0, nr;        // rows of this tile within the group: [r0, r0 + nr), nr = 1..256
  int row0;          // kRaggedRows: first row of the segment
  int k0, krows;     // kRaggedK: first k row and number of k rows
  int kb0, kb1;      // K blocks [kb0, kb1)
  bool triangle;     // a symmetric product's mirror image is stored too
  int part, slot;    // part of the split, split-tile index (-1: whole)
};

__device__ __forceinline__ void segment(const Params& p, int g, int& row0, int& rows, bool& bad) {
  const int a = p.offsets[g], b = p.offsets[g + 1];
  row0 = min(max(a, 0), p.M_total);
  const int end = min(max(b, row0), p.M_total);
  rows = end - row0;
  bad = row0 != a || end != b;
}

// Tiles of a group of `rows` rows, at most 2^lr of them in a tile (256, 128 or 64).  Of a symmetric
// product only the lower triangle of 256 x 256 tiles is computed, but all of the smaller tiles.
constexpr int kMostLr = 8, kLeastLr = 6;
constexpr bool symmetric(int epi) { return epi == kGram || epi == kPoly; }
template <int EPI>
__host__ __device__ inline int tiles_of(int rows, int ct, int lr) {
  const int rt = (rows + (1 << lr) - 1) >> lr;
  if (symmetric(EPI) && lr == kMostLr) return rt * (rt + 1) / 2;
  return rt * ct;
}

// n / d for quotients below 2^22, inv = 1 / d: the estimate is off by at most one (every role divides for every
// tile, and a tile of few K blocks is worth only some thousand cycles)
__device__ __forceinline__ int divide(int n, int d, float inv, int& rem) {
  int q = (int)((float)n * inv);
  rem = n - q * d;
  if (rem < 0) --q, rem += d;
  if (rem >= d) ++q, rem -= d;
  return q;
}

// Rows of a tile of a group.  They are dealt evenly over its rt row tiles, in 16s: a tile of few rows costs
// nearly half a full one, for the columns' operand comes in whole.  The symmetric products keep square tiles.
template <int EPI>
__host__ __device__ constexpr int step_of(int rows, int rt, int lr) {
  if (symmetric(EPI) || rt <= 1) return 1 << lr;
  return ((rows + rt - 1) / rt + 15) / 16 * 16;
}
static_assert(step_of<kOut16>(0, 0, kMostLr) > 0, "no rows (every launch of ragged rows asks): no division by no tiles");

// tab: kRaggedRows, kRaggedK: first row and rows of each group; kRaggedRows: then the first tile of each
template <int RAGGED, int EPI>
__device__ __forceinline__ Item item_of(const Params& p, const int* tab, const Sched& sc, int i) {
  Item x;
  int t = i;
  int parts = 1;
  x.part = 0;
  x.slot = -1;
  if (i >= sc.full && sc.split > 1) {
    x.slot = divide(i - sc.full, sc.split, sc.inv_split, x.part);
    t = sc.full + x.slot;
    parts = sc.split;
  }
  int rows = p.rows, local;
  x.row0 = 0, x.k0 = 0, x.krows = 0;
  if constexpr (RAGGED == kRaggedRows) {
    const int* tile_start = tab + 2 * p.G;
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile_start[mid] <= t) lo = mid; else hi = mid - 1;
    }
    x.g = lo;
    x.row0 = tab[2 * lo];
    rows = tab[2 * lo + 1];
    local = t - tile_start[lo];
  } else {
    x.g = divide(t, sc.per, sc.inv_per, local);
    if constexpr (RAGGED == kRaggedK) {
      if (p.G <= table_groups(EPI)) {
        x.k0 = tab[2 * x.g];
        x.krows = tab[2 * x.g + 1];
      } else {
        bool bad;
        segment(p, x.g, x.k0, x.krows, bad);
      }
    }
  }
  const int rt = (rows + (1 << p.lr) - 1) >> p.lr;
  x.triangle = symmetric(EPI) && p.lr == kMostLr;
  if (x.triangle) {
    // lower triangle, row by row
    int r = (int)((sqrtf(8.0f * (float)local + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1) / 2 > local) --r;
    while ((r + 1) * (r + 2) / 2 <= local) ++r;
    x.rt = r;
    x.ct = local - r * (r + 1) / 2;
  } else {
    // bands of 8 row tiles, rows fastest inside a band: the ~74 tiles in flight share about 8 row
    // blocks and 9 column blocks through L2 (bands of 4 and 16: within 3% of it either way)
    int rem, in_band;
    const int band = divide(local, kBand * p.ct, sc.inv_band, rem);
    const int rb = min(kBand, rt - kBand * band);
    x.ct = divide(rem, rb, __fdividef(1.0f, (float)rb), in_band);
    x.rt = kBand * band + in_band;
  }
  const int step = RAGGED == kRaggedRows ? step_of<EPI>(rows, rt, p.lr) : sc.step;
  x.r0 = x.rt * step;
  x.nr = min(step, rows - x.r0);
  const int kb = RAGGED == kRaggedK ? (x.krows + kBK - 1) / kBK : (p.K + kBK - 1) / kBK;
  x.kb0 = 0, x.kb1 = kb;
  if (parts > 1) {
    x.kb0 = split_begin(kb, x.part, parts);
    x.kb1 = split_end(kb, x.part, parts);
  }
  return x;
}

// rows of B each CTA multiplies: half of the tile's rows rounded up to 16
__device__ __forceinline__ int half_of(int nr) { return ((nr + 15) / 16) * 8; }

// kRaggedK: the K block at kx ends behind the segment and inside a 16-long instruction
__device__ __forceinline__ bool ragged_tail(int krows, int kx) { return kx + kBK > krows && ((krows - kx) & 15) != 0; }

// ------------------------------------------------------------------------------ epilogue
__device__ __forceinline__ uint16_t half_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ float half_val(uint16_t b) { return __half2float(__ushort_as_half(b)); }

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_half(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// 32 bytes of a lane: one sector
__device__ __forceinline__ void load_sector(const uint16_t* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store_sector(uint16_t* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Where the output's rows are the tile's columns (kApply and kApplyLast by the choice of operands, the symmetric
// products by symmetry) a lane's 32 values are 64 contiguous bytes of its own row, and nothing goes through shared
// memory, which the operands of the MMAs keep busy (with chunks turned there, and the low-order part alone added,
// kApply took 420 us on 8 matrices of 2048 x 7168 and 49 on 6 of 2001 x 999, so 378 and 35).  Pitches are multiples of 16
// elements, so whole sectors move, and so are the rows of a tile or they end in zeros.
__device__ __forceinline__ long long lane_row(const Params& p, const Item& x, int rows, int j0, int col) {
  return ((long long)x.g * rows + col) * p.ld + x.r0 + j0;
}
__device__ __forceinline__ void store_lane_row(uint16_t* o, const uint32_t (&w)[16], int nj) {
  store_sector(o, w);
  if (nj > 16) store_sector(o + 16, w + 8);
}

// X's low-order part is no operand of a product, so it lies as the epilogues take it: blocks of 32 rows x 16
// columns, one row's 16 (a lane's sector) after the other, and a warp's load or store is 1 KB in one piece.  In rows, as
// hi, each touches 32 lines, and their number is what bounds these epilogues: 6 x [2001, 999] took 425 us so and takes
// 380, 8 x [1024, 4096] 1038 and 950, 8 x [2048, 7168] 3590 and 3405.  Index of an element of matrix g:
__device__ __forceinline__ long long low_index(int g, int row, int column, int rows, int ld) {
  return (((long long)g * ((rows + 31) / 32) + row / 32) * (ld / 16) + column / 16) * 512 + row % 32 * 16 + column % 16;
}
inline long long low_elements(int groups, int rows, int ld) { return (long long)groups * ((rows + 31) / 32 * 32) * ld; }

// what kPoly, kApply and kApplyLast add to a chunk: read one chunk ahead
template <int EPI>
struct Addend {
  uint32_t hi[16];
  uint32_t lo[applies(EPI) ? 16 : 1];
  float diag;  // P X: of this lane's row of X; X P: of column j0 + lane of X
};
template <int EPI, bool PX>
__device__ __forceinline__ void load_addend(const Params& p, const Item& x, Addend<EPI>& s, int j0, int col, int lane) {
  const int rows = EPI == kPoly ? p.rows : p.cols;
  if (j0 >= x.nr) return;
  const bool two = x.nr - j0 > 16;
  if (col < rows) {
    const long long at = lane_row(p, x, rows, j0, col);
    load_sector(p.src + at, s.hi);
    if (two) load_sector(p.src + at + 16, s.hi + 8);
    if constexpr (applies(EPI)) {
      const uint16_t* lo = p.src_lo + low_index(x.g, col, x.r0 + j0, rows, p.ld);
      load_sector(lo, s.lo);
      if (two) load_sector(lo + 512, s.lo + 8);
    }
  }
  if constexpr (applies(EPI)) {
    const int i = PX ? col : x.r0 + j0 + lane;
    s.diag = i < (PX ? p.cols : p.cols_out) ? __ldcg(p.diag + (long long)x.g * p.diag_ld + i) : 0.0f;
  }
}

// A warp's 16-bit chunk, w[i] = rows 2 i and 2 i + 1 of this lane's column, turned through shared memory and
// stored 16 bytes a lane (a store per element made this half of the epilogue's 6000 cycles a tile).  o: the
// first row's place at the chunk's first column; limit: columns that exist from there on, a multiple of 8.
__device__ __forceinline__ void store_turned(uint16_t* o, int pitch, uint8_t* buf, const uint32_t (&w)[16], int nj,
                                             int limit, int lane) {
  uint32_t* b = reinterpret_cast<uint32_t*>(buf);
#pragma unroll
  for (int i = 0; i < 16; ++i) b[i * 32 + lane] = w[i];
  __syncwarp();
  const int c8 = (lane & 3) * 8;  // eight columns of a pair of rows
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int pair = (lane >> 2) + 8 * i;
    const uint4 l = *reinterpret_cast<const uint4*>(b + pair * 32 + c8);
    const uint4 h = *reinterpret_cast<const uint4*>(b + pair * 32 + c8 + 4);
    if (c8 < limit) {
      uint16_t* at = o + (long long)(2 * pair) * pitch + c8;
      if (2 * pair < nj)
        *reinterpret_cast<uint4*>(at) = make_uint4(__byte_perm(l.x, l.y, 0x5410), __byte_perm(l.z, l.w, 0x5410),
                                                   __byte_perm(h.x, h.y, 0x5410), __byte_perm(h.z, h.w, 0x5410));
      if (2 * pair + 1 < nj)
        *reinterpret_cast<uint4*>(at + pitch) = make_uint4(__byte_perm(l.x, l.y, 0x7632), __byte_perm(l.z, l.w, 0x7632),
                                                           __byte_perm(h.x, h.y, 0x7632), __byte_perm(h.z, h.w, 0x7632));
    }
  }
  __syncwarp();  // the buffer is written again
}

// A warp's chunk of kApplyLast, w[i] = elements j0 + 2 i and + 1 of row col of X (this lane's), turned through
// shared memory (16 bytes at a time, permuted within a row so that no two lanes meet in a bank) so that a
// row's 64 bytes lie side by side in a store: 417 -> 376 us of this launch for 8 x [2048, 7168], against 16 bytes of
// each lane's own row.  Of another pitch than whole 16 bytes, an element a lane, a row at a time.
__device__ __forceinline__ void store_rows(const Params& p, const Item& x, uint8_t* buf, const uint32_t (&w)[16], int j0,
                                           int nj, int col, int lane) {
  const int pitch = p.cols_out, c0 = x.r0 + j0;
  const int limit = min(nj, pitch - c0), rows = min(32, p.cols - (col - lane));  // that exist
  uint16_t* o = static_cast<uint16_t*>(p.out) + ((long long)x.g * p.cols + col - lane) * pitch + c0;
  uint4* b = reinterpret_cast<uint4*>(buf);
#pragma unroll
  for (int u = 0; u < 4; ++u)
    b[lane * 4 + (u ^ ((lane >> 1) & 3))] = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
  __syncwarp();
  if ((pitch & 7) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (lane >> 2) + 8 * i, u = lane & 3;
      const uint4 v = b[r * 4 + (u ^ ((r >> 1) & 3))];
      if (r < rows && 8 * u < limit) *reinterpret_cast<uint4*>(o + (long long)r * pitch + 8 * u) = v;
    }
  } else {
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      const uint16_t v = reinterpret_cast<const uint16_t*>(b)[r * 32 + (((lane >> 3) ^ ((r >> 1) & 3)) * 8) + (lane & 7)];
      if (r < rows && lane < limit) o[(long long)r * pitch + lane] = v;
    }
  }
  __syncwarp();  // the buffer is written again
}

// One warp's 32 rows x 32 columns, v[j] = accumulator of row j0 + j and column col (this lane's), s its
// addend; nj rows are valid.  PX: X is multiplied from the left.
template <int RAGGED, int EPI, bool PX>
__device__ __forceinline__ void emit(const Params& p, const Item& x, uint8_t* buf, const float (&v)[32],
                                     const Addend<EPI>& s, int j0, int nj, int col, int lane) {
  const int row_in = x.r0 + j0;  // row within the group
  const long long row = (RAGGED == kRaggedRows ? (long long)x.row0 : (long long)x.g * p.rows) + row_in;
  uint16_t* const out = static_cast<uint16_t*>(p.out);
  if constexpr (EPI == kOut32) {  // a row of 32 columns is one store of a warp
    if (col >= p.cols) return;
    float* o = static_cast<float*>(p.out) + row * p.cols + col;
    if (nj == 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[(long long)j * p.cols] = v[j];
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < nj) o[(long long)j * p.cols] = v[j];
    }
  } else if constexpr (applies(EPI)) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {  // two at a time: only the conversions of pairs run at full rate
      const float2 a = unpack_half(s.hi[i]), b = unpack_half(s.lo[i]);
      const float d0 = PX ? s.diag : __shfl_sync(0xffffffffu, s.diag, 2 * i);
      const float d1 = PX ? s.diag : __shfl_sync(0xffffffffu, s.diag, 2 * i + 1);
      const float w0 = v[2 * i] * p.c1 + d0 * a.x + p.c2 * b.x;
      const float w1 = v[2 * i + 1] * p.c1 + d1 * a.y + p.c2 * b.y;
      if constexpr (EPI == kApplyLast) {
        hi[i] = pack_bf16(w0 * p.c0, w1 * p.c0);
      } else {
        hi[i] = pack_half(w0, w1);
        const float2 f = unpack_half(hi[i]);
        lo[i] = pack_half((w0 - f.x) * 2048.0f, (w1 - f.y) * 2048.0f);
      }
    }
    if constexpr (EPI == kApplyLast) {
      store_rows(p, x, buf, hi, j0, nj, col, lane);
    } else if (col < p.cols) {
      store_lane_row(out + lane_row(p, x, p.cols, j0, col), hi, nj);
      uint16_t* o = p.out_lo + low_index(x.g, col, x.r0 + j0, p.cols, p.ld);
      store_sector(o, lo);
      if (nj > 16) store_sector(o + 512, lo + 8);
    }
  } else {
    uint32_t w[16];
    if constexpr (EPI == kPoly) {
      const int at = col - row_in;  // the row of the diagonal's element
      float d = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 a = unpack_half(s.hi[i]);
        const float w0 = v[2 * i] * p.c1 + a.x * p.c0, w1 = v[2 * i + 1] * p.c1 + a.y * p.c0;
        d = at == 2 * i ? w0 : at == 2 * i + 1 ? w1 : d;
        w[i] = pack_half(at == 2 * i ? 0.0f : w0, at == 2 * i + 1 ? 0.0f : w1);
      }
      if (at >= 0 && at < nj && col < p.rows) p.diag[(long long)x.g * p.diag_ld + col] = p.c2 + d * (1.0f / 4096.0f);
    } else if (EPI == kOut16 && p.out_bf16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    } else {
      const float c = EPI == kGram ? p.c1 : 1.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = pack_half(v[2 * i] * c, v[2 * i + 1] * c);
    }
    if constexpr (symmetric(EPI)) {  // the tile's transpose, and itself where no other tile is its transpose
      if (col < p.rows) store_lane_row(out + lane_row(p, x, p.rows, j0, col), w, nj);
      if (x.triangle && x.rt != x.ct) store_turned(out + row * p.ld + col - lane, p.ld, buf, w, nj, p.ld - (col - lane), lane);
    } else {
      store_turned(out + row * p.cols + col - lane, p.cols, buf, w, nj, p.cols - (col - lane), lane);
    }
  }
}

// kGrad: rows j0 + [0, nj) leave as one box of 32 x 32 (16 x 32 at the end of a tile) from the buffer
// whose last store was the last but one; what lies past the matrix is not written
__device__ __forceinline__ void emit_grad(const Params& p, const Item& x, uint8_t* buf, uint32_t& stored,
                                          const float (&v)[32], int j0, int nj, int col, int lane) {
  float* b = reinterpret_cast<float*>(buf + (stored++ & 1) * 2 * kChunkBytes);
  if (lane == 0) bulk_wait_read_but_one();
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 32; ++j) b[j * 32 + lane] = v[j];
  fence_async();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(nj > 16 ? &p.out_map : &p.out16_map, b, col - lane, x.r0 + j0, x.g);
    bulk_commit();
  }
}

// the sum of a split tile's parts over rows j0 + [0, 32), in the order of the parts, ROWS x PARTS loads in
// flight at a time (past the last row or part: the last again)
template <int ROWS, int PARTS>
__device__ __forceinline__ void add_parts(const float* first, size_t pitch, int parts, int nj, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; j += ROWS) {
    if (j < nj) {
#pragma unroll 1
      for (int s = 0; s < parts; s += PARTS) {
        float t[PARTS][ROWS];
#pragma unroll
        for (int u = 0; u < PARTS; ++u)
#pragma unroll
          for (int i = 0; i < ROWS; ++i)
            t[u][i] = __ldcg(first + min(s + u, parts - 1) * pitch + (size_t)min(j + i, nj - 1) * 128);
#pragma unroll
        for (int u = 0; u < PARTS; ++u)
#pragma unroll
          for (int i = 0; i < ROWS; ++i) v[j + i] += s + u < parts && j + i < nj ? t[u][i] : 0.0f;
      }
    }
  }
}

__device__ __forceinline__ float* part_ptr(const Params& p, int slot, int split, int part, int rank) {
  return p.partial + (((size_t)slot * split + part) * 2 + rank) * (size_t)p.prows * 128;
}

// ------------------------------------------------------------------------------ the kernel
template <bool A_MN, bool B_MN, int RAGGED, int EPI>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Params p) {
  constexpr bool kPromote = EPI == kOut32 || EPI == kGrad, kAdds = EPI == kPoly || applies(EPI);
  constexpr bool kPX = B_MN;  // kApply, kApplyLast: X is the MN-major operand where it is contracted over its rows
  constexpr int kStages = stages_of(EPI);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);  // even CTA: both halves landed
  uint64_t* empty = full + kStages;                                           // both CTAs: stage consumed
  uint64_t* acc_full = empty + kStages;                                       // both CTAs: accumulator ready
  uint64_t* acc_empty = acc_full + 2;                                         // even CTA: both epilogues done
  uint64_t* tail_bar = acc_empty + 2;                                         // kRaggedK: this CTA's tail block landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail_bar + kStages);
  uint8_t* staging = smem + kStages * kStageBytes + kBarBytes;
  int* sched_smem = reinterpret_cast<int*>(staging + kEpiWarps * staging_of(EPI));
  volatile uint32_t* progress = reinterpret_cast<uint32_t*>(sched_smem + 3);  // kRaggedK: see the tail blocks
  int* tab = sched_smem + 4;  // item_of's table

  // the parameters' lines are fetched while the barriers are set up, not one by one where they are used
  asm volatile("" ::"r"(p.G), "r"(p.rows), "r"(p.cols), "r"(p.K), "r"(p.ld), "r"(p.prows), "r"(p.kb_typ), "l"(p.err));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    if (RAGGED == kRaggedK) *progress = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], RAGGED == kRaggedK ? 2 : 1);  // kRaggedK: see the tail blocks below
      mbar_init(&empty[s], 1);
      mbar_init(&tail_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    fence_barrier_init();
    prefetch_tensormap(&p.a);
    for (int i = 0; i < (B_MN ? 1 : kBoxes); ++i) prefetch_tensormap(&p.b[i]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * kTile);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // both CTAs' barriers and tensor memory are ready before either is used remotely
  tc_fence_after();
  // Segments are read from memory that the kernel before may have written; the schedule of equal groups is
  // not, so there the producer and the epilogue wait before their own first access: 136 -> 128 us for
  // 16 x [512, 256].
  if constexpr (RAGGED != kDense) pdl_wait();
  pdl_trigger();
  if constexpr (RAGGED != kDense) {
    for (int g = threadIdx.x; g < p.G; g += kThreads) {
      int row0, rows;
      bool bad;
      segment(p, g, row0, rows, bad);
      if (bad && blockIdx.x == 0) set_error(p.err, kErrBadIndex);
      if (p.G <= table_groups(EPI)) {
        tab[2 * g] = row0;
        tab[2 * g + 1] = rows;
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    int all = p.tiles, split = p.split;
    if constexpr (RAGGED == kRaggedRows) {  // exclusive scan of the groups' tile counts
      const int per = (p.G + 31) / 32;
      const int lo = min(p.G, lane * per), hi = min(p.G, lo + per);
      int own = 0;
      for (int g = lo; g < hi; ++g) own += tiles_of<EPI>(tab[2 * g + 1], p.ct, p.lr);
      int run = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run += v;
      }
      all = __shfl_sync(0xffffffffu, run, 31);
      run -= own;
      for (int g = lo; g < hi; ++g) {
        tab[2 * p.G + g] = run;
        run += tiles_of<EPI>(tab[2 * g + 1], p.ct, p.lr);
      }
      split = split_of(all % n_clusters, n_clusters, p.kb_typ, min(p.rows_typ, 1 << p.lr), lane);
    }
    if (lane == 0) {
      const int r = all % n_clusters;
      sched_smem[0] = split > 1 ? all - r : all;
      sched_smem[1] = split;
      sched_smem[2] = split > 1 ? all - r + r * split : all;
    }
  }
  __syncthreads();
  const uint32_t tmem_base = *tmem_slot;
  Sched sc;
  sc.full = sched_smem[0], sc.split = sched_smem[1], sc.items = sched_smem[2];
  sc.per = RAGGED == kRaggedRows ? 1 : tiles_of<EPI>(p.rows, p.ct, p.lr);
  sc.step = step_of<EPI>(p.rows, (p.rows + (1 << p.lr) - 1) >> p.lr, p.lr);
  sc.inv_split = __frcp_rn((float)sc.split), sc.inv_band = __frcp_rn((float)(kBand * p.ct)), sc.inv_per = __frcp_rn((float)sc.per);

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int i = cluster_id; i < sc.items && ok; i += n_clusters) {
        const Item x = item_of<RAGGED, EPI>(p, tab, sc, i);
        if (RAGGED == kDense && i == cluster_id) pdl_wait();
        const int half = half_of(x.nr);
        const int box = B_MN ? 0 : box_of(half);
        const CUtensorMap* bmap = &p.b[box];
        const uint32_t bytes = (uint32_t)kTileA + (B_MN ? (half > 64 ? 16384u : 8192u) : (uint32_t)box_rows(box) * 128u);
        const int acol = x.ct * kTile + (int)rank * 128;
        const int brow = (RAGGED == kRaggedRows ? x.row0 : 0) + x.r0 + (int)rank * half;
        const int ag = RAGGED == kRaggedK ? 0 : x.g;
        const int bg = RAGGED == kDense ? x.g : 0;
        for (int kb = x.kb0; kb < x.kb1; ++kb, ++it) {
          const int stage = it % kStages;
          if (!sleep_wait(&empty[stage], ((it / kStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (RAGGED == kRaggedK && (it & 0xffff) == 0) *progress = it;
          uint8_t* sa = smem + stage * kStageBytes;
          uint8_t* sb = sa + kTileA;
          const int kx = kb * kBK;
          const int ky = x.k0 + kx;  // k as a row of an MN-major operand (x.k0 = 0 unless kRaggedK)
          if (RAGGED == kRaggedK && ragged_tail(x.krows, kx)) {
            // lands on this CTA's own barrier; warp 10 hands it on
            mbar_arrive_expect_tx(&tail_bar[stage], bytes);
            tma_3d(&p.a, &tail_bar[stage], sa, acol, ky, ag);
            tma_3d(&p.a, &tail_bar[stage], sa + 8192, acol + 64, ky, ag);
            tma_3d(bmap, &tail_bar[stage], sb, brow, ky, bg);
            if (half > 64) tma_3d(bmap, &tail_bar[stage], sb + 8192, brow + 64, ky, bg);
            continue;
          }
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          if (leader) {
            mbar_arrive_expect_tx(&full[stage], 2u * bytes);
            if (RAGGED == kRaggedK) mbar_arrive(&full[stage]);
          }
          if (leader && p.withhold_first_load && it == 0) continue;
          if constexpr (A_MN) {
            tma_3d_pair(&p.a, bar, sa, acol, ky, ag);
            tma_3d_pair(&p.a, bar, sa + 8192, acol + 64, ky, ag);
          } else {
            tma_3d_pair(&p.a, bar, sa, kx, acol, ag);
          }
          if constexpr (B_MN) {
            tma_3d_pair(bmap, bar, sb, brow, ky, bg);
            if (half > 64) tma_3d_pair(bmap, bar, sb + 8192, brow + 64, ky, bg);
          } else {
            tma_3d_pair(bmap, bar, sb, kx, brow, bg);
          }
        }
      }
      if (!ok) set_error(p.err, kErrTimeout);
      // every stage this CTA filled must be consumed (the even CTA: landed) before shared memory is
      // released; after one expired wait the copies still in flight have long landed
      for (int s = 0; s < kStages; ++s) {
        if ((uint32_t)s >= it) break;
        const uint32_t last = it - 1 - ((it - 1 - s) % kStages);
        if (!sleep_wait(leader ? &full[s] : &empty[s], (last / kStages) & 1)) {
          set_error(p.err, kErrTimeout);
          break;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (even CTA)
    if (leader && lane == 0) {
      uint32_t it = 0, use = 0;
      bool ok = true;
      for (int i = cluster_id; i < sc.items && ok; i += n_clusters) {
        const Item x = item_of<RAGGED, EPI>(p, tab, sc, i);
        const uint32_t idesc = p.idesc | ((uint32_t)(2 * half_of(x.nr)) >> 3 << 17) | (16u << 24);
        int kb = x.kb0;
        do {  // one use of an accumulator: the whole item, or one drain's K blocks; at least one
          const uint32_t buf = use & 1;
          if (!sleep_wait(&acc_empty[buf], ((use >> 1) & 1) ^ 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + buf * kTile;
          const int end = kPromote ? min(x.kb1, kb + kPromoteBlocks) : x.kb1;
          uint32_t accumulate = 0;
          for (; kb < end; ++kb, ++it) {
            const int stage = it % kStages;
            // acquiring from the other CTA's threads costs about 800 cycles: only where they wrote
            const bool landed = RAGGED == kRaggedK && ragged_tail(x.krows, kb * kBK)
                                    ? sleep_wait<true>(&full[stage], (it / kStages) & 1)
                                    : sleep_wait(&full[stage], (it / kStages) & 1);
            if (!landed) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * kStageBytes), sb = sa + kTileA;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) {
              if (RAGGED == kRaggedK && kb * kBK + kk * 16 >= x.krows) break;  // behind the segment
              const uint64_t ad = A_MN ? mn_desc(sa + kk * 2048) : sw128_kmajor_desc(sa + kk * 32);
              const uint64_t bd = B_MN ? mn_desc(sb + kk * 2048) : sw128_kmajor_desc(sb + kk * 32);
              umma_bf16_pair(d, ad, bd, idesc, accumulate);
              accumulate = 1;
            }
            umma_commit_pair(&empty[stage], 0x3);
          }
          if (!ok) break;
          umma_commit_pair(&acc_full[buf], 0x3);  // also after no MMA at all: the epilogue takes zeros
          ++use;
        } while (kb < x.kb1);
      }
      if (!ok) set_error(p.err, kErrTimeout);
      if (it > 0) {  // the last commit covers every MMA issued before it
        const uint32_t last = it - 1;
        if (!sleep_wait(&empty[last % kStages], (last / kStages) & 1)) set_error(p.err, kErrTimeout);
      }
    }
  } else if (warp == 2 + kEpiWarps) {
    // ------------------------------------------------------------------ tail blocks (kRaggedK, both CTAs)
    // The rows of a segment's last block past its end belong to the next segment, and an infinity or
    // NaN of theirs must not meet a zero.  Both operands are MN-major: k row r of a box is the 128 bytes
    // at r * 128 (the swizzle permutes within a row), so once the block has landed its rows up to the
    // next multiple of 16 are zeroed in both operands and the stage is handed to the MMA; the producer
    // has gone on meanwhile.  Of the full barrier's two arrivals each CTA makes one here; for the other
    // blocks the even CTA's producer makes both, so that no arrival crosses the pair.  A tile of a segment
    // of 10^8 rows can take longer than one wait may, so a wait that has expired is made again if the
    // producer has come on by 2^16 blocks (some 30 ms) in it.
    if constexpr (RAGGED == kRaggedK) {
      uint32_t it = 0, phases = 0;
      bool ok = true;
      for (int i = cluster_id; i < sc.items && ok; i += n_clusters) {
        const Item x = item_of<RAGGED, EPI>(p, tab, sc, i);
        const int count = x.kb1 - x.kb0, kx = (x.kb1 - 1) * kBK;
        it += count;
        if (count <= 0 || !ragged_tail(x.krows, kx)) continue;
        const int stage = (it - 1) % kStages;
        uint32_t seen = *progress;
        while (!(ok = __all_sync(0xffffffffu, sleep_wait(&tail_bar[stage], (phases >> stage) & 1)))) {
          const uint32_t now = __shfl_sync(0xffffffffu, *progress, 0);
          if (__shfl_sync(0xffffffffu, seen, 0) == now) break;
          seen = now;
        }
        phases ^= 1u << stage;
        if (!ok) break;
        uint8_t* sa = smem + stage * kStageBytes;
        const int valid = x.krows - kx, end = (valid + 15) / 16 * 16;
        for (int o = valid * 128 + lane * 16; o < end * 128; o += 512) {
#pragma unroll
          for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(sa + q * 8192 + o) = make_uint4(0, 0, 0, 0);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&full[stage]);
          else mbar_arrive_cluster(mapa_shared(smem_u32(&full[stage]), 0));
        }
      }
      if (!ok && lane == 0) set_error(p.err, kErrTimeout);
    }
  } else {
    // ------------------------------------------------------------------ epilogue (warps 2..9, both CTAs)
    const int q = warp & 3;         // TMEM lane quarter this warp may read
    const int h = (warp - 2) >> 2;  // which half of the tile's rows, in chunks of 32
    uint32_t use = 0;
    bool ok = true;
    uint8_t* const buf0 = staging + (warp - 2) * staging_of(EPI);
    uint32_t stored = 0;  // kGrad: chunks stored, alternately from two buffers
    Addend<EPI> next;     // the next chunk's addend
    for (int i = cluster_id; i < sc.items && ok; i += n_clusters) {
      const Item x = item_of<RAGGED, EPI>(p, tab, sc, i);
      if (RAGGED == kDense && i == cluster_id) pdl_wait();
      const int col = x.ct * kTile + (int)rank * 128 + q * 32 + lane;
      const bool none = x.kb1 <= x.kb0;
      const bool split = x.slot >= 0;
      float* mine = split ? part_ptr(p, x.slot, sc.split, x.part, (int)rank) + q * 32 + lane : nullptr;
      // chunks of 32 rows with valid rows; of kGrad none where no column is valid
      const int all = (x.nr + 31) / 32, first = h * ((all + 1) / 2);
      const int chunks = EPI == kGrad && col - lane >= p.ld ? 0 : h == 0 ? (all + 1) / 2 : all / 2;
      const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16) + first * 32;
      // what becomes of rows j0 + [0, nj) in v
      auto finish = [&](const float (&v)[32], int c) {
        const int j0 = (first + c) * 32;
        const int nj = min(32, x.nr - j0);
        if (split) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < nj) __stcg(mine + (size_t)(j0 + j) * 128, v[j]);
        } else if constexpr (EPI == kGrad) {
          emit_grad(p, x, buf0, stored, v, j0, nj, col, lane);
        } else if constexpr (kAdds) {
          const Addend<EPI> s = next;
          load_addend<EPI, kPX>(p, x, next, c + 1 < chunks ? j0 + 32 : x.nr, col, lane);
          emit<RAGGED, EPI, kPX>(p, x, buf0, v, s, j0, nj, col, lane);
        } else {
          emit<RAGGED, EPI, kPX>(p, x, buf0, v, next, j0, nj, col, lane);
        }
      };
      if (kPromote && x.kb1 - x.kb0 > kPromoteBlocks) {
        float acc[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c][j] = 0.0f;
        for (int kb = x.kb0; kb < x.kb1; kb += kPromoteBlocks, ++use) {
          const uint32_t buf = use & 1;
          ok = __all_sync(0xffffffffu, sleep_wait(&acc_full[buf], (use >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c < chunks) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {  // 16 at a time: 128 sums and 16 addends fit the registers
                uint32_t r[16];
                tmem_ld_32x32b_x16(tlane + buf * kTile + c * 32 + u * 16, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[c][u * 16 + j] += __uint_as_float(r[j]);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_even(&acc_empty[buf]);
        }
        if (!ok) {
          if (lane == 0) set_error(p.err, kErrTimeout);
          break;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) finish(acc[c], c);
      } else {
        const uint32_t buf = use & 1;
        if constexpr (kAdds)
          if (!split && chunks > 0) load_addend<EPI, kPX>(p, x, next, first * 32, col, lane);
        ok = __all_sync(0xffffffffu, sleep_wait(&acc_full[buf], (use >> 1) & 1));
        if (!ok) {
          if (lane == 0) set_error(p.err, kErrTimeout);
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(tlane + buf * kTile + c * 32, r);
          tmem_ld_wait();
          if (c + 1 == chunks) {  // the accumulator has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_even(&acc_empty[buf]);
          }
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = none ? 0.0f : __uint_as_float(r[j]);
          finish(v, c);
        }
        if (chunks == 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive_even(&acc_empty[buf]);
        }
        ++use;
      }
      if (split) {
        // the last of the parts to store this warp's share (its lanes, its half of the rows) adds them up
        __threadfence();
        __syncwarp();
        int* counter = p.counters + (x.slot * 2 + (int)rank) * kEpiWarps + (warp - 2);
        int before = 0;
        if (lane == 0) before = atomicAdd(counter, 1);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before == sc.split - 1) {
          __threadfence();
          if (lane == 0) *counter = 0;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            const int j0 = (first + c) * 32;
            const int nj = min(32, x.nr - j0);
            if constexpr (kAdds) load_addend<EPI, kPX>(p, x, next, j0, col, lane);
            const float* part0 = part_ptr(p, x.slot, sc.split, 0, (int)rank) + (size_t)j0 * 128 + q * 32 + lane;
            const size_t pitch = 2 * (size_t)p.prows * 128;
            float v[32];
            if (nj <= 4) add_parts<4, 16>(part0, pitch, sc.split, nj, v);
            else add_parts<8, 8>(part0, pitch, sc.split, nj, v);
            if constexpr (EPI == kGrad) emit_grad(p, x, buf0, stored, v, j0, nj, col, lane);
            else emit<RAGGED, EPI, kPX>(p, x, buf0, v, next, j0, nj, col, lane);
          }
        }
      }
    }
    if constexpr (EPI == kGrad)
      if (lane == 0) bulk_wait();
  }

  tc_fence_before();
  __syncthreads();
  __syncwarp();
  // neither CTA leaves (or frees TMEM) while its partner may still signal its barriers or the pair's
  // MMAs may still write its tensor memory
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kTile);
  }
}

// ------------------------------------------------------------------------------ host side
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(ptr);
  });
  return fn;
}

// row-major [groups, rows, inner] tensor, box of box_inner elements x box_rows rows of one group, 128-byte
// swizzle for an operand, none for what the epilogue loads or stores; what lies past inner or rows reads as
// zero and is not written.  A row is a multiple of 16 bytes.
inline bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t rows,
                     uint64_t groups, uint32_t box_inner, uint32_t box_rows, bool swizzle) {
  EncodeFn enc = encode_fn();
  if (enc == nullptr || inner == 0 || rows == 0 || groups == 0) return false;
  const uint64_t size = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  cuuint64_t dims[3] = {inner, rows, groups};
  cuuint64_t strides[2] = {inner * size, inner * rows * size};
  cuuint32_t box[3] = {box_inner, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the current device is one this library runs on
inline moe_status_t device_status() {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_NO_DEVICE;
  }
  return major == 10 ? MOE_OK : MOE_ERR_NO_DEVICE;
}

inline moe_status_t launch_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

struct OperandHost {
  const void* base;
  uint64_t inner, rows, groups;  // as stored
};

// Fills the operand maps and the descriptor's types.  bf16 selects the type of both operands.
template <bool A_MN, bool B_MN>
bool set_operands(Params& p, const OperandHost& a, const OperandHost& b, bool bf16) {
  const uint32_t ty = bf16 ? 1u : 0u;
  p.idesc = (1u << 4) | (ty << 7) | (ty << 10) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16);
  const CUtensorMapDataType type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!make_map(&p.a, type, a.base, a.inner, a.rows, a.groups, 64, A_MN ? 64 : 128, true)) return false;
  for (int i = 0; i < (B_MN ? 1 : kBoxes); ++i)
    if (!make_map(&p.b[i], type, b.base, b.inner, b.rows, b.groups, 64, B_MN ? 64 : box_rows(i), true)) return false;
  return true;
}

// kGrad's maps of its fp32 [groups, rows, inner] output
inline bool set_output(Params& p, const OperandHost& t) {
  return make_map(&p.out_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, t.base, t.inner, t.rows, t.groups, 32, 32, false) &&
         make_map(&p.out16_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, t.base, t.inner, t.rows, t.groups, 32, 16, false);
}

// Tile size and parts (see cost_of).  kRaggedRows: for the mean segment of the groups that have rows
template <int RAGGED, int EPI>
void choose(Params& p, int clusters) {
  p.ct = (p.cols + kTile - 1) / kTile;
  const int groups = RAGGED == kRaggedRows && p.M_total < p.G ? p.M_total : p.G;
  const int rows = RAGGED == kRaggedRows ? (p.M_total + groups - 1) / groups : p.rows;
  float best = 1e30f;
  for (int lr = kMostLr; lr >= kLeastLr; --lr) {
    const long long tiles = (long long)groups * tiles_of<EPI>(rows, p.ct, lr);
    if (lr < kMostLr && tiles > 8 * clusters) break;  // large products: whole tiles
    const int t = (int)(tiles < (1LL << 30) ? tiles : 1LL << 30), most = most_parts(t % clusters, p.kb_typ);
    for (int s = 1; s == 1 || s <= most; ++s) {
      const float c = cost_of(t, clusters, p.kb_typ, rows < 1 << lr ? rows : 1 << lr, s);
      if (c < best) {
        best = c;
        p.lr = lr;
        p.tiles = t;
        p.split = s;
      }
    }
  }
}

template <bool A_MN, bool B_MN, int RAGGED, int EPI>
cudaError_t launch(Params& p, cudaStream_t s) {
  auto kernel = product_kernel<A_MN, B_MN, RAGGED, EPI>;
  static std::atomic<int> cached[64];  // clusters that fit on the device at once, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(EPI);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  int clusters = dev >= 0 && dev < 64 ? cached[dev].load() : 0;
  if (clusters == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(EPI));
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2);
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters <= 0) return cudaErrorInvalidConfiguration;
    clusters = clusters > kMaxParts / 2 ? kMaxParts / 2 : clusters;
    if (dev >= 0 && dev < 64) cached[dev].store(clusters);
  }
  choose<RAGGED, EPI>(p, clusters);
  cfg.gridDim = dim3(2 * clusters);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace product
}  // namespace moe
