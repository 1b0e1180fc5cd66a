// product_sm100.cuh -- the tcgen05 kernel of the grouped products (grouped_product.cu) and of the
// Newton-Schulz iteration (orthogonalize.cu).  For every group g it computes
//
//     out_g[r][c] = sum_k B_g[r][k] * A_g[c][k]        rows r, contiguous columns c
//
// with 16-bit operands (both bf16 or both fp16) and fp32 accumulators in tensor memory.  The
// contiguous output dimension is the MMA's M side (operand A), the rows are its N side (operand B),
// so a ragged last row tile costs its own rows rounded up to 16 instead of a whole tile, and a TMEM
// lane is an output column: a warp stores 32 neighbouring columns of one row per instruction.
// Each operand is K-major (stored [index][k]) or MN-major (stored [k][index]); both come in by TMA
// with the 128-byte swizzle and only the descriptors differ, so no operand is ever transposed in
// memory.
//
// One tile is 256 columns x up to 256 rows on a cluster of two CTAs (tcgen05.mma.cta_group::2, M = 256):
// each CTA loads its own 128 columns and its half of the rows, 32 KB per 64-wide K block for a
// 128 x 256 x 64 product -- 64 bytes per cycle and SM at the tensor pipe's rate, where a one-CTA tile
// would need 96.  No load is multicast.
//
// Kernel layout (persistent clusters of two, 320 threads per CTA):
//   warp 0     TMA producer: 6 stages of 32 KB.
//   warp 1     TMEM allocation; in the even CTA one thread issues the pair's MMAs.
//   warps 2-9  epilogue: four TMEM lane quarters x two halves of the rows.
// Tiles are dealt round-robin.  The tiles of the last, partly filled round are split along K when
// that shortens the round (few rows, one token: split_of); each part stores its fp32 accumulators and
// the last part to arrive (an atomic counter per warp's share, no waiting) adds them in the order of
// the parts, so results do not depend on timing.
//
// Rounding.  The tensor core truncates when it aligns an addend to its accumulator, which biases a
// long sum towards zero: about 1e-9 of the sum for every k (measured on this GPU through a library
// product with fp32 results: 1e-6 at k = 1024, 4.4e-6 at 4096, 1.9e-5 at 16384).  Where the result stays
// fp32 (PROMOTE), the accumulator is therefore drained every 512 k into registers and added there,
// rounded to nearest; a 16-bit result, 2^-9 wide, does not see it.
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
  kPoly = 3,      // symmetric: out = fp16(c0 * src + acc * c1), and its mirror image
  kApply = 4,     // x = c0 * (src + src_lo / 2048) + acc * c1; out = fp16(x), out_lo = fp16(2048 (x - out))
  kApplyLast = 5  // out = bf16(the same x * c2), rows of ld_out elements
};

constexpr int kTile = 256;               // rows (N) and columns (M) of a pair's tile
constexpr int kBK = 64;                  // K per stage
constexpr int kStages = 6;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kTileA = 128 * kBK * 2;    // 16 KB: this CTA's columns
constexpr int kTileB = 128 * kBK * 2;    // 16 KB: this CTA's rows, at most
constexpr int kStageBytes = kTileA + kTileB;
constexpr int kPromoteBlocks = 8;        // K blocks per accumulator drain (512 k)
constexpr int kMaxGroups = 1024;
constexpr int kBarBytes = 256;
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + kBarBytes + 4 * (kMaxGroups + 4);
static_assert(kSmemBytes <= 232448, "shared memory budget");

// workspace of a launch: error word, counters (zero between launches), split-K partial sums
constexpr int kMaxParts = 148;           // split tiles x parts
constexpr int kMaxSplit = 16;
constexpr size_t kCounterBytes = 8192;   // 16 per split tile; fewer split tiles than clusters (<= 74)
constexpr size_t kPartialOffset = kWsHeader + kCounterBytes;
inline int partial_rows(long long rows) { return rows >= kTile ? kTile : (int)((rows + 31) / 32 * 32); }
inline size_t partial_bytes(int prows) { return (size_t)kMaxParts * 2 * 128 * 4 * (size_t)prows; }

struct alignas(64) Params {
  CUtensorMap a;    // K-major: box 64 k x 128 columns; MN-major: box 64 columns x 64 k
  CUtensorMap b;    // K-major: box 64 k x 128 rows;    MN-major: box 64 rows x 64 k
  CUtensorMap b32;  // K-major only: the same tensor, boxes of 32 and 8 rows for ragged halves
  CUtensorMap b8;
  const int32_t* offsets;  // kRaggedRows / kRaggedK: segment bounds [G + 1]
  int G;                   // groups
  int M_total;             // rows of the ragged tensor
  int rows, cols, K;       // rows (not kRaggedRows), columns and K (not kRaggedK) of a group
  uint32_t idesc;          // instruction descriptor without M and N
  int out_bf16;            // kOut16: bf16 instead of fp16
  int ld, ld_out;          // row pitch of src / src_lo / out / out_lo; of the last output
  int cols_out;            // kApplyLast: columns that are stored
  void* out;
  uint16_t* out_lo;
  const uint16_t* src;
  const uint16_t* src_lo;
  float c0, c1, c2;
  float* partial;
  int* counters;
  int prows;               // rows per partial tile
  int kb_typ;              // K blocks of a typical tile (the split's cost model)
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
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// as mbar_wait, seeing what the other CTA wrote before its arrival
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait_cluster(a, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_cluster(a, parity)) {
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
  return true;
}
// UMMA descriptor of an MN-major operand: 64-element chunks 8 KB apart, 8-k groups 1 KB apart
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// ------------------------------------------------------------------------------ schedule
struct Sched {
  int full;   // tiles dealt whole
  int split;  // parts of each later tile
  int items;
};

// Parts of each of the r < clusters tiles of the last round.  Cost in K blocks: rounds of parts, each
// with a fixed share for filling the pipeline and for the epilogue, and the reading of the parts.
// Without the split a one-token product of 4 experts x [5760, 2880] leaves 3/4 of the clusters idle in
// its second round.
__device__ __forceinline__ int split_of(int r, int clusters, int kb) {
  if (r <= 0) return 1;
  const int most = min(kMaxSplit, min(kb / 2, kMaxParts / r));
  int best = 1;
  float cost = 1e30f;
  for (int s = 1; s <= most || s == 1; ++s) {
    const float rounds = (float)((r * s + clusters - 1) / clusters);
    const float c = rounds * ((float)kb / (float)s + 4.0f) + (s > 1 ? 2.0f + 0.5f * (float)s : 0.0f);
    if (c < cost) cost = c, best = s;
  }
  return best;
}

struct Item {
  int g;
  int rt, ct;        // row tile, column tile
  int nr;            // rows of this tile (1..256)
  int row0;          // kRaggedRows: first row of the segment
  int k0, krows;     // kRaggedK: first k row and number of k rows
  int kb0, kb1;      // K blocks [kb0, kb1)
  int part, slot;    // part of the split, split-tile index (-1: whole)
};

__device__ __forceinline__ void segment(const Params& p, int g, int& row0, int& rows, bool& bad) {
  const int a = p.offsets[g], b = p.offsets[g + 1];
  row0 = min(max(a, 0), p.M_total);
  const int end = min(max(b, row0), p.M_total);
  rows = end - row0;
  bad = row0 != a || end != b;
}

template <int RAGGED, int EPI>
__device__ __forceinline__ int tiles_of(const Params& p, int rows) {
  const int rt = (rows + kTile - 1) / kTile;
  if constexpr (EPI == kGram || EPI == kPoly) return rt * (rt + 1) / 2;
  return rt * ((p.cols + kTile - 1) / kTile);
}

template <int RAGGED, int EPI>
__device__ __forceinline__ Item item_of(const Params& p, const int* tile_start, const Sched& sc, int i) {
  Item x;
  int t = i;
  int parts = 1;
  x.part = 0;
  x.slot = -1;
  if (i >= sc.full && sc.split > 1) {
    x.slot = (i - sc.full) / sc.split;
    x.part = (i - sc.full) - x.slot * sc.split;
    t = sc.full + x.slot;
    parts = sc.split;
  }
  int rows = p.rows, local;
  x.row0 = 0, x.k0 = 0, x.krows = 0;
  bool bad;
  if constexpr (RAGGED == kRaggedRows) {
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile_start[mid] <= t) lo = mid; else hi = mid - 1;
    }
    x.g = lo;
    segment(p, lo, x.row0, rows, bad);
    local = t - tile_start[lo];
  } else {
    const int per = tiles_of<RAGGED, EPI>(p, p.rows);
    x.g = t / per;
    local = t - x.g * per;
    if constexpr (RAGGED == kRaggedK) segment(p, x.g, x.k0, x.krows, bad);
  }
  const int rt = (rows + kTile - 1) / kTile;
  if constexpr (EPI == kGram || EPI == kPoly) {
    // lower triangle, row by row
    int r = (int)((sqrtf(8.0f * (float)local + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1) / 2 > local) --r;
    while ((r + 1) * (r + 2) / 2 <= local) ++r;
    x.rt = r;
    x.ct = local - r * (r + 1) / 2;
  } else {
    // bands of 8 row tiles, rows fastest inside a band: the ~74 tiles in flight share about 8 row
    // blocks and 9 column blocks through L2
    const int ct = (p.cols + kTile - 1) / kTile;
    const int band = local / (8 * ct);
    const int rem = local - band * 8 * ct;
    const int rb = min(8, rt - 8 * band);
    x.ct = rem / rb;
    x.rt = 8 * band + (rem - x.ct * rb);
  }
  x.nr = min(kTile, rows - x.rt * kTile);
  const int kb = RAGGED == kRaggedK ? (x.krows + kBK - 1) / kBK : (p.K + kBK - 1) / kBK;
  x.kb0 = split_begin(kb, x.part, parts);
  x.kb1 = split_end(kb, x.part, parts);
  return x;
}

// rows of B each CTA holds: half of the tile's rows rounded up to 16 (an MN-major B: always 128, the
// rows past the tensor read as zero)
template <bool B_MN>
__device__ __forceinline__ int half_of(int nr) {
  return B_MN ? 128 : ((nr + 15) / 16) * 8;
}

// ------------------------------------------------------------------------------ epilogue
__device__ __forceinline__ uint16_t half_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ float half_val(uint16_t b) { return __half2float(__ushort_as_half(b)); }

// v[j] = accumulator of row j0 + j and column col (this lane's) of the item; nj rows are valid
template <int RAGGED, int EPI>
__device__ __forceinline__ void emit(const Params& p, const Item& x, const float (&v)[32], int j0, int nj, int col) {
  const int row_in = x.rt * kTile + j0;  // row within the group
  const long long row = (RAGGED == kRaggedRows ? (long long)x.row0 : (long long)x.g * p.rows) + row_in;
  if constexpr (EPI == kOut16) {
    if (col >= p.cols) return;
    uint16_t* o = static_cast<uint16_t*>(p.out) + row * p.cols + col;
    const bool bf = p.out_bf16 != 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j < nj) {
        const uint16_t h = bf ? __bfloat16_as_ushort(__float2bfloat16_rn(v[j])) : half_bits(v[j]);
        o[(long long)j * p.cols] = h;
      }
    }
  } else if constexpr (EPI == kOut32) {
    if (col >= p.cols) return;
    float* o = static_cast<float*>(p.out) + row * p.cols + col;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < nj) o[(long long)j * p.cols] = v[j];
  } else if constexpr (EPI == kGram || EPI == kPoly) {
    uint16_t h[32];
    const long long base = (long long)x.g * p.rows * p.ld;
    const uint16_t* s = p.src + base + (long long)row_in * p.ld + col;
    uint16_t* o = static_cast<uint16_t*>(p.out) + base + (long long)row_in * p.ld + col;
    const bool col_ok = col < p.ld;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float w = v[j] * p.c1;
      if constexpr (EPI == kPoly) w += (col_ok && j < nj) ? p.c0 * half_val(s[(long long)j * p.ld]) : 0.0f;
      h[j] = half_bits(w);
      if (col_ok && j < nj) o[(long long)j * p.ld] = h[j];
    }
    if (x.rt != x.ct && col < p.rows) {  // the mirror image: row `col`, columns row_in ..
      uint16_t* m = static_cast<uint16_t*>(p.out) + base + (long long)col * p.ld + row_in;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (row_in + 8 * u + 8 <= p.ld) {
          uint4 w;
          w.x = (uint32_t)h[8 * u] | (uint32_t)h[8 * u + 1] << 16;
          w.y = (uint32_t)h[8 * u + 2] | (uint32_t)h[8 * u + 3] << 16;
          w.z = (uint32_t)h[8 * u + 4] | (uint32_t)h[8 * u + 5] << 16;
          w.w = (uint32_t)h[8 * u + 6] | (uint32_t)h[8 * u + 7] << 16;
          *reinterpret_cast<uint4*>(m + 8 * u) = w;
        }
      }
    }
  } else {
    if (col >= p.ld) return;
    const long long at = row * p.ld + col;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j < nj) {
        const long long i = at + (long long)j * p.ld;
        const float w = p.c0 * (half_val(p.src[i]) + half_val(p.src_lo[i]) * (1.0f / 2048.0f)) + v[j] * p.c1;
        if constexpr (EPI == kApply) {
          const uint16_t h = half_bits(w);
          static_cast<uint16_t*>(p.out)[i] = h;
          p.out_lo[i] = half_bits((w - half_val(h)) * 2048.0f);
        } else if (col < p.cols_out) {
          static_cast<uint16_t*>(p.out)[(row + j) * p.ld_out + col] =
              __bfloat16_as_ushort(__float2bfloat16_rn(w * p.c2));
        }
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
  constexpr bool kPromote = EPI == kOut32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);  // even CTA: both halves landed
  uint64_t* empty = full + kStages;                                           // both CTAs: stage consumed
  uint64_t* acc_full = empty + kStages;                                       // both CTAs: accumulator ready
  uint64_t* acc_empty = acc_full + 2;                                         // even CTA: both epilogues done
  uint64_t* tail_bar = acc_empty + 2;                                         // kRaggedK: this CTA's tail block landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail_bar + 1);
  int* sched_smem = reinterpret_cast<int*>(smem + kStages * kStageBytes + kBarBytes);
  int* tile_start = sched_smem + 3;  // kRaggedRows: [G + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], RAGGED == kRaggedK ? 2 : 1);  // kRaggedK: each CTA's producer arrives
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(tail_bar, 1);
    fence_barrier_init();
    prefetch_tensormap(&p.a);
    prefetch_tensormap(&p.b);
    if constexpr (!B_MN) {
      prefetch_tensormap(&p.b32);
      prefetch_tensormap(&p.b8);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * kTile);
    tmem_relinquish_pair();
  }
  pdl_wait();
  pdl_trigger();
  if constexpr (RAGGED != kDense) {
    for (int g = threadIdx.x; g < p.G; g += kThreads) {
      int row0, rows;
      bool bad;
      segment(p, g, row0, rows, bad);
      if (bad && blockIdx.x == 0) set_error(p.err, kErrBadIndex);
      if constexpr (RAGGED == kRaggedRows) tile_start[g] = tiles_of<RAGGED, EPI>(p, rows);
    }
  }
  __syncthreads();
  if (warp == 0) {
    int total;
    if constexpr (RAGGED == kRaggedRows) {  // exclusive scan of the groups' tile counts
      const int per = (p.G + 31) / 32;
      const int lo = min(p.G, lane * per), hi = min(p.G, lo + per);
      int sum = 0;
      for (int g = lo; g < hi; ++g) sum += tile_start[g];
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      int run = incl - sum;
      for (int g = lo; g < hi; ++g) {
        const int c = tile_start[g];
        tile_start[g] = run;
        run += c;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
    } else {
      total = p.G * tiles_of<RAGGED, EPI>(p, p.rows);
    }
    if (lane == 0) {
      const int r = total % n_clusters;
      const int split = p.partial != nullptr ? split_of(r, n_clusters, p.kb_typ) : 1;
      sched_smem[0] = split > 1 ? total - r : total;
      sched_smem[1] = split;
      sched_smem[2] = split > 1 ? total - r + r * split : total;
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // both CTAs' barriers and tensor memory are ready before either is used remotely
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Sched sc = {sched_smem[0], sched_smem[1], sched_smem[2]};

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    if (RAGGED == kRaggedK || lane == 0) {
      uint32_t it = 0, tails = 0;
      bool ok = true;
      for (int i = cluster_id; i < sc.items && ok; i += n_clusters) {
        const Item x = item_of<RAGGED, EPI>(p, tile_start, sc, i);
        const int half = half_of<B_MN>(x.nr);
        const uint32_t bytes = (uint32_t)kTileA + (uint32_t)half * 128u;
        const int acol = x.ct * kTile + (int)rank * 128;
        const int brow = (RAGGED == kRaggedRows ? x.row0 : 0) + x.rt * kTile + (int)rank * half;
        const int ag = RAGGED == kRaggedK ? 0 : x.g;
        const int bg = RAGGED == kDense ? x.g : 0;
        for (int kb = x.kb0; kb < x.kb1; ++kb, ++it) {
          const int stage = it % kStages;
          bool free_ = mbar_wait(&empty[stage], ((it / kStages) & 1) ^ 1, kWaitLimitNs);
          if constexpr (RAGGED == kRaggedK) free_ = __all_sync(0xffffffffu, free_);
          if (!free_) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * kStageBytes;
          uint8_t* sb = sa + kTileA;
          const int kx = kb * kBK;
          const int ky = x.k0 + kx;  // k as a row of an MN-major operand (x.k0 = 0 unless kRaggedK)
          // kRaggedK: the rows of the last block past the segment belong to the next one
          const bool tail = RAGGED == kRaggedK && kx + kBK > x.krows;
          if (!tail) {
            if (lane == 0) {
              const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
              if (leader) mbar_arrive_expect_tx(&full[stage], 2u * bytes);
              else if (RAGGED == kRaggedK) mbar_arrive_cluster(bar);
              if (!(leader && p.withhold_first_load && it == 0)) {
                if constexpr (A_MN) {
                  tma_3d_pair(&p.a, bar, sa, acol, ky, ag);
                  tma_3d_pair(&p.a, bar, sa + 8192, acol + 64, ky, ag);
                } else {
                  tma_3d_pair(&p.a, bar, sa, kx, acol, ag);
                }
                if constexpr (B_MN) {
                  tma_3d_pair(&p.b, bar, sb, brow, ky, bg);
                  tma_3d_pair(&p.b, bar, sb + 8192, brow + 64, ky, bg);
                } else if (half == 128) {
                  tma_3d_pair(&p.b, bar, sb, kx, brow, bg);
                } else {
                  int r = 0;
                  for (; r + 32 <= half; r += 32) tma_3d_pair(&p.b32, bar, sb + r * 128, kx, brow + r, bg);
                  for (; r < half; r += 8) tma_3d_pair(&p.b8, bar, sb + r * 128, kx, brow + r, bg);
                }
              }
            }
          } else {
            // Both operands are MN-major: k row r of a box is the 128 bytes at r * 128 (the swizzle
            // permutes within a row).  The block lands on this CTA's own barrier, its rows past the
            // segment are zeroed in both operands (an infinity or NaN of the next segment must not
            // meet a zero), and only then is the stage handed to the MMA.
            const int valid = x.krows - kx;
            if (lane == 0) {
              mbar_arrive_expect_tx(tail_bar, bytes);
              tma_3d(&p.a, tail_bar, sa, acol, ky, ag);
              tma_3d(&p.a, tail_bar, sa + 8192, acol + 64, ky, ag);
              tma_3d(&p.b, tail_bar, sb, brow, ky, bg);
              tma_3d(&p.b, tail_bar, sb + 8192, brow + 64, ky, bg);
            }
            bool landed = mbar_wait(tail_bar, tails & 1, kWaitLimitNs);
            ++tails;
            landed = __all_sync(0xffffffffu, landed);
            if (!landed) {
              ok = false;
              break;
            }
            for (int o = valid * 128 + lane * 16; o < 8192; o += 512) {
#pragma unroll
              for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(sa + q * 8192 + o) = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the tensor core reads them
            __syncwarp();
            if (lane == 0) {
              if (leader) mbar_arrive(&full[stage]);
              else mbar_arrive_cluster(mapa_shared(smem_u32(&full[stage]), 0));
            }
          }
        }
      }
      if (!ok && lane == 0) set_error(p.err, kErrTimeout);
      // every stage this CTA filled must be consumed (the even CTA: landed) before shared memory is
      // released; after one expired wait the copies still in flight have long landed
      if (lane == 0) {
        const uint32_t issued = it;
        for (int s = 0; s < kStages; ++s) {
          if ((uint32_t)s >= issued) break;
          const uint32_t last = issued - 1 - ((issued - 1 - s) % kStages);
          const bool done = leader ? mbar_wait(&full[s], (last / kStages) & 1, kWaitLimitNs)
                                   : mbar_wait(&empty[s], (last / kStages) & 1, kWaitLimitNs);
          if (!done) {
            set_error(p.err, kErrTimeout);
            break;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (even CTA)
    if (leader && lane == 0) {
      uint32_t it = 0, use = 0;
      bool ok = true;
      for (int i = cluster_id; i < sc.items && ok; i += n_clusters) {
        const Item x = item_of<RAGGED, EPI>(p, tile_start, sc, i);
        const uint32_t idesc = p.idesc | ((uint32_t)(2 * half_of<B_MN>(x.nr)) >> 3 << 17) | (16u << 24);
        int kb = x.kb0;
        do {  // one use of an accumulator: the whole item, or one drain's K blocks; at least one
          const uint32_t buf = use & 1;
          if (!mbar_wait(&acc_empty[buf], ((use >> 1) & 1) ^ 1, kWaitLimitNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + buf * kTile;
          const int end = kPromote ? min(x.kb1, kb + kPromoteBlocks) : x.kb1;
          uint32_t accumulate = 0;
          for (; kb < end; ++kb, ++it) {
            const int stage = it % kStages;
            const bool landed = RAGGED == kRaggedK ? mbar_wait_cluster(&full[stage], (it / kStages) & 1, kWaitLimitNs)
                                                   : mbar_wait(&full[stage], (it / kStages) & 1, kWaitLimitNs);
            if (!landed) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * kStageBytes), sb = sa + kTileA;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) {
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
        if (!mbar_wait(&empty[last % kStages], (last / kStages) & 1, kWaitLimitNs)) set_error(p.err, kErrTimeout);
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue (warps 2..9, both CTAs)
    const int q = warp & 3;         // TMEM lane quarter this warp may read
    const int h = (warp - 2) >> 2;  // which 128 of the tile's rows
    uint32_t use = 0;
    bool ok = true;
    for (int i = cluster_id; i < sc.items && ok; i += n_clusters) {
      const Item x = item_of<RAGGED, EPI>(p, tile_start, sc, i);
      const int col = x.ct * kTile + (int)rank * 128 + q * 32 + lane;
      const bool none = x.kb1 <= x.kb0;
      const bool split = x.slot >= 0;
      float* mine = split ? part_ptr(p, x.slot, sc.split, x.part, (int)rank) + q * 32 + lane : nullptr;
      const int chunks = max(0, min(4, (x.nr - h * 128 + 31) / 32));  // chunks of 32 rows with valid rows
      if constexpr (kPromote) {
        float acc[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c][j] = 0.0f;
        int kb = x.kb0;
        do {
          const uint32_t buf = use & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (use >> 1) & 1, kWaitLimitNs));
          if (!ok) break;
          tc_fence_after();
          const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + buf * kTile + h * 128;
          if (!none) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c < chunks) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(tacc + c * 32, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[c][j] += __uint_as_float(r[j]);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[buf]), 0));
          ++use;
          kb += kPromoteBlocks;
        } while (kb < x.kb1);
        if (!ok) {
          if (lane == 0) set_error(p.err, kErrTimeout);
          break;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j0 = h * 128 + c * 32;
          const int nj = min(32, x.nr - j0);
          if (c < chunks) {
            if (!split) {
              emit<RAGGED, EPI>(p, x, acc[c], j0, nj, col);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j < nj) __stcg(mine + (size_t)(j0 + j) * 128, acc[c][j]);
            }
          }
        }
      } else {
        const uint32_t buf = use & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (use >> 1) & 1, kWaitLimitNs));
        if (!ok) {
          if (lane == 0) set_error(p.err, kErrTimeout);
          break;
        }
        tc_fence_after();
        const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + buf * kTile + h * 128;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          const int j0 = h * 128 + c * 32;
          const int nj = min(32, x.nr - j0);
          float v[32];
          if (!none) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tacc + c * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.0f;
          }
          if (!split) {
            emit<RAGGED, EPI>(p, x, v, j0, nj, col);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < nj) __stcg(mine + (size_t)(j0 + j) * 128, v[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[buf]), 0));
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
            const int j0 = h * 128 + c * 32;
            const int nj = min(32, x.nr - j0);
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.0f;
#pragma unroll 1
            for (int s = 0; s < sc.split; ++s) {
              const float* src = part_ptr(p, x.slot, sc.split, s, (int)rank) + (size_t)j0 * 128 + q * 32 + lane;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j < nj) v[j] += __ldcg(src + (size_t)j * 128);
            }
            emit<RAGGED, EPI>(p, x, v, j0, nj, col);
          }
        }
      }
    }
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

// 16-bit row-major [groups, rows, inner] tensor, box of 64 elements x box_rows rows of one group,
// 128-byte swizzle; what lies past inner or rows reads as zero.  inner is a multiple of 8.
inline bool make_map(CUtensorMap* m, bool bf16, const void* base, uint64_t inner, uint64_t rows, uint64_t groups,
                     uint32_t box_rows) {
  EncodeFn enc = encode_fn();
  if (enc == nullptr || inner == 0 || rows == 0 || groups == 0) return false;
  cuuint64_t dims[3] = {inner, rows, groups};
  cuuint64_t strides[2] = {inner * 2, inner * rows * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  if (!make_map(&p.a, bf16, a.base, a.inner, a.rows, a.groups, A_MN ? 64 : 128)) return false;
  if (!make_map(&p.b, bf16, b.base, b.inner, b.rows, b.groups, B_MN ? 64 : 128)) return false;
  if (!B_MN && (!make_map(&p.b32, bf16, b.base, b.inner, b.rows, b.groups, 32) ||
                !make_map(&p.b8, bf16, b.base, b.inner, b.rows, b.groups, 8)))
    return false;
  return true;
}

template <bool A_MN, bool B_MN, int RAGGED, int EPI>
cudaError_t launch(const Params& p, cudaStream_t s) {
  auto kernel = product_kernel<A_MN, B_MN, RAGGED, EPI>;
  static std::atomic<int> cached[64];  // clusters that fit on the device at once, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
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
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2);
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters <= 0) return cudaErrorInvalidConfiguration;
    clusters = clusters > kMaxParts / 2 ? kMaxParts / 2 : clusters;
    if (dev >= 0 && dev < 64) cached[dev].store(clusters);
  }
  cfg.gridDim = dim3(2 * clusters);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace product
}  // namespace moe
