// orthogonalize.cu -- the Newton-Schulz orthogonalisation of a batch of matrices, the update of an
// optimiser that steps along the nearest semi-orthogonal matrix of each weight's gradient instead of
// the gradient itself.  It takes what the layer's backward pass or moe_grouped_gemm_wgrad returns for
// every expert.  For one matrix g [M, N] (Frobenius norm s):
//     X_0 = g / s (0 if s = 0);  X <- a X + (b A + c A A) X,  A = X X^T;  `steps` times
// with (a, b, c) = (3.4445, -4.7750, 2.0315): every singular value of X_0 in [0, 1] goes through
// f(v) = a v + b v^3 + c v^5, which stays in [0, 1.2025] and pulls all but the smallest to about 1.
// p(X X^T) X = X p(X^T X), so the Gram matrix of the shorter side is used: [m, m] with m = min(M, N).
//
// Each step is three launches of the kernel of product_sm100.cuh over a batch of matrices:
//     A  = X X^T  (M <= N) or X^T X       symmetric: the lower tiles, each stored with its mirror image
//     P  = a I + b A + c A A              symmetric
//     X <- P X  or  X P
// 3 m^2 n + m^3 products per step for n = max(M, N), a quarter to a third below the plain form's.
//
// Numerics.  Operands are fp16 scaled by 2^12 (not bf16: the same tensor-core rate with 1/8 of the
// rounding; |X| <= 1.2025, |A| <= 1.45, |P - a I| <= 2.81, so nothing overflows, and values down to 2^-36
// keep a bit).  A singular value v grows by up to a^steps = 485, and so does what rounding adds along
// directions that the matrix does not have; gradients of experts with few tokens are of such low rank.
// Two roundings would do that, and are not made:
//   X is kept as hi + lo * 2^-11 (22 bits): the tensor core multiplies hi, and a lo * 2^-11 is added.
//   P's diagonal, which a I makes larger than all the rest, stays in fp32 beside it (the fp16 P has zeros
//   there) and multiplies hi in the epilogue; lo meets a alone, for the rest of P has not met it either.
// In a simulation of exactly these roundings over thirteen spectra, 65 x 3000 to 384 x 768, the last iterate is
// off by at most this share of its Frobenius norm, before its rounding to bf16 takes another 1.7e-3: rank 1, 4
// and 8 and one value over a tail of 1e-5 6e-4 to 8e-4, full rank, rank 64, polynomial and geometric decay and one huge
// entry 4e-4 to 1.4e-3, a diagonal matrix with geometric decay 2.9e-3 (A's own rounding).  With a I inside the
// fp16 P rank 1 and the tail are 2.4e-3 off, without lo 4e-2, with bf16 operands 3e-1 (rank 8).  P uses
// the rounded A in both terms: its error is then that of a nearby X, which the iteration damps (with the unrounded
// A in b A it is twice as large).
// The norm is summed in 64 bits, so fp32 inputs of any magnitude neither overflow nor vanish.
#include "product_sm100.cuh"

using namespace moe;
using namespace moe::product;

namespace {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr float kScale = 4096.0f, kUnscale = 1.0f / 4096.0f;
constexpr int kNormParts = 128;
constexpr int kPrepThreads = 256;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// What these kernels read, the caller's matrices too, the kernel before may write while they are resident already
// (programmatic launch), and the short-side product runs in place.  All of it is therefore read by ordinary loads,
// never as memory that nobody writes: no __ldg, no const __restrict__.
__device__ __forceinline__ float load_value(const float* p) { return *p; }
__device__ __forceinline__ float load_value(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// eight values from p, which is 16-byte aligned
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// the first n of eight values from any p, zeros for the others
template <typename T>
__device__ __forceinline__ void load8_tail(const T* p, int n, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? load_value(p + i) : 0.0f;
}

// partial[matrix][part] = sum of squares of the part's elements, in 64 bits and a fixed order.  Bound by
// reading g once; `wide`: every matrix starts on 16 bytes.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) norm_kernel(const T* g, long long count, int wide,
                                                            double* __restrict__ partial) {
  __shared__ double warp_sum[kPrepThreads / 32];
  pdl_wait();
  pdl_trigger();
  const T* m = g + (long long)blockIdx.y * count;
  const long long groups = (count + 7) / 8;
  double sum = 0.0;
#pragma unroll 4
  for (long long i = (long long)blockIdx.x * kPrepThreads + threadIdx.x; i < groups; i += (long long)gridDim.x * kPrepThreads) {
    float v[8];
    const long long left = count - 8 * i;
    if (wide && left >= 8) load8(m + 8 * i, v);
    else load8_tail(m + 8 * i, left < 8 ? (int)left : 8, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)v[j] * (double)v[j];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < kPrepThreads / 32; ++w) t += warp_sum[w];
    partial[(size_t)blockIdx.y * kNormParts + blockIdx.x] = t;
  }
}

// the parts of every matrix's sum of squares; g is on 16 bytes, and so is every matrix whose length is a
// multiple of 16 bytes
template <typename T>
cudaError_t norms_of(const T* g, int count, int M, int N, double* norms, int& parts, cudaStream_t s) {
  const long long n = (long long)M * N, most = (n + 16 * kPrepThreads - 1) / (16 * kPrepThreads);
  parts = most < kNormParts ? (int)most : kNormParts;
  return launch_pdl(norm_kernel<T>, dim3((unsigned)parts, (unsigned)count), dim3(kPrepThreads), 0, s, g, n,
                    n % (16 / (int)sizeof(T)) == 0 ? 1 : 0, norms);
}

#include "orthogonalize_small.cuh"

// hi + lo * 2^-11 = 2^12 g / ||g||, rows padded with zeros to the pitch, lo in low_index's order; bound by reading
// g and writing as many bytes.  `wide`: every row of g starts on 16 bytes.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) scale_kernel(const T* g, int M, int N, int ld, int wide,
                                                             const double* partial, int parts,
                                                             uint16_t* __restrict__ hi, uint16_t* __restrict__ lo) {
  __shared__ double inv;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) {
    double t = 0.0;
    for (int i = threadIdx.x; i < parts; i += 32) t += partial[(size_t)blockIdx.y * kNormParts + i];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    if (threadIdx.x == 0) inv = t == 0.0 ? 0.0 : (double)kScale / sqrt(t);
  }
  __syncthreads();
  const double f = inv;
  const T* m = g + (long long)blockIdx.y * M * N;
  const long long base = (long long)blockIdx.y * M * ld;
  const unsigned per = (unsigned)ld / 8;  // groups of 8 per row
  const unsigned groups = (unsigned)M * per;
#pragma unroll 2
  for (unsigned i = blockIdx.x * kPrepThreads + threadIdx.x; i < groups; i += gridDim.x * kPrepThreads) {
    const unsigned r = i / per, c = (i - r * per) * 8;
    const T* at = m + (long long)r * N + c;
    float v[8];
    if (wide && (int)c < N) load8(at, v);
    else load8_tail(at, min(8, N - (int)c), v);
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = 0, l[j] = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float w = (float)((double)v[2 * j + u] * f);
        const uint16_t hb = half_bits(w);
        h[j] |= (uint32_t)hb << 16 * u;
        l[j] |= (uint32_t)half_bits((w - half_val(hb)) * 2048.0f) << 16 * u;
      }
    }
    *reinterpret_cast<uint4*>(hi + base + 8LL * i) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(lo + low_index((int)blockIdx.y, (int)r, (int)c, M, ld)) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

struct Layout {
  int low, lp, np;   // shorter side, its pitch, the pitch of X's rows
  int batch;         // matrices per round of launches
  int prows;
  size_t norms, hi0, hi1, lo, gram, poly, diag, total;
};

// Enough matrices side by side that the launch with the fewest tiles, the Gram matrix's, fills eight rounds
// of 74 clusters, within 768 MB of X.  With one round's worth 300 x [128, 128] took 546 us, with four 323, with
// eight 237; 8 x [2048, 7168] 4225, 3670 and 3680 (one build, before the low-order part's present order).
constexpr long long kTargetTiles = 592;
constexpr long long kBatchBytes = 3LL << 28;

bool layout_of(int B, int M, int N, Layout& l) {
  if (B <= 0 || M <= 0 || N <= 0 || M > 65536 || N > 65536) return false;
  l.low = M < N ? M : N;
  l.lp = (l.low + 15) / 16 * 16;
  l.np = (N + 15) / 16 * 16;
  const long long rt = (l.low + kTile - 1) / kTile, tiles = rt * (rt + 1) / 2;
  long long batch = (kTargetTiles + tiles - 1) / tiles;
  const long long fits = kBatchBytes / (4LL * M * l.np + 2 * low_elements(1, M, l.np));
  if (batch > fits) batch = fits > 1 ? fits : 1;
  l.batch = B < batch ? B : (int)batch;
  l.prows = partial_rows(M > l.np ? M : l.np);
  size_t at = align_up(kPartialOffset + partial_bytes(l.prows), 256);
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = align_up(at + bytes, 256);
    return was;
  };
  const size_t x = (size_t)l.batch * M * l.np * 2, s = (size_t)l.batch * l.low * l.lp * 2;
  l.norms = take((size_t)l.batch * kNormParts * sizeof(double));
  l.hi0 = take(x);
  l.hi1 = take(x);
  l.lo = take((size_t)low_elements(l.batch, M, l.np) * 2);
  l.gram = take(s);
  l.poly = take(s);
  l.diag = take((size_t)l.batch * l.lp * sizeof(float));
  l.total = at;
  return true;
}

template <typename T>
cudaError_t prepare(const T* g, int count, int M, int N, const Layout& l, uint8_t* b, cudaStream_t s) {
  double* norms = reinterpret_cast<double*>(b + l.norms);
  int parts = 0;
  const cudaError_t e = norms_of(g, count, M, N, norms, parts, s);
  if (e != cudaSuccess) return e;
  long long blocks = ((long long)M * (l.np / 8) + 2 * kPrepThreads - 1) / (2 * kPrepThreads);
  if (blocks > 1024) blocks = 1024;
  return launch_pdl(scale_kernel<T>, dim3((unsigned)blocks, (unsigned)count), dim3(kPrepThreads), 0, s, g, M, N, l.np,
                    N % 8 == 0 ? 1 : 0, (const double*)norms, parts, reinterpret_cast<uint16_t*>(b + l.hi0),
                    reinterpret_cast<uint16_t*>(b + l.lo));
}

// the iteration over `count` matrices whose X_0 lies in hi0 / lo
cudaError_t iterate(int count, int M, int N, int steps, const Layout& l, uint16_t* out, uint8_t* b, cudaStream_t s) {
  const bool tall = M > N;
  const uint64_t G = (uint64_t)count;
  Params base;
  memset(&base, 0, sizeof(base));
  base.G = count;
  base.err = reinterpret_cast<int*>(b);
  base.counters = reinterpret_cast<int*>(b + kWsHeader);
  base.partial = reinterpret_cast<float*>(b + kPartialOffset);
  base.prows = l.prows;
  uint16_t* lo = reinterpret_cast<uint16_t*>(b + l.lo);
  uint16_t* hi[2] = {reinterpret_cast<uint16_t*>(b + l.hi0), reinterpret_cast<uint16_t*>(b + l.hi1)};
  uint16_t* gram = reinterpret_cast<uint16_t*>(b + l.gram);
  uint16_t* poly = reinterpret_cast<uint16_t*>(b + l.poly);
  base.diag = reinterpret_cast<float*>(b + l.diag);
  base.diag_ld = l.lp;
  const OperandHost og = {gram, (uint64_t)l.lp, (uint64_t)l.low, G};
  const OperandHost op = {poly, (uint64_t)l.lp, (uint64_t)l.low, G};
  for (int k = 0; k < steps; ++k) {
    const bool last = k == steps - 1;
    const OperandHost ox = {hi[k & 1], (uint64_t)l.np, (uint64_t)M, G};
    cudaError_t e;

    Params p = base;  // 2^12 A = 2^-12 (2^12 X)(2^12 X)^T
    p.withhold_first_load = k == 0 && test_withhold_this_launch() ? 1 : 0;
    p.rows = p.cols = l.low;
    p.ld = l.lp;
    p.K = tall ? M : l.np;
    p.kb_typ = (p.K + kBK - 1) / kBK;
    p.out = gram;
    p.c1 = kUnscale;
    if (tall) {
      if (!set_operands<true, true>(p, ox, ox, false)) return cudaErrorInvalidValue;
      e = launch<true, true, kDense, kGram>(p, s);
    } else {
      if (!set_operands<false, false>(p, ox, ox, false)) return cudaErrorInvalidValue;
      e = launch<false, false, kDense, kGram>(p, s);
    }
    if (e != cudaSuccess) return e;

    p = base;
    p.rows = p.cols = l.low;
    p.ld = l.lp;
    p.K = l.lp;
    p.kb_typ = (p.K + kBK - 1) / kBK;
    p.out = poly;
    p.src = gram;
    p.c0 = kNsB;
    p.c1 = kNsC * kUnscale;
    p.c2 = kNsA;
    if (!set_operands<false, false>(p, og, og, false)) return cudaErrorInvalidValue;
    if ((e = launch<false, false, kDense, kPoly>(p, s)) != cudaSuccess) return e;

    p = base;
    p.K = l.lp;
    p.kb_typ = (p.K + kBK - 1) / kBK;
    p.rows = p.ld = l.np;  // the product's rows and columns are exchanged
    p.cols = M;
    p.cols_out = N;
    p.src = hi[k & 1];
    p.src_lo = lo;
    p.out = last ? out : hi[(k + 1) & 1];
    p.out_lo = lo;
    p.c0 = kUnscale;
    p.c1 = kUnscale;
    p.c2 = kNsA / 2048.0f;
    if (tall) {  // X P
      if (!set_operands<false, false>(p, ox, op, false)) return cudaErrorInvalidValue;
      e = last ? launch<false, false, kDense, kApplyLast>(p, s) : launch<false, false, kDense, kApply>(p, s);
    } else {     // P X: X is contracted over its rows
      if (!set_operands<false, true>(p, op, ox, false)) return cudaErrorInvalidValue;
      e = last ? launch<false, true, kDense, kApplyLast>(p, s) : launch<false, true, kDense, kApply>(p, s);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

extern "C" {

size_t moe_orthogonalize_workspace_size(int B, int M, int N) {
  Layout l;
  if (!layout_of(B, M, N, l)) return 0;
  return small_side(M, N) ? small_workspace(B, M, N) : l.total;
}

moe_status_t moe_orthogonalize(const void* g, int g_dtype, int B, int M, int N, int steps, moe_bf16_t* out, void* ws,
                               size_t ws_bytes, moe_stream_t stream) {
  if (B < 0 || M <= 0 || N <= 0 || steps < 1 || steps > 16) return MOE_ERR_INVALID_ARG;
  if (g_dtype != MOE_DTYPE_FP32 && g_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (M > 65536 || N > 65536) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return MOE_OK;
  if (!g || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(g, 16) || !aligned(out, 16) || !aligned(ws, 256)) return MOE_ERR_ALIGNMENT;
  Layout l;
  if (!layout_of(B, M, N, l)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (ws_bytes < moe_orthogonalize_workspace_size(B, M, N)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const moe_status_t st = device_status();
  if (st != MOE_OK) return st;
  uint8_t* b = static_cast<uint8_t*>(ws);
  cudaStream_t s = (cudaStream_t)stream;
  if (small_side(M, N)) {
    const SmallLayout sl = small_layout(B, M, N, steps > kSmallSteps);
    for (int at = 0; at < B; at += sl.batch) {
      const int count = B - at < sl.batch ? B - at : sl.batch;
      const long long skip = (long long)at * M * N;
      const cudaError_t e =
          g_dtype == MOE_DTYPE_FP32
              ? small_orthogonalize(static_cast<const float*>(g) + skip, count, M, N, steps, sl, out + skip, b, s)
              : small_orthogonalize(static_cast<const uint16_t*>(g) + skip, count, M, N, steps, sl, out + skip, b, s);
      if (e != cudaSuccess) return launch_status(e);
    }
    return MOE_OK;
  }
  const int rounds = (B + l.batch - 1) / l.batch, most = (B + rounds - 1) / rounds;  // dealt evenly
  for (int at = 0; at < B; at += most) {
    const int count = B - at < most ? B - at : most;
    const long long skip = (long long)at * M * N;
    cudaError_t e = g_dtype == MOE_DTYPE_FP32
                        ? prepare(static_cast<const float*>(g) + skip, count, M, N, l, b, s)
                        : prepare(static_cast<const uint16_t*>(g) + skip, count, M, N, l, b, s);
    if (e == cudaSuccess) e = iterate(count, M, N, steps, l, out + skip, b, s);
    if (e != cudaSuccess) return launch_status(e);
  }
  return MOE_OK;
}

}  // extern "C"
