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
//     P  = b A + c A A                    symmetric
//     X <- a X + P X  or  a X + X P
// 3 m^2 n + m^3 products per step for n = max(M, N), a quarter to a third below the plain form's.
//
// Numerics.  Operands are fp16 scaled by 2^12 (not bf16: the same tensor-core rate with 1/8 of the
// rounding; |X| <= 1.2025, |A| <= 1.45, |P| <= 2.81, so nothing overflows, and values down to 2^-36
// keep a bit).  A singular value v grows by up to a^steps = 485, and so does what rounding adds along
// directions that the matrix does not have; gradients of experts with few tokens are of such low
// rank.  X is therefore kept as hi + lo * 2^-11 (22 bits): the tensor core multiplies hi, and the
// term a X, which alone carries small singular values, adds both.  In a simulation of exactly these
// roundings over ten spectra (full rank, rank 8 and 64, polynomial and geometric decay, one huge
// entry) the result is 2e-4 to 1.7e-3 off in the 2-norm, less than its rounding to bf16; without lo
// 4e-2, with bf16 operands 3e-1 (rank 8).  P uses the rounded A in both terms: its error is then that
// of a nearby X, which the iteration damps (with the unrounded A in b A it is twice as large).
// The norm is summed in 64 bits, so fp32 inputs of any magnitude neither overflow nor vanish.
#include "product_sm100.cuh"

using namespace moe;
using namespace moe::product;

namespace {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr float kScale = 4096.0f, kUnscale = 1.0f / 4096.0f;
constexpr int kNormParts = 64;
constexpr int kPrepThreads = 256;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename T>
__device__ __forceinline__ float load_value(const T* p);
template <>
__device__ __forceinline__ float load_value<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float load_value<uint16_t>(const uint16_t* p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }

// partial[matrix][part] = sum of squares of the part's elements, in 64 bits and a fixed order
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) norm_kernel(const T* __restrict__ g, long long count,
                                                            double* __restrict__ partial) {
  __shared__ double warp_sum[kPrepThreads / 32];
  pdl_wait();
  pdl_trigger();
  const T* m = g + (long long)blockIdx.y * count;
  double sum = 0.0;
  for (long long i = (long long)blockIdx.x * kPrepThreads + threadIdx.x; i < count; i += (long long)gridDim.x * kPrepThreads) {
    const double v = load_value(m + i);
    sum += v * v;
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

// hi + lo * 2^-11 = 2^12 g / ||g||, rows padded with zeros to the pitch
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) scale_kernel(const T* __restrict__ g, int M, int N, int ld,
                                                             const double* __restrict__ partial, int parts,
                                                             uint16_t* __restrict__ hi, uint16_t* __restrict__ lo) {
  __shared__ double inv;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < parts; ++i) t += partial[(size_t)blockIdx.y * kNormParts + i];
    inv = t == 0.0 ? 0.0 : (double)kScale / sqrt(t);
  }
  __syncthreads();
  const double f = inv;
  const T* m = g + (long long)blockIdx.y * M * N;
  const long long base = (long long)blockIdx.y * M * ld;
  const long long total = (long long)M * ld;
  for (long long i = (long long)blockIdx.x * kPrepThreads + threadIdx.x; i < total; i += (long long)gridDim.x * kPrepThreads) {
    const int r = (int)(i / ld), c = (int)(i - (long long)r * ld);
    const float v = c < N ? (float)((double)load_value(m + (long long)r * N + c) * f) : 0.0f;
    const uint16_t h = half_bits(v);
    hi[base + i] = h;
    lo[base + i] = half_bits((v - half_val(h)) * 2048.0f);
  }
}

struct Layout {
  int low, lp, np;   // shorter side, its pitch, the pitch of X's rows
  int batch;         // matrices per round of launches
  int prows;
  size_t norms, hi0, hi1, lo, gram, poly, total;
};

// Enough matrices side by side to fill several rounds of clusters with X's tiles, no more: what is in
// flight then stays small next to memory, and for small matrices in L2.
constexpr int kTargetTiles = 592;  // 8 rounds of 74 clusters

bool layout_of(int B, int M, int N, Layout& l) {
  if (B <= 0 || M <= 0 || N <= 0 || M > 65536 || N > 65536) return false;
  l.low = M < N ? M : N;
  l.lp = (l.low + 7) / 8 * 8;
  l.np = (N + 7) / 8 * 8;
  const long long tiles = (long long)((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  const long long batch = (kTargetTiles + tiles - 1) / tiles;
  l.batch = B < batch ? B : (int)batch;
  l.prows = partial_rows(M);
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
  l.lo = take(x);
  l.gram = take(s);
  l.poly = take(s);
  l.total = at;
  return true;
}

template <typename T>
cudaError_t prepare(const T* g, int count, int M, int N, const Layout& l, uint8_t* b, cudaStream_t s) {
  const long long n = (long long)M * N;
  long long parts = (n + 16 * kPrepThreads - 1) / (16 * kPrepThreads);
  if (parts > kNormParts) parts = kNormParts;
  double* norms = reinterpret_cast<double*>(b + l.norms);
  cudaError_t e = launch_pdl(norm_kernel<T>, dim3((unsigned)parts, (unsigned)count), dim3(kPrepThreads), 0, s, g, n, norms);
  if (e != cudaSuccess) return e;
  long long blocks = ((long long)M * l.np + 8 * kPrepThreads - 1) / (8 * kPrepThreads);
  if (blocks > 1024) blocks = 1024;
  return launch_pdl(scale_kernel<T>, dim3((unsigned)blocks, (unsigned)count), dim3(kPrepThreads), 0, s, g, M, N, l.np,
                    (const double*)norms, (int)parts, reinterpret_cast<uint16_t*>(b + l.hi0),
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
  base.src_lo = base.out_lo = reinterpret_cast<uint16_t*>(b + l.lo);
  uint16_t* hi[2] = {reinterpret_cast<uint16_t*>(b + l.hi0), reinterpret_cast<uint16_t*>(b + l.hi1)};
  uint16_t* gram = reinterpret_cast<uint16_t*>(b + l.gram);
  uint16_t* poly = reinterpret_cast<uint16_t*>(b + l.poly);
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
    p.src = gram;
    p.out = poly;
    p.c0 = kNsB;
    p.c1 = kNsC * kUnscale;
    if (!set_operands<false, false>(p, og, og, false)) return cudaErrorInvalidValue;
    if ((e = launch<false, false, kDense, kPoly>(p, s)) != cudaSuccess) return e;

    p = base;
    p.rows = M;
    p.cols = l.np;
    p.ld = l.np;
    p.K = l.lp;
    p.kb_typ = (p.K + kBK - 1) / kBK;
    p.src = hi[k & 1];
    p.out = last ? out : hi[(k + 1) & 1];
    p.ld_out = p.cols_out = N;
    p.c0 = kNsA;
    p.c1 = kUnscale;
    p.c2 = kUnscale;
    if (tall) {  // X P: P's rows are the columns, X's rows the rows
      if (!set_operands<false, false>(p, op, ox, false)) return cudaErrorInvalidValue;
      e = last ? launch<false, false, kDense, kApplyLast>(p, s) : launch<false, false, kDense, kApply>(p, s);
    } else {     // P X: X is contracted over its rows
      if (!set_operands<true, false>(p, ox, op, false)) return cudaErrorInvalidValue;
      e = last ? launch<true, false, kDense, kApplyLast>(p, s) : launch<true, false, kDense, kApply>(p, s);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

extern "C" {

size_t moe_orthogonalize_workspace_size(int B, int M, int N) {
  Layout l;
  return layout_of(B, M, N, l) ? l.total : 0;
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
  if (ws_bytes < l.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const moe_status_t st = device_status();
  if (st != MOE_OK) return st;
  uint8_t* b = static_cast<uint8_t*>(ws);
  cudaStream_t s = (cudaStream_t)stream;
  for (int at = 0; at < B; at += l.batch) {
    const int count = B - at < l.batch ? B - at : l.batch;
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
