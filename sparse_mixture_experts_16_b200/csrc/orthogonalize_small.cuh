// orthogonalize_small.cuh -- the Newton-Schulz iterate of matrices whose shorter side is at most 64
// (router weights, low-rank factors, heads).  The products of the general path would fill a corner of a
// tile each, and its launches, three per step, cost 65 to 340 us whatever the work.  Both paths measured, there and
// here, us: 13 x [202, 29] 73 and 19, 1 x [64, 64] 65 and 48, 9 x [32, 6645] 226 and 48, 300 x [64, 64] 156 and 125,
// 60 x [2000, 40] 197 and 153, 700 x [40, 56] 325 and 242, 64 x [7168, 64] 643 and 347, 512 x [16, 7168] 5400 and 880.
// Every iterate is a polynomial of A_0 = X_0 X_0^T times X_0, so the iteration runs on [L, L] matrices alone
// (L = 32 or 64):
//     Q = I, A = A_0;  P = a I + b A + c A A;  Q <- P Q;  A <- P A P;  ...;  X = Q X_0
// and the long side is read twice: for the Gram matrix and for the product with Q.  Four launches in all:
// norm, Gram (parts of the long side, added in a fixed order), iteration (a block per matrix), product.
//
// Numerics, fp32 (FFMA).  The matrices commute only up to rounding: where A has no component a rounding grows
// by a = 3.4445 per step and side, so the order of the factors matters.  A stays P A P (P (P A) grows by
// a^2 on one side), and only the symmetric A and P are read by rows in the place of columns: with Q read
// so, the result is up to 0.4 off.  What rounds A_0 itself grows likewise, and one fp32 chain over a long side
// rounds it with every term: 4e-3 (8 x 900) to 1.2e-2 (16 x 7168) off, one direction and 1e-2 or 1e-3 of noise.  Its sums
// are therefore drained every 64 terms into 64 bits, over the parts too, and rounded to fp32 at the end of a part and of
// all.  In simulation the result is then at most 1e-3 off after five steps, whatever the length and the number of
// parts (2 x 2 to 64 x 900, rank 4, polynomial and geometric decay; one direction and noise to 8 x 65536: 5.4e-4), but
// after sixteen it has diverged.  More than five steps are therefore made in rounds of five, each from the Gram
// matrix of the X that the last one left in fp32: X is bounded.
//
// Included by orthogonalize.cu, whose norm partials it uses.
#pragma once

constexpr int kSmallSide = 64, kSmallSteps = 5;
constexpr int kSmallThreads = 256;     // 16 x 16 threads, a micro tile each
constexpr int kSmallChunk = 64;        // of the long side
constexpr int kSmallBlocks = 592;      // 4 per SM: parts of the Gram matrices, slices of the products
constexpr long long kSmallXBytes = 1LL << 26;  // of the fp32 X between rounds; one matrix has at most 2^24 bytes

struct SmallLayout {
  int L, chunks, batch, parts;
  size_t norms, scale, partial, q, x, total;
};

inline bool small_side(int M, int N) { return (M < N ? M : N) <= kSmallSide; }

// Matrices side by side and their places in the workspace.  `rounds`: more than kSmallSteps steps, with an X in
// fp32 between them, and so few matrices at a time that X is bounded (and stays in L2).
inline SmallLayout small_layout(int B, int M, int N, bool rounds) {
  SmallLayout l;
  const int low = M < N ? M : N, high = M < N ? N : M;
  l.L = low <= 32 ? 32 : 64;
  l.chunks = (high + kSmallChunk - 1) / kSmallChunk;
  const long long fits = kSmallXBytes / (4LL * M * N);
  l.batch = B < kSmallBlocks ? B : kSmallBlocks;
  if (rounds && l.batch > fits) l.batch = (int)fits;
  l.parts = kSmallBlocks / l.batch;
  if (l.parts > 32) l.parts = 32;  // one block adds them up
  if (l.parts > l.chunks) l.parts = l.chunks;
  size_t at = align_up(kPartialOffset, 256);
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = align_up(at + bytes, 256);
    return was;
  };
  l.norms = take((size_t)l.batch * kNormParts * sizeof(double));
  l.scale = take((size_t)l.batch * sizeof(float2));
  l.partial = take((size_t)l.batch * l.parts * l.L * l.L * sizeof(float));
  l.q = take((size_t)l.batch * l.L * l.L * sizeof(float));
  l.x = take(rounds ? (size_t)l.batch * M * N * sizeof(float) : 0);
  l.total = at;
  return l;
}

// for any number of steps
inline size_t small_workspace(int B, int M, int N) {
  const size_t once = small_layout(B, M, N, false).total, rounds = small_layout(B, M, N, true).total;
  return once > rounds ? once : rounds;
}

template <int R>
__device__ __forceinline__ void read_row(const float* p, float (&v)[R]) {
  if constexpr (R == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
  } else {
    const float2 t = *reinterpret_cast<const float2*>(p);
    v[0] = t.x, v[1] = t.y;
  }
}

// acc[i][j] += sum_k x[k][RX ty + i] y[k][RY tx + j], k < K
template <int RX, int RY, int K>
__device__ __forceinline__ void micro(const float* x, int px, const float* y, int py, int ty, int tx, float (&acc)[RX][RY]) {
#pragma unroll 8
  for (int k = 0; k < K; ++k) {
    float a[RX], b[RY];
    read_row<RX>(x + k * px + RX * ty, a);
    read_row<RY>(y + k * py + RY * tx, b);
#pragma unroll
    for (int i = 0; i < RX; ++i)
#pragma unroll
      for (int j = 0; j < RY; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
  }
}

// 1 / ||g|| from the norm's parts (0 for a zero matrix), 1 without parts; a whole warp
__device__ __forceinline__ double small_scale(const double* norms, int parts, int lane) {
  if (parts == 0) return 1.0;
  double t = 0.0;
  for (int i = lane; i < parts; i += 32) t += norms[i];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  return t == 0.0 ? 0.0 : 1.0 / sqrt(t);
}

// f as two fp32 factors, the first a power of two: v * p.x * p.y rounds once for every v and f (neither
// overflows on the way for values of one matrix), without the conversions of a 64-bit product
__device__ __forceinline__ float2 two_factors(double f) {
  int e = 0;
  frexp(f, &e);
  const float x = f > 0.0 && f < 1e300 ? ldexpf(1.0f, e / 2) : 1.0f;
  return make_float2(x, (float)(f / (double)x));
}

// A chunk of the long side: neighbouring threads read neighbouring elements, all of a thread's in flight (past
// the edge the last element again: a condition around a load puts a wait behind it)
template <typename T, bool TALL, int L>
__device__ __forceinline__ void fetch_chunk(const T* m, int low, int high, int n0, float (&v)[kSmallChunk * L / kSmallThreads],
                                            int tid) {
#pragma unroll
  for (int u = 0; u < kSmallChunk * L / kSmallThreads; ++u) {
    const int e = tid + u * kSmallThreads;
    const int i = min(TALL ? e % L : e / kSmallChunk, low - 1), n = min(n0 + (TALL ? e / L : e % kSmallChunk), high - 1);
    v[u] = load_value(m + (TALL ? (long long)n * low + i : (long long)i * high + n));
  }
}
// the same scaled, as to[n * pitch_n + i * pitch_i] for element i of the short side at position n0 + n; zeros
// past the matrix
template <bool TALL, int L>
__device__ __forceinline__ void place_chunk(const float (&v)[kSmallChunk * L / kSmallThreads], int low, int high, int n0,
                                            float2 f, float* to, int pitch_n, int pitch_i, int tid) {
#pragma unroll
  for (int u = 0; u < kSmallChunk * L / kSmallThreads; ++u) {
    const int e = tid + u * kSmallThreads;
    const int i = TALL ? e % L : e / kSmallChunk, n = TALL ? e / L : e % kSmallChunk;
    to[n * pitch_n + i * pitch_i] = i < low && n0 + n < high ? v[u] * f.x * f.y : 0.0f;
  }
}

// partial[matrix][part] = the part's share of X_0 X_0^T
template <typename T, bool TALL, int L>
__global__ void __launch_bounds__(kSmallThreads) small_gram_kernel(const T* g, int low, int high, int chunks,
                                                                   const double* norms, int norm_parts,
                                                                   float* __restrict__ partial) {
  constexpr int R = L / 16, kPitch = L + 4;
  __shared__ __align__(16) float xs[kSmallChunk * kPitch];
  __shared__ float2 scale;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  if (tid < 32) {
    const double f = small_scale(norms + (size_t)blockIdx.y * kNormParts, norm_parts, tid);
    if (tid == 0) scale = two_factors(f);
  }
  __syncthreads();
  const float2 f = scale;
  const T* m = g + (long long)blockIdx.y * low * high;
  double sum[R][R] = {};
  const int c0 = (int)((long long)chunks * blockIdx.x / gridDim.x), c1 = (int)((long long)chunks * (blockIdx.x + 1) / gridDim.x);
  float v[kSmallChunk * L / kSmallThreads];
  fetch_chunk<T, TALL, L>(m, low, high, c0 * kSmallChunk, v, tid);
  for (int c = c0; c < c1; ++c) {
    __syncthreads();
    place_chunk<TALL, L>(v, low, high, c * kSmallChunk, f, xs, kPitch, 1, tid);
    __syncthreads();
    if (c + 1 < c1) fetch_chunk<T, TALL, L>(m, low, high, (c + 1) * kSmallChunk, v, tid);
    float acc[R][R] = {};
    micro<R, R, kSmallChunk>(xs, kPitch, xs, kPitch, ty, tx, acc);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) sum[i][j] += (double)acc[i][j];
  }
  float* to = partial + ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * L * L;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < R; ++j) to[(R * ty + i) * L + R * tx + j] = (float)sum[i][j];
}

// Q^T of each matrix from the parts of its Gram matrix, and the scale of X_0
template <int L>
__global__ void __launch_bounds__(kSmallThreads) small_iterate_kernel(const float* partial, int parts, int steps,
                                                                      const double* norms, int norm_parts,
                                                                      float* __restrict__ q, float2* __restrict__ scales) {
  constexpr int R = L / 16, kPitch = L + 4, kEach = L * L / kSmallThreads;
  extern __shared__ __align__(16) float small_smem[];
  float *A = small_smem, *P = A + L * kPitch, *Q = P + L * kPitch, *W = Q + L * kPitch;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  if (tid < 32) {
    const double f = small_scale(norms + (size_t)blockIdx.x * kNormParts, norm_parts, tid);
    if (tid == 0) scales[blockIdx.x] = two_factors(f);
  }
  const float* from = partial + (size_t)blockIdx.x * parts * L * L;
  constexpr int kQuads = kEach / 4;
  double sum[kQuads][4] = {};
#pragma unroll 1
  for (int t = 0; t < parts; t += 4) {  // in the order of the parts; past the last: the last again, not added
    float4 v[4][kQuads];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
        v[u][i] = __ldcg(reinterpret_cast<const float4*>(from + (size_t)min(t + u, parts - 1) * L * L) + tid + i * kSmallThreads);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (t + u < parts)
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
          sum[i][0] += v[u][i].x, sum[i][1] += v[u][i].y, sum[i][2] += v[u][i].z, sum[i][3] += v[u][i].w;
  }
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const int e = 4 * (tid + i * kSmallThreads);
    *reinterpret_cast<float4*>(A + e / L * kPitch + e % L) =
        make_float4((float)sum[i][0], (float)sum[i][1], (float)sum[i][2], (float)sum[i][3]);
  }
  __syncthreads();
  auto product = [&](const float* x, const float* y, float (&acc)[R][R]) {  // x^T y
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) acc[i][j] = 0.0f;
    micro<R, R, L>(x, kPitch, y, kPitch, ty, tx, acc);
  };
  auto put = [&](float* to, const float (&acc)[R][R]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) to[(R * ty + i) * kPitch + R * tx + j] = acc[i][j];
  };
  float acc[R][R];
  for (int k = 0; k < steps; ++k) {
    product(A, A, acc);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int r = R * ty + i, c = R * tx + j;
        acc[i][j] = kNsB * A[r * kPitch + c] + kNsC * acc[i][j] + (r == c ? kNsA : 0.0f);
      }
    put(P, acc);
    if (k == 0) {
      put(Q, acc);
      __syncthreads();
    } else {
      __syncthreads();
      product(P, Q, acc);
      __syncthreads();
      put(Q, acc);
    }
    if (k + 1 < steps) {
      product(P, A, acc);  // P A, kept transposed
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) W[(R * tx + j) * kPitch + R * ty + i] = acc[i][j];
      __syncthreads();
      product(W, P, acc);
      put(A, acc);
    }
    __syncthreads();
  }
  float* to = q + (size_t)blockIdx.x * L * L;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = tid + i * kSmallThreads;
    to[e] = Q[e % L * kPitch + e / L];
  }
}

// out = Q X_0, or X_0 Q^T of tall matrices, in bf16 or fp32; q holds Q^T.  out may be g: a chunk is read whole
// before any of it is written, by the same block
template <typename T, bool TALL, int L, typename OUT>
__global__ void __launch_bounds__(kSmallThreads) small_apply_kernel(const T* g, int low, int high, int chunks,
                                                                    const float* q,
                                                                    const float2* scales,
                                                                    OUT* out) {
  constexpr int R = L / 16, kPitch = L + 4, kXPitch = kSmallChunk + 4;
  __shared__ __align__(16) float qs[L * kPitch];
  __shared__ __align__(16) float xs[L * kXPitch];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const float2 f = scales[blockIdx.y];
#pragma unroll
  for (int i = 0; i < L * L / kSmallThreads; ++i) {
    const int e = tid + i * kSmallThreads;
    qs[e / L * kPitch + e % L] = q[(size_t)blockIdx.y * L * L + e];
  }
  const T* m = g + (long long)blockIdx.y * low * high;
  OUT* o = out + (long long)blockIdx.y * low * high;
  auto store = [](OUT* at, float v) {
    if constexpr (sizeof(OUT) == 4) *at = v;
    else *at = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  };
  float v[kSmallChunk * L / kSmallThreads];
  fetch_chunk<T, TALL, L>(m, low, high, blockIdx.x * kSmallChunk, v, tid);
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int n0 = c * kSmallChunk;
    __syncthreads();
    place_chunk<TALL, L>(v, low, high, n0, f, xs, 1, kXPitch, tid);
    __syncthreads();
    if (c + (int)gridDim.x < chunks) fetch_chunk<T, TALL, L>(m, low, high, (c + (int)gridDim.x) * kSmallChunk, v, tid);
    if constexpr (TALL) {
      float acc[4][R] = {};
      micro<4, R, L>(xs, kXPitch, qs, kPitch, ty, tx, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 4 * ty + i;
#pragma unroll
        for (int j = 0; j < R; ++j)
          if (n < high && R * tx + j < low) store(o + (long long)n * low + R * tx + j, acc[i][j]);
      }
    } else {
      float acc[R][4] = {};
      micro<R, 4, L>(qs, kPitch, xs, kXPitch, ty, tx, acc);
      const int n = n0 + 4 * tx;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = R * ty + i;
        if (r >= low) continue;
        OUT* at = o + (long long)r * high + n;
        if (sizeof(OUT) == 2 && (high & 3) == 0 && n + 4 <= high) {
          *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16(acc[i][0], acc[i][1]), pack_bf16(acc[i][2], acc[i][3]));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < high) store(at + j, acc[i][j]);
        }
      }
    }
  }
}

// one round of at most kSmallSteps steps from g: into out, or as fp32 into x if it is not the last
template <typename T, bool TALL, int L>
cudaError_t small_round(const T* g, int count, int low, int high, int steps, int norm_parts, bool last, const SmallLayout& l,
                        uint16_t* out, uint8_t* b, cudaStream_t s) {
  constexpr int kSmem = 4 * L * (L + 4) * (int)sizeof(float);
  const double* norms = reinterpret_cast<const double*>(b + l.norms);
  float2* scale = reinterpret_cast<float2*>(b + l.scale);
  float* partial = reinterpret_cast<float*>(b + l.partial);
  float* q = reinterpret_cast<float*>(b + l.q);
  cudaError_t e = cudaFuncSetAttribute(small_iterate_kernel<L>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(small_gram_kernel<T, TALL, L>, dim3((unsigned)l.parts, (unsigned)count), dim3(kSmallThreads), 0, s, g, low,
                 high, l.chunks, norms, norm_parts, partial);
  if (e != cudaSuccess) return e;
  e = launch_pdl(small_iterate_kernel<L>, dim3((unsigned)count), dim3(kSmallThreads), kSmem, s, (const float*)partial, l.parts,
                 steps, norms, norm_parts, q, scale);
  if (e != cudaSuccess) return e;
  int slices = (2 * kSmallBlocks + count - 1) / count;
  if (slices > l.chunks) slices = l.chunks;
  const dim3 grid((unsigned)slices, (unsigned)count);
  if (last)
    return launch_pdl(small_apply_kernel<T, TALL, L, uint16_t>, grid, dim3(kSmallThreads), 0, s, g, low, high, l.chunks,
                      (const float*)q, (const float2*)scale, out);
  return launch_pdl(small_apply_kernel<T, TALL, L, float>, grid, dim3(kSmallThreads), 0, s, g, low, high, l.chunks,
                    (const float*)q, (const float2*)scale, reinterpret_cast<float*>(b + l.x));
}

template <bool TALL, int L, typename T>
cudaError_t small_rounds(const T* g, int count, int low, int high, int steps, int norm_parts, const SmallLayout& l,
                         uint16_t* out, uint8_t* b, cudaStream_t s) {
  const int first = steps < kSmallSteps ? steps : kSmallSteps;
  cudaError_t e = small_round<T, TALL, L>(g, count, low, high, first, norm_parts, first == steps, l, out, b, s);
  for (int k = first; k < steps && e == cudaSuccess; k += kSmallSteps) {
    const int n = steps - k < kSmallSteps ? steps - k : kSmallSteps;
    e = small_round<float, TALL, L>(reinterpret_cast<const float*>(b + l.x), count, low, high, n, 0, k + n == steps, l, out, b, s);
  }
  return e;
}

template <typename T>
cudaError_t small_orthogonalize(const T* g, int count, int M, int N, int steps, const SmallLayout& l, uint16_t* out,
                                uint8_t* b, cudaStream_t s) {
  int norm_parts = 0;
  const cudaError_t e = norms_of(g, count, M, N, reinterpret_cast<double*>(b + l.norms), norm_parts, s);
  if (e != cudaSuccess) return e;
  const bool tall = M > N;
  const int low = tall ? N : M, high = tall ? M : N;
  if (l.L == 32)
    return tall ? small_rounds<true, 32>(g, count, low, high, steps, norm_parts, l, out, b, s)
                : small_rounds<false, 32>(g, count, low, high, steps, norm_parts, l, out, b, s);
  return tall ? small_rounds<true, 64>(g, count, low, high, steps, norm_parts, l, out, b, s)
              : small_rounds<false, 64>(g, count, low, high, steps, norm_parts, l, out, b, s);
}
