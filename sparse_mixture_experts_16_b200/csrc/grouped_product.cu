// grouped_product.cu -- products grouped by expert over ragged row segments, the plain linear layer
// of an expert and its two gradients (the grouped backend of keryc.com "Mixture of Experts optimiza
// Transformers y LLMs", section "Ejecucion eficiente: backends de expertos", without the SwiGLU that
// moe_grouped_swiglu_ffn fuses in).  Segment e holds rows [offsets[e], offsets[e+1]):
//     gemm   y[r]  = x[r] W_e^T      A = W_e (K-major),  B = x (K-major)
//     dgrad  dx[r] = dy[r] W_e       A = W_e (MN-major), B = dy (K-major)
//     wgrad  dW_e  = dy_e^T x_e      A = x (MN-major),   B = dy (MN-major), contracted over the segment
// in the notation of product_sm100.cuh, whose kernel computes them; this file checks the arguments and
// fills in the operands.
#include "product_sm100.cuh"

using namespace moe;
using namespace moe::product;

namespace {

// rows that can be rounded up to whole tiles, K blocks or means of segments within 32 bits
constexpr int kMostRows = 0x7fffffff - 65535;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

moe_status_t shape_status(int M, int E, int N, int K, int dtype) {
  if (M < 0 || E <= 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_ERR_INVALID_ARG;
  // rows of 16-bit elements that TMA can step over, and coordinates and tile counts within 32 bits
  if (N % 8 != 0 || K % 8 != 0 || N > 65536 || K > 65536 || E > kMaxGroups) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (M > kMostRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  // whatever the offsets are: clamped, each segment has at most M rows
  const long long tiles = ((long long)M / kTile + 1) * E * ((N > K ? N : K) / kTile + 1);
  if (tiles >= (1LL << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// the workspace's share of a launch
void set_workspace(Params& p, void* ws, int prows) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  p.err = reinterpret_cast<int*>(b);
  p.counters = reinterpret_cast<int*>(b + kWsHeader);
  p.partial = reinterpret_cast<float*>(b + kPartialOffset);
  p.prows = prows;
}

size_t workspace_bytes(int prows) { return align_up(kPartialOffset + partial_bytes(prows), 256); }

// gemm (W_MN = false: rows of N weights, contracted over K) and dgrad (W_MN = true: contracted over N)
template <bool W_MN>
moe_status_t rows_product(const void* x, const int32_t* offsets, const void* w, int M, int E, int N, int K, int dtype,
                          int out_dtype, void* out, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = shape_status(M, E, N, K, dtype);
  if (st != MOE_OK) return st;
  if (out_dtype != dtype && out_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (!offsets || !w || !ws || (M > 0 && (!x || !out))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(offsets, 4) || !aligned(ws, 256))
    return MOE_ERR_ALIGNMENT;
  if (ws_bytes < moe_grouped_gemm_workspace_size(M)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = device_status()) != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  Params p;
  memset(&p, 0, sizeof(p));
  p.offsets = offsets;
  p.G = E;
  p.M_total = M;
  p.cols = W_MN ? K : N;
  p.K = W_MN ? N : K;
  p.kb_typ = (p.K + kBK - 1) / kBK;
  p.rows_typ = M / E;  // the mean segment
  p.out = out;
  p.out_bf16 = dtype == MOE_DTYPE_BF16;
  p.withhold_first_load = test_withhold_this_launch() ? 1 : 0;
  set_workspace(p, ws, partial_rows(M));
  const OperandHost a = {w, (uint64_t)K, (uint64_t)N, (uint64_t)E};
  const OperandHost b = {x, (uint64_t)p.K, (uint64_t)M, 1};
  if (!set_operands<W_MN, false>(p, a, b, dtype == MOE_DTYPE_BF16)) return MOE_ERR_CUDA;
  const cudaError_t e = out_dtype == MOE_DTYPE_FP32 ? launch<W_MN, false, kRaggedRows, kOut32>(p, (cudaStream_t)stream)
                                                    : launch<W_MN, false, kRaggedRows, kOut16>(p, (cudaStream_t)stream);
  return launch_status(e);
}

}  // namespace

extern "C" {

size_t moe_grouped_gemm_workspace_size(int M) { return M < 0 ? 0 : workspace_bytes(partial_rows(M)); }

moe_status_t moe_grouped_gemm(const void* x, const int32_t* offsets, const void* w, int M, int E, int N, int K,
                              int dtype, int out_dtype, void* y, void* ws, size_t ws_bytes, moe_stream_t stream) {
  return rows_product<false>(x, offsets, w, M, E, N, K, dtype, out_dtype, y, ws, ws_bytes, stream);
}

moe_status_t moe_grouped_gemm_dgrad(const void* dy, const int32_t* offsets, const void* w, int M, int E, int N, int K,
                                    int dtype, int out_dtype, void* dx, void* ws, size_t ws_bytes,
                                    moe_stream_t stream) {
  return rows_product<true>(dy, offsets, w, M, E, N, K, dtype, out_dtype, dx, ws, ws_bytes, stream);
}

size_t moe_grouped_gemm_wgrad_workspace_size(int N) { return N <= 0 ? 0 : workspace_bytes(partial_rows(N)); }

moe_status_t moe_grouped_gemm_wgrad(const void* dy, const void* x, const int32_t* offsets, int M, int E, int N, int K,
                                    int dtype, float* dw, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = shape_status(M, E, N, K, dtype);
  if (st != MOE_OK) return st;
  if (!dw || !ws || !offsets || (M > 0 && (!dy || !x))) return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16) || !aligned(offsets, 4) || !aligned(ws, 256))
    return MOE_ERR_ALIGNMENT;
  if (ws_bytes < moe_grouped_gemm_wgrad_workspace_size(N)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = device_status()) != MOE_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (M == 0) return launch_status(cudaMemsetAsync(dw, 0, (size_t)E * N * K * sizeof(float), s));
  Params p;
  memset(&p, 0, sizeof(p));
  p.offsets = offsets;
  p.G = E;
  p.M_total = M;
  p.rows = N;
  p.cols = K;
  p.kb_typ = (M / E + kBK - 1) / kBK;  // the mean segment
  p.ld = K;
  const OperandHost out = {dw, (uint64_t)K, (uint64_t)N, (uint64_t)E};
  if (!set_output(p, out)) return MOE_ERR_CUDA;
  p.withhold_first_load = test_withhold_this_launch() ? 1 : 0;
  set_workspace(p, ws, partial_rows(N));
  const OperandHost a = {x, (uint64_t)K, (uint64_t)M, 1};
  const OperandHost b = {dy, (uint64_t)N, (uint64_t)M, 1};
  if (!set_operands<true, true>(p, a, b, dtype == MOE_DTYPE_BF16)) return MOE_ERR_CUDA;
  return launch_status(launch<true, true, kRaggedK, kGrad>(p, s));
}

}  // extern "C"
