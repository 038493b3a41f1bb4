// Host side of the scoring entry points declared in include/flkl.h: e4m3
// quantisers, the block-scaled product, token log-probabilities.

#include <cmath>
#include <type_traits>

#include "../../include/flkl.h"
#include "fp8_kernels.cuh"
#include "token_logprobs.cuh"

namespace flkl {
namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int d) { return d == FLKL_DTYPE_F32 || d == FLKL_DTYPE_BF16; }
size_t elem_size(int d) { return d == FLKL_DTYPE_F32 ? 4 : 2; }
flkl_status launched() {
  return cudaGetLastError() == cudaSuccess ? FLKL_OK : FLKL_ERR_CUDA;
}

template <typename T>
flkl_status quantize(const void* src, int64_t rows, int64_t cols, int block_rows, void* q,
                     float* scale, cudaStream_t st) {
  const int64_t kb = (cols + kScaleBlock - 1) / kScaleBlock;
  const int64_t ctas = block_rows == 1 ? (rows * kb + 15) / 16
                                       : (rows + kScaleBlock - 1) / kScaleBlock * kb;
  if (ctas >= kMaxDim) return FLKL_ERR_UNSUPPORTED;
  auto kern = block_rows == 1 ? k_quantize_rows<T> : k_quantize_blocks<T>;
  kern<<<static_cast<unsigned>(ctas), 256, 0, st>>>(static_cast<const T*>(src), rows,
                                                    static_cast<int>(cols),
                                                    static_cast<uint8_t*>(q), scale);
  return launched();
}

}  // namespace
}  // namespace flkl

using namespace flkl;

extern "C" {

flkl_status flkl_fp8_quantize(const void* src, int64_t rows, int64_t cols, int dtype,
                              int block_rows, void* q, float* scale, void* stream) {
  if (!dtype_ok(dtype) || rows < 0 || cols < 1) return FLKL_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != kScaleBlock) return FLKL_ERR_INVALID_ARG;
  if (cols % 16 != 0 || rows >= kMaxDim || cols >= kMaxDim) return FLKL_ERR_UNSUPPORTED;
  if (rows == 0) return FLKL_OK;
  if (src == nullptr || q == nullptr || scale == nullptr) return FLKL_ERR_INVALID_ARG;
  if (!aligned(src, 16) || !aligned(q, 16) || !aligned(scale, 4)) return FLKL_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == FLKL_DTYPE_BF16
             ? quantize<__nv_bfloat16>(src, rows, cols, block_rows, q, scale, st)
             : quantize<float>(src, rows, cols, block_rows, q, scale, st);
}

flkl_status flkl_fp8_block_matmul(const void* A, const float* a_scale, const void* B,
                                  const float* b_scale, const void* bias, int64_t M, int64_t N,
                                  int64_t K, int out_dtype, void* D, void* stream) {
  if (!dtype_ok(out_dtype) || M < 0 || N < 0 || K < 1) return FLKL_ERR_INVALID_ARG;
  if (K % 16 != 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return FLKL_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return FLKL_OK;
  if (A == nullptr || B == nullptr || a_scale == nullptr || b_scale == nullptr || D == nullptr)
    return FLKL_ERR_INVALID_ARG;
  const size_t e = elem_size(out_dtype);
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, e) || !aligned(a_scale, 4) ||
      !aligned(b_scale, 4) || !aligned(bias, e))
    return FLKL_ERR_UNSUPPORTED;
  Fp8Args a{};
  a.A = static_cast<const uint8_t*>(A);
  a.sa = a_scale;
  a.B = static_cast<const uint8_t*>(B);
  a.sb = b_scale;
  a.bias = bias;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.KB = static_cast<int>((K + kScaleBlock - 1) / kScaleBlock);
  a.D = D;
  const int64_t mt = (M + 63) / 64;
  if (mt > 65535) return FLKL_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>((N + 63) / 64), static_cast<unsigned>(mt));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (out_dtype == FLKL_DTYPE_BF16) k_fp8_simt<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  else k_fp8_simt<float><<<grid, 256, 0, st>>>(a);
  return launched();
}

flkl_status flkl_token_logprobs_forward(const void* logits, int64_t row_stride,
                                        const int64_t* target, int64_t ignore_index,
                                        int64_t rows, int64_t V, int dtype, float temperature,
                                        int top_k, float* logp, float* entropy, float* lse,
                                        float* stats, float* top_logp, int64_t* top_ids,
                                        void* stream) {
  if (!dtype_ok(dtype) || rows < 0 || V < 1 || top_k < 0 || row_stride < V)
    return FLKL_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !(temperature < INFINITY)) return FLKL_ERR_INVALID_ARG;
  if (top_k > LP_MAX_K || top_k > V || rows >= kMaxDim || V >= kMaxDim ||
      row_stride >= (int64_t(1) << 40))
    return FLKL_ERR_UNSUPPORTED;
  if (rows == 0) return FLKL_OK;
  if (logits == nullptr || entropy == nullptr || lse == nullptr || stats == nullptr ||
      (target != nullptr) != (logp != nullptr) ||
      (top_k > 0 && (top_logp == nullptr || top_ids == nullptr)))
    return FLKL_ERR_INVALID_ARG;
  if (!aligned(logits, elem_size(dtype)) || !aligned(target, 8) || !aligned(top_ids, 8) ||
      !aligned(stats, 8) || !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(lse, 4) ||
      !aligned(top_logp, 4))
    return FLKL_ERR_UNSUPPORTED;
  LpFwdArgs a{};
  a.logits = logits;
  a.ld = row_stride;
  a.target = target;
  a.ignore_index = ignore_index;
  a.rows = static_cast<int>(rows);
  a.V = static_cast<int>(V);
  a.temperature = temperature;
  a.k = top_k;
  a.logp = logp;
  a.entropy = entropy;
  a.lse = lse;
  a.stats = reinterpret_cast<float2*>(stats);
  a.top_logp = top_logp;
  a.top_ids = top_ids;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(rows);
  const bool bf = dtype == FLKL_DTYPE_BF16;
  if (top_k > 0) {
    if (bf) k_token_logprobs<__nv_bfloat16, true><<<grid, LP_NT, 0, st>>>(a);
    else k_token_logprobs<float, true><<<grid, LP_NT, 0, st>>>(a);
  } else {
    if (bf) k_token_logprobs<__nv_bfloat16, false><<<grid, LP_NT, 0, st>>>(a);
    else k_token_logprobs<float, false><<<grid, LP_NT, 0, st>>>(a);
  }
  return launched();
}

flkl_status flkl_token_logprobs_backward(const void* logits, int64_t row_stride,
                                         const int64_t* target, int64_t ignore_index,
                                         int64_t rows, int64_t V, int dtype, float temperature,
                                         int top_k, const float* stats, const float* entropy,
                                         const int64_t* top_ids, const float* dlogp,
                                         const float* dentropy, const float* dtop_logp,
                                         void* dlogits, int64_t d_row_stride, void* stream) {
  if (!dtype_ok(dtype) || rows < 0 || V < 1 || top_k < 0 || row_stride < V || d_row_stride < V)
    return FLKL_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !(temperature < INFINITY)) return FLKL_ERR_INVALID_ARG;
  if (top_k > LP_MAX_K || top_k > V || rows >= kMaxDim || V >= kMaxDim ||
      row_stride >= (int64_t(1) << 40) || d_row_stride >= (int64_t(1) << 40))
    return FLKL_ERR_UNSUPPORTED;
  if (rows == 0) return FLKL_OK;
  if (logits == nullptr || stats == nullptr || entropy == nullptr || dlogits == nullptr ||
      (dlogp != nullptr && target == nullptr) ||
      (dtop_logp != nullptr && (top_k == 0 || top_ids == nullptr)))
    return FLKL_ERR_INVALID_ARG;
  if (!aligned(logits, elem_size(dtype)) || !aligned(dlogits, elem_size(dtype)) ||
      !aligned(target, 8) || !aligned(top_ids, 8) || !aligned(stats, 8) ||
      !aligned(entropy, 4) || !aligned(dlogp, 4) || !aligned(dentropy, 4) ||
      !aligned(dtop_logp, 4))
    return FLKL_ERR_UNSUPPORTED;
  LpBwdArgs a{};
  a.logits = logits;
  a.ld = row_stride;
  a.target = target;
  a.ignore_index = ignore_index;
  a.rows = static_cast<int>(rows);
  a.V = static_cast<int>(V);
  a.temperature = temperature;
  a.k = top_k;
  a.stats = reinterpret_cast<const float2*>(stats);
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.dtop = dtop_logp;
  a.dlogits = dlogits;
  a.dld = d_row_stride;
  const int64_t ctas = rows * ((V + LPB_CHUNK - 1) / LPB_CHUNK);
  if (ctas >= kMaxDim) return FLKL_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(ctas);
  if (dtype == FLKL_DTYPE_BF16) k_token_logprobs_bwd<__nv_bfloat16><<<grid, LPB_NT, 0, st>>>(a);
  else k_token_logprobs_bwd<float><<<grid, LPB_NT, 0, st>>>(a);
  return launched();
}

}  // extern "C"
