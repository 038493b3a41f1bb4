// Host side of the scoring entry points declared in include/flkl.h: e4m3
// quantisers, the block-scaled product, token log-probabilities.

#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cudaTypedefs.h>

#include "../../include/flkl.h"
#include "fp8_gemm.cuh"
#include "fp8_kernels.cuh"
#include "token_logprobs.cuh"

namespace flkl {

extern unsigned long long g_wait_limit_ns;  // flkl_api.cu

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int d) { return d == FLKL_DTYPE_F32 || d == FLKL_DTYPE_BF16; }
// (1 / temperature has to be a number too)
bool temperature_ok(float t) { return t > 0x1p-120f && t < INFINITY; }
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

// ---------------------------------------------------------------- product
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// Byte matrix [rows][K], box {128, box_rows}, 128-byte swizzle, zeros outside.
bool fp8_map(CUtensorMap* m, const void* base, int64_t K, int64_t rows, uint32_t box_rows) {
  const auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {128, box_rows}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output matrix [M][N] of bf16 or fp32, box 128 bytes x 32 rows, 128-byte swizzle.
template <typename TO>
bool out_map(CUtensorMap* m, void* base, int64_t M, int64_t N) {
  const auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * sizeof(TO)};
  const cuuint32_t box[2] = {128 / sizeof(TO), 32}, estr[2] = {1, 1};
  return fn(m, sizeof(TO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
            2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;
constexpr size_t kMaxSmem = 227 * 1024;

// Per device: SMs, and whether a kernel's shared memory limit has been raised.
int device_sms() {
  static int cache[kMaxDevices] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  if (cache[dev] > 0) return cache[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    n = 148;
  return cache[dev] = n;
}

template <typename K>
bool raise_smem(K kern, bool (&done)[kMaxDevices]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  if (!done[dev])
    done[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(kMaxSmem)) == cudaSuccess;
  return done[dev];
}

// Clusters of `size` CTAs, one CTA to an SM, that are resident at once (a cluster
// sits inside one GPC, and these differ): 148 SMs hold fewer than 148 / size.
int resident_clusters(int size) {
  static int cache[kMaxDevices][S8_MAX_CLUSTER + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 1;
  if (cache[dev][size] > 0) return cache[dev][size];
  static bool done[kMaxDevices];
  int n = 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(size * device_sms()));
  cfg.blockDim = dim3(s8_threads<16>());
  cfg.dynamicSmemBytes = kMaxSmem;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(size);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (!raise_smem(k_fp8_skinny<float, 16, false>, done) ||
      cudaOccupancyMaxActiveClusters(&n, k_fp8_skinny<float, 16, false>, &cfg) != cudaSuccess ||
      n < 1)
    n = 1;
  return cache[dev][size] = n;
}

struct Fp8Call {
  const void *A, *B;
  int64_t K;
  Fp8Gemm g;
  cudaStream_t st;
};

template <typename TO, int BN, bool HOLD>
flkl_status launch_pair(const Fp8Call& c) {
  static bool done[kMaxDevices];
  if (!raise_smem(k_fp8_pair<TO, BN, HOLD>, done)) return FLKL_ERR_CUDA;
  Fp8Gemm g = c.g;
  g.m_tiles = (g.M - 1) / 256 + 1;
  g.n_tiles = (g.N - 1) / BN + 1;
  g.vec = (size_t(g.N) * sizeof(TO)) % 16 == 0 && aligned(g.D, 16);
  const int64_t tiles = int64_t(g.m_tiles) * g.n_tiles;
  if (tiles >= (int64_t(1) << 30)) return FLKL_ERR_UNSUPPORTED;
  CUtensorMap ma, mb, md;
  if (!fp8_map(&ma, c.A, c.K, g.M, 128) || !fp8_map(&mb, c.B, c.K, g.N, BN / 2))
    return FLKL_ERR_CUDA;
  md = ma;  // (not used where the rows of D are not on 16-byte boundaries)
  if (g.vec && !out_map<TO>(&md, g.D, g.M, g.N)) return FLKL_ERR_CUDA;
  const int pairs = static_cast<int>(std::min<int64_t>(resident_clusters(2), tiles));
  k_fp8_pair<TO, BN, HOLD><<<2 * pairs, P8_THREADS, P8<BN>::SMEM, c.st>>>(ma, mb, md, g);
  return launched();
}

template <typename TO, int BN, bool HOLD>
flkl_status launch_skinny(const Fp8Call& c, int cluster) {
  static bool done[kMaxDevices];
  if (!raise_smem(k_fp8_skinny<TO, BN, HOLD>, done)) return FLKL_ERR_CUDA;
  Fp8Gemm g = c.g;
  g.m_tiles = (g.M - 1) / BN + 1;
  g.n_tiles = (g.N - 1) / 128 + 1;
  const size_t fixed = s8_smem_fixed<BN>((g.KB + cluster - 1) / cluster);
  const size_t stages = std::min<size_t>((kMaxSmem - fixed) / s8_stage_bytes<BN>(), S8_MAX_STAGES);
  g.stages = static_cast<int>(stages);
  CUtensorMap mx, mw;
  if (!fp8_map(&mx, c.A, c.K, g.M, BN) || !fp8_map(&mw, c.B, c.K, g.N, 128)) return FLKL_ERR_CUDA;
  const int tiles = g.n_tiles * g.m_tiles;
  const int ctas =
      cluster == 1 && g.m_tiles == 1 ? std::min(device_sms(), tiles) : tiles * cluster;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(s8_threads<BN>());
  cfg.dynamicSmemBytes = fixed + stages * s8_stage_bytes<BN>();
  cfg.stream = c.st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(cluster);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_fp8_skinny<TO, BN, HOLD>, mx, mw, g) == cudaSuccess
             ? FLKL_OK
             : FLKL_ERR_CUDA;
}

// Which kernel.  Up to 64 rows there is one token tile and the weight is streamed
// at HBM's rate (64 x 128256 x 4096: 104 us, pairs 133).  Beyond, the pairs' tiles
// hold 4 or 8 of the small kernel's 128 x 64 ones on two SMs and take about as long
// per block of K: they win from a dozen large tiles on (256 x 4096 x 4096, 16
// tiles: 18.8 against 23.5 us; 129 x 1000 x 8192, 4 tiles: 36 against 18 us).
template <typename TO, bool HOLD>
flkl_status fp8_matmul(const Fp8Call& c) {
  const int M = c.g.M, KB = c.g.KB, sms = device_sms();
  const int64_t pair_tiles = int64_t((M - 1) / 256 + 1) * ((c.g.N - 1) / 256 + 1);
  if (M <= 64 || pair_tiles <= sms / 12) {
    // CTAs that share a tile, each with a part of K: as many as run at once
    const int64_t tiles = int64_t((c.g.N - 1) / 128 + 1) * ((M - 1) / 64 + 1);
    int cluster = static_cast<int>(std::min<int64_t>({S8_MAX_CLUSTER, sms / tiles, KB}));
    while (cluster > 1 && resident_clusters(cluster) < tiles) --cluster;
    cluster = std::max(cluster, 1);
    // (the tokens' scales have to leave room for a ring, which later holds the
    // cluster's parts)
    if (s8_smem_fixed<64>((KB + cluster - 1) / cluster) + 4 * s8_stage_bytes<64>() <= kMaxSmem) {
      if (M <= 16) return launch_skinny<TO, 16, HOLD>(c, cluster);
      if (M <= 32) return launch_skinny<TO, 32, HOLD>(c, cluster);
      return launch_skinny<TO, 64, HOLD>(c, cluster);
    }
  }
  // Tiles of 128 weight rows where they all run at once: a wave of them takes 0.7
  // of the larger ones' (300 x 4096 x 4096: 18.8 against 24.2 us; two waves of them
  // against one lose: 777 x 4096 x 4096 28.7 against 24.6).
  if (pair_tiles <= resident_clusters(2) / 2) return launch_pair<TO, 128, HOLD>(c);
  return launch_pair<TO, 256, HOLD>(c);
}

// --------------------------------------------------------- log-probabilities
template <typename T, bool TOP, int NT>
flkl_status launch_logprobs_nt(const LpFwdArgs& a, int parts, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(int64_t(a.rows) * parts));
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(parts);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_token_logprobs<T, TOP, NT>, a) == cudaSuccess ? FLKL_OK
                                                                                 : FLKL_ERR_CUDA;
}

template <typename T, bool TOP>
flkl_status launch_logprobs(const LpFwdArgs& a, cudaStream_t st) {
  // CTAs per row: a power of two up to 8, doubled while all rows' CTAs are no more
  // than the SMs and each has a tile of its own (4 x 128256 bf16: 8 us on the
  // device).  An SM holds four such CTAs, so that a few hundred rows, one CTA each,
  // leave places empty: 300 x 128256 with 5 alternatives takes 31 us (2.5 TB/s).
  int parts = 1;
  while (parts < 8 && int64_t(a.rows) * parts * 2 <= 2 * device_sms() &&
         a.V / (parts * 2) >= 256 * 16 / static_cast<int>(sizeof(T)))
    parts *= 2;
  if (parts == 1 && int64_t(a.V) * sizeof(T) <= 160 * 1024)
    return launch_logprobs_nt<T, TOP, 128>(a, 1, st);
  return launch_logprobs_nt<T, TOP, 256>(a, parts, st);
}

// flkl_fp8_block_matmul, with a role of its kernels that stops after a number of blocks.
flkl_status block_matmul(const void* A, const float* a_scale, const void* B, const float* b_scale,
                         const void* bias, int64_t M, int64_t N, int64_t K, int out_dtype, void* D,
                         void* stream, unsigned long long limit_ns, int hold, uint32_t hold_at) {
  if (!dtype_ok(out_dtype) || M < 0 || N < 0 || K < 1) return FLKL_ERR_INVALID_ARG;
  if (K % 16 != 0 || M > kMaxDim / 2 || N > kMaxDim / 2 || K > kMaxDim / 2)
    return FLKL_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return FLKL_OK;
  if (A == nullptr || B == nullptr || a_scale == nullptr || b_scale == nullptr || D == nullptr)
    return FLKL_ERR_INVALID_ARG;
  const size_t e = elem_size(out_dtype);
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, e) || !aligned(a_scale, 4) ||
      !aligned(b_scale, 4) || !aligned(bias, e))
    return FLKL_ERR_UNSUPPORTED;
  Fp8Call c{};
  c.A = A;
  c.B = B;
  c.K = K;
  c.st = static_cast<cudaStream_t>(stream);
  c.g.sa = a_scale;
  c.g.sb = b_scale;
  c.g.bias = bias;
  c.g.D = D;
  c.g.M = static_cast<int>(M);
  c.g.N = static_cast<int>(N);
  c.g.KB = static_cast<int>((K + kScaleBlock - 1) / kScaleBlock);
  c.g.wait_limit_ns = limit_ns;
  c.g.hold = hold;
  c.g.hold_at = hold_at;
  if (hold != FP8_HOLD_NONE) return fp8_matmul<__nv_bfloat16, true>(c);
  return out_dtype == FLKL_DTYPE_BF16 ? fp8_matmul<__nv_bfloat16, false>(c)
                                      : fp8_matmul<float, false>(c);
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
  return block_matmul(A, a_scale, B, b_scale, bias, M, N, K, out_dtype, D, stream,
                      g_wait_limit_ns, FP8_HOLD_NONE, 0);
}

flkl_status flkl_fp8_wait_selftest(const void* A, const float* a_scale, const void* B,
                                   const float* b_scale, int64_t M, int64_t N, int64_t K, void* D,
                                   int role, unsigned int blocks, unsigned int limit_ms,
                                   void* stream) {
  if (role < FP8_HOLD_MMA || role > FP8_HOLD_LOAD_ODD || limit_ms < 1 || limit_ms > 1000)
    return FLKL_ERR_INVALID_ARG;
  return block_matmul(A, a_scale, B, b_scale, nullptr, M, N, K, FLKL_DTYPE_BF16, D, stream,
                      limit_ms * 1000000ull, role, blocks);
}

flkl_status flkl_fp8_device_status(void* stream) {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_fp8_status) != cudaSuccess) return FLKL_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int h = 0;
  if (cudaMemcpyAsync(&h, p, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return FLKL_ERR_CUDA;
  if (h != 0 && (cudaMemsetAsync(p, 0, sizeof(int), st) != cudaSuccess ||
                 cudaStreamSynchronize(st) != cudaSuccess))
    return FLKL_ERR_CUDA;
  return static_cast<flkl_status>(h);
}

flkl_status flkl_token_logprobs_forward(const void* logits, int64_t row_stride,
                                        const int64_t* target, int64_t ignore_index,
                                        int64_t rows, int64_t V, int dtype, float temperature,
                                        int top_k, float* logp, float* entropy, float* lse,
                                        float* stats, float* top_logp, int64_t* top_ids,
                                        void* stream) {
  if (!dtype_ok(dtype) || rows < 0 || V < 1 || top_k < 0 || row_stride < V)
    return FLKL_ERR_INVALID_ARG;
  if (!temperature_ok(temperature)) return FLKL_ERR_INVALID_ARG;
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
  if (dtype == FLKL_DTYPE_BF16)
    return top_k > 0 ? launch_logprobs<__nv_bfloat16, true>(a, st)
                     : launch_logprobs<__nv_bfloat16, false>(a, st);
  return top_k > 0 ? launch_logprobs<float, true>(a, st) : launch_logprobs<float, false>(a, st);
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
  if (!temperature_ok(temperature)) return FLKL_ERR_INVALID_ARG;
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
