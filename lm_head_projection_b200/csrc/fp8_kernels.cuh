// Quantisers to e4m3 with scales, and the block-scaled product
//
//   D[m][n] = sum over blocks kb of  sa[m][kb] sb[n / 128][kb]
//                 sum over k in block kb of A[m][k] B[n][k]   (+ bias[n])
//
// with A [M][K], B [N][K] in e4m3, blocks of 128 along K (the last may be
// short), fp32 sums.
#pragma once

#include "fp8.cuh"

namespace flkl {

// ------------------------------------------------------------- quantisers
// One scale per row and 128 columns: a half warp per block, 8 columns a lane.
template <typename T>
__global__ void __launch_bounds__(256) k_quantize_rows(const T* __restrict__ src, long long rows,
                                                       int cols, uint8_t* __restrict__ q,
                                                       float* __restrict__ scale) {
  const int kb = (cols + kScaleBlock - 1) / kScaleBlock;
  const long long g = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 4;
  const int l = threadIdx.x & 15;
  const long long row = g / kb;
  const int b = static_cast<int>(g % kb), c = b * kScaleBlock + l * 8;
  const bool ok = row < rows && c < cols;
  float v[8] = {};
  if (ok) Vec8<T>::load(src + row * cols + c, v);
  const float s = e4m3_scale(half_warp_max(amax8(v)));
  if (!ok) return;
  *reinterpret_cast<uint2*>(q + row * cols + c) = e4m3_pack8(v, 1.f / s);
  if (l == 0) scale[row * kb + b] = s;
}

// One scale per 128 x 128 block: a CTA per block, held in registers between
// its maximum and its codes.
template <typename T>
__global__ void __launch_bounds__(256) k_quantize_blocks(const T* __restrict__ src,
                                                         long long rows, int cols,
                                                         uint8_t* __restrict__ q,
                                                         float* __restrict__ scale) {
  __shared__ float red[8];
  const int kb = (cols + kScaleBlock - 1) / kScaleBlock;
  const long long br = blockIdx.x / kb;
  const int b = static_cast<int>(blockIdx.x % kb);
  const int c = b * kScaleBlock + (threadIdx.x & 15) * 8;
  const long long r0 = br * kScaleBlock + (threadIdx.x >> 4);
  float v[8][8] = {};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < rows && c < cols) {
      Vec8<T>::load(src + (r0 + 16 * i) * cols + c, v[i]);
      m = fmaxf(m, amax8(v[i]));
    }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
  const float s = e4m3_scale(m);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < rows && c < cols)
      *reinterpret_cast<uint2*>(q + (r0 + 16 * i) * cols + c) = e4m3_pack8(v[i], 1.f / s);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
}

// ---------------------------------------------------------------- product
struct Fp8Args {
  const uint8_t* A;
  const float* sa;  // [M][KB]
  const uint8_t* B;
  const float* sb;  // [ceil(N / 128)][KB]
  const void* bias; // [N] in the output's type, or null
  int M, N, K, KB;
  void* D;  // [M][N]
};

template <typename T>
__device__ __forceinline__ T fp8_out(float v);
template <>
__device__ __forceinline__ float fp8_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 fp8_out<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Plain tiles: 64 x 64 outputs per CTA, 4 x 4 per thread, 16 columns of K a step.
template <typename TO>
__global__ void __launch_bounds__(256) k_fp8_simt(const Fp8Args a) {
  __shared__ float As[16][65], Bs[16][65];
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int lr = threadIdx.x >> 2, lc = (threadIdx.x & 3) * 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 16) {
    const int kb = k0 / kScaleBlock;
    auto fill = [&](float (&dst)[16][65], const uint8_t* src, int r, int lim, float s) {
      uint32_t w = 0;
      if (r < lim) w = *reinterpret_cast<const uint32_t*>(src + static_cast<size_t>(r) * a.K + k0 + lc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __nv_fp8_e4m3 e;
        e.__x = static_cast<uint8_t>(w >> (8 * i));
        dst[lc + i][lr] = static_cast<float>(e) * s;
      }
    };
    const int ra = m0 + lr, rb = n0 + lr;
    fill(As, a.A, ra, a.M, ra < a.M ? a.sa[static_cast<size_t>(ra) * a.KB + kb] : 0.f);
    fill(Bs, a.B, rb, a.N, rb < a.N ? a.sb[static_cast<size_t>(rb / kScaleBlock) * a.KB + kb] : 0.f);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + ty * 4 + i;
    if (m >= a.M) break;
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= a.N) break;
      float v = acc[i][j];
      if (a.bias != nullptr) v += static_cast<float>(static_cast<const TO*>(a.bias)[n]);
      static_cast<TO*>(a.D)[static_cast<size_t>(m) * a.N + n] = fp8_out<TO>(v);
    }
  }
}

}  // namespace flkl
