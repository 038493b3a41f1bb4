// Quantisers to e4m3 with scales.
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
  const float m = half_warp_max(amax8(v));
  if (!ok) return;
  *reinterpret_cast<uint2*>(q + row * cols + c) =
      e4m3_pack8(v, e4m3_tiny(m) ? 1.f : e4m3_inverse(m));
  if (l == 0) scale[row * kb + b] = e4m3_scale(m);
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
  const float inv = e4m3_tiny(m) ? 1.f : e4m3_inverse(m);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < rows && c < cols)
      *reinterpret_cast<uint2*>(q + (r0 + 16 * i) * cols + c) = e4m3_pack8(v[i], inv);
  if (threadIdx.x == 0) scale[blockIdx.x] = e4m3_scale(m);
}

}  // namespace flkl
