// e4m3 codes with fp32 scales: what the norm's 8-bit output, the quantisers
// and the block-scaled product share.
//
// A block's scale is its largest magnitude / 448 (the largest e4m3 number), so
// that the block's extreme keeps its value; a code is the value over the scale,
// rounded to nearest even.  A block below 2^-100 throughout (all zeros, as a
// rule) has the scale 1 and codes 0: its reciprocal scale would overflow.
#pragma once

#include <cuda_fp8.h>

#include "vec8.cuh"

namespace flkl {

constexpr float kE4m3Max = 448.f;
constexpr int kScaleBlock = 128;  // columns (and, for weights, rows) that share a scale

__device__ __forceinline__ float e4m3_scale(float amax) {
  return amax < 0x1p-100f ? 1.f : amax / kE4m3Max;
}
// 1 / scale for the codes, within 3 of its last places (a true division per
// block costs more than the rest of a block's arithmetic; a code moves only
// where a value lies that close to the middle of two).
__device__ __forceinline__ float e4m3_inv_scale(float amax) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(amax * (1.f / kE4m3Max)));
  return amax < 0x1p-100f ? 1.f : r;
}

// 8 values times inv -> 8 codes (out-of-range values saturate, NaN stays NaN).
__device__ __forceinline__ uint2 e4m3_pack8(const float (&v)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float a = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
  return a;
}

// Largest value over the 16 lanes of a half warp, which hold one block of 128
// columns when every lane has 8.  All 32 lanes call.
__device__ __forceinline__ float half_warp_max(float a) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

}  // namespace flkl
