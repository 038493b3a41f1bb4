// e4m3 codes with fp32 scales: what the norm's 8-bit output, the quantisers
// and the block-scaled product share.
//
// A block's scale is its largest magnitude m / 448 (the largest e4m3 number), so
// that the block's extreme keeps its value; a code is 448 v / m, rounded to
// nearest even.  A block below 2^-100 throughout (all zeros, as a rule) has the
// scale 1 and codes 0: its reciprocal scale would overflow.
//
// Ties.  bf16 values (and the norm's products h w of two of them) are short, so
// that 448 v / m lies exactly between two codes time and again (one of 170 values
// of random bf16 rows).  A quotient from a reciprocal is off by up to 2^-22 of
// itself and would land on either side; it is therefore rounded to 21 bits first,
// which a tie (5 bits) is the nearest such number to.  Nothing else comes that
// close: with v = V 2^a and m = M 2^b of 16 bits, 448 v / m differs from a tie k 2^j
// (k < 32) by at least 1 / (16 M) > 2^-20 of the tie's leading bit, half a step of
// 21 bits is 2^-21 and the error less than that.  fp32 values have more bits and no
// such gap: theirs may go either way within 2^-21 of a tie.
#pragma once

#include <cuda_fp8.h>

#include "vec8.cuh"

namespace flkl {

constexpr float kE4m3Max = 448.f;
constexpr int kScaleBlock = 128;  // columns (and, for weights, rows) that share a scale

__device__ __forceinline__ bool e4m3_tiny(float amax) { return amax < 0x1p-100f; }
__device__ __forceinline__ float e4m3_scale(float amax) {
  return e4m3_tiny(amax) ? 1.f : amax / kE4m3Max;
}
// 448 / m, off by at most 3 * 2^-24 of itself (the reciprocal 2^-23, then one
// rounding; a true division per block costs more than the rest of a block's
// arithmetic).  2^-8 m has a normal reciprocal for every finite m above 2^-101.
__device__ __forceinline__ float e4m3_inverse(float m) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(m * 0x1p-8f));
  return r * (448.f * 0x1p-8f);
}

// 8 values times inv -> 8 codes (out-of-range values saturate, NaN stays NaN).
// The quotients are cut to 21 bits by Veltkamp's splitting: with t = (2^3 + 1) q,
// t - (t - q) is q rounded to its upper 24 - 3 bits.
__device__ __forceinline__ uint2 e4m3_pack8(const float (&v)[8], float inv) {
  const uint64_t i2 = f2_pack(inv, inv), k2 = f2_pack(9.f, 9.f), n2 = f2_pack(-1.f, -1.f);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t q = f2_mul(f2_pack(v[2 * i], v[2 * i + 1]), i2);
    const uint64_t t = f2_mul(q, k2);
    h[i] = __nv_cvt_float2_to_fp8x2(f2_unpack(f2_fma(f2_fma(q, n2, t), n2, t)), __NV_SATFINITE,
                                    __NV_E4M3);
  }
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
