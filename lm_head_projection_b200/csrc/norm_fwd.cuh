// RMSNorm of h = x + residual, with h passed on and y in the input's type or
// in e4m3 with one fp32 scale per row and 128 columns:
//
//   h = round(x + residual),  r = 1 / sqrt(mean(h^2) + eps),  y = h r w,
//   scale = max |y| over the block / 448,  code = e4m3(y / scale).
//
// y is formed from the rounded h, the value that the residual stream keeps, so
// that the backward pass, which reads h, differentiates what was computed.
// The 8-bit output is rounded once: r falls out of y / max |y|, so that codes are
// formed from p = 2^e h w, with 2^e the power of two in r.  p has y's size and,
// where the row is bf16, is exact, so that codes are the nearest ones and exact
// ties go to even (fp8.cuh); the scale is max |p| r / 2^e / 448.
//
// HBM-bound (bf16 in, e4m3 out: 7 bytes per element and nothing to reuse), so a
// row is read once into registers, 8 columns per thread and vector, and every
// output leaves from there.  A row of at most 256 columns is one warp's (4 rows
// per CTA, no barrier); wider rows are one CTA's.  Measured: 8192 x 8192 bf16 to
// e4m3 79 us (470 MB, 5.9 TB/s; a copy reaches 6.5), to bf16 84 us (6.4 TB/s);
// 512 threads x 2 vectors took 88 us for what 256 x 4 did in 98 and 1024 x 1 in
// 108, and a register limit that lets 2048 threads stand on an SM brought it to 79
// (bf16; fp32 rows, whose loads are twice as wide, run best without).
#pragma once

#include "fp8.cuh"
#include "norm_bwd.cuh"

namespace flkl {

struct NormFwdArgs {
  const void* X;
  const void* R;  // residual, or null (then Hs is null)
  const void* W;
  int rows, H;
  float eps;
  void* Y;       // T, or e4m3 codes with QUANT
  float* scale;  // [rows][ceil(H / 128)] with QUANT
  void* Hs;
};

// G threads per row, VPT vectors of 8 columns per thread (H <= 8 G VPT);
// NT threads per CTA, NT / G rows.
template <typename T, int NT, int G, int VPT, bool QUANT>
__global__ void __launch_bounds__(NT, sizeof(T) == 2 ? 2048 / NT : 1)
    k_add_rms_norm(const NormFwdArgs a) {
  constexpr int NW = G / 32;
  __shared__ float red[NW > 1 ? NW : 1];
  const int lane = threadIdx.x & 31;
  const int t = threadIdx.x % G;
  const int row = blockIdx.x * (NT / G) + threadIdx.x / G;
  if (G == 32 && row >= a.rows) return;  // (a whole warp; with G = NT every row exists)
  const int H = a.H;
  const size_t off = static_cast<size_t>(row) * H;
  const T* X = static_cast<const T*>(a.X) + off;
  const T* R = static_cast<const T*>(a.R) + off;
  T* Hs = static_cast<T*>(a.Hs) + off;
  float h[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * G + t) * 8;
    if (c < H) {
      Vec8<T>::load(X + c, h[v]);
      if (a.R != nullptr) {
        float r[8];
        Vec8<T>::load(R + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = Vec8<T>::round(h[v][i] + r[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = 0.f;
    }
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * G + t) * 8;
    if (c < H && a.R != nullptr) Vec8<T>::store(Hs + c, h[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if constexpr (NW > 1) {
    if (lane == 0) red[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = red[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) ss += red[i];
  }
  const float rinv = rsqrtf(ss / static_cast<float>(H) + a.eps);
  // 8 bits: 2^e, and what is left of rinv (infinity and NaN are passed on whole)
  float factor = rinv, rest = 1.f;
  if constexpr (QUANT) {
    if (rinv < INFINITY) {
      factor = __uint_as_float(__float_as_uint(rinv) & 0x7F800000u);
      rest = rinv * __uint_as_float(0x7F000000u - __float_as_uint(factor));
    }
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) h[v][i] *= factor;
  const T* W = static_cast<const T*>(a.W);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * G + t) * 8;
    if (c < H) {
      float w[8];
      Vec8<T>::load(W + c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] *= w[i];
    }
    if constexpr (QUANT) {
      // columns [128 j, 128 j + 128) are one half warp's (G is a multiple of 32)
      const float m = half_warp_max(amax8(h[v])), ymax = m * rest;
      if (c < H) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.Y) + off + c) =
            e4m3_pack8(h[v], e4m3_tiny(ymax) ? 1.f : e4m3_inverse(m));
        if ((lane & 15) == 0)
          a.scale[static_cast<size_t>(row) * ((H + 127) / 128) + c / 128] = e4m3_scale(ymax);
      }
    } else {
      if (c < H) Vec8<T>::store(static_cast<T*>(a.Y) + off + c, h[v]);
    }
  }
}

template <typename T, int NT, int G, int VPT>
cudaError_t launch_norm_fwd_w(const NormFwdArgs& a, bool quant, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((a.rows + NT / G - 1) / (NT / G));
  if (quant) k_add_rms_norm<T, NT, G, VPT, true><<<grid, NT, 0, st>>>(a);
  else k_add_rms_norm<T, NT, G, VPT, false><<<grid, NT, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_norm_fwd(const NormFwdArgs& a, bool quant, cudaStream_t st) {
  if (a.H <= 256) return launch_norm_fwd_w<T, 128, 32, 1>(a, quant, st);
  if (a.H <= 1024) return launch_norm_fwd_w<T, 128, 128, 1>(a, quant, st);
  if (a.H <= 2048) return launch_norm_fwd_w<T, 128, 128, 2>(a, quant, st);
  if (a.H <= 4096) return launch_norm_fwd_w<T, 256, 256, 2>(a, quant, st);
  return launch_norm_fwd_w<T, 512, 512, 2>(a, quant, st);
}

}  // namespace flkl
