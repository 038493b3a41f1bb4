// The block-scaled e4m3 product on the tensor cores:
//
//   D[m][n] = sum_kb sa[m][kb] sb[n / 128][kb] (A B^T over block kb)[m][n]  (+ bias[n])
//
// The scales are arbitrary fp32 numbers, so each block of 128 along K is one
// product of its own in TMEM (four tcgen05.mma.kind::f8f6f4 of K = 32, the first
// overwriting), read back while the next block's runs into another TMEM
// buffer, and added with its scales into fp32 registers.  Rows, columns and
// the end of K that the tiles overhang are zeros that TMA fills in.
//
//   k_fp8_pair    many tokens: 256 tokens x 256 (or 128) weight rows per CTA pair
//                 (cta_group::2), a TMEM lane holds one token; bound by the
//                 tensor cores' rate.
//   k_fp8_skinny  few tokens: the weight's rows are the MMA's M side, 128 per
//                 tile, the tokens its N side (16 .. 64 columns), so that each
//                 weight byte is read once and little of an MMA is padding;
//                 bound by HBM.  Also more tokens, in tiles of 64, where the
//                 pairs' tiles would leave most SMs idle.
//
// What bounds the pairs: a 256 x 256 block is 512 clocks of MMAs, 256 of TMEM reads
// and 256 of additions per SM quarter, which would fit side by side; but a buffer's
// way round (commit, wake, read, arrival in the other CTA, wake: about 700 clocks
// beside the 450 of the read) has only two buffers to hide behind, as 512 columns
// of TMEM hold no third of 256 (three of 160 were not measured).  1024 x 128256 x
// 4096 takes 857 clocks a block (635 without additions and stores) and 490 - 507 us
// (2120 TFLOP/s and more) in a burst; back to back the power limit holds the clock
// at 1.3 - 1.5 GHz (577 - 592 us).  What made it so: two issuing threads instead of
// one (585 -> 551 us), reads of 16 columns with the next on its way (551 -> 528), a
// relaxed arrival (a cluster-scope release cost 1100 clocks a block), the scales of
// four blocks in one load.  Measured and left: tokens on the
// N side (their scales then come from shared memory, 512 bytes a load: 892 us),
// 16 epilogue warps, two MMAs of half the width, packed additions, a deeper ring.
//
// The small kernel: 1 x 128256 x 4096 92 us (525 MB, 5.7 TB/s; 1002 tiles on 148
// SMs are 6.8 waves, the last one short); 40 x 4096 x 4096 about 6 us on the device.
//
// Every wait is bounded; on a timeout the CTA stops computing, waits (bounded
// again) until the loads that it has issued have landed and its MMAs are done,
// frees TMEM and returns, and the status word says so.
#pragma once

#include "ptx.cuh"

namespace flkl {

// 0 or FLKL_ERR_TIMEOUT, read and cleared by flkl_fp8_device_status.
__device__ int g_fp8_status;

struct Fp8Gemm {
  const float* sa;   // [M][KB]
  const float* sb;   // [ceil(N / 128)][KB]
  const void* bias;  // [N] in D's type, or null
  void* D;           // [M][N]
  int M, N, KB;
  int m_tiles, n_tiles;  // token tiles (k_fp8_pair), weight tiles
  int vec;               // k_fp8_pair: D's rows start on 16-byte boundaries
  int stages;            // k_fp8_skinny: ring depth
  unsigned long long wait_limit_ns;
  int hold;              // Fp8Hold: a role that stops, so that the others' waits run out
  uint32_t hold_at;      // after this many blocks
};
// (kernels with HOLD, which flkl_fp8_wait_selftest launches; in the others not even
// looked at: the comparison per block cost 1 %)
enum Fp8Hold { FP8_HOLD_NONE = 0, FP8_HOLD_MMA = 1, FP8_HOLD_LOAD = 2, FP8_HOLD_LOAD_ODD = 3 };

template <typename T>
__device__ __forceinline__ T fp8_out(float v);
template <>
__device__ __forceinline__ float fp8_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 fp8_out<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// ------------------------------------------------------------------ pairs
// Roles of the 12 warps of each CTA: 0 TMA producer, 1 (which owns the TMEM) and
// 2 the MMA issuers (even CTA), 4 .. 11 the two column halves of the four TMEM
// lane quarters.  CTA r stages tokens [128 r, 128 r + 128) and weight rows
// [BN / 2 r, BN / 2 (r + 1)) of the tile, and holds its tokens' outputs.  Tiles go
// round the pairs, tokens fastest, so that the pairs at work share weight tiles in
// L2.
constexpr int P8_A = 128 * 128;  // bytes of tokens per CTA and stage
constexpr int P8_THREADS = 384;
constexpr int P8_EPI_WARPS = 8;
constexpr int P8_ROW = 256;          // bytes of a row that are written at a time, at most
constexpr int P8_OUT = P8_ROW + 16;  // a lane's shared memory: a copy may start inside a unit

template <int BN>
struct P8 {
  static constexpr int B = BN / 2 * 128;  // bytes of weight rows per CTA and stage
  static constexpr int STAGE = P8_A + B;
  static constexpr int STAGES = BN == 256 ? 4 : 6;  // (256: 6 measured the same)
  static constexpr int BUFS = 512 / BN;  // TMEM buffers
  static constexpr int HN = BN / 2;      // columns of an epilogue warp
  static constexpr int SMEM = STAGES * STAGE + P8_EPI_WARPS * 32 * P8_OUT + 256 + 1024;
};

// A warp's outputs leave through its shared memory, by copies that run while the
// next tile is computed.  (A lane that stored its row itself would touch 32 lines
// an instruction; rows written by whole warps cost more instructions than the
// tile's additions when N is odd.)
//
// Where D's rows start on 16-byte boundaries: BOXES boxes of 32 rows x 128
// bytes, a row's 16-byte units permuted by the row as TMA's 128-byte swizzle has
// them.  Called by all lanes (lane = row); v holds the lane's outputs.
template <typename TO, int BOXES>
__device__ __forceinline__ void p8_write_boxes(const CUtensorMap* map, const Fp8Gemm& g,
                                               uint8_t* buf, const float* v, int row0, int col,
                                               int lane) {
  constexpr int COLS = 128 / static_cast<int>(sizeof(TO));
  if (lane == 0) bulk_wait_read();  // the last copies have left the buffer
  __syncwarp();
#pragma unroll
  for (int q = 0; q < BOXES; ++q) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float* x = v + q * COLS + u * (COLS / 8);
      uint4 w;
      if constexpr (sizeof(TO) == 2)
        w = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                       pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      else
        w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                       __float_as_uint(x[3]));
      *reinterpret_cast<uint4*>(buf + q * 4096 + lane * 128 + ((u ^ (lane & 7)) * 16)) = w;
    }
  }
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
#pragma unroll
    for (int q = 0; q < BOXES; ++q)
      if (col + q * COLS < g.N) tma_store_2d(map, buf + q * 4096, col + q * COLS, row0);
    bulk_commit();
  }
}

// Elsewhere: `count` consecutive outputs of one row (W words at most), v, to d.  The lane puts them
// into its own piece of shared memory, at the place in a 16-byte unit that they
// have in D, and hands the whole units to one copy; what fills no unit is stored
// directly.
template <typename TO, int W>
__device__ __forceinline__ void p8_write_row(TO* d, uint8_t* buf, const float* v, int count) {
  uint32_t w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (sizeof(TO) == 2) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    else w[i] = __float_as_uint(v[i]);
  }
  const uint32_t ph = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(d)) & 15u;
  bulk_wait_read();  // the lane's last copy has left the buffer
  uint32_t* b = reinterpret_cast<uint32_t*>(buf) + (ph >> 2);
  if constexpr (sizeof(TO) == 2) {
    // between two words: each takes a half of its neighbour
    const uint32_t sel = (ph & 2u) ? 0x5432u : 0x7654u;
    b[0] = __byte_perm(0u, w[0], sel);
#pragma unroll
    for (int i = 1; i < W; ++i) b[i] = __byte_perm(w[i - 1], w[i], sel);
    b[W] = w[W - 1] >> 16;  // (counts where the row starts between two words)
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) b[i] = w[i];
  }
  uint8_t* base = reinterpret_cast<uint8_t*>(d) - ph;  // of the unit that d lies in
  const uint32_t end = ph + static_cast<uint32_t>(count) * sizeof(TO);
  const uint32_t first = ph ? 16u : 0u, last = end & ~15u;
  if (last > first) {
    fence_proxy_async_shared();
    bulk_store_1d(base + first, buf + first, last - first);
  }
  bulk_commit();
  auto piece = [&](uint32_t at, uint32_t n) {  // n = 2, 4 or 8 bytes, aligned to n
    if (n == 8) *reinterpret_cast<uint2*>(base + at) = *reinterpret_cast<const uint2*>(buf + at);
    else if (n == 4)
      *reinterpret_cast<uint32_t*>(base + at) = *reinterpret_cast<const uint32_t*>(buf + at);
    else *reinterpret_cast<uint16_t*>(base + at) = *reinterpret_cast<const uint16_t*>(buf + at);
  };
  if (ph != 0 && end >= 16u) {  // up to the first boundary: 2, 4, 8 as they fit
    uint32_t at = ph;
#pragma unroll
    for (uint32_t n = sizeof(TO); n <= 8; n *= 2)
      if (at & n) {
        piece(at, n);
        at += n;
      }
  }
  uint32_t at = end >= 16u ? last : ph;  // from the last boundary (or all of it)
  if (end >= 16u || ph == 0) {
#pragma unroll
    for (uint32_t n = 8; n >= sizeof(TO); n /= 2)
      if (end & n) {
        piece(at, n);
        at += n;
      }
  } else {  // within one unit, from its middle
    for (; at < end; at += sizeof(TO)) piece(at, sizeof(TO));
  }
}

// What the CTAs of a pair tell one another where both have given up.
struct P8Leave {
  uint32_t peer_loads;  // 1 + the stages that the other CTA has filled
  uint32_t landed;      // (odd CTA) the even one has seen both CTAs' loads land
};
// A CTA's loading thread that has given up, `mine` stages filled: returns once both
// CTAs' loads have landed.  These count on the even CTA's barriers, which expect them
// in pairs: the halves that one of the two has not issued are evened out.  If the
// other CTA has not given up, all its loads have been consumed, and so this one's; it
// says nothing, and the wait for its word (which comes within one limit: it waits
// for what this CTA waited for) runs out.  Off the pair's way out on purpose: one look
// at a flag between the last two barriers cost small products 0.8 us.
__device__ __noinline__ void p8_leave(volatile P8Leave* l, uint64_t* full, uint32_t stages,
                                      uint32_t half, uint32_t rank, uint32_t mine,
                                      unsigned long long limit_ns) {
  const uint32_t other_l = mapa_shared(smem_u32(const_cast<P8Leave*>(l)), rank ^ 1u);
  st_shared_cluster_u32(other_l, mine + 1);
  const uint64_t t0 = globaltimer_ns();
  while ((rank == 0 ? l->peer_loads : l->landed) == 0)
    if (globaltimer_ns() - t0 > 3 * limit_ns) return;
  if (rank != 0) return;
  const uint32_t other = l->peer_loads - 1, n = max(mine, other);
  for (uint32_t i = min(mine, other); i < n; ++i) {
    if (mine < other) mbar_arrive_expect_tx(&full[i % stages], half);
    else mbar_complete_tx(&full[i % stages], half);
  }
  ring_land(full, stages, n, limit_ns);
  st_shared_cluster_u32(other_l + 4, 1);
}

template <typename TO, int BN, bool HOLD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P8_THREADS, 1)
    k_fp8_pair(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
               const __grid_constant__ CUtensorMap mapD, const __grid_constant__ Fp8Gemm g) {
  using C = P8<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;  // stage: tokens, then weight rows
  uint8_t* outs = ring + C::STAGES * C::STAGE;
  // even CTA's are used
  uint64_t* full = reinterpret_cast<uint64_t*>(outs + P8_EPI_WARPS * 32 * P8_OUT);
  uint64_t* empty = full + C::STAGES;   // each CTA
  uint64_t* tfull = empty + C::STAGES;  // [BUFS] each CTA
  uint64_t* tempty = tfull + C::BUFS;   // [BUFS] even CTA's are used
  uint64_t* drain = tempty + C::BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile P8Leave* leave = reinterpret_cast<volatile P8Leave*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_cta_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = g.m_tiles * g.n_tiles;  // (below 2^30: checked by the host)

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < C::BUFS; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * P8_EPI_WARPS);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    leave->peer_loads = leave->landed = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapA);
    tma_prefetch_desc(&mapB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{abort_flag, &g_fp8_status, g.wait_limit_ns};

  // registers: 128 (56 + 2 x 224) = 384 x 168, what the block was launched with
  if (warp < 4) {
    reg_dealloc<56>();
    if (warp == 0 && lane == 0) {
      const uint32_t stop =
          HOLD && g.hold == (leader ? FP8_HOLD_LOAD : FP8_HOLD_LOAD_ODD) ? g.hold_at : ~0u;
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        const int m0 = (t % g.m_tiles) * 256 + static_cast<int>(rank) * 128;
        const int n0 = (t / g.m_tiles) * BN + static_cast<int>(rank) * C::HN;
        for (int kb = 0; kb < g.KB; ++kb) {
          if ((HOLD && issued == stop) || !mbar_wait(&empty[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          const uint32_t fbar = mapa_shared(smem_u32(&full[stage]), 0);
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * C::STAGE);
          uint8_t* dst = ring + stage * C::STAGE;
          tma_load_2d_pair(&mapA, fbar, dst, kb * 128, m0);
          tma_load_2d_pair(&mapB, fbar, dst + P8_A, kb * 128, n0);
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every stage this CTA filled has been consumed before it leaves, or has landed
      int s = stage;
      uint32_t ph = phase;
      for (uint32_t i = 0; i < C::STAGES && i < issued; ++i) {
        if (--s < 0) {
          s = C::STAGES - 1;
          ph ^= 1u;
        }
        if (!mbar_wait(&empty[s], ph, wc)) {
          ok = false;
          break;
        }
      }
      if (!ok) p8_leave(leave, full, C::STAGES, C::STAGE, rank, issued, g.wait_limit_ns);
    } else if ((warp == 1 || warp == 2) && lane == 0 && leader) {
      // warp 1 the even blocks, warp 2 the odd: their buffers differ, so nothing
      // orders the two, and the waits of one pass while the other's MMAs run
      constexpr uint32_t idesc = idesc_e4m3_f32(256, BN);
      const uint64_t d0 = smem_desc_sw128(0, 16u, 1024u);
      const uint64_t hi = d0 & ~uint64_t(0xFFFFFFFFu);
      const uint32_t r0 = static_cast<uint32_t>(d0) + ((smem_u32(ring) & 0x3FFFFu) >> 4);
      uint32_t buf = warp - 1;
      long long total =
          static_cast<long long>((tiles - pair + pairs - 1) / pairs) * g.KB;  // of this pair
      if (HOLD && g.hold == FP8_HOLD_MMA && g.hold_at < total) total = g.hold_at;
      int stage = warp - 1;
      uint32_t phase = 0, tphase = 1;
      for (long long it = warp - 1; it < total; it += 2) {
        if (!mbar_wait(&full[stage], phase, wc) || !mbar_wait(&tempty[buf], tphase, wc)) break;
        tc_fence_after();
        const uint32_t a = r0 + stage * (C::STAGE >> 4);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          tc_mma_pair_f8(tmem + buf * BN, hi | (a + 2 * k), hi | (a + (P8_A >> 4) + 2 * k),
                         idesc, k);
        tc_commit_pair(&tfull[buf], 0x3);
        tc_commit_pair(&empty[stage], 0x3);
        buf += 2;
        if (buf >= C::BUFS) {
          buf -= C::BUFS;
          tphase ^= 1u;
        }
        stage += 2;
        if (stage >= C::STAGES) {
          stage -= C::STAGES;
          phase ^= 1u;
        }
      }
      tc_commit_pair(&drain[warp - 1], 0x1);
      mbar_drain_wait(&drain[warp - 1], 0, g.wait_limit_ns);
    }
    __syncwarp();
  } else {
    reg_alloc<224>();
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * C::HN;
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
    const int nb_last = (g.N - 1) / 128;
    // (boxes start on 1024-byte boundaries, a lane's rows on 16-byte ones)
    uint8_t* out = outs + (g.vec ? (warp - 4) * 32 * P8_ROW : ((warp - 4) * 32 + lane) * P8_OUT);
    uint32_t it = 0;
    bool ok = true;
    // a token's scales times its weight block's, four blocks at a time, loaded
    // while the four before them are used (rows and columns past the end take
    // the last one's; not stored)
    const bool vec4 = g.KB % 4 == 0 && (reinterpret_cast<uintptr_t>(g.sa) & 15) == 0 &&
                      (reinterpret_cast<uintptr_t>(g.sb) & 15) == 0;
    const float *pa, *pb;
    int row0, col0;
    auto place = [&](int t) {
      const int nt = t / g.m_tiles, mt = t - nt * g.m_tiles;
      row0 = mt * 256 + static_cast<int>(rank) * 128 + quad * 32;
      col0 = nt * BN + half * C::HN;
      pa = g.sa + static_cast<size_t>(min(row0 + lane, g.M - 1)) * g.KB;
      pb = g.sb + static_cast<size_t>(min(col0 / 128, nb_last)) * g.KB;
    };
    float4 na, nb;
    auto load4 = [&](int kb) {
      if (vec4) {
        na = __ldg(reinterpret_cast<const float4*>(pa + kb));
        nb = __ldg(reinterpret_cast<const float4*>(pb + kb));
      } else {
        const int k1 = min(kb + 1, g.KB - 1), k2 = min(kb + 2, g.KB - 1),
                  k3 = min(kb + 3, g.KB - 1);
        na = make_float4(__ldg(pa + kb), __ldg(pa + k1), __ldg(pa + k2), __ldg(pa + k3));
        nb = make_float4(__ldg(pb + kb), __ldg(pb + k1), __ldg(pb + k2), __ldg(pb + k3));
      }
    };
    if (pair < tiles) {
      place(pair);
      load4(0);
    }
    for (int t = pair; t < tiles && ok; t += pairs) {
      float acc[C::HN];
#pragma unroll
      for (int i = 0; i < C::HN; ++i) acc[i] = 0.f;
      const int out_row = row0, out_col = col0;
      for (int k4 = 0; k4 < g.KB && ok; k4 += 4) {
        const float s4[4] = {na.x * nb.x, na.y * nb.y, na.z * nb.z, na.w * nb.w};
        if (k4 + 4 < g.KB) {
          load4(k4 + 4);
        } else if (t + pairs < tiles) {
          place(t + pairs);
          load4(0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (k4 + j >= g.KB) break;
          const uint32_t buf = it % C::BUFS;
          ok = mbar_wait(&tfull[buf], (it / C::BUFS) & 1, wc);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t r[2][16];  // one piece on its way while the other is added
          tmem_ld16_async(tl + buf * BN, r[0]);
#pragma unroll
          for (int c = 0; c < C::HN / 16; ++c) {
            tmem_wait16(r[c & 1]);
            if (c + 1 < C::HN / 16) {
              tmem_ld16_async(tl + buf * BN + (c + 1) * 16, r[(c + 1) & 1]);
            } else {
              // the buffer is read: the MMAs may have it back
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + buf * 8);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[16 * c + i] =
                  fmaf(__uint_as_float(r[c & 1][i]), s4[j], acc[16 * c + i]);
          }
          ++it;
        }
      }
      const int cols = min(C::HN, g.N - out_col);
      if (ok && out_row < g.M && cols > 0) {
        if (g.bias != nullptr) {
          const TO* b = static_cast<const TO*>(g.bias) + out_col;
#pragma unroll
          for (int i = 0; i < C::HN; ++i)
            if (i < cols) acc[i] += static_cast<float>(b[i]);
        }
        constexpr int E = static_cast<int>(sizeof(TO));
        constexpr int COLS = P8_ROW / E < C::HN ? P8_ROW / E : C::HN;
        TO* d = static_cast<TO*>(g.D) + static_cast<size_t>(out_row + lane) * g.N + out_col;
#pragma unroll
        for (int c = 0; c < C::HN / COLS; ++c) {
          if (c * COLS >= cols) break;
          if (g.vec)
            p8_write_boxes<TO, COLS * E / 128>(&mapD, g, out, acc + c * COLS, out_row,
                                               out_col + c * COLS, lane);
          else if (out_row + lane < g.M)
            p8_write_row<TO, COLS * E / 4>(d + c * COLS, out, acc + c * COLS,
                                           min(COLS, cols - c * COLS));
        }
      }
      __syncwarp();
    }
    bulk_wait();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ----------------------------------------------------------------- skinny
// Warps: 0 TMA producer, 1 TMEM owner and MMA issuer, from 2 on the epilogue, four
// (one per TMEM lane quarter; lane = weight row, column = token) for each group of
// s8_cols columns: with 64 tokens, one group's work on a block would take longer
// than the block's load (113 against 95 us with 128256 x 4096).  The
// tokens' scales stand in shared memory for the whole call, [kb][BN].  CTAs
// take tiles of 128 weight rows in turn; more than one token tile makes one CTA
// (or cluster) per tile.  Where there are too few tiles to
// keep the SMs reading, a cluster of CTAs shares one tile: CTA r takes its
// r-th part of K, and the parts' fp32 sums are added in rank order through the
// cluster's shared memory.
constexpr int S8_W = 128 * 128;  // weight bytes per stage
constexpr int S8_MAX_STAGES = 16;
constexpr int S8_BUFS = 4;       // TMEM buffers of BN columns
constexpr int S8_MAX_CLUSTER = 8;

template <int BN>
__host__ __device__ constexpr int s8_cols() { return BN > 32 ? 32 : BN; }
template <int BN>
__host__ __device__ constexpr int s8_threads() { return 64 + 128 * (BN / s8_cols<BN>()); }
template <int BN>
__host__ __device__ constexpr int s8_stage_bytes() { return S8_W + BN * 128; }
template <int BN>
__host__ __device__ constexpr int s8_tmem_cols() {  // a power of two
  int n = 32;
  while (n < BN * S8_BUFS) n *= 2;
  return n;
}
// Shared memory besides the ring: barriers, the tokens' scales of kbs blocks,
// alignment.
template <int BN>
__host__ __device__ constexpr size_t s8_smem_fixed(size_t kbs) {
  return (2 * S8_MAX_STAGES + 2 * S8_BUFS + 2) * 8 + 16 + kbs * BN * 4 + 1024;
}

template <typename TO, int BN, bool HOLD>
__global__ void __launch_bounds__(s8_threads<BN>(), 1)
    k_fp8_skinny(const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapW,
                 const __grid_constant__ Fp8Gemm g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = g.stages;
  uint8_t* ring = smem;  // stage: weight rows, then tokens
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + S * s8_stage_bytes<BN>());
  uint64_t* empty = full + S8_MAX_STAGES;
  uint64_t* tfull = empty + S8_MAX_STAGES;  // [S8_BUFS]
  uint64_t* tempty = tfull + S8_BUFS;       // [S8_BUFS]
  uint64_t* drain = tempty + S8_BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // [this CTA's kb][BN], 16-byte aligned (the barriers before it are an even number)
  float* xs = reinterpret_cast<float*>(drain + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t cs, rank = cluster_cta_rank();
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
  const int kb0 = static_cast<int>(static_cast<long long>(g.KB) * rank / cs);
  const int kb1 = static_cast<int>(static_cast<long long>(g.KB) * (rank + 1) / cs);
  const int first = blockIdx.x / cs, step = gridDim.x / cs;
  const int tiles = g.n_tiles * g.m_tiles;
  const int m0 = first % g.m_tiles * BN;  // (more than one token tile: one tile per CTA)
  constexpr int kCols = s8_tmem_cols<BN>();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < S8_BUFS; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4 * (BN / s8_cols<BN>()));
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapX);
    tma_prefetch_desc(&mapW);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  if (warp >= 2) {
    for (int i = threadIdx.x - 64; i < (kb1 - kb0) * BN; i += blockDim.x - 64) {
      const int c = i % BN, kb = i / BN;
      xs[i] = m0 + c < g.M ? g.sa[static_cast<size_t>(m0 + c) * g.KB + kb0 + kb] : 0.f;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{abort_flag, &g_fp8_status, g.wait_limit_ns};

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t stop = HOLD && g.hold == FP8_HOLD_LOAD ? g.hold_at : ~0u;
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if ((HOLD && issued == stop) || !mbar_wait(&empty[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          uint8_t* dst = ring + stage * s8_stage_bytes<BN>();
          mbar_arrive_expect_tx(&full[stage], s8_stage_bytes<BN>());
          tma_load_2d(&mapW, &full[stage], dst, kb * 128, t / g.m_tiles * 128);
          tma_load_2d(&mapX, &full[stage], dst + S8_W, kb * 128, m0);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every stage has been consumed, or has landed, before the CTA goes on
      int s = stage;
      uint32_t ph = phase;
      for (uint32_t i = 0; i < S && i < issued; ++i) {
        if (--s < 0) {
          s = S - 1;
          ph ^= 1u;
        }
        if (!mbar_wait(&empty[s], ph, wc)) break;
      }
      if (*abort_flag) ring_land(full, S, issued, g.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(128, BN);
      const uint64_t d0 = smem_desc_sw128(0, 16u, 1024u);
      const uint32_t hi = static_cast<uint32_t>(d0 >> 32);
      const uint32_t r0 = static_cast<uint32_t>(d0) + ((smem_u32(ring) & 0x3FFFFu) >> 4);
      const uint32_t stop = HOLD && g.hold == FP8_HOLD_MMA ? g.hold_at : ~0u;
      int stage = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const uint32_t buf = it % S8_BUFS;
          if ((HOLD && it == stop) || !mbar_wait(&tempty[buf], ((it / S8_BUFS) & 1) ^ 1u, wc) ||
              !mbar_wait(&full[stage], phase, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w = r0 + stage * (s8_stage_bytes<BN>() >> 4);
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k)
            tc_mma_f8(tmem + buf * BN, (static_cast<uint64_t>(hi) << 32) | (w + 2 * k),
                      (static_cast<uint64_t>(hi) << 32) | (w + (S8_W >> 4) + 2 * k), idesc, k);
          tc_commit(&empty[stage]);
          tc_commit(&tfull[buf]);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      tc_commit(drain);
      mbar_drain_wait(drain, 0, g.wait_limit_ns);
    }
    __syncwarp();
  }
  bool ok = true;
  constexpr int CN = s8_cols<BN>();
  uint64_t acc[CN / 2];
  const int quad = warp & 3, col0 = (warp - 2) / 4 * CN;
  if (warp >= 2) {
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    uint32_t it = 0;
    for (int t = first; t < tiles && ok; t += step) {
      const float* sb = g.sb + static_cast<size_t>(t / g.m_tiles) * g.KB;
#pragma unroll
      for (int i = 0; i < CN / 2; ++i) acc[i] = 0;
      float s_next = __ldg(sb + kb0);
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t buf = it % S8_BUFS;
        const uint64_t s = f2_pack(s_next, s_next);
        if (kb + 1 < kb1) s_next = __ldg(sb + kb + 1);
        ok = mbar_wait(&tfull[buf], (it / S8_BUFS) & 1, wc);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const ulonglong2* x2 = reinterpret_cast<const ulonglong2*>(xs + (kb - kb0) * BN + col0);
        uint32_t r[2][16];
        tmem_ld16_async(tl + buf * BN, r[0]);
#pragma unroll
        for (int c = 0; c < CN / 16; ++c) {
          tmem_wait16(r[c & 1]);
          if (c + 1 < CN / 16) {
            tmem_ld16_async(tl + buf * BN + (c + 1) * 16, r[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const ulonglong2 x = x2[c * 4 + i];
            const uint32_t* q = &r[c & 1][4 * i];
            acc[8 * c + 2 * i] =
                f2_fma(f2_pack(__uint_as_float(q[0]), __uint_as_float(q[1])),
                       f2_mul(x.x, s), acc[8 * c + 2 * i]);
            acc[8 * c + 2 * i + 1] =
                f2_fma(f2_pack(__uint_as_float(q[2]), __uint_as_float(q[3])),
                       f2_mul(x.y, s), acc[8 * c + 2 * i + 1]);
          }
        }
      }
      if (cs == 1 && ok) {
        const int n = t / g.m_tiles * 128 + quad * 32 + lane;
        if (n < g.N) {
          const float b =
              g.bias != nullptr ? static_cast<float>(static_cast<const TO*>(g.bias)[n]) : 0.f;
          const int m = m0 + col0;
          TO* d = static_cast<TO*>(g.D) + static_cast<size_t>(m) * g.N + n;
#pragma unroll
          for (int i = 0; i < CN / 2; ++i) {
            const float2 p = f2_unpack(acc[i]);
            if (m + 2 * i < g.M) d[static_cast<size_t>(2 * i) * g.N] = fp8_out<TO>(p.x + b);
            if (m + 2 * i + 1 < g.M) d[static_cast<size_t>(2 * i + 1) * g.N] = fp8_out<TO>(p.y + b);
          }
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  if (cs > 1) {
    // the ring is free (every MMA has read it): [BN][128] sums of this part
    float* part = reinterpret_cast<float*>(ring);
    if (warp >= 2) {
#pragma unroll
      for (int i = 0; i < CN / 2; ++i) {
        const float2 p = f2_unpack(acc[i]);
        part[(col0 + 2 * i) * 128 + quad * 32 + lane] = p.x;
        part[(col0 + 2 * i + 1) * 128 + quad * 32 + lane] = p.y;
      }
    }
    cluster_sync();
    // CTA r adds and stores tokens r, r + cs, ... of each group
    if (warp >= 2 && ok) {
      const int l = quad * 32 + lane, n = first / g.m_tiles * 128 + l;
      if (n < g.N) {
        const float b =
            g.bias != nullptr ? static_cast<float>(static_cast<const TO*>(g.bias)[n]) : 0.f;
        // 4 tokens at a time: their loads from the other CTAs fly together
        for (int c0 = static_cast<int>(rank) + col0; c0 < col0 + CN && m0 + c0 < g.M;
             c0 += 4 * static_cast<int>(cs)) {
          float p[4][S8_MAX_CLUSTER];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = c0 + q * static_cast<int>(cs);
            const uint32_t at = smem_u32(part + (c < col0 + CN ? c : c0) * 128 + l);
#pragma unroll
            for (uint32_t r = 0; r < S8_MAX_CLUSTER; ++r) {
              p[q][r] = 0.f;
              if (r < cs)
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(p[q][r])
                             : "r"(mapa_shared(at, r)));
            }
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = c0 + q * static_cast<int>(cs);
            float v = p[q][0];
#pragma unroll
            for (int r = 1; r < S8_MAX_CLUSTER; ++r) v += p[q][r];
            if (c < col0 + CN && m0 + c < g.M)
              static_cast<TO*>(g.D)[static_cast<size_t>(m0 + c) * g.N + n] = fp8_out<TO>(v + b);
          }
        }
      }
    }
    cluster_sync();  // nobody leaves while its part is read
  }
}

}  // namespace flkl
