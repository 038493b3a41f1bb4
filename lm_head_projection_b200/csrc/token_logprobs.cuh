// Log-probabilities of given tokens, entropy and best alternatives of rows of
// logits, in one pass over them, and the gradient in a second.
//
//   u = z / T,  m = max z,  t = (z - m) log2(e) / T,  S = sum 2^t,  A = sum 2^t t
//   logp    = (z_y - m) / T - ln S          (y the given token)
//   entropy = ln S - A ln2 / S              (= - sum p ln p)
//   lse     = m / T + ln S
//   top     = the k largest z, ties to the lower index, as (z - m) / T - ln S
//
// m is a running maximum: S and A are carried to a new one by S' = S 2^d,
// A' = (A + d S) 2^d with d = (m - m') log2(e) / T.  z - m is formed before it is
// scaled, so that a row of the type's lowest values stays finite, and t is cut
// at -200, below which 2^t is 0 in fp32 (0 times -infinity would not be).
//
// The k best: a thread compares the largest of each of its vectors with a
// bound that at least k of the row's logits reach; what passes is appended to
// a list in shared memory, as a 64-bit key (ordered value, then the lower
// index first), and the list is cut to its k best (the bound is then the k-th)
// as it grows.  The first bound is the k-th largest of a warp's 32 lane maxima.
// A random row appends a few hundred of its 128k logits; a tile that overflows
// the list (a row of equal logits, or one that ascends) is appended in rounds
// of one vector per thread, each cut before the next.
#pragma once

#include "ptx.cuh"

namespace flkl {

constexpr int LP_NT = 256;          // threads per CTA
constexpr int LP_U = 4;             // 16-byte vectors per thread and tile
constexpr int LP_MAX_K = 32;        // alternatives at most (one per lane)
constexpr int LP_TRIG = 64;         // appended keys above k that make a cut worth it
constexpr int LP_CAP = LP_NT * 8 + LP_MAX_K + LP_TRIG + 32;  // keys the list holds

struct LpFwdArgs {
  const void* logits;
  long long ld;  // elements between rows
  const int64_t* target;  // or null
  long long ignore_index;
  int rows, V;
  float temperature;
  int k;
  float* logp;      // [rows] (with target)
  float* entropy;   // [rows]
  float* lse;       // [rows]
  float2* stats;    // [rows] (m, ln S), read by the backward pass
  float* top_logp;  // [rows][k]
  int64_t* top_ids; // [rows][k]
};

// Value -> key order: -0 equals +0, NaN is above everything (as in torch's sort).
__device__ __forceinline__ uint32_t lp_ord(float z) {
  if (z != z) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(z + 0.f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float lp_unord(uint32_t o) {
  return __uint_as_float((o >> 31) ? (o ^ 0x80000000u) : ~o);
}
__device__ __forceinline__ unsigned long long lp_key(float z, uint32_t idx) {
  return (static_cast<unsigned long long>(lp_ord(z)) << 32) | (0xFFFFFFFFu - idx);
}

// max that keeps NaN
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float t) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

template <typename T>
struct LpVec;
template <>
struct LpVec<__nv_bfloat16> {
  static constexpr int E = 8;
  __device__ static uint4 empty() { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
  __device__ static void unpack(const uint4& u, float (&f)[8]) { unpack8_bf16(u, f); }
  __device__ static float max(const uint4& u) {
    uint32_t a, b, c;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(u.x), "r"(u.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(u.z), "r"(u.w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return fmax_nan(bf16lo(c), bf16hi(c));
  }
  __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct LpVec<float> {
  static constexpr int E = 4;
  __device__ static uint4 empty() { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }
  __device__ static void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  __device__ static float max(const uint4& u) {
    return fmax_nan(fmax_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                    fmax_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  __device__ static float one(const float* p) { return *p; }
};

// Running softmax sums of one thread (base 2; c = log2(e) / T).
struct LpSums {
  float m, S, A;
  __device__ void init() { m = -INFINITY; S = A = 0.f; }
  __device__ void raise(float nm, float c) {  // nm > m
    const float d = fmaxf((m - nm) * c, -200.f);
    const float f = ex2(d);
    A = fmaf(d, S, A) * f;
    S *= f;
    m = nm;
  }
  __device__ void add(float z, float c) {  // z <= m, or NaN
    const float t = fmax_nan((z - m) * c, -200.f);
    const float e = ex2(t);
    S += e;
    A = fmaf(e, t, A);
  }
  __device__ void merge(float om, float oS, float oA, float c) {
    if (om > m) raise(om, c);
    if (om > -INFINITY) {
      const float d = fmaxf((om - m) * c, -200.f);
      const float f = ex2(d);
      A = fmaf(fmaf(d, oS, oA), f, A);
      S = fmaf(oS, f, S);
    } else if (oS != oS) {
      S = oS;  // a NaN among -infinities
    }
  }
};

__device__ __forceinline__ unsigned long long shfl_xor64(unsigned long long v, int o) {
  return __shfl_xor_sync(0xffffffffu, v, o);
}
// Keys of a warp into descending order (lane 0 the largest): bitonic sort.
template <typename K>
__device__ __forceinline__ K warp_sort_desc(K v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o >= 1; o >>= 1) {
      const K w = __shfl_xor_sync(0xffffffffu, v, o);
      // a lane keeps the larger when it is the lower of its pair in a
      // descending run (bit `size` of the lane clear)
      const bool larger = ((lane & o) == 0) == ((lane & size) == 0 || size == 32);
      v = larger ? (v > w ? v : w) : (v > w ? w : v);
    }
  return v;
}
// The 32 largest of two descending lists, descending (v this lane's entry of
// one, w_rev the other's entry 31 - lane): their elementwise maximum is
// bitonic, five steps sort it.
__device__ __forceinline__ unsigned long long warp_merge_desc(unsigned long long v,
                                                              unsigned long long w_rev, int lane) {
  v = v > w_rev ? v : w_rev;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const unsigned long long w = shfl_xor64(v, o);
    v = (lane & o) == 0 ? (v > w ? v : w) : (v > w ? w : v);
  }
  return v;
}

struct LpTopSmem {
  unsigned long long buf[LP_CAP];
  unsigned long long part[LP_NT / 32][32];
  int cnt;
  uint32_t bound[LP_NT / 32];
};

// Cuts the list to its k best, buf[0..k) descending (0 where there are fewer).
// Called by all threads; a barrier before it makes the appended keys visible.
// Ends with a barrier.
__device__ __forceinline__ void lp_cut(LpTopSmem& s, int c, int k) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long best = 0;
  for (int b = warp * 32; b < c; b += LP_NT) {
    unsigned long long v = b + lane < c ? s.buf[b + lane] : 0ull;
    v = warp_sort_desc(v, lane);
    best = warp_merge_desc(best, __shfl_sync(0xffffffffu, v, 31 - lane), lane);
  }
  s.part[warp][lane] = best;
  __syncthreads();
  // the warps' lists pairwise
#pragma unroll
  for (int n = LP_NT / 64; n >= 1; n >>= 1) {
    if (warp < n) {
      best = warp_merge_desc(best, s.part[warp + n][31 - lane], lane);
      s.part[warp][lane] = best;
    }
    __syncthreads();
  }
  if (warp == 0 && lane < k) s.buf[lane] = best;
  if (threadIdx.x == 0) s.cnt = k;
  __syncthreads();
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(LP_NT) k_token_logprobs(const LpFwdArgs a) {
  using VT = LpVec<T>;
  constexpr int E = VT::E;
  __shared__ float3 red[LP_NT / 32];
  __shared__ typename std::conditional<TOP, LpTopSmem, int>::type top_mem;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x;
  const long long y = a.target != nullptr ? a.target[row] : -1;
  if (a.target != nullptr && y == a.ignore_index) {  // the whole CTA
    if (tid == 0) {
      a.logp[row] = 0.f;
      a.entropy[row] = 0.f;
      a.lse[row] = 0.f;
      a.stats[row] = make_float2(-INFINITY, 0.f);
    }
    if (TOP && tid < a.k) {
      a.top_logp[static_cast<size_t>(row) * a.k + tid] = 0.f;
      a.top_ids[static_cast<size_t>(row) * a.k + tid] = -1;
    }
    return;
  }
  const T* z = static_cast<const T*>(a.logits) + static_cast<long long>(row) * a.ld;
  const float c = 1.4426950408889634f / a.temperature;
  // the row as [head][vectors of 16 aligned bytes][tail]
  const int head = min(a.V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) /
                                static_cast<int>(sizeof(T)));
  const int nvec = (a.V - head) / E;
  const int tail0 = head + nvec * E;
  const uint4* zv = reinterpret_cast<const uint4*>(z + head);

  LpSums sum;
  sum.init();
  float bound = -INFINITY;      // what a vector's largest has to reach to be looked at
  uint32_t bound_ord = 0;       // keys from here on are appended
  int count = 0;                // keys in the list when the tile begins (uniform)
  if constexpr (TOP) {
    if (tid == 0) top_mem.cnt = 0;
  }
  // head and tail: at most 2 (E - 1) logits, one per thread
  const int extra = head + (a.V - tail0);
  float xz = -INFINITY;
  int xi = -1;
  if (tid < extra) {
    xi = tid < head ? tid : tail0 + tid - head;
    xz = VT::one(z + xi);
    if (xz > sum.m) sum.raise(xz, c);
    if (sum.m > -INFINITY) sum.add(xz, c);
    else if (xz != xz) sum.S = xz;
  }

  for (int t0 = 0; t0 < nvec || t0 == 0; t0 += LP_NT * LP_U) {
    uint4 raw[LP_U];
#pragma unroll
    for (int u = 0; u < LP_U; ++u) {
      const int i = t0 + u * LP_NT + tid;
      raw[u] = i < nvec ? ld_nc_v4(zv + i) : VT::empty();
    }
    float vm[LP_U], tm = -INFINITY;
#pragma unroll
    for (int u = 0; u < LP_U; ++u) {
      vm[u] = VT::max(raw[u]);
      tm = fmax_nan(tm, vm[u]);
    }
    if (tm > sum.m) sum.raise(tm, c);
    if (tm != tm) sum.S = tm;
    if (sum.m > -INFINITY) {
#pragma unroll
      for (int u = 0; u < LP_U; ++u) {
        float f[E];
        VT::unpack(raw[u], f);
#pragma unroll
        for (int i = 0; i < E; ++i) sum.add(f[i], c);
      }
    }
    if constexpr (TOP) {
      const bool first = t0 == 0;
      if (first) {
        // a bound that at least k logits of the tile reach
        uint32_t o = warp_sort_desc(lp_ord(tm), lane);
        o = __shfl_sync(0xffffffffu, o, a.k - 1);
        if (lane == 0) top_mem.bound[warp] = o;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < LP_NT / 32; ++w) bound_ord = max(bound_ord, top_mem.bound[w]);
        bound = bound_ord == 0xFFFFFFFFu ? INFINITY : lp_unord(bound_ord);
      }
      auto append = [&](float f, int idx) {
        if (lp_ord(f) < bound_ord) return false;
        const int p = atomicAdd(&top_mem.cnt, 1);
        if (p < LP_CAP) top_mem.buf[p] = lp_key(f, static_cast<uint32_t>(idx));
        return true;
      };
      auto append_vec = [&](int u) {
        const int i0 = t0 + u * LP_NT + tid;
        bool any = false;
        if (!(vm[u] < bound) && i0 < nvec) {
          float f[E];
          VT::unpack(raw[u], f);
#pragma unroll
          for (int i = 0; i < E; ++i) any |= append(f[i], head + i0 * E + i);
        }
        return any;
      };
      // after the list is cut: the bound is its k-th key, later equals lose
      auto lower = [&]() {
        const unsigned long long kth = top_mem.buf[a.k - 1];
        if (kth != 0) {
          const uint32_t o = static_cast<uint32_t>(kth >> 32);
          bound = o == 0xFFFFFFFFu ? INFINITY : lp_unord(o);
          bound_ord = o == 0xFFFFFFFFu ? o : o + 1;
        }
      };
      bool any = false;
#pragma unroll
      for (int u = 0; u < LP_U; ++u) any |= append_vec(u);
      if (first && xi >= 0) any |= append(xz, xi);
      if (__syncthreads_or(any)) {
        int n = top_mem.cnt;
        __syncthreads();
        if (n > LP_CAP) {
          // too many for the list: one vector per thread at a time
          if (tid == 0) top_mem.cnt = count;
          __syncthreads();
          for (int u = 0; u < LP_U; ++u) {
            append_vec(u);
            if (u == 0 && first && xi >= 0) append(xz, xi);
            __syncthreads();
            n = top_mem.cnt;
            __syncthreads();
            lp_cut(top_mem, n, a.k);
            lower();
            __syncthreads();
          }
          count = a.k;
        } else if (first || n > a.k + LP_TRIG) {
          lp_cut(top_mem, n, a.k);
          lower();
          __syncthreads();
          count = a.k;
        } else {
          count = n;
        }
      }
    }
  }

  // sums of the CTA, warps in order
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, sum.m, o);
    const float oS = __shfl_xor_sync(0xffffffffu, sum.S, o);
    const float oA = __shfl_xor_sync(0xffffffffu, sum.A, o);
    sum.merge(om, oS, oA, c);
  }
  if (lane == 0) red[warp] = make_float3(sum.m, sum.S, sum.A);
  __syncthreads();
  if constexpr (TOP) lp_cut(top_mem, top_mem.cnt, a.k);
  if (warp != 0) return;
  sum.init();
#pragma unroll
  for (int w = 0; w < LP_NT / 32; ++w) sum.merge(red[w].x, red[w].y, red[w].z, c);
  // a row that holds no token: logp -inf, entropy 0
  const bool none = sum.m == -INFINITY && sum.S == 0.f;
  const float lnS = none ? 0.f : logf(sum.S);
  if (lane == 0) {
    a.stats[row] = make_float2(sum.m, lnS);
    a.entropy[row] = none ? 0.f : lnS - sum.A / sum.S * 0.693147180559945309f;
    a.lse[row] = none ? -INFINITY : sum.m / a.temperature + lnS;
    if (a.logp != nullptr) {
      float lp = 0.f;
      if (y >= 0 && y < a.V)
        lp = none ? -INFINITY : (VT::one(z + y) - sum.m) / a.temperature - lnS;
      a.logp[row] = lp;
    }
  }
  if constexpr (TOP) {
    if (lane < a.k) {
      const unsigned long long key = top_mem.buf[lane];
      const uint32_t idx = 0xFFFFFFFFu - static_cast<uint32_t>(key);
      const size_t o = static_cast<size_t>(row) * a.k + lane;
      a.top_ids[o] = idx;
      a.top_logp[o] = none ? -INFINITY : (VT::one(z + idx) - sum.m) / a.temperature - lnS;
    }
  }
}

// --------------------------------------------------------------- gradient
//   d/dz_v = [ gl 1(v = y) + sum_j gt_j 1(v = i_j)
//              - (gl + sum_j gt_j) p_v - ge p_v (ln p_v + H) ] / T
// One pass: read z, write dz; the given token and the alternatives (at most
// k + 1 entries of a row) are written afterwards by one thread each, with all
// that falls on the entry in one fp32 sum.
struct LpBwdArgs {
  const void* logits;
  long long ld;
  const int64_t* target;
  long long ignore_index;
  int rows, V;
  float temperature;
  int k;
  const float2* stats;
  const float* entropy;
  const int64_t* top_ids;
  const float* dlogp;     // [rows] or null
  const float* dentropy;  // [rows] or null
  const float* dtop;      // [rows][k] or null
  void* dlogits;
  long long dld;
};

constexpr int LPB_NT = 256;
constexpr int LPB_CHUNK = LPB_NT * 8 * 8;  // logits of a row per CTA

template <typename T>
__global__ void __launch_bounds__(LPB_NT) k_token_logprobs_bwd(const LpBwdArgs a) {
  using VT = LpVec<T>;
  constexpr int E = VT::E;
  const int tid = threadIdx.x;
  const int chunks = (a.V + LPB_CHUNK - 1) / LPB_CHUNK;
  const int row = static_cast<int>(blockIdx.x / chunks);
  const int lo = static_cast<int>(blockIdx.x % chunks) * LPB_CHUNK;
  const int hi = min(a.V, lo + LPB_CHUNK);
  const T* z = static_cast<const T*>(a.logits) + static_cast<long long>(row) * a.ld;
  T* dz = static_cast<T*>(a.dlogits) + static_cast<long long>(row) * a.dld;
  long long y = a.target != nullptr ? a.target[row] : -1;
  const float2 st = a.stats[row];
  // dropped rows and rows without a token: 0
  const bool none = (a.target != nullptr && y == a.ignore_index) ||
                    (st.x == -INFINITY && st.y == 0.f);
  if (y >= a.V) y = -1;
  const float invT = 1.f / a.temperature;
  const float c = 1.4426950408889634f * invT;
  const float m = st.x, l2 = st.y * 1.4426950408889634f;
  const float gl = (a.dlogp != nullptr && y >= 0) ? a.dlogp[row] : 0.f;
  const float ge = a.dentropy != nullptr ? a.dentropy[row] : 0.f;
  float gsum = gl;
  if (a.dtop != nullptr)
    for (int j = 0; j < a.k; ++j) gsum += a.dtop[static_cast<size_t>(row) * a.k + j];
  // dz = p (alpha + beta log2 p)
  const float alpha = -(gsum + ge * a.entropy[row]) * invT;
  const float beta = -ge * 0.693147180559945309f * invT;
  auto grad = [&](float zz) {
    const float lp2 = fmax_nan(fmaf(zz - m, c, -l2), -200.f);
    return ex2(lp2) * fmaf(beta, lp2, alpha);
  };
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(z + lo) & 15);
  const bool same = shift == static_cast<int>(reinterpret_cast<uintptr_t>(dz + lo) & 15);
  // [head][aligned vectors][tail]; all head where the two rows' alignments differ
  const int head =
      same ? min(hi - lo, ((16 - shift) & 15) / static_cast<int>(sizeof(T))) : hi - lo;
  const int nvec = (hi - lo - head) / E;
  auto store1 = [&](int i, float g) {
    if constexpr (sizeof(T) == 2) dz[i] = __float2bfloat16_rn(g);
    else dz[i] = g;
  };
  for (int i = lo + tid; i < lo + head; i += LPB_NT)
    store1(i, none ? 0.f : grad(VT::one(z + i)));
  for (int i = lo + head + nvec * E + tid; i < hi; i += LPB_NT)
    store1(i, none ? 0.f : grad(VT::one(z + i)));
  const uint4* zv = reinterpret_cast<const uint4*>(z + lo + head);
  uint4* dv = reinterpret_cast<uint4*>(dz + lo + head);
#pragma unroll 4
  for (int i = tid; i < nvec; i += LPB_NT) {
    float f[E];
    uint4 o = make_uint4(0, 0, 0, 0);
    if (!none) {
      VT::unpack(ld_nc_v4(zv + i), f);
#pragma unroll
      for (int j = 0; j < E; ++j) f[j] = grad(f[j]);
      if constexpr (sizeof(T) == 2) {
        o.x = pack_bf16x2(f[0], f[1]);
        o.y = pack_bf16x2(f[2], f[3]);
        o.z = pack_bf16x2(f[4], f[5]);
        o.w = pack_bf16x2(f[6], f[7]);
      } else {
        o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                       __float_as_uint(f[3]));
      }
    }
    dv[i] = o;
  }
  if (none) return;
  __syncthreads();
  // entry tid of [token, alternatives]: the whole gradient of that logit
  const int64_t* ids = a.dtop != nullptr ? a.top_ids + static_cast<size_t>(row) * a.k : nullptr;
  const float* gt = a.dtop != nullptr ? a.dtop + static_cast<size_t>(row) * a.k : nullptr;
  const int n = ids != nullptr ? a.k : 0;
  if (tid <= n) {
    const long long v = tid == 0 ? y : ids[tid - 1];
    if (v >= lo && v < hi) {
      float g = v == y ? gl : 0.f;
      for (int j = 0; j < n; ++j)
        if (ids[j] == v) g += gt[j];
      store1(static_cast<int>(v), fmaf(g, invT, grad(VT::one(z + v))));
    }
  }
}

}  // namespace flkl
