// sq_lora.cu -- low-rank adapters of many requests at once, beside a shared
// projection (sm_100a):
//
//   y[t] = base[t] + scale_a B_a (A_a x_t),   a = ids[t],
//
// A_a [rank_a][K], B_a [N][rank_a] in binary32, binary16 or bfloat16, x, base and
// y in binary32.  Products and sums keep a binary32 sum's accuracy, on the tensor
// cores (the paragraph on precision below says how).
//
// Few tokens (a decode step): one launch.  A cluster of 8 or 16 CTAs serves up
// to kGroup tokens that share an adapter (found from the ids by ballots): each CTA
// forms its channels' part of v = A x, the parts meet over distributed shared
// memory, and each CTA adds its columns of B v.  Both products run on the tensor
// cores with the weights as MMA rows and the tokens as columns, each weight word
// loaded once, from memory into operand registers.  The adapter is read once, by
// the cluster, and there is no second launch to wait for.  Bound by latency (two
// chains of loads): 5.8 us for one token (rank 16, 4096 -> 4096), 23 us for 64 tokens
// over 32 adapters of rank up to 64, 4096 -> 12288 (42 MB).
//
// More tokens: the tokens are sorted by adapter, and two tensor-core kernels
// (mma.sync) follow.  Shrink: 16 tokens of one adapter per CTA (per cluster, where
// that leaves SMs idle), its warps split rank and channels; the parts are summed in
// a fixed order.  Expand: a tile of 64 tokens and a span of columns per CTA; a warp
// holds 16 tokens' v as MMA operands and streams over the columns.  By their bytes
// both are bound by memory (x once; base and y once: the products have a few
// dozen terms per byte); measured, 2048 tokens, rank 64, 4096 -> 14336 in binary16
// take 92 us (44 at a copy's rate): sort and shrink 35 to 40 us, chains of loads, the
// expand kernel the rest, of which 48 us go to copying base and y alone.
// Precision: bfloat16 weights are taken as they are, and x, cut by truncation into
// three bfloat16 parts that sum to it exactly (8 significand bits each).  binary16 and
// binary32 operands of the shrink and decode kernels are cut into tf32 parts (11 bits
// rounded, and the rest, read in 11 bits: 2^-23; a binary16 weight is one part); of two cut
// operands the product of the two rests, below 2^-22, is left out: at most 2^-21 of a product in all.
// The expand kernel does the same for binary32 weights; a binary16 weight it takes as it is, and v,
// scaled by a power of two per token into binary16's range, as two binary16 parts (rounded: 2^-23
// of a value, or 2^-38 of the token's largest where that is more).  The products of parts are
// summed by the tensor cores over at most 32 channels (or of the rank), those sums in binary32 with
// rounding (add_step).  Measured against 64 bits, rms of the error over that of B A x: 1.6 to 2.2e-7
// at K = 4096, 2.3 to 3.4e-7 at 14336 (rank 128 and 256), 5.9 to 6.1e-7 at 65536.
// binary32 weights take the kernels to the limit of 128 registers: shrink and expand spill
// 32 to 72 bytes a thread.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "sq_grouped.cuh"
#include "sq_internal.h"

namespace cg = cooperative_groups;

namespace sq {
namespace {

constexpr int kCluster = 8;        // CTAs per cluster (the portable size)
constexpr int kDecodeCluster = 16; // of the decode kernel
constexpr int kDecodeThreads = 256;
constexpr int kGroup = 8;          // tokens per cluster of the decode kernel (MMA columns)
constexpr int kTile = 64;          // tokens per tile of the expand kernel

struct Params {
  const void* A;
  const void* B;
  const float* scale;
  const int32_t* rank;
  int S, R, K, N;
  const float* x;
  int M;
  const int32_t* ids;
  const float* base;
  int64_t ldb;
  float* y;
  int64_t ldy;
  const int32_t* offsets;
  const int32_t* order;
  float* v;   // [M][Rp], in place order
  int Rp;     // R rounded up to 32
  int32_t* status;
  int cluster;  // CTAs per cluster
  int span;   // expand: columns per CTA
  int self_sort;  // the shrink kernel sorts the ids
  int tiles;  // expand: CTAs along the tiles (the rest copy rows without adapter)
};

__device__ __forceinline__ int adapter_rank(const Params& p, int a) {
  return p.rank ? min(max(__ldg(p.rank + a), 0), p.R) : p.R;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A step's sums into the running ones.  The tensor cores add with truncation, always
// towards zero, so an accumulator that stays there drifts with the number of steps
// (rank 128: 1.3e-5 of the result at K = 14336, rank 256: 1.2e-4 at 65536); sums of one
// step, added here with rounding, do not (the rms of the error is that of a binary32 sum).
__device__ __forceinline__ void add_step(float (&acc)[4], const float (&t)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] += t[i];
}
// low: the products of the operands' lesser parts, kept from the larger sum.
__device__ __forceinline__ void add_step(float (&acc)[4], const float (&t)[4], const float (&low)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] += t[i] + low[i];
}

// One k8 step on tf32 operands (the tensor cores read the upper 19 bits of each).
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Upper halves of two binary32 values as a pair of bfloat16 (first in the low half).
__device__ __forceinline__ uint32_t upper_pair(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float below_upper(float v) { return v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }

// Eight values as three bfloat16 parts (by truncation; exact), four pairs each.
__device__ __forceinline__ void cut8(float (&v)[8], uint32_t (&o)[3][4]) {
#pragma unroll
  for (int s = 0; s < 3; ++s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[s][i] = upper_pair(v[2 * i], v[2 * i + 1]);
    if (s < 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = below_upper(v[i]);
    }
  }
}

// Which products a weight type takes: bfloat16 ones as it is, tf32 ones with a binary16
// weight as one part, or with a binary32 weight cut in two.
template <class W>
constexpr bool kBf16 = std::is_same<W, __nv_bfloat16>::value;
template <class W>
constexpr bool kCutWeight = std::is_same<W, float>::value;

// Eight neighbouring elements as they lie in memory, under a mask (all ones or
// zero: what is masked may hold anything, NaN included).  The
// loads of a step are issued together, without branches; a row without vector
// alignment is gathered element by element instead.
template <class T>
struct Raw8 {
  static constexpr int kWords = (int)sizeof(T) * 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
  // elements i0 .. i0 + 7 of a row of `len`, 0 past its end
  __device__ __forceinline__ void gather(const T* row, int i0, int len) {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i0 + i < len ? row[i0 + i] : T(0.0f);
    __builtin_memcpy(w, v, sizeof(v));
  }
  // elements from n on become zero
  __device__ __forceinline__ void keep(int n) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int e = i * 4 / (int)sizeof(T);  // first element of the word
      uint32_t m = e < n ? 0xffffffffu : 0u;
      if (sizeof(T) == 2 && e + 1 >= n) m &= 0x0000ffffu;
      w[i] &= m;
    }
  }
  __device__ __forceinline__ void floats(float (&v)[8]) const {
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
};
// Elements i0 .. i0 + 7 of row `row` of a matrix of rows `ld` apart, `len` long; zero
// unless `live`.  base points at a readable row in any case.  In two halves, so that
// a load can be issued long before its use.
template <bool VEC, class T>
__device__ __forceinline__ void issue_masked(Raw8<T>& r, const T* row, int i0, int len, bool live) {
  if constexpr (VEC) r.load(row + (i0 < len ? i0 : 0));  // a vector lies inside the row or outside it, or crosses `len`
  else r.gather(row, i0, live ? len : 0);
}
template <bool VEC, class T>
__device__ __forceinline__ void finish_masked(Raw8<T>& r, int i0, int len, bool live) {
  if constexpr (VEC) r.keep(live ? len - i0 : 0);
}
template <bool VEC, class T>
__device__ __forceinline__ void load_masked(Raw8<T>& r, const T* row, int i0, int len, bool live) {
  issue_masked<VEC>(r, row, i0, len, live);
  finish_masked<VEC>(r, i0, len, live);
}

// The MMA's k index is free as long as both operands agree: over 32 channels lane
// tid4 holds channels 8 tid4 .. 8 tid4 + 7, the first four in one k16 step and the
// last four in the next, so that every load is 16 bytes or more of a row.
// ---- few tokens: one launch -------------------------------------------------------
// Weights are the MMA's rows (16 of A's rank, or 16 columns of y), the group's
// tokens its eight columns.  A lane holds the activations (then v) of token gid.
// Each weight word is loaded once, from memory straight into operand registers.

// acc += A x over one 32-channel step: rows w0 (gid) and w1 (gid + 8), columns'
// operand parts x.
template <class W>
struct Columns;
template <>
struct Columns<__nv_bfloat16> {
  uint32_t p[3][4];
  __device__ __forceinline__ void set(float (&v)[8]) { cut8(v, p); }
  __device__ __forceinline__ void mma(float (&acc)[4], const Raw8<__nv_bfloat16>& w0,
                                      const Raw8<__nv_bfloat16>& w1) const {
    float t[4] = {}, low[4] = {};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t a[4] = {w0.w[2 * q], w1.w[2 * q], w0.w[2 * q + 1], w1.w[2 * q + 1]};
      mma_bf16(low, a, p[2][2 * q], p[2][2 * q + 1]);
      mma_bf16(low, a, p[1][2 * q], p[1][2 * q + 1]);
      mma_bf16(t, a, p[0][2 * q], p[0][2 * q + 1]);
    }
    add_step(acc, t, low);
  }
};
template <class W>
struct Columns32 {  // tf32 parts
  uint32_t h[8], l[8];
  __device__ __forceinline__ void set(float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cut_tf32(v[i], h[i], l[i]);
  }
  __device__ __forceinline__ void mma(float (&acc)[4], const Raw8<W>& w0, const Raw8<W>& w1) const {
    float t[4] = {}, low[4] = {};
    float f0[8], f1[8];
    w0.floats(f0);
    w1.floats(f1);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t a[4] = {__float_as_uint(f0[2 * q]), __float_as_uint(f1[2 * q]), __float_as_uint(f0[2 * q + 1]),
                       __float_as_uint(f1[2 * q + 1])};
      if constexpr (kCutWeight<W>) {
        uint32_t b[4];
        cut_tf32(f0[2 * q], a[0], b[0]);
        cut_tf32(f1[2 * q], a[1], b[1]);
        cut_tf32(f0[2 * q + 1], a[2], b[2]);
        cut_tf32(f1[2 * q + 1], a[3], b[3]);
        mma_tf32(low, b[0], b[1], b[2], b[3], h[2 * q], h[2 * q + 1]);
      }
      mma_tf32(low, a[0], a[1], a[2], a[3], l[2 * q], l[2 * q + 1]);
      mma_tf32(t, a[0], a[1], a[2], a[3], h[2 * q], h[2 * q + 1]);
    }
    add_step(acc, t, low);
  }
};
template <>
struct Columns<__half> : Columns32<__half> {};
template <>
struct Columns<float> : Columns32<float> {};

template <class W, bool VECK, bool VECR>
__global__ void __launch_bounds__(kDecodeThreads, 2) k_lora_decode(const Params p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int members[kGroup], n_members, adapter;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = p.cluster, c = (int)cluster.block_rank(), u = blockIdx.y;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid4 = lane & 3;
  constexpr int kWarps = kDecodeThreads / 32;
  pdl_wait();
  pdl_launch_dependents();
  // Tokens that share an adapter form groups of up to kGroup, in token order; cluster
  // u takes the u-th group, the clusters behind the groups one token without an
  // adapter each, and the rest of the grid has nothing to do (it comes last, so it
  // keeps no SM from a group).
  if (warp == 0) {
    static_assert(kLoraDecodeTokens == 64, "two tokens a lane");
    int id[2], before[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = lane + 32 * h;
      const int a = k < p.M ? __ldg(p.ids + k) : -2;
      id[h] = a >= 0 && a < p.S ? a : k < p.M ? -1 : -2;
      if (k < p.M && id[h] < 0 && a != -1) set_status(p.status, SQ_ERR_INVALID_ARG);
      before[h] = __popc(__match_any_sync(0xffffffffu, id[h]) & ((1u << lane) - 1u));
    }
    for (int i = 0; i < 32; ++i) before[1] += __shfl_sync(0xffffffffu, id[0], i) == id[1];
    uint32_t lead[2], none[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lead[h] = __ballot_sync(0xffffffffu, id[h] >= 0 && before[h] % kGroup == 0);
      none[h] = __ballot_sync(0xffffffffu, id[h] == -1);
    }
    const int groups = __popc(lead[0]) + __popc(lead[1]);
    int want = u, a = -1, n = -1, first = 0;  // the want-th set bit of lead (or none)
    const uint32_t* bits = u < groups ? lead : none;
    if (u >= groups) want -= groups;
    const int half = want >= __popc(bits[0]) ? 1 : 0;
    if (half) want -= __popc(bits[0]);
    const uint32_t word = bits[half];
    const bool mine = (word >> lane & 1u) && __popc(word & ((1u << lane) - 1u)) == want;
    const uint32_t at = __ballot_sync(0xffffffffu, mine);
    if (at) {
      const int src = __ffs(at) - 1;
      a = __shfl_sync(0xffffffffu, half ? id[1] : id[0], src);
      first = __shfl_sync(0xffffffffu, half ? before[1] : before[0], src);
      n = 0;
      if (a < 0 && lane == 0) members[0] = src + 32 * half;
    }
    if (a >= 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = id[h] == a && before[h] >= first && before[h] < first + kGroup;
        if (in) members[before[h] - first] = lane + 32 * h;
        n += __popc(__ballot_sync(0xffffffffu, in));
      }
    }
    if (lane == 0) {
      adapter = a;
      n_members = n;  // 0: a token without an adapter; -1: nothing to do
    }
  }
  __syncthreads();
  const int nm = n_members, a = adapter;
  // this CTA's columns, in blocks of 16
  const int nb = (p.N + 15) / 16;
  const int n0 = nb * c / nc * 16, n1 = min(p.N, nb * (c + 1) / nc * 16);
  if (nm <= 0) {
    const int64_t t = members[0];  // no adapter: the base row as it is
    if (nm == 0 && p.base != p.y)
      for (int n = n0 + threadIdx.x; n < n1; n += kDecodeThreads)
        p.y[t * p.ldy + n] = p.base ? p.base[t * p.ldb + n] : 0.0f;
    return;  // (the whole cluster)
  }
  const int rank = adapter_rank(p, a), R16 = (p.R + 15) & ~15;
  const W* Ba = static_cast<const W*>(p.B) + (int64_t)a * p.N * p.R;
  float* part = sm;                             // [kWarps][R16][8]: v of each warp, then [R16][8] of the CTA
  float* vs = part + kWarps * R16 * 8;          // [R16 rounded up to 32][8]: v
  // ---- v = A x: warp slices of the channels, 32 at a time
  {
    const float* xrow = p.x + (int64_t)members[min(gid, nm - 1)] * p.K;
    const W* Aa = static_cast<const W*>(p.A) + (int64_t)a * p.R * p.K;
    const int steps = (p.K + 31) / 32, slice = c * kWarps + warp, slices = nc * kWarps;
    const int s0 = (int)((int64_t)steps * slice / slices), s1 = (int)((int64_t)steps * (slice + 1) / slices);
    for (int r0 = 0; r0 < rank; r0 += 64) {
      float acc[4][4] = {};
      for (int s = s0; s < s1; ++s) {
        const int k = 32 * s + 8 * tid4;
        Raw8<float> xr;
        load_masked<VECK>(xr, xrow, k, p.K, true);
        Raw8<W> w[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = r0 + 16 * j + gid + 8 * h;
            if (r0 + 16 * j < rank) load_masked<VECK>(w[j][h], Aa + (int64_t)min(r, rank - 1) * p.K, k, p.K, r < rank);
          }
        float xf[8];
        xr.floats(xf);
        Columns<W> x;
        x.set(xf);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r0 + 16 * j < rank) x.mma(acc[j], w[j][0], w[j][1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r0 + 16 * j < rank) {
          float* o = part + (warp * R16 + r0 + 16 * j + gid) * 8 + 2 * tid4;
          *reinterpret_cast<float2*>(o) = make_float2(acc[j][0], acc[j][1]);
          *reinterpret_cast<float2*>(o + 64) = make_float2(acc[j][2], acc[j][3]);
        }
    }
  }
  __syncthreads();
  const int live = (rank + 15) / 16 * 16 * 8;  // values computed
  for (int i = threadIdx.x; i < live; i += kDecodeThreads) {
    float v = part[i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += part[w * R16 * 8 + i];
    part[i] = v;
  }
  cluster.sync();
  bool bad = false;
  const float sc = __ldg(p.scale + a);
  const int steps = (rank + 31) / 32;
  for (int i = threadIdx.x; i < steps * 32 * 8; i += kDecodeThreads) {
    float v = 0.0f;
    if (i < live) {
#pragma unroll 8
      for (int d = 0; d < nc; ++d) v += cluster.map_shared_rank(part, d)[i];
      bad |= (i & 7) < nm && !isfinite(v);
      v *= sc;
    }
    vs[i] = v;
  }
  if (bad) set_status(p.status, SQ_ERR_NONFINITE);
  // the parts have been read: no CTA leaves before every other has got here
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  __syncthreads();
  // ---- y += B v: 16 columns at a time, two blocks' weights in flight
  const float* by[2];
  float* yy[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // the accumulators' tokens
    const int64_t row = members[min(2 * tid4 + i, nm - 1)];
    by[i] = p.base ? p.base + row * p.ldb : nullptr;
    yy[i] = p.y + row * p.ldy;
  }
  constexpr int kAhead = 2;
  for (int b0 = n0 + 16 * kAhead * warp; b0 < n1; b0 += 16 * kAhead * kWarps) {
    float b[kAhead][4], acc[kAhead][4] = {};
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = b0 + 16 * u + gid + 8 * (i >> 1);
        b[u][i] = by[i & 1] && n < n1 && 2 * tid4 + (i & 1) < nm ? by[i & 1][n] : 0.0f;
      }
    constexpr int kSteps = sizeof(W) == 2 ? 2 : 1;  // steps of the rank loaded together
    for (int s0 = 0; s0 < steps; s0 += kSteps) {
      Raw8<W> w[kSteps][kAhead][2];
#pragma unroll
      for (int e = 0; e < kSteps; ++e)
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            load_masked<VECR>(w[e][u][h], Ba + (int64_t)min(b0 + 16 * u + gid + 8 * h, n1 - 1) * p.R,
                              32 * (s0 + e) + 8 * tid4, rank, true);
#pragma unroll
      for (int e = 0; e < kSteps; ++e) {
        if (s0 + e >= steps) break;
        float vf[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) vf[i] = vs[(32 * (s0 + e) + 8 * tid4 + i) * 8 + gid];
        Columns<W> v;
        v.set(vf);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) v.mma(acc[u], w[e][u][0], w[e][u][1]);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = b0 + 16 * u + gid + 8 * (i >> 1);
        if (n < n1 && 2 * tid4 + (i & 1) < nm) yy[i & 1][n] = b[u][i] + acc[u][i];
      }
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ---- many tokens ------------------------------------------------------------------------
// Shrink: a cluster (of one CTA where there are tokens enough) takes 16 tokens of one
// adapter; a warp has 32 of the rank and a slice of the channels (of 16 warps, Rp / 32
// share a slice, so that its x comes from the first-level cache).  The next step's x
// and weights are loaded as soon as this step's have left their registers.  The
// parts meet in shared memory, then over the cluster, and are summed in a fixed
// order.  What bounds it is the latency of those loads: with 64 of the rank per warp
// the accumulators and parts spilled, and 2048 tokens, rank 64, 4096 -> 14336 took
// 104 us against 95 (both kernels).
constexpr int kShrinkThreads = 512, kShrinkWarps = kShrinkThreads / 32;
constexpr int kGroupTokens = 16;

// Without a sort from the caller, up to this many tokens: every CTA of the shrink kernel
// finds its group in the ids by itself (a count per adapter, one scan, one pass for
// the members), and the groups together write the sort that the expand kernel reads.
// 333 tokens over 5 adapters take 28.4 us so, 30.1 with a sorting launch before them; 512 over
// 100 32.6 and 34.3, 512 over 8 34.8 and 35.4; 1000 over 300 36.6 and 35.4.
constexpr int kSelfSortTokens = 512;

struct Group {
  int a, p0, cnt;  // adapter (-1: none), first place, tokens
};
// Group u of the ids; its tokens in members[].  counts: [S] ints, part: one per warp.
// All threads of the CTA call it; the first CTA writes the offsets.
__device__ Group find_group(const Params& p, int u, bool writes_order, int* counts, int* part, int* members) {
  __shared__ Group found;
  static_assert(2 * kShrinkThreads >= kMaxSegments && kSelfSortTokens <= 32767, "two adapters a thread, packed sums");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int s = threadIdx.x; s < p.S; s += kShrinkThreads) counts[s] = 0;
  if (threadIdx.x == 0) found.a = -1;
  __syncthreads();
  const int span = (p.M + kShrinkThreads - 1) / kShrinkThreads * 32;  // tokens per warp
  const int lo = min(p.M, warp * span), hi = min(p.M, lo + span);
  auto id_of = [&](int i) {
    const int id = i < hi ? __ldg(p.ids + i) : -1;
    return id >= 0 && id < p.S ? id : id == -1 ? -1 : -2;
  };
  bool bad = false;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int id = id_of(i0 + lane);
    bad |= id == -2;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    if (id >= 0 && __ffs(same) - 1 == lane) atomicAdd(&counts[id], __popc(same));  // (a count: the order does not matter)
  }
  if (bad && blockIdx.x == 0) set_status(p.status, SQ_ERR_INVALID_ARG);
  __syncthreads();
  // exclusive sums of (groups << 16 | tokens) over the adapters, two a thread
  int n[2], v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int s = 2 * threadIdx.x + h;
    n[h] = s < p.S ? counts[s] : 0;
    v[h] = ((n[h] + kGroupTokens - 1) / kGroupTokens) << 16 | n[h];
  }
  int incl = v[0] + v[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  int excl = incl - v[0] - v[1];
  for (int w = 0; w < warp; ++w) excl += part[w];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int s = 2 * threadIdx.x + h, g = u - (excl >> 16);
    if (blockIdx.x == 0 && s <= p.S) const_cast<int32_t*>(p.offsets)[s] = excl & 0xffff;
    if (n[h] > 0 && g >= 0 && g * kGroupTokens < n[h])
      found = Group{s, (excl & 0xffff) + g * kGroupTokens, min(kGroupTokens, n[h] - g * kGroupTokens)};
    if (n[h] > 0 && g >= 0 && g * kGroupTokens < n[h]) members[kGroupTokens] = g * kGroupTokens;  // rank of its first
    excl += v[h];
  }
  if (blockIdx.x == 0 && threadIdx.x == kShrinkThreads - 1 && p.S >= 2 * kShrinkThreads)
    const_cast<int32_t*>(p.offsets)[p.S] = excl & 0xffff;
  __syncthreads();
  const Group f = found;
  if (f.a < 0) return f;
  const int first = members[kGroupTokens];
  int mine = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) mine += __popc(__ballot_sync(0xffffffffu, id_of(i0 + lane) == f.a));
  if (lane == 0) part[warp] = mine;
  __syncthreads();
  int at = -first;
  for (int w = 0; w < warp; ++w) at += part[w];
  for (int i0 = lo; i0 < hi && at < kGroupTokens; i0 += 32) {
    const bool is = id_of(i0 + lane) == f.a;
    const uint32_t all = __ballot_sync(0xffffffffu, is);
    const int r = at + __popc(all & ((1u << lane) - 1u));
    if (is && r >= 0 && r < kGroupTokens) {
      members[r] = i0 + lane;
      if (writes_order) const_cast<int32_t*>(p.order)[f.p0 + r] = i0 + lane;
    }
    at += __popc(all);
  }
  __syncthreads();
  return f;
}

template <class W, bool VEC>
__global__ void __launch_bounds__(kShrinkThreads) k_lora_shrink(const Params p) {
  extern __shared__ __align__(16) float sm[];  // [slices][16][Rp], then the tile sums [S + 1]
  __shared__ int part_i[kShrinkThreads / 32], members[kGroupTokens + 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = p.cluster, c = (int)cluster.block_rank(), u = (int)blockIdx.x / nc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tid4 = lane & 3;
  const int rgroups = p.Rp / 32, warps = kShrinkWarps / rgroups;  // slices of the channels in this CTA
  const int part = warp / rgroups, r0 = 32 * (warp % rgroups);    // this warp's (a warp past them idles)
  int* pre = reinterpret_cast<int*>(sm + warps * kGroupTokens * p.Rp);
  pdl_wait();
  pdl_launch_dependents();
  Group group;
  if (p.self_sort) {
    group = find_group(p, u, c == 0, pre, part_i, members);
    if (group.a < 0) return;  // (the whole cluster)
  } else {
    const int units = segment_units(p.offsets, p.S, p.M, p.status, kGroupTokens, pre, part_i);
    if (u >= units) return;
    group.a = unit_expert(pre, p.S, u);
    const int2 seg = segment_bounds(p.offsets, p.M, group.a, p.status);
    group.p0 = seg.x + (u - pre[group.a]) * kGroupTokens;
    group.cnt = min(kGroupTokens, seg.y - group.p0);
  }
  const int a = group.a, p0 = group.p0, cnt = group.cnt;
  const int rank = adapter_rank(p, a);
  const int steps = (p.K + 31) / 32, slice = c * warps + part, slices = nc * warps;
  const int s0 = (int)((int64_t)steps * slice / slices), s1 = (int)((int64_t)steps * (slice + 1) / slices);
  float* mine = sm + part * kGroupTokens * p.Rp;
  if (part < warps) {
    const float* xr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = min(gid + 8 * h, cnt - 1);
      int t = p.self_sort ? members[at] : __ldg(p.order + p0 + at);
      if (t < 0 || t >= p.M) {
        set_status(p.status, SQ_ERR_INVALID_ARG);
        t = 0;
      }
      xr[h] = p.x + (int64_t)t * p.K;
    }
    const W* Aa = static_cast<const W*>(p.A) + (int64_t)a * p.R * p.K;
    constexpr int NT = 4;
    float acc[NT][4] = {};
    if (r0 < rank && s0 < s1) {
      Raw8<float> xr8[2];
      Raw8<W> wr8[NT];
      int wrow[NT];  // (R K < 2^25)
#pragma unroll
      for (int j = 0; j < NT; ++j) wrow[j] = min(r0 + 8 * j + gid, rank - 1) * p.K;
      auto issue_x = [&](int k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) issue_masked<VEC>(xr8[h], xr[h], k, p.K, true);
      };
      auto issue_w = [&](int j, int k) { issue_masked<VEC>(wr8[j], Aa + wrow[j], k, p.K, r0 + 8 * j + gid < rank); };
      constexpr bool AHEAD = !kCutWeight<W>;  // (no registers for it with binary32 weights)
      issue_x(32 * s0 + 8 * tid4);
      if constexpr (AHEAD) {
#pragma unroll
        for (int j = 0; j < NT; ++j) issue_w(j, 32 * s0 + 8 * tid4);
      }
      for (int s = s0; s < s1; ++s) {
        const int k = 32 * s + 8 * tid4, next = min(s + 1, s1 - 1) * 32 + 8 * tid4;
        if constexpr (!AHEAD) {
#pragma unroll
          for (int j = 0; j < NT; ++j) issue_w(j, k);
        }
        const bool inside = 32 * s + 32 <= p.K;  // (the whole warp's)
        if (!inside) {
#pragma unroll
          for (int h = 0; h < 2; ++h) finish_masked<VEC>(xr8[h], k, p.K, true);
        }
        if constexpr (kBf16<W>) {
          uint32_t xa[2][3][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[8];
            xr8[h].floats(v);
            cut8(v, xa[h]);
          }
          issue_x(next);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (r0 + 8 * j >= rank) break;
            if (!inside || r0 + 8 * j + 8 > rank) finish_masked<VEC>(wr8[j], k, p.K, r0 + 8 * j + gid < rank);
            float t[4] = {};
#pragma unroll
            for (int i = 2; i >= 0; --i)  // small products first
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t av[4] = {xa[0][i][2 * q], xa[1][i][2 * q], xa[0][i][2 * q + 1], xa[1][i][2 * q + 1]};
                mma_bf16(t, av, wr8[j].w[2 * q], wr8[j].w[2 * q + 1]);
              }
            add_step(acc[j], t);
            issue_w(j, next);
          }
        } else {
          // k8 step q: channels 2q, 2q + 1 of the lane's eight
          uint32_t xh[2][8], xl[2][8];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i) cut_tf32(__uint_as_float(xr8[h].w[i]), xh[h][i], xl[h][i]);
          issue_x(next);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (r0 + 8 * j >= rank) break;
            if (!inside || r0 + 8 * j + 8 > rank) finish_masked<VEC>(wr8[j], k, p.K, r0 + 8 * j + gid < rank);
            float wv[8];
            wr8[j].floats(wv);
            if constexpr (AHEAD) issue_w(j, next);
            float t[4] = {}, low[4] = {};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t h0 = __float_as_uint(wv[2 * q]), h1 = __float_as_uint(wv[2 * q + 1]);
              if constexpr (kCutWeight<W>) {
                uint32_t l0, l1;
                cut_tf32(wv[2 * q], h0, l0);
                cut_tf32(wv[2 * q + 1], h1, l1);
                mma_tf32(low, xh[0][2 * q], xh[1][2 * q], xh[0][2 * q + 1], xh[1][2 * q + 1], l0, l1);
              }
              mma_tf32(low, xl[0][2 * q], xl[1][2 * q], xl[0][2 * q + 1], xl[1][2 * q + 1], h0, h1);
              mma_tf32(t, xh[0][2 * q], xh[1][2 * q], xh[0][2 * q + 1], xh[1][2 * q + 1], h0, h1);
            }
            add_step(acc[j], t, low);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float* o = mine + gid * p.Rp + r0 + 8 * j + 2 * tid4;
      *reinterpret_cast<float2*>(o) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(o + 8 * p.Rp) = make_float2(acc[j][2], acc[j][3]);
    }
  }
  __syncthreads();
  // the CTA's parts summed into the first warp's, then the cluster's, CTA c taking
  // its share of the values
  const int total = cnt * p.Rp;
  for (int i = threadIdx.x; i < total; i += blockDim.x) {
    float v = sm[i];
    for (int w = 1; w < warps; ++w) v += sm[w * kGroupTokens * p.Rp + i];
    sm[i] = v;
  }
  if (nc > 1) cluster.sync();
  else __syncthreads();
  const int i0 = (int)((int64_t)total * c / nc), i1 = (int)((int64_t)total * (c + 1) / nc);
  const float sc = __ldg(p.scale + a);
  bool bad = false;
  for (int i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
    float v = 0.0f;
    for (int d = 0; d < nc; ++d) v += nc > 1 ? cluster.map_shared_rank(sm, d)[i] : sm[i];
    bad |= !isfinite(v);
    p.v[(int64_t)p0 * p.Rp + i] = v * sc;
  }
  if (bad) set_status(p.status, SQ_ERR_NONFINITE);
  if (nc > 1) cluster.sync();  // no CTA leaves while its parts may be read
}

constexpr int kExpandThreads = 128;
constexpr int kBlockCols = 64;  // columns of y per warp pass
constexpr int kRing = 4;        // units of the weight ring

// 16-byte words a lane holds of v per 32 of the rank in the expand kernel: three
// bfloat16 parts for bfloat16 weights, two binary16 parts for binary16 ones; for
// binary32 weights v itself, cut into tf32 parts when it is read.
template <class W>
constexpr int kVWords = kBf16<W> ? 6 : 4;

// Expand: CTA = one tile of 64 tokens (16 per warp) and a span of columns.  The
// warp's v lies in shared memory in operand order ([k32 step][part][two 16-byte
// words per lane]).  Of each 16 columns, one MMA takes columns 4i, 4i+1 and one
// 4i+2, 4i+3 (i = 0..3), so that a lane's accumulators are four neighbouring
// columns and base and y move in 16-byte words.  The next 64 columns of base are
// copied into shared memory (each lane its own words) under the products of these.
template <class W, bool VEC, bool VECY>
__global__ void __launch_bounds__(kExpandThreads, 4) k_lora_expand(const Params p) {
  constexpr int NV = kVWords<W>;
  constexpr bool BF = kBf16<W>, HALF = std::is_same<W, __half>::value;
  // [4 warps][Rp / 32][NV][32] of v, [4 warps][8][32] of base, the weight ring, the tile sums
  extern __shared__ __align__(16) uint4 vsm[];
  constexpr int kUnitWords = kBlockCols * 32 * (int)sizeof(W) / 16;  // 16-byte words of a ring unit
  __shared__ int part_i[kExpandThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tid4 = lane & 3;
  const int u = blockIdx.y;
  const int n0 = blockIdx.x * p.span, n1 = min(p.N, n0 + p.span);
  pdl_wait();
  pdl_launch_dependents();
  if (u >= p.tiles) {  // rows without an adapter
    if (p.base == p.y) return;
    for (int t = (u - p.tiles) * 4 + warp; t < p.M; t += ((int)gridDim.y - p.tiles) * 4) {
      const int a = __ldg(p.ids + t);
      if (a >= 0 && a < p.S) continue;
      for (int n = n0 + lane; n < n1; n += 32) p.y[t * p.ldy + n] = p.base ? p.base[t * p.ldb + n] : 0.0f;
    }
    return;
  }
  const int steps_all = p.Rp / 32;
  uint4* ring = vsm + 4 * (steps_all * NV + 8) * 32;
  int* pre = reinterpret_cast<int*>(ring + (VEC ? kRing * kUnitWords : 0));
  const int units = segment_units(p.offsets, p.S, p.M, p.status, kTile, pre, part_i);
  if (u >= units) return;
  const int a = unit_expert(pre, p.S, u);
  const int2 seg = segment_bounds(p.offsets, p.M, a, p.status);
  // (a warp without tokens repeats the tile's last: it helps copying the weights)
  const int pt = seg.x + (u - pre[a]) * kTile, p0 = min(pt + 16 * warp, seg.y - 1), cnt = min(16, seg.y - (pt + 16 * warp));
  const int rank = adapter_rank(p, a), steps = (rank + 31) / 32;
  uint4* vw = vsm + warp * steps_all * NV * 32;
  uint4* bw = vsm + 4 * steps_all * NV * 32 + warp * 256 + lane;
  float back[2] = {1.0f, 1.0f};  // binary16 parts: 2^e of the two rows
  int64_t row[2];
  const float* vrow[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = min(p0 + gid + 8 * h, seg.y - 1);
    int t = __ldg(p.order + at);
    if (t < 0 || t >= p.M) t = 0;  // (reported by the shrink kernel)
    row[h] = t;
    vrow[h] = p.v + (int64_t)at * p.Rp;
  }
  float to[2] = {1.0f, 1.0f};
  if constexpr (HALF) {
    float m[2] = {0.0f, 0.0f};
    for (int s = 0; s < steps; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 f = *reinterpret_cast<const float4*>(vrow[h] + 32 * s + 8 * tid4 + 4 * i);
          m[h] = fmaxf(m[h], fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w))));
        }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 1));
      m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 2));
      // the largest |v| to [2^13, 2^14): exponent field of the power is 267 - its own,
      // kept inside the normal range (a row of zeros or of tiny values stays below)
      const int ex = (int)(__float_as_uint(m[h]) >> 23);
      const int f = min(max(267 - ex, 1), 253);
      to[h] = __uint_as_float((uint32_t)f << 23);
      back[h] = __uint_as_float((uint32_t)(254 - f) << 23);
    }
  }
  for (int s = 0; s < steps; ++s) {
    uint4* o4 = vw + s * NV * 32 + lane;
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(vrow[h] + 32 * s + 8 * tid4 + 4 * i);
        v[h][4 * i] = f.x; v[h][4 * i + 1] = f.y; v[h][4 * i + 2] = f.z; v[h][4 * i + 3] = f.w;
      }
    if constexpr (BF || HALF) {
      uint32_t o[2][3][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (HALF) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x0 = v[h][2 * i] * to[h], x1 = v[h][2 * i + 1] * to[h];
            const __half2 hi = __floats2half2_rn(x0, x1);
            const float2 hf = __half22float2(hi);
            const __half2 lo = __floats2half2_rn(x0 - hf.x, x1 - hf.y);
            o[h][0][i] = *reinterpret_cast<const uint32_t*>(&hi);
            o[h][1][i] = *reinterpret_cast<const uint32_t*>(&lo);
          }
        } else {
          cut8(v[h], o[h]);
        }
      }
#pragma unroll
      for (int i = 0; i < NV / 2; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          o4[(i * 2 + q) * 32] = make_uint4(o[0][i][2 * q], o[1][i][2 * q], o[0][i][2 * q + 1], o[1][i][2 * q + 1]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o4[q * 32] = make_uint4(__float_as_uint(v[0][2 * q]), __float_as_uint(v[1][2 * q]), __float_as_uint(v[0][2 * q + 1]),
                                __float_as_uint(v[1][2 * q + 1]));
    }
  }
  __syncwarp();
  const W* Ba = static_cast<const W*>(p.B) + (int64_t)a * p.N * p.R;
  const int col = 4 * (gid >> 1) + (gid & 1);  // this lane's B column of each 16 (and + 2)
  const bool staged = VECY && p.base != nullptr;
  // this lane's words of base of the 64 columns from c0
  auto stage_base = [&](int c0) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = c0 + 16 * j + 4 * tid4;
        if (gid + 8 * h >= cnt || n >= n1) continue;
        uint4* dst = bw + (j * 2 + h) * 32;
        const float* src = p.base + row[h] * p.ldb + n;
        if (n + 4 <= n1) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
        } else {
          float* d = reinterpret_cast<float*>(dst);
          for (int i = 0; n + i < n1; ++i) d[i] = src[i];
        }
      }
  };
  // ring unit i: 32 of the rank (step i % steps) of the 64 columns of block i / steps,
  // column by column, copied by the whole CTA, kRing - 1 units ahead of its use
  const int units_w = steps * ((n1 - n0 + kBlockCols - 1) / kBlockCols);
  int next_c0 = n0, next_s = 0, issued = 0;
  auto stage_weights = [&] {
    if (VEC && issued < units_w) {
      uint4* dst = ring + (issued % kRing) * kUnitWords;
      constexpr int kWordElems = 16 / (int)sizeof(W), kRowWords = 32 / kWordElems;
#pragma unroll
      for (int i = 0; i < kUnitWords / kExpandThreads; ++i) {
        const int w = threadIdx.x + i * kExpandThreads, n = w / kRowWords, e = 32 * next_s + (w % kRowWords) * kWordElems;
        const W* src = Ba + (int64_t)min(next_c0 + n, n1 - 1) * p.R + (e < p.R ? e : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst + w)), "l"(src) : "memory");
      }
      if (++next_s == steps) {
        next_s = 0;
        next_c0 += kBlockCols;
      }
    }
    ++issued;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kRing - 1; ++i) stage_weights();
  int unit = 0;
  for (int c0 = n0; c0 < n1; c0 += kBlockCols) {
    if (staged) stage_base(c0);  // (with the next weight unit's group)
    float acc[8][4] = {};
    for (int s = 0; s < steps; ++s) {
      Raw8<W> wr8[8];
      if constexpr (VEC) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
        __syncthreads();  // every thread's copies of this unit have landed, and the unit before is used
        stage_weights();
        const uint4* wu = ring + (unit % kRing) * kUnitWords;
        ++unit;
        constexpr int kLaneWords = (int)sizeof(W) / 2;  // 16-byte words of a lane's eight
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4* src = wu + (16 * (j >> 1) + col + 2 * (j & 1)) * 4 * kLaneWords + tid4 * kLaneWords;
#pragma unroll
          for (int i = 0; i < kLaneWords; ++i) {
            const uint4 f = src[i];
            wr8[j].w[4 * i] = f.x; wr8[j].w[4 * i + 1] = f.y; wr8[j].w[4 * i + 2] = f.z; wr8[j].w[4 * i + 3] = f.w;
          }
          if (32 * s + 32 > rank) wr8[j].keep(rank - 32 * s - 8 * tid4);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n = c0 + 16 * (j >> 1) + col + 2 * (j & 1);
          wr8[j].gather(Ba + (int64_t)min(n, n1 - 1) * p.R, 32 * s + 8 * tid4, rank);
        }
      }
      uint4 va[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) va[i] = vw[(s * NV + i) * 32 + lane];
      if constexpr (BF || HALF) {
        // (four columns' sums side by side: one after another, their chains of MMAs cost 5 us more)
#pragma unroll
        for (int j0 = 0; j0 < 8; j0 += 4) {
          float t[4][4] = {};
#pragma unroll
          for (int i = NV / 2 - 1; i >= 0; --i)  // small products first
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint4 f = va[i * 2 + q];
              const uint32_t av[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if constexpr (HALF) mma_f16(t[j], av, wr8[j0 + j].w[2 * q], wr8[j0 + j].w[2 * q + 1]);
                else mma_bf16(t[j], av, wr8[j0 + j].w[2 * q], wr8[j0 + j].w[2 * q + 1]);
              }
            }
#pragma unroll
          for (int j = 0; j < 4; ++j) add_step(acc[j0 + j], t[j]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t vh[4], vl[4];
          cut_tf32(__uint_as_float(va[q].x), vh[0], vl[0]);
          cut_tf32(__uint_as_float(va[q].y), vh[1], vl[1]);
          cut_tf32(__uint_as_float(va[q].z), vh[2], vl[2]);
          cut_tf32(__uint_as_float(va[q].w), vh[3], vl[3]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t h0, h1, l0, l1;
            cut_tf32(__uint_as_float(wr8[j].w[2 * q]), h0, l0);
            cut_tf32(__uint_as_float(wr8[j].w[2 * q + 1]), h1, l1);
            float t[4] = {};
            mma_tf32(t, vh[0], vh[1], vh[2], vh[3], l0, l1);
            mma_tf32(t, vl[0], vl[1], vl[2], vl[3], h0, h1);
            mma_tf32(t, vh[0], vh[1], vh[2], vh[3], h0, h1);
            add_step(acc[j], t);
          }
        }
      }
    }
    // base went out with the group of this block's first unit: steps - 1 groups are newer
    if (staged) {
      if (!VEC || steps < 2) asm volatile("cp.async.wait_all;" ::: "memory");
      else if (steps == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 2;" ::: "memory");
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = c0 + 16 * j + 4 * tid4;
        if (gid + 8 * h >= cnt || n >= n1) continue;
        float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (staged) {
          const float4 f = *reinterpret_cast<const float4*>(bw + (j * 2 + h) * 32);
          b[0] = f.x; b[1] = f.y; b[2] = f.z; b[3] = f.w;
        } else if (p.base) {
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = n + i < n1 ? p.base[row[h] * p.ldb + n + i] : 0.0f;
        }
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fmaf(acc[2 * j + (i >> 1)][2 * h + (i & 1)], back[h], b[i]);
        float* yr = p.y + row[h] * p.ldy + n;
        if (VECY && n + 4 <= n1) {
          *reinterpret_cast<float4*>(yr) = make_float4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < n1) yr[i] = o[i];
        }
      }
  }
}

cudaError_t launch(void (*fn)(const Params), dim3 grid, int threads, int smem, int cluster, bool pdl, cudaStream_t stream,
                   const Params& p) {
  const cudaError_t e = ensure_smem_attr((const void*)fn, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

bool aligned(const void* q, int64_t stride_elems, int elem, int bytes) {
  return reinterpret_cast<uintptr_t>(q) % bytes == 0 && stride_elems * elem % bytes == 0;
}

template <class W>
cudaError_t launch_type(Params p, void* sort_ws, int32_t* sort_arrays, int sm_count, cudaStream_t stream) {
  // rows of A and x (B) start at addresses that allow 8-element vectors
  const bool veck = p.K % 8 == 0 && aligned(p.A, p.K, sizeof(W), 16) && aligned(p.x, p.K, 4, 16);
  const bool vecr = p.R % 8 == 0 && aligned(p.B, p.R, sizeof(W), 16);
  if (p.M <= kLoraDecodeTokens) {
    const int R16 = (int)round_up(p.R, 16);
    const int smem = 4 * 8 * (kDecodeThreads / 32 * R16 + (int)round_up(p.R, 32));
    // 16 CTAs a cluster for few tokens (5.8 against 6.6 us for one), but only some 16
    // such clusters run at a time (64 tokens over 32 adapters: 37 against 27 us).  16 : 8
    // CTAs, rank 64, 4096 -> 12288, cold, us: each token another adapter, at 8, 12, 16 and 32
    // tokens 22.6 : 24.7, 22.5 : 24.6, 36.8 : 28.7, 55.3 : 32.8; 8 adapters, 16 tokens 22.6 : 24.6.
    // This kernel against the two below at 64 tokens: 64 adapters 57 : 174, 8 adapters
    // 27 : 51, one 25 : 37.
    p.cluster = p.M <= 16 ? kDecodeCluster : kCluster;
    auto* fn = veck ? (vecr ? k_lora_decode<W, true, true> : k_lora_decode<W, true, false>)
                    : (vecr ? k_lora_decode<W, false, true> : k_lora_decode<W, false, false>);
    // clusters above the portable size: allowed once per kernel and device
    static std::atomic<uint64_t> allowed[4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<uint64_t>& mask = allowed[(veck ? 2 : 0) + (vecr ? 1 : 0)];
    if (p.cluster > kCluster && !(mask.load() >> dev & 1u)) {
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      mask.fetch_or(1ull << dev);
    }
    return launch(fn, dim3(p.cluster, p.M), kDecodeThreads, smem, p.cluster, true, stream, p);
  }
  if (!p.offsets) {
    int32_t* offsets = sort_arrays;
    int32_t* order = offsets + round_up(p.S + 1, 4);
    int32_t* place = order + round_up(p.M, 4);
    p.self_sort = p.M <= kSelfSortTokens ? 1 : 0;
    if (!p.self_sort) {
      const cudaError_t e = launch_segment(p.ids, p.M, p.S, offsets, order, place, sort_ws, p.status, stream);
      if (e != cudaSuccess) return e;
    }
    p.offsets = offsets;
    p.order = order;
  }
  // tiles: at most one partial tile per adapter
  const int tiles = (int)(p.M / kTile + std::min(p.S, p.M));
  const int tables = (int)round_up(4 * (p.S + 1), 16);
  {
    // clusters only where 16 tokens a CTA leave SMs without work
    const int64_t units = ceil_div(p.M, kGroupTokens);
    p.cluster = 1;
    while (p.cluster < kCluster && units * p.cluster * 2 <= sm_count) p.cluster *= 2;
    const int smem = kShrinkWarps / (p.Rp / 32) * kGroupTokens * p.Rp * 4 + tables;
    auto* fn = veck ? k_lora_shrink<W, true> : k_lora_shrink<W, false>;
    const int groups = (int)(p.M / kGroupTokens + std::min(p.S, p.M));
    const cudaError_t e = launch(fn, dim3(p.cluster * groups), kShrinkThreads, smem, p.cluster, true, stream, p);
    if (e != cudaSuccess) return e;
  }
  // columns per CTA: a few CTAs per SM over all tiles
  const int64_t live = ceil_div(p.M, kTile);
  p.span = (int)std::max<int64_t>(kBlockCols, round_up(ceil_div((int64_t)p.N * live, 8 * (int64_t)sm_count), kBlockCols));
  p.tiles = tiles;
  const int copies = p.base == p.y ? 0 : (int)std::min<int64_t>(ceil_div(p.M, 64), 64);
  const bool vecy = aligned(p.y, p.ldy, 4, 16) && (!p.base || aligned(p.base, p.ldb, 4, 16));
  const int smem = 4 * ((p.Rp / 32) * kVWords<W> + 8) * 32 * 16 + (vecr ? kRing * kBlockCols * 32 * (int)sizeof(W) : 0) + tables;
  auto* fn = vecr ? (vecy ? k_lora_expand<W, true, true> : k_lora_expand<W, true, false>)
                  : (vecy ? k_lora_expand<W, false, true> : k_lora_expand<W, false, false>);
  return launch(fn, dim3((unsigned)ceil_div(p.N, p.span), tiles + copies), kExpandThreads, smem, 1, true, stream, p);
}

struct Carve {
  size_t arrays, sort, v, total;
};
Carve carve(int M, int S, int R) {
  Carve c;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (size_t)round_up((int64_t)(off + bytes), 256);
    return at;
  };
  c.arrays = take(4 * (size_t)(round_up(S + 1, 4) + 2 * round_up(M, 4)));
  c.sort = take(segment_workspace_bytes(M, S, 1, false));
  c.v = take((size_t)M * round_up(R, 32) * 4);
  c.total = off;
  return c;
}

}  // namespace

size_t lora_workspace_bytes(int M, int S, int R) { return M <= kLoraDecodeTokens ? 0 : carve(M, S, R).total; }

cudaError_t launch_lora(const sq_lora_bank& bank, const float* x, int M, const int32_t* ids, const int32_t* offsets,
                        const int32_t* order, const float* base, int64_t ldb, float* y, int64_t ldy, void* workspace,
                        int32_t* status, int sm_count, cudaStream_t stream) {
  Params p = {};
  p.A = bank.A;
  p.B = bank.B;
  p.scale = bank.scale;
  p.rank = bank.rank;
  p.S = bank.S;
  p.R = bank.R;
  p.K = bank.K;
  p.N = bank.N;
  p.x = x;
  p.M = M;
  p.ids = ids;
  p.base = base;
  p.ldb = ldb;
  p.y = y;
  p.ldy = ldy;
  p.offsets = offsets;
  p.order = order;
  p.Rp = (int)round_up(bank.R, 32);
  p.status = status;
  void* sort_ws = nullptr;
  int32_t* arrays = nullptr;
  if (M > kLoraDecodeTokens) {
    const Carve c = carve(M, bank.S, bank.R);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    arrays = reinterpret_cast<int32_t*>(w + c.arrays);
    sort_ws = w + c.sort;
    p.v = reinterpret_cast<float*>(w + c.v);
  }
  if (bank.type == SQ_TYPE_F16) return launch_type<__half>(p, sort_ws, arrays, sm_count, stream);
  if (bank.type == SQ_TYPE_BF16) return launch_type<__nv_bfloat16>(p, sort_ws, arrays, sm_count, stream);
  return launch_type<float>(p, sort_ws, arrays, sm_count, stream);
}

}  // namespace sq
