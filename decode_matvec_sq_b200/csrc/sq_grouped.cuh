// sq_grouped.cuh -- arguments and segment bookkeeping shared by the two kernels
// of the expert-grouped linear layer.
#pragma once

#include <stdint.h>

#include "sq_common.cuh"
#include "sq_internal.h"
#include "sq_layout.h"

namespace sq {

// E experts of N rows (rbe = ceil(N/16) row blocks each) stacked in one tiled
// weight; n places, the activations' row of place p is order[p] / div (or p).
struct GroupedArgs {
  const int8_t* res;
  const uint32_t* sign;
  const uint32_t* mask;
  const float* alpha;
  const float* scale;
  const int32_t* zero;
  int E, N, K, tpr, rbe;
  const int8_t* xq;
  int xs;  // row stride of xq
  const float* sx;
  const float* xout;
  const int32_t* idx;
  int n_out;
  int rows;             // activation rows
  const int32_t* order; // may be null
  int div;
  const int32_t* offsets;
  int n;
  float* y;
  int32_t* status;
  int pdl;
  int zero_rest;        // rows of y behind the last segment become 0
  // for the tests (include/sq_testing.h): the limit of the many-token kernel's waits,
  // and a channel group whose weights are never requested (-1: none)
  uint64_t wait_ns;
  int skip_group;
};

// a / b for 0 <= a, 0 < b, in 32 bits where a allows it (a 64-bit division costs
// hundreds of clocks, and the walks over the tiles begin with several).
__device__ __forceinline__ int64_t fast_div(int64_t a, int b) {
  if ((a >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
  return pred != 0;
}

// Byte k = 0xFF if bit 8k+7 of x is set, else 0.
__device__ __forceinline__ uint32_t sign_bytes(uint32_t x) {
  uint32_t d;
  asm("prmt.b32 %0, %1, 0, 0xBA98;" : "=r"(d) : "r"(x));
  return d;
}
// Channels 4w .. 4w+3 of a lane's 32 as +1 / -1 bytes, 0 outside the mask.
template <bool MASK>
__device__ __forceinline__ uint32_t trunk_word(uint32_t sign, uint32_t mask, int w) {
  const uint32_t t = ~sign_bytes(sign << (7 - w)) | 0x01010101u;
  return MASK ? t & sign_bytes(mask << (7 - w)) : t;
}
// The bits of words w and w ^ 4 exchanged (bit 8c + w is channel 4w + c).
__device__ __forceinline__ uint32_t swap_halves(uint32_t b) {
  return ((b >> 4) & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
}

// Bounds of segment e of a sort of n entries, clamped to them (offsets that do
// not ascend in [0, n] are reported; no access leaves the arrays).
__device__ __forceinline__ int2 segment_bounds(const int32_t* offsets, int n, int e, int32_t* status) {
  const int a = __ldg(offsets + e), b = __ldg(offsets + e + 1);
  const int ca = min(max(a, 0), n), cb = min(max(b, ca), n);
  if (ca != a || cb != b) set_status(status, SQ_ERR_INVALID_ARG);
  return make_int2(ca, cb);
}

// Activation row of place `at`; a row outside the activations is reported and
// taken as 0.
__device__ __forceinline__ int source_row(const GroupedArgs& p, int at) {
  int r = at;
  if (p.order) {
    r = __ldg(p.order + at);
    // (the number of choices is mostly a power of two)
    if (r > 0) r = (p.div & (p.div - 1)) == 0 ? r >> (__ffs(p.div) - 1) : r / p.div;
  }
  if (r < 0 || r >= p.rows) {
    set_status(p.status, SQ_ERR_INVALID_ARG);
    r = 0;
  }
  return r;
}

// The rows of y behind the last segment set to 0, one CTA a row (all threads of every
// CTA call it; rows of no segment, so nothing else writes them).
__device__ __forceinline__ void zero_rest(const GroupedArgs& p) {
  const int live = min(max(__ldg(p.offsets + p.E), 0), p.n);
  for (int64_t r = (int64_t)live + blockIdx.x; r < p.n; r += gridDim.x)
    for (int c = threadIdx.x; c < p.N; c += blockDim.x) p.y[r * p.N + c] = 0.0f;
}

// Exclusive sums over the experts of ceil(segment / unit), into pre[0 .. E]
// (shared memory; all threads of the CTA call it; part: one int per warp).
__device__ inline int segment_units(const int32_t* offsets, int E, int n, int32_t* status, int unit, int* pre, int* part) {
  const int THREADS = blockDim.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += THREADS) {
    const int e = e0 + (int)threadIdx.x;
    int v = 0;
    if (e < E) {
      const int2 b = segment_bounds(offsets, n, e, status);
      v = (b.y - b.x + unit - 1) / unit;
    }
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int before = carry, total = carry;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += part[w];
      total += part[w];
    }
    if (e < E) pre[e] = before + incl - v;
    carry = total;
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[E] = carry;
  __syncthreads();
  return carry;
}

// The expert whose units hold unit u: the last e with pre[e] <= u.
__device__ __forceinline__ int unit_expert(const int* pre, int E, int u) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace sq
