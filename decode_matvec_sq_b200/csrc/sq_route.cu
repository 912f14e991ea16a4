// sq_route.cu -- which tokens meet which weight: the top-k router gate, the
// stable sort of (token, choice) entries into one segment per expert (or per
// adapter), and the weighted sum that brings the experts' rows back to their
// tokens (sm_100a).
//
// Gate: per token the k largest logits, ties to the lower expert, by k rounds
// of a warp-wide maximum (redux) over logits held in registers as ordered integers,
// neighbouring experts in one lane, so that the first lane with the maximum is the
// choice; softmax over the chosen, or over all, experts with the row maximum
// subtracted.
// Segments: a counting sort.  Every warp owns a contiguous span of a chunk of
// entries; a lane's rank among equal ids of its 32 is a popcount of the
// match mask, earlier batches and warps add their counts, so the order within a
// segment is that of the entries whatever the timing (no atomic decides a
// place).  Up to kSmallTokens tokens / one chunk of entries run in one CTA and
// one launch (the latency of a decode step: 4.1 us for 16 tokens of 64 experts,
// k = 4); more take two launches: counts per chunk, then places, every CTA summing
// the chunks' counts itself.
// What bounds them: latency.  8192 tokens of 128 experts, k = 8, take 16.8 us
// (10 MB in and out would be 1 us): two launches, in each a chain of load, sort
// and store.  Experts spread over the lanes (lane + 32 i) took a second reduction
// per choice, and the chunks' counts read after the chunk's own sort, 23.5 us.
// Above 524288 entries the reads of the chunks' counts dominate, with the square of the chunks:
// 524288 ids of 1024 take 49 us, 2097152 453 us, 16777216 21 ms.
// Combine: one pass, bound by memory (4099 tokens, k = 4, 4096 columns: 6.3 TB/s).
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "sq_common.cuh"
#include "sq_internal.h"

namespace sq {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
// Entries of one chunk (one CTA).
constexpr int kMaxChunk = 4096;
// Tokens routed by the single-CTA kernel (a warp then routes at most 8).
constexpr int kSmallTokens = 256;

struct SegParams {
  const int32_t* ids;  // [n] (segment calls; null where the router forms them)
  int n, S;
  int chunk, chunks;   // entries per CTA, CTAs
  int32_t* offsets;    // [S + 1]
  int32_t* order;      // [n]
  int32_t* place;      // [n]
  int32_t* counts;     // workspace [chunks][S] (chunks > 1)
  int32_t* status;
};

struct RouteParams {
  const float* logits;
  int T, E, k, all;    // all: softmax over all experts
  int32_t* ids;
  float* gates;
  int32_t* status;
};

// Shared memory of a CTA that sorts a chunk: ids and ranks of its entries,
// per-warp counts, segment bases and totals.
__host__ __device__ inline int seg_smem_ints(int chunk, int S) { return 2 * chunk + kWarps * S + 2 * S + kWarps + 1; }

struct SegSmem {
  int *id, *rank, *wcount, *base, *total, *scan;
  __device__ SegSmem(int* s, int chunk, int S)
      : id(s), rank(s + chunk), wcount(s + 2 * chunk), base(wcount + kWarps * S), total(base + S), scan(total + S) {}
};

// Exclusive sum of `total` over the S segments into `base` (in place of its
// previous content, which is added); returns the grand total to all threads.
__device__ int scan_totals(const SegSmem& sm, int S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int v = threadIdx.x < S ? sm.total[threadIdx.x] : 0;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = sm.scan[lane], wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += u;
    }
    sm.scan[lane] = wi - w;
    if (lane == 31) sm.scan[32] = wi;
  }
  __syncthreads();
  if (threadIdx.x < S) {
    sm.total[threadIdx.x] = sm.scan[warp] + incl - v;  // offsets[s]
    sm.base[threadIdx.x] += sm.total[threadIdx.x];
  }
  return sm.scan[32];
}

// Counts and ranks of the chunk's entries (ids in sm.id, -1: none): per warp
// and segment in sm.wcount, the entry's rank in its warp in sm.rank; then the
// counts become exclusive sums over the warps and sm.total the chunk's counts.
__device__ void count_chunk(const SegSmem& sm, int n, int S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kWarps * S; i += kThreads) sm.wcount[i] = 0;
  __syncthreads();
  const int span = ((n + kThreads - 1) / kThreads) * 32;  // entries per warp
  const int lo = min(n, warp * span), hi = min(n, lo + span);
  int* wc = sm.wcount + warp * S;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const int id = i < hi ? sm.id[i] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    if (id >= 0) {
      const int before = __popc(same & ((1u << lane) - 1u));
      const int at = wc[id];
      sm.rank[i] = at + before;
      __syncwarp(same);
      if (before == 0) wc[id] = at + __popc(same);
    }
    __syncwarp();
  }
  __syncthreads();
  for (int s = threadIdx.x; s < S; s += kThreads) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int c = sm.wcount[w * S + s];
      sm.wcount[w * S + s] = sum;
      sum += c;
    }
    sm.total[s] = sum;
  }
  __syncthreads();
}

// Places of the chunk's entries [e0, e0 + n), sm.base holding the place of each
// segment's first entry of this chunk.
__device__ void place_chunk(const SegSmem& sm, const SegParams& p, int e0, int n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int span = ((n + kThreads - 1) / kThreads) * 32;
  const int lo = min(n, warp * span), hi = min(n, lo + span);
  for (int i = lo + lane; i < hi; i += 32) {
    const int id = sm.id[i];
    int at = -1;
    if (id >= 0) {
      at = sm.base[id] + sm.wcount[warp * p.S + id] + sm.rank[i];
      p.order[at] = e0 + i;
    }
    p.place[e0 + i] = at;
  }
}

// ids of entries [e0, e0 + n) into shared memory; ids outside [-1, S) count as
// none and are reported.
__device__ void load_ids(const SegSmem& sm, const SegParams& p, int e0, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    int id = p.ids[e0 + i];
    if (id < -1 || id >= p.S) {
      set_status(p.status, SQ_ERR_INVALID_ARG);
      id = -1;
    }
    sm.id[i] = id;
  }
}

// Order-preserving integer of a logit; both zeros equal, NaN below every expert
// that can be chosen.  kMasked: -inf (and NaN); 0: no expert / already chosen.
constexpr uint32_t kMasked = 0x007FFFFFu;
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (v != v) return kMasked;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.0f : expf(v - m); }

__device__ __forceinline__ float key_logit(uint32_t key) {  // (of a key above kMasked)
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// Routes token t by one warp; I neighbouring logits per lane (expert I lane + i, so
// that among equal keys the first lane, and its first, is the lower expert).  Lane
// j < k returns the j-th choice (-1: fewer than k experts unmasked).
template <int I>
__device__ int route_token(const RouteParams& p, int t) {
  const int lane = threadIdx.x & 31;
  const float* l = p.logits + (int64_t)t * p.E + I * lane;
  float v[I];
  uint32_t key[I];
  bool bad = false;
  if (I >= 4 && (p.E & 3) == 0) {  // (rows are 16-byte aligned)
#pragma unroll
    for (int i = 0; i < I; i += 4) {
      const float4 f = I * lane + i < p.E ? __ldg(reinterpret_cast<const float4*>(l + i))
                                          : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      const float g[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int u = 0; u < 4 && i + u < I; ++u) v[i + u] = g[u];
    }
  } else {
#pragma unroll
    for (int i = 0; i < I; ++i) v[i] = I * lane + i < p.E ? __ldg(l + i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < I; ++i) {
    key[i] = logit_key(v[i]);
    bad |= v[i] != v[i] || v[i] == INFINITY;
  }
  if (bad) set_status(p.status, SQ_ERR_NONFINITE);
  int id = -1;
  uint32_t chosen = 0u, first = 0u;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < I; ++i) best = max(best, key[i]);
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    if (m <= kMasked) break;
    const int src = __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
    int at = 0;
    bool open = lane == src;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const bool hit = open && key[i] == m;
      if (hit) {
        at = i;
        key[i] = 0u;
        open = false;
      }
    }
    const int e = I * src + __shfl_sync(0xffffffffu, at, src);
    if (j == 0) first = m;
    if (lane == j) {
      id = e;
      chosen = m;
    }
  }
  const float top = key_logit(first), val = key_logit(chosen);
  float sum = 0.0f;
  if (p.all) {
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (v[i] > -INFINITY) sum += exp_below(v[i], top);  // (false for NaN)
  } else if (id >= 0) {
    sum = exp_below(val, top);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < p.k) {
    p.ids[(int64_t)t * p.k + lane] = id;
    p.gates[(int64_t)t * p.k + lane] = id >= 0 ? exp_below(val, top) / sum : 0.0f;
  }
  return id;
}

// Tokens [t0, t1) of a CTA: their choices to memory and to sm.id.
template <int I>
__device__ void route_tokens(const RouteParams& p, const SegSmem& sm, int t0, int t1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t = t0 + warp; t < t1; t += kWarps) {
    const int id = route_token<I>(p, t);
    if (lane < p.k) sm.id[(t - t0) * p.k + lane] = id;
  }
}

// One chunk holds every entry: sort it and write everything.
__device__ void finish_single(const SegSmem& sm, const SegParams& p) {
  count_chunk(sm, p.n, p.S);
  if (threadIdx.x < p.S) sm.base[threadIdx.x] = 0;
  const int live = scan_totals(sm, p.S);
  if (threadIdx.x < p.S) p.offsets[threadIdx.x] = sm.total[threadIdx.x];
  if (threadIdx.x == 0) p.offsets[p.S] = live;
  __syncthreads();
  place_chunk(sm, p, 0, p.n);
  for (int i = live + threadIdx.x; i < p.n; i += kThreads) p.order[i] = -1;
}

template <int I>
__global__ void __launch_bounds__(kThreads, 1) k_route_one(const RouteParams r, const SegParams p) {
  extern __shared__ int smem[];
  const SegSmem sm(smem, p.chunk, p.S);
  pdl_wait();
  pdl_launch_dependents();
  route_tokens<I>(r, sm, 0, r.T);
  __syncthreads();
  finish_single(sm, p);
}

__global__ void __launch_bounds__(kThreads, 1) k_segment_one(const SegParams p) {
  extern __shared__ int smem[];
  const SegSmem sm(smem, p.chunk, p.S);
  pdl_wait();
  pdl_launch_dependents();
  load_ids(sm, p, 0, p.n);
  __syncthreads();
  finish_single(sm, p);
}

// First launch over many entries: (route the chunk's tokens,) count its
// entries per segment.
template <int I>
__global__ void __launch_bounds__(kThreads, 1) k_count(const RouteParams r, const SegParams p) {
  extern __shared__ int smem[];
  const SegSmem sm(smem, p.chunk, p.S);
  pdl_wait();
  const int e0 = blockIdx.x * p.chunk, n = min(p.chunk, p.n - e0);
  for (int i = threadIdx.x; i < p.S; i += kThreads) sm.total[i] = 0;
  if constexpr (I > 0) {
    __syncthreads();
    route_tokens<I>(r, sm, e0 / r.k, (e0 + n) / r.k);
  } else {
    load_ids(sm, p, e0, n);
  }
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const int id = i < n ? sm.id[i] : -1;
    if (id >= 0) atomicAdd(&sm.total[id], 1);  // (a count: the order does not matter)
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.S; s += kThreads) p.counts[(int64_t)blockIdx.x * p.S + s] = sm.total[s];
  pdl_launch_dependents();
}

// Second launch: every CTA sums the chunks' counts and places its own entries.
__global__ void __launch_bounds__(kThreads, 1) k_place(const SegParams p) {
  extern __shared__ int smem[];
  const SegSmem sm(smem, p.chunk, p.S);
  pdl_wait();
  pdl_launch_dependents();
  const int e0 = blockIdx.x * p.chunk, n = min(p.chunk, p.n - e0);
  // segment totals over all chunks, and over the chunks before this one: loaded
  // first, summed in shared memory when the chunk's own counts are done
  const int S32 = (p.S + 31) & ~31, groups = kThreads / S32;  // S <= 1024
  const int g = threadIdx.x / S32, s = threadIdx.x % S32;
  int total = 0, before = 0;
  if (g < groups && s < p.S) {
#pragma unroll 16
    for (int c = g; c < p.chunks; c += groups) {
      const int v = __ldg(p.counts + (int64_t)c * p.S + s);
      total += v;
      if (c < (int)blockIdx.x) before += v;
    }
  }
  load_ids(sm, p, e0, n);
  __syncthreads();
  count_chunk(sm, n, p.S);
  for (int i = threadIdx.x; i < p.S; i += kThreads) {
    sm.total[i] = 0;
    sm.base[i] = 0;
  }
  __syncthreads();
  if (g < groups && s < p.S) {
    atomicAdd(&sm.total[s], total);
    atomicAdd(&sm.base[s], before);
  }
  __syncthreads();
  const int live = scan_totals(sm, p.S);
  if (blockIdx.x == 0) {
    if (threadIdx.x < p.S) p.offsets[threadIdx.x] = sm.total[threadIdx.x];
    if (threadIdx.x == 0) p.offsets[p.S] = live;
  }
  __syncthreads();
  place_chunk(sm, p, e0, n);
  for (int i = max(live, e0) + (int)threadIdx.x; i < e0 + n; i += kThreads) p.order[i] = -1;
}

// ---- the weighted sum of each token's rows -----------------------------------------
// One pass: a thread sums its four columns (VEC; else one) of one token over
// the token's k rows, the loads of up to four rows in flight.
template <bool VEC>
__global__ void __launch_bounds__(256) k_combine(const float* __restrict__ z, int rows, const float* __restrict__ gates,
                                                 const int32_t* __restrict__ place, int k, int N,
                                                 const float* base, float* out, int32_t* status) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x;
  const int c = (blockIdx.y * 256 + threadIdx.x) * (VEC ? 4 : 1);
  if (c >= N) return;
  const int32_t* pl = place + (int64_t)t * k;
  const float* gt = gates + (int64_t)t * k;
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < k; j0 += 4) {
    float w[4], v[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = j0 + u < k ? __ldg(pl + j0 + u) : -1;
      const bool ok = at >= 0 && at < rows;
      if (at < -1 || at >= rows) set_status(status, SQ_ERR_INVALID_ARG);
      w[u] = ok ? __ldg(gt + j0 + u) : 0.0f;
      const float* zr = z + (int64_t)(ok ? at : 0) * N + c;
      if constexpr (VEC) {
        const float4 f = ok ? __ldg(reinterpret_cast<const float4*>(zr)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        v[u][0] = f.x;
        v[u][1] = f.y;
        v[u][2] = f.z;
        v[u][3] = f.w;
      } else {
        v[u][0] = ok ? __ldg(zr) : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < (VEC ? 4 : 1); ++i) a[i] = fmaf(w[u], v[u][i], a[i]);
  }
  const int64_t o = (int64_t)t * N + c;
  if constexpr (VEC) {
    if (base) {
      const float4 b = *reinterpret_cast<const float4*>(base + o);
      a[0] += b.x;
      a[1] += b.y;
      a[2] += b.z;
      a[3] += b.w;
    }
    *reinterpret_cast<float4*>(out + o) = make_float4(a[0], a[1], a[2], a[3]);
  } else {
    out[o] = base ? base[o] + a[0] : a[0];
  }
}

// Every kernel here begins by waiting for the one before it, so its launch may always
// be brought forward (programmatic dependent launch).
template <class... Args>
cudaError_t launch(void (*fn)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream, Args... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = ensure_smem_attr((const void*)fn, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// Calls f(integral_constant<I>) with the logits per lane for E experts.
template <class F>
cudaError_t with_lanes(int E, F f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

// Entries per chunk of a two-launch sort, a multiple of `unit`: at most kChunks chunks
// (each of the second launch's CTAs reads every chunk's counts) up to kChunks full chunks;
// more entries take more chunks, and the reads of counts grow with their square.
constexpr int kChunks = 128;
int longest_chunk(int unit) { return kMaxChunk / unit * unit; }  // (unit <= kMaxChoices)
int chunk_entries(int64_t n, int unit) {
  const int64_t want = std::max<int64_t>(256, ceil_div(n, kChunks));
  return (int)std::min<int64_t>(longest_chunk(unit), round_up(want, unit));
}

}  // namespace

size_t segment_workspace_bytes(int64_t n, int S, int unit, bool route) {
  if (route ? n / unit <= kSmallTokens && n <= kMaxChunk : n <= kMaxChunk) return 0;
  // (the chunks themselves can be fewer for a longer sort, where rounding to `unit` makes
  // them longer; a workspace for the longest batch serves every shorter one)
  return (size_t)std::max<int64_t>(kChunks, ceil_div(n, longest_chunk(unit))) * S * sizeof(int32_t);
}

cudaError_t launch_route(const float* logits, int T, int E, int k, bool all, int32_t* ids, float* gates,
                         int32_t* offsets, int32_t* order, int32_t* place, void* workspace, int32_t* status,
                         cudaStream_t stream) {
  RouteParams r{logits, T, E, k, all ? 1 : 0, ids, gates, status};
  SegParams p{ids, T * k, E, T * k, 1, offsets, order, place, static_cast<int32_t*>(workspace), status};
  if (segment_workspace_bytes(p.n, E, k, true) == 0) {
    const int smem = 4 * seg_smem_ints(p.chunk, E);
    return with_lanes(E, [&](auto I) {
      return launch(k_route_one<decltype(I)::value>, dim3(1), kThreads, smem, stream, r, p);
    });
  }
  p.chunk = chunk_entries(p.n, k);
  p.chunks = (int)ceil_div(p.n, p.chunk);
  const int smem = 4 * seg_smem_ints(p.chunk, E);
  const cudaError_t e = with_lanes(E, [&](auto I) {
    return launch(k_count<decltype(I)::value>, dim3(p.chunks), kThreads, smem, stream, r, p);
  });
  if (e != cudaSuccess) return e;
  return launch(k_place, dim3(p.chunks), kThreads, smem, stream, p);
}

cudaError_t launch_segment(const int32_t* ids, int n, int S, int32_t* offsets, int32_t* order, int32_t* place,
                           void* workspace, int32_t* status, cudaStream_t stream) {
  SegParams p{ids, n, S, n, 1, offsets, order, place, static_cast<int32_t*>(workspace), status};
  if (segment_workspace_bytes(n, S, 1, false) == 0)
    return launch(k_segment_one, dim3(1), kThreads, 4 * seg_smem_ints(n, S), stream, p);
  p.chunk = chunk_entries(n, 1);
  p.chunks = (int)ceil_div(n, p.chunk);
  const int smem = 4 * seg_smem_ints(p.chunk, S);
  const cudaError_t e =
      launch(k_count<0>, dim3(p.chunks), kThreads, smem, stream, RouteParams{}, p);
  if (e != cudaSuccess) return e;
  return launch(k_place, dim3(p.chunks), kThreads, smem, stream, p);
}

cudaError_t launch_combine(const float* z, int rows, const float* gates, const int32_t* place, int T, int k, int N,
                           const float* base, float* out, int32_t* status, cudaStream_t stream) {
  if ((N & 3) == 0)
    return launch(k_combine<true>, dim3(T, (unsigned)ceil_div(N, 1024)), 256, 0, stream, z, rows, gates, place, k,
                  N, base, out, status);
  return launch(k_combine<false>, dim3(T, (unsigned)ceil_div(N, 256)), 256, 0, stream, z, rows, gates, place, k, N,
                base, out, status);
}

}  // namespace sq
