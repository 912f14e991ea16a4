// sq_grouped.cu -- the linear layer grouped by expert, for the few tokens per
// expert of a decode step (sm_100a).
//
//   y[p] = What_e x[row(p)]   for the places p of segment e,
// with the products of sq_linear: exact int8 tensor-core sums (mma.sync
// m16n8k32) of the residual codes per 128-channel group and of the trunk over
// the row, combined in binary32, outlier channels in binary32.
//
// The experts' tiles lie behind one another in the stack, so an expert is a range
// of row blocks.  A segment is cut into groups of up to 8 NT tokens, which share
// one read of the expert's weights; the (group, row block) pairs, group-major,
// are split evenly over the CTAs and a CTA's tiles over its 16 warps, exactly as
// the decode kernel of one weight splits its own.  Nothing is read for an expert
// without tokens, and the host needs no counts: every CTA forms the groups from
// the device's offsets.
// What bounds it: the weight stream.  Each warp keeps 2 D tiles (2.3 KB each) in
// flight by bulk copies into its shared-memory ring, two tiles to a slot, one
// mbarrier per slot.
// Measured: one token through 2 of 8 experts, 4096 -> 14336, 26 to 28 us, 4.8 to 5.2 TB/s
// of the packed weights, 0.74 to 0.79 of a copy's rate (what is missing: the launch, the
// walk over the offsets and the drain, 5 us); 16 tokens, 2 of 8 each, 14336 -> 4096,
// 72 outlier channels, 101 to 108 us, 5.0 to 5.3 TB/s.
// The trunk operand is +-1 (0 outside the mask) bytes made from the bits by one
// shift, one sign-replicating byte permute and one three-input logic operation
// per four channels, so T needs one MMA where bits as 0/-1 need two.
// A lane's 64 code bytes are read as four 16-byte words; lanes 2 and 3 of a quad
// take them in the order 2, 3, 0, 1 (with their activation words and sign bits
// swapped alike), which halves the bank conflicts of the unpadded tile.
#include <stdint.h>

#include <algorithm>

#include "sq_grouped.cuh"

namespace sq {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxDepth = 2;  // (16 rings of three slots and the partial sums do not fit)
constexpr int kPair = 2;   // tiles per ring slot: neighbours in memory, copied together

struct Params {
  GroupedArgs a;
  int depth;
  int off_ring, off_part, off_pre, off_ostart, off_idx;  // shared-memory offsets (bytes)
};

// One ring slot: kPair tiles, array by array.
template <bool MASK, bool ASYM>
struct Slot {
  static constexpr int kSign = kPair * 2048;
  static constexpr int kMask = kSign + kPair * 256;
  static constexpr int kScale = MASK ? kMask + kPair * 256 : kMask;
  static constexpr int kZero = kScale + kPair * 64;
  static constexpr int kTile = 2048 + 256 + 64 + (MASK ? 256 : 0) + (ASYM ? 64 : 0);
  static constexpr int kBytes = kPair * kTile;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The tokens of one group: lane l holds those of token l % (8 NT).
template <int NT>
struct Tokens {
  const int8_t* x[NT];   // this lane's B column (token gid of each eight), at its 32 channels
  int row;               // activation row and scale of token l
  float sx;
  int p0, cnt;           // first place, tokens
};

template <int NT>
__device__ __forceinline__ void load_tokens(Tokens<NT>& tk, const GroupedArgs& a, int p0, int cnt, int lane) {
  tk.p0 = p0;
  tk.cnt = cnt;
  // (columns past the group repeat its last token; they are not written)
  tk.row = source_row(a, p0 + min(lane & (8 * NT - 1), cnt - 1));
  tk.sx = __ldg(a.sx + tk.row);
#pragma unroll
  for (int g = 0; g < NT; ++g)
    tk.x[g] = a.xq + (int64_t)__shfl_sync(0xffffffffu, tk.row, (lane >> 2) + 8 * g) * a.xs + (lane & 3) * 32;
}

template <bool MASK, bool ASYM, int NT>
__global__ void __launch_bounds__(kThreads, 1) k_grouped(const Params p) {
  using SL = Slot<MASK, ASYM>;
  constexpr int TG = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps * kMaxDepth];
  __shared__ int part_i[kWarps];
  const GroupedArgs& a = p.a;
  float* part = reinterpret_cast<float*>(smem + p.off_part);  // [kWarps][2][16][TG]
  int* pre = reinterpret_cast<int*>(smem + p.off_pre);
  int* ostart = reinterpret_cast<int*>(smem + p.off_ostart);  // first outlier of each channel group
  int* idx_s = reinterpret_cast<int*>(smem + p.off_idx);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid4 = lane & 3;
  const int D = p.depth;

  if (lane == 0)
    for (int d = 0; d < D; ++d) mbar_init(&bars[warp * kMaxDepth + d], 1);
  fence_barrier_init();
  if (!a.pdl) pdl_wait();
  // the outlier list (with SQ_LAUNCH_PDL fixed, and read before the wait)
  const int i0 = threadIdx.x;
  const int jv = i0 < a.n_out ? __ldg(a.idx + i0) : 0, jp = i0 > 0 && i0 < a.n_out ? __ldg(a.idx + i0 - 1) : -1;
  if (a.pdl) pdl_wait();
  pdl_launch_dependents();
  // Segments: with at most 32 experts every warp keeps expert `lane`'s in registers
  // (no barrier before the first copies), else the CTA forms them in shared memory.
  const bool few = a.E <= 32;
  int2 seg = make_int2(0, 0);
  int first = 0, groups;
  if (few) {
    if (lane < a.E) seg = segment_bounds(a.offsets, a.n, lane, a.status);
    const int v = (seg.y - seg.x + TG - 1) / TG;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    first = incl - v;
    groups = __shfl_sync(0xffffffffu, incl, 31);
  } else {
    groups = segment_units(a.offsets, a.E, a.n, a.status, TG, pre, part_i);
  }
  // expert of group u, its first group and its places
  struct Group {
    int e, first;
    int2 seg;
  };
  auto group_at = [&](int u) -> Group {
    Group g;
    if (few) {
      g.e = 31 - __clz(__ballot_sync(0xffffffffu, lane < a.E && first <= u));
      g.first = __shfl_sync(0xffffffffu, first, g.e);
      g.seg = make_int2(__shfl_sync(0xffffffffu, seg.x, g.e), __shfl_sync(0xffffffffu, seg.y, g.e));
    } else {
      g.e = unit_expert(pre, a.E, u);
      g.first = pre[g.e];
      g.seg = segment_bounds(a.offsets, a.n, g.e, nullptr);
    }
    return g;
  };

  // the CTA's (group, row block) pairs: the largest share that one CTA per SM
  // gives for as many CTAs as it takes, so that no CTA finishes alone
  const int64_t V = (int64_t)groups * a.rbe;
  const int64_t share = fast_div(V + gridDim.x - 1, (int)gridDim.x), v0 = blockIdx.x * share;
  if (v0 >= V) {
    if (a.zero_rest) zero_rest(a);
    return;
  }
  // tiles: in 32 bits by the host's check of n, unless bad offsets (reported) let
  // segments overlap; the rest of such a share is left out
  const int len = (int)min(min(share, V - v0) * a.tpr, (int64_t)0x7fffffff);
  const int t0 = (int)(((int64_t)warp * len) >> 4), t1 = (int)(((int64_t)(warp + 1) * len) >> 4);
  static_assert(kWarps == 16, "the split over the warps");
  // this warp's first tile: row block rb of the expert of group u, channel group cg
  const int lrb0 = t0 / a.tpr;
  int cg = t0 - lrb0 * a.tpr, u = (int)fast_div(v0 + lrb0, a.rbe), rb = (int)(v0 + lrb0 - (int64_t)u * a.rbe);
  Group grp = group_at(min(u, groups - 1));
  const int per_group = a.rbe * a.tpr;

  // producer cursor: the next tile to copy
  uint8_t* ring = smem + p.off_ring + warp * D * SL::kBytes;
  const uint32_t ring_u = smem_u32(ring), bar_u = smem_u32(&bars[warp * kMaxDepth]);
  int ct = t0, cu = u, cleft = per_group - rb * a.tpr - cg;  // tile; group, its tiles left
  int64_t ctile = (int64_t)grp.e * per_group + rb * a.tpr + cg;  // tile in the stack
  // the next slot: kPair tiles, or one at the end of a group or of the range
  auto copy = [&](int slot) {
    if (ct >= t1) return;
    if (cleft == 0) {
      ctile = (int64_t)group_at(++cu).e * per_group;
      cleft = per_group;
    }
    const uint32_t c = cleft >= kPair && ct + kPair <= t1 ? kPair : 1;
    const uint32_t dst = ring_u + slot * SL::kBytes, bar = bar_u + 8 * slot;
    if (elect_one()) {
      mbar_arrive_expect_tx(&bars[warp * kMaxDepth + slot], c * SL::kTile);
      bulk_load(dst, a.res + ctile * 2048, c * 2048, bar);
      bulk_load(dst + SL::kSign, a.sign + ctile * 64, c * 256, bar);
      bulk_load(dst + SL::kScale, a.scale + ctile * 16, c * 64, bar);
      if (MASK) bulk_load(dst + SL::kMask, a.mask + ctile * 64, c * 256, bar);
      if (ASYM) bulk_load(dst + SL::kZero, a.zero + ctile * 16, c * 64, bar);
    }
    __syncwarp();
    ct += c;
    ctile += c;
    cleft -= c;
  };
  // the group's tokens and the row block's scales
  Tokens<NT> tk;
  int64_t erow = 0;  // first row of the expert in the stack
  int gleft = 0;     // tiles left in the group
  float al[2] = {0.0f, 0.0f};
  auto enter_group = [&] {
    const int p0 = grp.seg.x + (u - grp.first) * TG;
    load_tokens<NT>(tk, a, p0, min(TG, grp.seg.y - p0), lane);
    erow = (int64_t)grp.e * a.rbe * kTileRows;
  };
  auto enter_rows = [&] {
    al[0] = __ldg(a.alpha + erow + rb * kTileRows + gid);
    al[1] = __ldg(a.alpha + erow + rb * kTileRows + gid + 8);
  };
  if (t0 < t1) {
    gleft = per_group - rb * a.tpr - cg;
    // (before the copies, whose queue these small loads would stand in)
    enter_group();
    enter_rows();
  }
  for (int d = 0; d < D; ++d) copy(d);
  if (a.zero_rest) zero_rest(a);

  // the outlier tables, while the first tiles are on their way
  bool bad = i0 < a.n_out && (jv < 0 || jv >= a.K || jp >= jv);
  for (int i = i0 + kThreads; i < a.n_out; i += kThreads) {
    const int j = __ldg(a.idx + i);
    bad |= j < 0 || j >= a.K || __ldg(a.idx + i - 1) >= j;
  }
  const int n_out = __syncthreads_or(bad) ? 0 : a.n_out;
  if (n_out < a.n_out && threadIdx.x == 0) set_status(a.status, SQ_ERR_INVALID_ARG);
  for (int i = i0; i < n_out; i += kThreads) {
    const int j = i < kThreads ? jv : __ldg(a.idx + i), jq = i == 0 ? -1 : i < kThreads ? jp : __ldg(a.idx + i - 1);
    idx_s[i] = j;
    for (int g = i > 0 ? (jq >> 7) + 1 : 0; g <= (j >> 7); ++g) ostart[g] = i;
    if (i == n_out - 1)
      for (int g = (j >> 7) + 1; g <= a.tpr; ++g) ostart[g] = n_out;
  }
  if (n_out == 0)
    for (int g = threadIdx.x; g <= a.tpr; g += kThreads) ostart[g] = 0;
  __syncthreads();

  const bool hi = tid4 >= 2;  // takes its code words in the order 2, 3, 0, 1
  const int cofs = lane * 64 + (hi ? 32 : 0), xofs = hi ? 16 : 0;
  int T[NT][4];
  float F[NT][4], U[NT][4];
  auto clear = [&] {
#pragma unroll
    for (int g = 0; g < NT; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        T[g][i] = 0;
        F[g][i] = U[g][i] = 0.0f;
      }
  };
  clear();
  bool head = cg == 0, timed_out = false;
  int slot = 0, sub = 0, in_slot = 0;  // tile of the slot, tiles in it
  uint32_t phase = 0;

  for (int t = t0; t < t1; ++t) {
    // activation words of this tile (the copies may still be on their way)
    uint32_t xw[NT][8];
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      const int8_t* xp = tk.x[g] + cg * kTileK;
      const int4 u = ldg_nc_v4(xp + xofs), v = ldg_nc_v4(xp + (16 - xofs));
      xw[g][0] = u.x; xw[g][1] = u.y; xw[g][2] = u.z; xw[g][3] = u.w;
      xw[g][4] = v.x; xw[g][5] = v.y; xw[g][6] = v.z; xw[g][7] = v.w;
    }
    const int o0 = ostart[cg], o1 = ostart[cg + 1];
    float xf[NT][2];  // the first outlier channel's activations, if the tile has one
#pragma unroll
    for (int g = 0; g < NT; ++g)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = __shfl_sync(0xffffffffu, tk.row, 2 * tid4 + c + 8 * g);
        xf[g][c] = o0 < o1 ? __ldg(a.xout + (int64_t)r * a.n_out + o0) : 0.0f;
      }
    if (sub == 0) {
      const bool landed = mbar_wait(&bars[warp * kMaxDepth + slot], (phase >> slot) & 1u);
      if (!__all_sync(0xffffffffu, landed)) {
        timed_out = true;
        break;
      }
      phase ^= 1u << slot;
      in_slot = gleft >= kPair && t + kPair <= t1 ? kPair : 1;
    }
    --gleft;
    const uint8_t* sl = ring + slot * SL::kBytes;
    const uint8_t* ql = sl + sub * 2048;
    const uint8_t* bl = sl + SL::kSign + sub * 256;
    const uint8_t* ml = sl + SL::kMask + sub * 256;
    uint32_t q[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint4 v = *reinterpret_cast<const uint4*>(ql + ((cofs ^ ((m & 2) << 4)) + (m & 1) * 16));
      q[m][0] = v.x; q[m][1] = v.y; q[m][2] = v.z; q[m][3] = v.w;
    }
    uint2 s = *reinterpret_cast<const uint2*>(bl + lane * 8);
    uint2 k = make_uint2(0u, 0u);
    if constexpr (MASK) k = *reinterpret_cast<const uint2*>(ml + lane * 8);
    const float c0 = *reinterpret_cast<const float*>(sl + SL::kScale + sub * 64 + gid * 4);
    const float c1 = *reinterpret_cast<const float*>(sl + SL::kScale + sub * 64 + gid * 4 + 32);
    if (hi) {
      s.x = swap_halves(s.x);
      s.y = swap_halves(s.y);
      if constexpr (MASK) {
        k.x = swap_halves(k.x);
        k.y = swap_halves(k.y);
      }
    }
    // R starts at the bits of 1.5 * 2^23, so that R (|R| < 2^22) is read as a float
    constexpr int kMagic = ASYM ? 0 : 0x4B400000;
    int R[NT][4], S[NT][4];
#pragma unroll
    for (int g = 0; g < NT; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        R[g][i] = kMagic;
        S[g][i] = 0;
      }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint32_t t0w = trunk_word<MASK>(s.x, k.x, 2 * m), t1w = trunk_word<MASK>(s.y, k.y, 2 * m);
      const uint32_t t2w = trunk_word<MASK>(s.x, k.x, 2 * m + 1), t3w = trunk_word<MASK>(s.y, k.y, 2 * m + 1);
#pragma unroll
      for (int g = 0; g < NT; ++g) {
        mma_s8(R[g], q[m][0], q[m][1], q[m][2], q[m][3], xw[g][2 * m], xw[g][2 * m + 1]);
        mma_s8(T[g], t0w, t1w, t2w, t3w, xw[g][2 * m], xw[g][2 * m + 1]);
        if constexpr (ASYM) {
          constexpr uint32_t one = 0x01010101u;
          mma_s8(S[g], one, one, one, one, xw[g][2 * m], xw[g][2 * m + 1]);
        }
      }
    }
    int z0 = 0, z1 = 0;
    if constexpr (ASYM) {
      z0 = *reinterpret_cast<const int*>(sl + SL::kZero + sub * 64 + gid * 4);
      z1 = *reinterpret_cast<const int*>(sl + SL::kZero + sub * 64 + gid * 4 + 32);
    }
#pragma unroll
    for (int g = 0; g < NT; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (ASYM) {
          // the zero-point's part is taken off in whole numbers (z may be large)
          const long long d = (long long)R[g][i] - (long long)(i < 2 ? z0 : z1) * (long long)S[g][i];
          F[g][i] = fmaf(i < 2 ? c0 : c1, (float)d, F[g][i]);
        } else {
          F[g][i] = fmaf(i < 2 ? c0 : c1, __int_as_float(R[g][i]) - 12582912.0f, F[g][i]);
        }
      }
    // outlier channels of this tile: the dequantized weight of the lane's two
    // rows from the slot, times its tokens' binary32 activations
    for (int o = o0; o < o1; ++o) {
      const int j = idx_s[o] & 127, w = (j & 31) >> 2;
      const int own = gid * 4 + (j >> 5);
      const int8_t* cb = reinterpret_cast<const int8_t*>(ql) + own * 64 + (w >> 1) * 16 + (w & 1) * 8 + (j & 3);
      const uint2 sb = *reinterpret_cast<const uint2*>(bl + own * 8);
      const int bit = tiled_bit_of(j & 31);
      float w0 = ((sb.x >> bit) & 1u) ? al[0] : -al[0], w1 = ((sb.y >> bit) & 1u) ? al[1] : -al[1];
      if constexpr (MASK) {
        const uint2 mb = *reinterpret_cast<const uint2*>(ml + own * 8);
        w0 = ((mb.x >> bit) & 1u) ? w0 : 0.0f;
        w1 = ((mb.y >> bit) & 1u) ? w1 : 0.0f;
      }
      w0 = fmaf(c0, (float)(cb[0] - z0), w0);
      w1 = fmaf(c1, (float)(cb[4] - z1), w1);
#pragma unroll
      for (int g = 0; g < NT; ++g) {
        const int r0 = __shfl_sync(0xffffffffu, tk.row, 2 * tid4 + 8 * g);
        const int r1 = __shfl_sync(0xffffffffu, tk.row, 2 * tid4 + 1 + 8 * g);
        const float x0 = o == o0 ? xf[g][0] : __ldg(a.xout + (int64_t)r0 * a.n_out + o);
        const float x1 = o == o0 ? xf[g][1] : __ldg(a.xout + (int64_t)r1 * a.n_out + o);
        U[g][0] = fmaf(w0, x0, U[g][0]);
        U[g][1] = fmaf(w0, x1, U[g][1]);
        U[g][2] = fmaf(w1, x0, U[g][2]);
        U[g][3] = fmaf(w1, x1, U[g][3]);
      }
    }
    if (++sub == in_slot) {
      __syncwarp();  // every lane has read the slot
      copy(slot);
      if (++slot == D) slot = 0;
      sub = 0;
    }

    const bool row_end = cg == a.tpr - 1;
    if (row_end || t + 1 == t1) {
      const bool whole = head && row_end;
#pragma unroll
      for (int g = 0; g < NT; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 2 * tid4 + (i & 1) + 8 * g, r = gid + (i >> 1) * 8;
          const float sx = __shfl_sync(0xffffffffu, tk.sx, c);
          const float v = fmaf(sx, fmaf(al[i >> 1], (float)T[g][i], F[g][i]), U[g][i]);
          if (c < tk.cnt) {
            if (whole) {
              if (rb * kTileRows + r < a.N) a.y[(int64_t)(tk.p0 + c) * a.N + rb * kTileRows + r] = v;
            } else {
              // slot 1: the piece that starts its row block; slot 0: one that continues it
              part[((warp * 2 + (head ? 1 : 0)) * 16 + r) * TG + c] = v;
            }
          }
        }
      clear();
      head = true;
      if (row_end && t + 1 < t1) {
        if (++rb == a.rbe) {
          rb = 0;
          grp = group_at(++u);
          gleft = per_group;
          enter_group();
        }
        enter_rows();
      }
    }
    if (++cg == a.tpr) cg = 0;
  }
  if (timed_out) {
    // the copies in flight end by themselves; wait (bounded) before the CTA leaves
    if (lane == 0) set_status(a.status, SQ_ERR_TIMEOUT);
    for (int d = 0; d < D; ++d) (void)mbar_wait(&bars[warp * kMaxDepth + d], (phase >> d) & 1u);
  }
  __syncthreads();
  if (t0 >= t1 || timed_out) return;
  // the row block that begins in this warp's range and ends past it: the later
  // warps' parts added in warp order
  const int last = (t1 - 1) / a.tpr;
  if (last * a.tpr >= t0 && t1 != (last + 1) * a.tpr) {
    const int end = (last + 1) * a.tpr;
    int w_hi = warp;
    while (w_hi + 1 < kWarps && (int)(((int64_t)(w_hi + 1) * len) >> 4) < end) ++w_hi;
#pragma unroll
    for (int g = 0; g < NT; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 2 * tid4 + (i & 1) + 8 * g, r = gid + (i >> 1) * 8;
        if (c >= tk.cnt) continue;
        float v = part[((warp * 2 + 1) * 16 + r) * TG + c];
        for (int w = warp + 1; w <= w_hi; ++w)
          if ((((int64_t)w * len) >> 4) < (((int64_t)(w + 1) * len) >> 4)) v += part[((w * 2) * 16 + r) * TG + c];
        if (rb * kTileRows + r < a.N) a.y[(int64_t)(tk.p0 + c) * a.N + rb * kTileRows + r] = v;
      }
  }
}

template <bool MASK, bool ASYM, int NT>
cudaError_t launch_nt(const GroupedArgs& a, int sm_count, cudaStream_t stream) {
  using SL = Slot<MASK, ASYM>;
  constexpr int TG = 8 * NT;
  Params p;
  p.a = a;
  const int part = kWarps * 2 * 16 * TG * 4;
  const int tables = (int)round_up(4 * (a.E + 1), 16) + (int)round_up(4 * (a.tpr + 1), 16) + (int)round_up(4 * (a.n_out + 1), 16);
  constexpr int kMax = 227 * 1024 - 2048;
  p.depth = std::min(kMaxDepth, (kMax - part - tables) / (kWarps * SL::kBytes));
  if (p.depth < 1) return cudaErrorInvalidValue;
  p.off_ring = 0;
  p.off_part = kWarps * p.depth * SL::kBytes;
  p.off_pre = p.off_part + part;
  p.off_ostart = p.off_pre + (int)round_up(4 * (a.E + 1), 16);
  p.off_idx = p.off_ostart + (int)round_up(4 * (a.tpr + 1), 16);
  const int smem = p.off_part + part + tables;
  auto* fn = k_grouped<MASK, ASYM, NT>;
  const cudaError_t e = ensure_smem_attr((const void*)fn, smem);
  if (e != cudaSuccess) return e;
  const int64_t groups = std::min<int64_t>(a.n, a.E + a.n / TG);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(sm_count, groups * a.rbe));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // (always: the kernel waits for the one before it, at its start or, with
  // SQ_LAUNCH_PDL, after the outlier list; only its launch is brought forward)
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

template <int NT>
cudaError_t launch_kind(const GroupedArgs& a, int sm_count, cudaStream_t stream) {
  if (a.zero)
    return a.mask ? launch_nt<true, true, NT>(a, sm_count, stream) : launch_nt<false, true, NT>(a, sm_count, stream);
  return a.mask ? launch_nt<true, false, NT>(a, sm_count, stream) : launch_nt<false, false, NT>(a, sm_count, stream);
}

}  // namespace

// Measured crossover, few-token kernel against the other, us at 16, 24 and 32 places per
// expert: 8 experts 4096 x 4096 54 : 63, 63 : 64, 92 : 64; 32 experts 2048 -> 1408 46 : 59,
// 64 : 60, 79 : 61; 4 experts 4096 -> 14336 93 : 117, 125 : 118, 138 : 118.  The host knows the
// average alone; with 60 % of the places at one expert the two meet there too (cold, at 20, 24
// and 32: 8 experts 4096 x 4096 65 : 70, 74 : 72, 92 : 74; 4 experts 4096 -> 14336 100 : 118,
// 109 : 117, 141 : 119).
bool grouped_many(int E, int64_t n) { return n >= 24 * (int64_t)E; }

size_t grouped_workspace_bytes(int E, int K, int64_t n, bool asym, int sm_count) {
  return grouped_many(E, n) && !asym ? grouped_tc5_workspace_bytes(K, n, sm_count) : 0;
}

cudaError_t launch_grouped(const GroupedArgs& a, void* workspace, int sm_count, cudaStream_t stream) {
  if (grouped_many(a.E, a.n) && grouped_tc5_supported(a.n_out, a.zero != nullptr))
    return launch_grouped_tc5(a, workspace, sm_count, stream);
  // Groups of 8 tokens up to 4 places per expert, of 16 above: the second eight
  // cost every tile 60 instructions, a second pass over the weights is rare at four
  // (16 tokens top-2 of 8 experts 14336 -> 4096: 115 against 139 us).  Groups of 8 : 16, cold, us
  // at 2, 4, 6, 8 and 12 random places per expert: 8 experts 4096 x 4096 47 : 49, 47 : 49, 55 : 55,
  // 59 : 53, 84 : 59; 4 experts 4096 -> 14336 59 : 59, 70 : 70, 94 : 88, 98 : 84, 148 : 82.
  if (a.n <= std::max(8, 4 * a.E)) return launch_kind<1>(a, sm_count, stream);
  return launch_kind<2>(a, sm_count, stream);
}

}  // namespace sq
