// sq_grouped_tc5.cu -- the linear layer grouped by expert for many tokens per
// expert, on the 5th-generation tensor cores (tcgen05.mma kind::i8, sm_100a).
//
// Same products as the few-token kernel: exact int32 sums of the residual codes
// per 128-channel group and of the +-1 trunk over the row,
//   y = sx (alpha T + sum_g s_g R_g) + sum_i What[r][idx_i] x_out[i].
//
// A tile is 128 weight rows of one expert (MMA M, one tensor-memory lane each)
// x up to 160 of its tokens (MMA N, a multiple of 32), so that a row's scales are
// one thread's scalars.  Persistent CTAs, one per SM, walk over the tiles of all
// experts, token tiles fastest (they share the weights in L2).
//   warp 0: tensor copies of a channel group's eight packed row blocks (codes, bits)
//     into the raw ring;
//   warp 2: TMA of the group's activation codes (rows in place order);
//   warps 4-11: turn the raw row blocks into the two K-major, 128-byte-swizzled
//     int8 operands, codes and +-1 (0 outside the mask) trunk bytes;
//   warp 3: picks the outlier channels' weights out of the raw row blocks as they
//     pass and dequantizes them, and fetches the token scales;
//   warp 1: per group, R into one of two tensor-memory buffers, and T;
//   warps 12-19: read each group's R and add s_g R to binary32 registers; at the
//     end of a tile read T, apply alpha and sx, add the outlier chunks and write y
//     (warps 12-15 the first half of the tile's tokens, 16-19 the second).
// Outlier channels are further steps of the same pipeline, 16 a step: What and x_out
// are cut into two tf32 parts each, and one stage holds [hi | hi] and [lo] of the
// weights (written by warps 4-11) and [hi | lo] of the activations (cut by the
// prologue kernel, brought by TMA); six kind::tf32 MMAs give all products but
// lo x lo: with the bits of lo that are not read, at most 2^-21 of a product is left out
// (the few-token kernel forms these products in binary32).  20 outlier channels cost 8 % of the time (4096
// places over 8 experts, 4096 -> 14336: 697 us without, 753 us with); on the CUDA
// cores of the promotion, a row of weights per lane, they cost 30 %.
// What bounds it: the hand-overs between five roles that have two operand stages and two R
// buffers.  A group takes 1300 clocks at 32 tokens and 1800 at 160.  Raw tile in and out, both
// operands in and out, activations in once and out twice are 160 KB a group through shared
// memory, 1250 clocks; but no unit is full: under ncu (8 experts, 4096 places) the tensor
// pipe is busy 31 % of the time, L1 and shared memory 48 %, DRAM 13 %.
// Hence the wide tile, one barrier per stage for both operands, and group scales
// that the promotion reads from memory itself.  At 758 us (the same weights again; 790 to 835
// with other weights at each call) that is 634 TFLOP/s of the layer's products, 0.16 of the
// int8 rate that the library's probe measures (4086 T op/s), 0.31 for the two products formed.
// The sums are integers because the tensor cores' binary32 sums are not exact
// enough: 16-bit operands accumulated over K = 4096 measured 4.4e-6 relative
// error (a truncation that grows with K; 1.6e-5 at 14336), the integer sums none.
// Every wait is bounded: one that runs out sets SQ_ERR_TIMEOUT and the CTA drains
// its copies and MMAs before it frees its tensor memory.
#include <stdint.h>

#include <algorithm>

#include "sq_grouped.cuh"
#include "sq_tcgen05.cuh"

namespace sq {
namespace {

using tc05::fence_after;
using tc05::fence_before;

constexpr int kThreads = 640;
constexpr int kLaunchRegs = 96;     // registers a thread at launch, as 640 threads allow
constexpr int kProducerRegs = 64, kOperandRegs = 64, kPromoteRegs = 144;
constexpr int kOperandWarps = 8;    // one row block each
constexpr int kSets = 2;            // warpgroups of the promotion, half of the tokens each
constexpr int kPromoteThreads = 128 * kSets;
constexpr int kRows = 128;          // weight rows per tile (MMA M)
constexpr int kTokens = 160;        // most tokens per tile (MMA N)
constexpr int kTokenUnit = 16 * kSets;  // MMA N is a multiple of this
constexpr int kCols = kTokens / kSets, kPieces = kCols / 16;
constexpr int kBlocks = kRows / kTileRows;
constexpr uint32_t kTmemCols = 512; // T [0, 160), R of group g at 160 + 160 (g % 2)
constexpr int kStages = 2;
constexpr int kABytes = kRows * kTileK;      // one operand: 16 KB
constexpr int kBBytes = kTokens * kTileK;    // 20 KB
constexpr int kStageBytes = 2 * kABytes + kBBytes;
static_assert(kStageBytes % 1024 == 0 && kCols % 16 == 0 && 3 * kTokens <= (int)kTmemCols, "tile layout");
constexpr int kMaxOut = 128;        // outlier channels this kernel takes
constexpr int kOutHeld = 32;        // of them held in shared memory under the tile's products
constexpr int kOutChunk = 16;       // of them in one stage

constexpr uint64_t kWaitNs = 1000000000ull;  // of the waits when winding down

template <bool MASK>
struct Raw {
  static constexpr int kSign = kBlocks * 2048;
  static constexpr int kMask = kSign + kBlocks * 256;
  static constexpr int kBytes = MASK ? kMask + kBlocks * 256 : kMask;
  static constexpr int kStages = MASK ? 3 : 4;  // of the ring
};
constexpr int kRawMost = 4;

struct Aux {
  uint64_t raw_full[kRawMost], raw_empty[kRawMost];
  uint64_t full[kStages], empty[kStages];
  uint64_t accf[2], acce[2];
  uint64_t t_full, t_empty, wo_full, wo_empty, drain;
  uint32_t tmem_base;
  int abort;
  int part[kThreads / 32];
};

// The stack's arrays as rows of row blocks, so that one tensor copy brings eight row
// blocks' tiles of a channel group (a bulk copy for each of the 24 pieces cost 90
// clocks of the issuing warp, 2200 a group).
struct WeightMaps {
  CUtensorMap codes, sign, mask;
};

struct Params {
  GroupedArgs a;
  const float* sxp;   // [n] token scales in place order
  float* wout;        // [CTAs][kMaxOut][kRows] outlier weights of the CTA's tile
  int rt;             // row tiles per expert
  int off_raw, off_sx, off_wh, off_aux, off_pre, off_ostart, off_oj;  // shared-memory offsets
};

// D (s32) (+)= A (s8) B (s8), both K-major; M = 128, N = n.  A K step of 32 bytes is
// 2 in a descriptor's address field.
__device__ __forceinline__ uint32_t idesc_of(int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0));
}

// D (f32) (+)= A (tf32) B (tf32); a K step of 8 is 32 bytes too.
__device__ __forceinline__ uint32_t idesc_tf32_of(int n) {
  return (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
__device__ __forceinline__ void mma_tf32(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0));
}

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Aux* aux, const Params& p) {
  // (the clock is read once in 32 tries: reading it at every one slows the SM)
  uint64_t t0 = 0;
  for (uint32_t n = 0;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 31u) == 31u) {
      const uint64_t now = global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > p.a.wait_ns) break;
    }
  }
  set_status(p.a.status, SQ_ERR_TIMEOUT);
  atomicExch(&aux->abort, 1);
  return false;
}
// The same for a whole warp, with a warp-uniform result (so that what follows may
// run on the uniform datapath).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Aux* aux, const Params& p) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, aux, p));
}
__device__ __forceinline__ bool aborted(const Aux* aux) {
  return *reinterpret_cast<const volatile int*>(&aux->abort) != 0;
}

// 16 consecutive TMEM columns of this thread's lane: the load, and the wait after
// which r may be used.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, int (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(int (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// f(c, r) for the 16-column pieces c of [0, h) (h <= kCols) from column `src`, two
// pieces' loads in flight per wait (columns past h are read, not used).
template <class F>
__device__ __forceinline__ void tmem_pieces(uint32_t src, int h, F f) {
#pragma unroll
  for (int c = 0; c < kPieces; c += 2) {
    if (16 * c < h) {
      int r[2][16];
      tmem_ld16(src + 16 * c, r[0]);
      if (c + 1 < kPieces) tmem_ld16(src + 16 * (c + 1), r[1]);
      tmem_wait16(r[0]);
      if (c + 1 < kPieces) tmem_wait16(r[1]);
      f(c, r[0]);
      if (c + 1 < kPieces && 16 * (c + 1) < h) f(c + 1, r[1]);
    }
  }
}
// Two binary32 values in a 64-bit register (first in the low half) and the packed
// operations on them: half the instructions of the promotion.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// One tile: an expert's 128 rows x up to kTokens of its places.
struct Tile {
  int rb0;       // first row block in the stack
  int blocks;    // row blocks of the expert in this tile (1..8)
  int row0;      // first row in the expert
  int p0, cnt;   // first place, tokens
  int n;         // MMA N: cnt rounded up to kTokenUnit
};
__device__ __forceinline__ Tile tile_at(const Params& p, const int* pre, int item) {
  const GroupedArgs& a = p.a;
  const int e = unit_expert(pre, a.E, item / p.rt);
  const int local = item - pre[e] * p.rt, ntt = pre[e + 1] - pre[e];
  const int tt = local % ntt, rt = local / ntt;
  const int2 seg = segment_bounds(a.offsets, a.n, e, nullptr);
  const int total = seg.y - seg.x;
  const int ts = ((total + ntt - 1) / ntt + kTokenUnit - 1) / kTokenUnit * kTokenUnit;  // (ntt - 1) ts < total
  Tile t;
  t.rb0 = e * a.rbe + rt * kBlocks;
  t.blocks = min(kBlocks, a.rbe - rt * kBlocks);
  t.row0 = rt * kRows;
  t.p0 = seg.x + tt * ts;
  t.cnt = min(ts, total - tt * ts);
  t.n = (t.cnt + kTokenUnit - 1) / kTokenUnit * kTokenUnit;
  return t;
}
template <bool MASK>
__global__ void __launch_bounds__(kThreads, 1)
    k_grouped_tc5(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ WeightMaps wm, const Params p) {
  using RW = Raw<MASK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Aux* aux = reinterpret_cast<Aux*>(smem + p.off_aux);
  int* pre = reinterpret_cast<int*>(smem + p.off_pre);
  int* ostart = reinterpret_cast<int*>(smem + p.off_ostart);
  uint8_t* oj = smem + p.off_oj;  // the outlier channels in their groups
  const GroupedArgs& a = p.a;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < RW::kStages; ++s) {
      mbar_init(&aux->raw_full[s], 1);
      mbar_init(&aux->raw_empty[s], kOperandWarps + 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&aux->full[s], kOperandWarps + 1);
      mbar_init(&aux->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&aux->accf[b], 1);
      mbar_init(&aux->acce[b], kPromoteThreads / 32);
    }
    mbar_init(&aux->t_full, 1);
    mbar_init(&aux->t_empty, kPromoteThreads / 32);
    mbar_init(&aux->wo_full, 1);
    mbar_init(&aux->wo_empty, kOperandWarps + kPromoteThreads / 32);
    mbar_init(&aux->drain, 1);
    aux->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc05::tmem_alloc(&aux->tmem_base, kTmemCols);
  // the outlier list; one that is not strictly ascending in [0, K) is reported
  // by the prologue kernel and taken as empty
  bool bad = false;
  for (int i = threadIdx.x; i < a.n_out; i += kThreads) {
    const int j = __ldg(a.idx + i), jp = i > 0 ? __ldg(a.idx + i - 1) : -1;
    bad |= j < 0 || j >= a.K || jp >= j;
  }
  const int n_out = __syncthreads_or(bad) ? 0 : a.n_out;
  const int steps = a.tpr + (n_out + kOutChunk - 1) / kOutChunk;  // of a tile: channel groups, outlier chunks
  for (int i = threadIdx.x; i < n_out; i += kThreads) {
    const int g0 = i > 0 ? (__ldg(a.idx + i - 1) >> 7) + 1 : 0, g1 = __ldg(a.idx + i) >> 7;
    for (int g = g0; g <= g1; ++g) ostart[g] = i;
    oj[i] = (uint8_t)(__ldg(a.idx + i) & 127);
  }
  for (int g = (n_out > 0 ? (__ldg(a.idx + n_out - 1) >> 7) + 1 : 0) + threadIdx.x; g <= a.tpr; g += kThreads)
    ostart[g] = n_out;
  pdl_wait();
  pdl_launch_dependents();
  const int units = segment_units(a.offsets, a.E, a.n, a.status, kTokens, pre, aux->part);
  const int items = units * p.rt;
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = aux->tmem_base;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp == 0) {
      // ---- raw producer: the tile's row blocks of each channel group
      uint32_t g = 0;
      int last[RW::kStages];
#pragma unroll
      for (int s = 0; s < RW::kStages; ++s) last[s] = -1;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const Tile t = tile_at(p, pre, item);
        for (int kb = 0; kb < a.tpr; ++kb, ++g) {
          const int s = (int)(g % RW::kStages);
          const uint32_t use = g / RW::kStages;
          if (g >= RW::kStages) ok = warp_wait(&aux->raw_empty[s], (use & 1u) ^ 1u, aux, p);
          ok = __all_sync(0xffffffffu, ok && !aborted(aux));
          if (!ok) break;
          if (kb == a.skip_group) continue;
          uint8_t* st = smem + p.off_raw + s * RW::kBytes;
          // (row blocks past the expert are the next expert's, past the stack zero;
          // their rows are not written)
          if (elect_one()) {
            mbar_arrive_expect_tx(&aux->raw_full[s], RW::kBytes);
            tc05::tma_load_2d(st, &wm.codes, kb * 256, t.rb0, &aux->raw_full[s]);
            tc05::tma_load_2d(st + RW::kSign, &wm.sign, kb * 32, t.rb0, &aux->raw_full[s]);
            if (MASK) tc05::tma_load_2d(st + RW::kMask, &wm.mask, kb * 32, t.rb0, &aux->raw_full[s]);
          }
          __syncwarp();
          last[s] = (int)use;
        }
      }
      if (aborted(aux)) {  // every requested stage must have landed
#pragma unroll
        for (int s = 0; s < RW::kStages; ++s)
          if (last[s] >= 0) (void)mbar_wait(&aux->raw_full[s], (uint32_t)last[s] & 1u, kWaitNs);
      }
    } else if (warp == 2) {
      // ---- activation producer: n rows of 128 codes per channel group, of 32
      // binary32 values per outlier chunk (16 channels' first parts, their second)
      uint32_t g = 0;
      int last[kStages];
#pragma unroll
      for (int s = 0; s < kStages; ++s) last[s] = -1;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const Tile t = tile_at(p, pre, item);
        for (int kb = 0; kb < steps; ++kb, ++g) {
          const int s = (int)(g % kStages);
          const uint32_t use = g / kStages;
          if (g >= kStages) ok = warp_wait(&aux->empty[s], (use & 1u) ^ 1u, aux, p);
          ok = __all_sync(0xffffffffu, ok && !aborted(aux));
          if (!ok) break;
          uint8_t* st = smem + s * kStageBytes + 2 * kABytes;
          if (elect_one()) {
            mbar_arrive_expect_tx(&aux->full[s], (uint32_t)t.n * kTileK);
            for (int r = 0; r < t.n; r += kTokenUnit)
              if (kb < a.tpr)
                tc05::tma_load_2d(st + r * kTileK, &tmB, kb * kTileK, t.p0 + r, &aux->full[s]);
              else
                tc05::tma_load_2d(st + r * kTileK, &tmX, 0, (kb - a.tpr) * a.n + t.p0 + r, &aux->full[s]);
          }
          __syncwarp();
          last[s] = (int)use;
        }
      }
      // winding down: every requested stage must have landed.  The stage's barrier
      // also counts the operand warps, which may have stopped: they arrive once
      // more for it when they leave
      if (aborted(aux)) {
#pragma unroll
        for (int s = 0; s < kStages; ++s)
          if (last[s] >= 0) (void)mbar_wait(&aux->full[s], (uint32_t)last[s] & 1u, kWaitNs);
      }
    } else if (warp == 3) {
      // ---- under the tile's products: its token scales, and the outlier channels'
      // dequantized weights as rows of the tile's 128 (the first kOutHeld of them in
      // shared memory, the rest in the CTA's scratch)
      float* sxh = reinterpret_cast<float*>(smem + p.off_sx);
      float* wh = reinterpret_cast<float*>(smem + p.off_wh);
      float* wout = p.wout + (int64_t)blockIdx.x * kMaxOut * kRows + lane;
      uint32_t g = 0, n_items = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x, ++n_items) {
        const Tile t = tile_at(p, pre, item);
        // this lane's rows: 32 i + lane of the tile; their trunk scales, and the group
        // scales of the next group, loaded a group ahead
        float al[4], sc[4];
        auto group_scales = [&](int kb) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sc[i] = __ldg(a.scale + ((t.rb0 + min(2 * i + (lane >> 4), t.blocks - 1)) * (int64_t)a.tpr + kb) * kTileRows + (lane & 15));
        };
#pragma unroll
        for (int i = 0; i < 4; ++i)
          al[i] = __ldg(a.alpha + (t.rb0 + min(2 * i + (lane >> 4), t.blocks - 1)) * (int64_t)kTileRows + (lane & 15));
        group_scales(0);
        if (n_items > 0) ok = warp_wait(&aux->wo_empty, (n_items & 1u) ^ 1u, aux, p);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kTokens / 32; ++i) {  // (waited for at the tile's end; zero past its tokens)
          const bool in = lane + 32 * i < t.cnt;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(sxh + lane + 32 * i)),
                       "l"(p.sxp + t.p0 + (in ? lane + 32 * i : 0)), "r"(in ? 4 : 0) : "memory");
        }
        for (int kb = 0; kb < a.tpr; ++kb, ++g) {
          const int s = (int)(g % RW::kStages);
          ok = warp_wait(&aux->raw_full[s], (g / RW::kStages) & 1u, aux, p) && !aborted(aux);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* st = smem + p.off_raw + s * RW::kBytes;
          for (int o = ostart[kb]; o < ostart[kb + 1]; ++o) {
            const int j = oj[o], w = (j & 31) >> 2, bit = tiled_bit_of(j & 31);
            const int own = (lane & 7) * 4 + (j >> 5), R = (lane >> 3) & 1;  // rows lane % 16 of a block
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int blk = 2 * i + (lane >> 4);
              const int code = reinterpret_cast<const int8_t*>(
                  st)[blk * 2048 + own * 64 + (w >> 1) * 16 + ((w & 1) * 2 + R) * 4 + (j & 3)];
              const uint32_t sb = *reinterpret_cast<const uint32_t*>(st + RW::kSign + blk * 256 + own * 8 + 4 * R);
              float tr = ((sb >> bit) & 1u) ? al[i] : -al[i];
              if constexpr (MASK) {
                const uint32_t mb = *reinterpret_cast<const uint32_t*>(st + RW::kMask + blk * 256 + own * 8 + 4 * R);
                if (!((mb >> bit) & 1u)) tr = 0.0f;
              }
              const float what = fmaf(sc[i], (float)code, tr);
              if (o < kOutHeld) wh[o * kRows + 32 * i + lane] = what;
              else wout[o * kRows + 32 * i] = what;
            }
          }
          if (kb + 1 < a.tpr) group_scales(kb + 1);
          __syncwarp();
          if (lane == 0) mbar_arrive(&aux->raw_empty[s]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&aux->wo_full);
      }
    } else if (warp == 1) {
      // ---- MMA issuer (the whole warp walks; one lane issues)
      uint32_t g = 0, n_items = 0;
      bool ok = true;
      const uint32_t s0 = smem_u32(smem);
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x, ++n_items) {
        const Tile t = tile_at(p, pre, item);
        const uint32_t idesc = idesc_of(t.n), idesc_x = idesc_tf32_of(t.n);
        for (int kb = 0; kb < steps; ++kb, ++g) {
          const int s = (int)(g % kStages), b = (int)(g & 1u);
          ok = warp_wait(&aux->full[s], (g / kStages) & 1u, aux, p) &&
               (g < 2 || warp_wait(&aux->acce[b], ((g >> 1) & 1u) ^ 1u, aux, p));
          if (!ok) break;
          fence_after();
          const uint64_t da = tc05::sw128_desc(s0 + s * kStageBytes);
          const uint64_t dt = da + (kABytes >> 4), db = da + (2 * kABytes >> 4);
          const uint32_t d = tmem + kTokens + kTokens * b;
          if (kb >= a.tpr) {  // What (first | first parts) x (first | second), What (second) x (first)
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mma_tf32(d, da + 2 * kk, db + 2 * kk, idesc_x, kk > 0);
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) mma_tf32(d, dt + 2 * kk, db + 2 * kk, idesc_x, true);
              tc05::mma_commit(&aux->accf[b]);
              tc05::mma_commit(&aux->empty[s]);
            }
            __syncwarp();
            continue;
          }
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_i8(d, da + 2 * kk, db + 2 * kk, idesc, kk > 0);
            tc05::mma_commit(&aux->accf[b]);
          }
          __syncwarp();
          if (kb == 0 && n_items > 0) {  // T of the tile before has been read
            ok = warp_wait(&aux->t_empty, (n_items & 1u) ^ 1u, aux, p);
            if (!ok) break;
            fence_after();
          }
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_i8(tmem, dt + 2 * kk, db + 2 * kk, idesc, kb > 0 || kk > 0);
            tc05::mma_commit(&aux->empty[s]);
            if (kb == a.tpr - 1) tc05::mma_commit(&aux->t_full);
          }
          __syncwarp();
        }
      }
      if (aborted(aux)) {  // the MMAs issued must be done before the tensor memory is freed
        if (elect_one()) tc05::mma_commit(&aux->drain);
        __syncwarp();
        (void)mbar_wait(&aux->drain, 0u, kWaitNs);
      }
    }
  } else if (warp < 4 + kOperandWarps) {
    // ---- operands: one row block of each group per warp
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOperandRegs));
    const int cw = warp - 4, gid = lane >> 2, tid4 = lane & 3;
    const bool hi = tid4 >= 2;  // takes its two 16-channel pieces in the other order
    const int odd = (gid & 1) * 16;
    uint32_t g = 0, rg = 0, n_items = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x, ++n_items) {
      for (int kb = 0; kb < a.tpr; ++kb, ++g, ++rg) {
        const int sr = (int)(rg % RW::kStages), sa = (int)(g % kStages);
        ok = warp_wait(&aux->raw_full[sr], (rg / RW::kStages) & 1u, aux, p);
        if (ok && g >= kStages) ok = warp_wait(&aux->empty[sa], ((g / kStages) & 1u) ^ 1u, aux, p);
        ok = __all_sync(0xffffffffu, ok && !aborted(aux));
        if (!ok) break;
        const uint8_t* st = smem + p.off_raw + sr * RW::kBytes;
        const uint8_t* cb = st + cw * 2048 + lane * 64;
        uint2 sg = *reinterpret_cast<const uint2*>(st + RW::kSign + cw * 256 + lane * 8);
        uint2 mk = make_uint2(0u, 0u);
        if constexpr (MASK) mk = *reinterpret_cast<const uint2*>(st + RW::kMask + cw * 256 + lane * 8);
        if (hi) {
          sg.x = swap_halves(sg.x);
          sg.y = swap_halves(sg.y);
          if constexpr (MASK) {
            mk.x = swap_halves(mk.x);
            mk.y = swap_halves(mk.y);
          }
        }
        // row gid (and gid + 8) of the block: 128 bytes in a 1024-byte atom of 8
        // rows, 16-byte chunk c at c ^ gid; channels 32 tid4 + 16 c' are chunk 2 tid4 + c'
        uint8_t* ao = smem + sa * kStageBytes + cw * 2048 + gid * 128;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = hi ? i ^ 1 : i;  // 16 channels: words 4c .. 4c + 3
          // (odd rows read the piece's two words in the other order, so that eight
          // neighbouring lanes read eight different 16-byte columns)
          const uint4 e0 = *reinterpret_cast<const uint4*>(cb + 32 * c + odd);
          const uint4 e1 = *reinterpret_cast<const uint4*>(cb + 32 * c + (odd ^ 16));
          const uint4 u = odd ? e1 : e0, v = odd ? e0 : e1;
          uint8_t* o = ao + (((2 * tid4 + c) ^ gid) << 4);
          *reinterpret_cast<uint4*>(o) = make_uint4(u.x, u.z, v.x, v.z);
          *reinterpret_cast<uint4*>(o + 1024) = make_uint4(u.y, u.w, v.y, v.w);
          // (the sign words are swapped alike, so the shifts are fixed)
          *reinterpret_cast<uint4*>(o + kABytes) =
              make_uint4(trunk_word<MASK>(sg.x, mk.x, 4 * i), trunk_word<MASK>(sg.x, mk.x, 4 * i + 1),
                         trunk_word<MASK>(sg.x, mk.x, 4 * i + 2), trunk_word<MASK>(sg.x, mk.x, 4 * i + 3));
          *reinterpret_cast<uint4*>(o + kABytes + 1024) =
              make_uint4(trunk_word<MASK>(sg.y, mk.y, 4 * i), trunk_word<MASK>(sg.y, mk.y, 4 * i + 1),
                         trunk_word<MASK>(sg.y, mk.y, 4 * i + 2), trunk_word<MASK>(sg.y, mk.y, 4 * i + 3));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&aux->full[sa]);
          mbar_arrive(&aux->raw_empty[sr]);
        }
      }
      if (!ok) break;
      // the outlier chunks: What of 16 channels cut in two, 8 channels of a row per thread
      ok = warp_wait(&aux->wo_full, n_items & 1u, aux, p);
      if (!ok) break;
      const float* wout = p.wout + (int64_t)blockIdx.x * kMaxOut * kRows;
      const float* wh = reinterpret_cast<const float*>(smem + p.off_wh);
      const int row = ((cw & 3) << 5) + lane, half = cw >> 2;
      for (int o0 = 8 * half; o0 < (steps - a.tpr) * kOutChunk; o0 += kOutChunk, ++g) {
        const int sa = (int)(g % kStages);
        if (g >= kStages) ok = warp_wait(&aux->empty[sa], ((g / kStages) & 1u) ^ 1u, aux, p);
        ok = __all_sync(0xffffffffu, ok && !aborted(aux));
        if (!ok) break;
        const float* src = (o0 < kOutHeld ? wh : wout) + o0 * kRows + row;
        float h[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) cut_tf32(o0 + i < n_out ? src[i * kRows] : 0.0f, h[i], l[i]);
        uint8_t* ao = smem + sa * kStageBytes + row * 128;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = ((2 * half + i) ^ (row & 7)) << 4;
          const float4 hv = make_float4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
          *reinterpret_cast<float4*>(ao + at) = hv;
          *reinterpret_cast<float4*>(ao + (at ^ 64)) = hv;
          *reinterpret_cast<float4*>(ao + kABytes + at) = make_float4(l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux->full[sa]);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&aux->wo_empty);
    }
    // winding down after a timeout: the activation producer waits for the copies of
    // the stages it has requested, on barriers that count these warps too
    if (aborted(aux) && lane == 0)
      for (int s = 0; s < kStages; ++s) mbar_arrive(&aux->full[s]);
  } else {
    // ---- promotion and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPromoteRegs));
    const int set = (warp - 4 - kOperandWarps) >> 2, q = warp & 3;  // half of the tokens; tensor-memory lane quarter
    const int my_row = 32 * q + lane;
    uint32_t g = 0, n_items = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x, ++n_items) {
      const Tile t = tile_at(p, pre, item);
      const int cols = t.n / kSets;
      f32x2 F[kCols / 2];  // this row's sums, two tokens each
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) F[i] = 0ull;
      // this row's group scales, two groups ahead
      const float* sp = a.scale + (int64_t)(t.rb0 + min(my_row >> 4, t.blocks - 1)) * a.tpr * kTileRows + (my_row & 15);
      float s_next[2] = {__ldg(sp), a.tpr > 1 ? __ldg(sp + kTileRows) : 0.0f};
      for (int kb = 0; kb < a.tpr; ++kb, ++g) {
        const int b = (int)(g & 1u);
        const float s1 = s_next[0];
        s_next[0] = s_next[1];
        s_next[1] = kb + 2 < a.tpr ? __ldg(sp + (kb + 2) * kTileRows) : 0.0f;
        ok = warp_wait(&aux->accf[b], (g >> 1) & 1u, aux, p);
        if (!ok) break;
        fence_after();
        const f32x2 s = pack2(s1, s1);
        const uint32_t src = tmem + ((uint32_t)(32 * q) << 16) + kTokens + kTokens * b + cols * set;
        tmem_pieces(src, cols, [&](int c, const int(&r)[16]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) F[8 * c + i] = fma2(s, pack2((float)r[2 * i], (float)r[2 * i + 1]), F[8 * c + i]);
        });
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux->acce[b]);
      }
      if (!ok) break;
      ok = warp_wait(&aux->t_full, n_items & 1u, aux, p) && warp_wait(&aux->wo_full, n_items & 1u, aux, p);
      if (!ok) break;
      fence_after();
      const int row = t.row0 + my_row;
      const bool live = my_row < t.blocks * kTileRows && row < a.N;
      const float al = __ldg(a.alpha + (int64_t)t.rb0 * kTileRows + min(my_row, t.blocks * kTileRows - 1));
      const int t0 = set * cols;                // this warp's tokens in the tile
      const int nt = max(0, min(cols, t.cnt - t0));
      const f32x2 al2 = pack2(al, al);
      tmem_pieces(tmem + ((uint32_t)(32 * q) << 16) + t0, cols, [&](int c, const int(&r)[16]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          F[8 * c + i] = fma2(al2, pack2((float)r[2 * i], (float)r[2 * i + 1]), F[8 * c + i]);
      });
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&aux->t_empty);
      const float* sxh = reinterpret_cast<const float*>(smem + p.off_sx) + t0;
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        if (16 * c >= cols) break;
        const ulonglong2* xr = reinterpret_cast<const ulonglong2*>(sxh + 16 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 x = xr[i];
          F[8 * c + 2 * i] = mul2(F[8 * c + 2 * i], x.x);
          F[8 * c + 2 * i + 1] = mul2(F[8 * c + 2 * i + 1], x.y);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&aux->wo_empty);
      for (int kb = a.tpr; kb < steps; ++kb, ++g) {  // the outlier chunks
        const int b = (int)(g & 1u);
        ok = warp_wait(&aux->accf[b], (g >> 1) & 1u, aux, p);
        if (!ok) break;
        fence_after();
        tmem_pieces(tmem + ((uint32_t)(32 * q) << 16) + kTokens + kTokens * b + t0, cols, [&](int c, const int(&r)[16]) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            F[8 * c + i] = add2(F[8 * c + i], pack2(__int_as_float(r[2 * i]), __int_as_float(r[2 * i + 1])));
        });
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux->acce[b]);
      }
      if (!ok) break;
      if (live) {
        float* yr = a.y + (int64_t)(t.p0 + t0) * a.N + row;
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
          const float2 v = unpack2(F[i]);
          if (2 * i < nt) yr[(int64_t)(2 * i) * a.N] = v.x;
          if (2 * i + 1 < nt) yr[(int64_t)(2 * i + 1) * a.N] = v.y;
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tc05::tmem_dealloc(tmem, kTmemCols);
  }
}

// Before the tiles: each place's activation codes (GATHER: rows in place order for
// the TMA), scale and outlier values (rows of a chunk's 16 channels,
// cut in two), one warp per place.
template <bool GATHER>
__global__ void __launch_bounds__(256) k_grouped_rows(const GroupedArgs a, int8_t* xs, float* sxp, float* xop) {
  const int lane = threadIdx.x & 31;
  if (a.pdl) pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    bool bad = false;
    for (int i = lane; i < a.n_out; i += 32) {
      const int j = __ldg(a.idx + i), jp = i > 0 ? __ldg(a.idx + i - 1) : -1;
      bad |= j < 0 || j >= a.K || jp >= j;
    }
    if (bad) set_status(a.status, SQ_ERR_INVALID_ARG);
  }
  if (a.zero_rest) zero_rest(a);
  const int live = min(max(__ldg(a.offsets + a.E), 0), a.n);
  for (int p = blockIdx.x * 8 + (threadIdx.x >> 5); p < live; p += gridDim.x * 8) {
    const int r = source_row(a, p);
    if (GATHER) {
      const int4* src = reinterpret_cast<const int4*>(a.xq + (int64_t)r * a.xs);
      int4* dst = reinterpret_cast<int4*>(xs + (int64_t)p * a.xs);
      for (int i = lane; i < a.xs / 16; i += 32) dst[i] = __ldg(src + i);
    }
    if (lane == 0) sxp[p] = __ldg(a.sx + r);
    for (int i = lane; i < (a.n_out + kOutChunk - 1) / kOutChunk * kOutChunk; i += 32) {
      float* dst = xop + ((int64_t)(i / kOutChunk) * a.n + p) * (2 * kOutChunk) + i % kOutChunk;
      cut_tf32(i < a.n_out ? __ldg(a.xout + (int64_t)r * a.n_out + i) : 0.0f, dst[0], dst[kOutChunk]);
    }
  }
}

struct Carve {
  size_t xs, sxp, xop, wout, total;
};
Carve carve(int K, int64_t n, int sm_count) {
  Carve c;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (size_t)round_up((int64_t)(off + bytes), 256);
    return at;
  };
  c.xs = take((size_t)n * xq_stride_of(K));
  c.sxp = take((size_t)n * 4);
  c.xop = take((size_t)n * kMaxOut * 8);
  c.wout = take((size_t)sm_count * kMaxOut * kRows * 4);
  c.total = off;
  return c;
}

template <bool MASK>
cudaError_t launch_tiles(const CUtensorMap& mb, const CUtensorMap& mx, const WeightMaps& wm, Params p, int grid, cudaStream_t stream) {
  p.off_raw = kStages * kStageBytes;
  p.off_sx = p.off_raw + Raw<MASK>::kStages * Raw<MASK>::kBytes;
  p.off_wh = p.off_sx + kTokens * 4;
  p.off_aux = p.off_wh + kOutHeld * kRows * 4;
  p.off_pre = p.off_aux + (int)round_up(sizeof(Aux), 16);
  p.off_ostart = p.off_pre + (int)round_up(4 * (p.a.E + 1), 16);
  p.off_oj = p.off_ostart + 4 * (p.a.tpr + 1);
  const int smem = (int)round_up(p.off_oj + kMaxOut, 16) + 1024;
  if (smem > 227 * 1024) return cudaErrorInvalidValue;
  auto* fn = k_grouped_tc5<MASK>;
  // the register split of the warpgroups must add up to the launch's registers
  static_assert(128 * kProducerRegs + 32 * kOperandWarps * kOperandRegs + kPromoteThreads * kPromoteRegs <= kThreads * kLaunchRegs, "register split");
  static const bool regs_ok = [&] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, fn) == cudaSuccess && at.numRegs == kLaunchRegs;
  }();
  if (!regs_ok) return cudaErrorInvalidKernelImage;
  const cudaError_t e = ensure_smem_attr((const void*)fn, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, mb, mx, wm, p);
}

}  // namespace

bool grouped_tc5_supported(int n_out, bool asym) {
  return !asym && n_out <= kMaxOut && tc05::encode_fn() != nullptr;
}

size_t grouped_tc5_workspace_bytes(int K, int64_t n, int sm_count) { return carve(K, n, sm_count).total; }

cudaError_t launch_grouped_tc5(const GroupedArgs& a, void* workspace, int sm_count, cudaStream_t stream) {
  const Carve c = carve(a.K, a.n, sm_count);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  Params p;
  p.a = a;
  int8_t* xs = reinterpret_cast<int8_t*>(w + c.xs);
  float* sxp = reinterpret_cast<float*>(w + c.sxp);
  float* xop = reinterpret_cast<float*>(w + c.xop);
  p.sxp = sxp;
  p.wout = reinterpret_cast<float*>(w + c.wout);
  p.rt = (int)ceil_div(a.rbe, kBlocks);
  // rows of the activation map: the places (in place order already without an
  // order), those past the last row read as zero
  CUtensorMap mb;
  const int64_t rows = a.order ? a.n : std::min(a.n, a.rows);
  if (!tc05::make_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.order ? xs : a.xq, (uint64_t)a.xs, (uint64_t)rows,
                      (uint64_t)a.xs, kTileK, kTokenUnit, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  CUtensorMap mx;  // rows of the outlier chunks
  if (!tc05::make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, xop, 8 * kOutChunk,
                      (uint64_t)a.n * std::max<int64_t>(1, ceil_div(a.n_out, kOutChunk)), 8 * kOutChunk, 8 * kOutChunk,
                      kTokenUnit, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  WeightMaps wm;
  const uint64_t blocks = (uint64_t)a.E * a.rbe;
  auto weight_map = [&](CUtensorMap* m, const void* base, int tile_bytes) {  // 8-byte elements
    return tc05::make_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, base, (uint64_t)a.tpr * tile_bytes / 8, blocks,
                          (uint64_t)a.tpr * tile_bytes, tile_bytes / 8, kBlocks, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  if (!weight_map(&wm.codes, a.res, 2048) || !weight_map(&wm.sign, a.sign, 256) ||
      !weight_map(&wm.mask, a.mask ? a.mask : a.sign, 256))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(ceil_div(a.n, 8), 4 * sm_count));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 1 : 0;
  const cudaError_t e = a.order ? cudaLaunchKernelEx(&cfg, k_grouped_rows<true>, a, xs, sxp, xop)
                                : cudaLaunchKernelEx(&cfg, k_grouped_rows<false>, a, xs, sxp, xop);
  if (e != cudaSuccess) return e;
  const int64_t tiles = std::min<int64_t>(a.n, a.E + a.n / kTokens) * p.rt;
  if (tiles >= INT32_MAX) return cudaErrorInvalidValue;
  const int grid = (int)std::min<int64_t>(tiles, sm_count);
  return a.mask ? launch_tiles<true>(mb, mx, wm, p, grid, stream) : launch_tiles<false>(mb, mx, wm, p, grid, stream);
}

}  // namespace sq
