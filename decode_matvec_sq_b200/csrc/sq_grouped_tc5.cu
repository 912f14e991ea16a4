// sq_grouped_tc5.cu -- the linear layer grouped by expert for many tokens per
// expert, on the 5th-generation tensor cores (tcgen05.mma kind::i8, sm_100a).
//
// Same products as the few-token kernel: exact int32 sums of the residual codes
// per 128-channel group and of the +-1 trunk over the row,
//   y = sx (alpha T + sum_g s_g R_g) + sum_i What[r][idx_i] x_out[i].
//
// A tile is 128 weight rows of one expert (MMA M, one tensor-memory lane each)
// x up to 256 of its tokens (MMA N, a multiple of 32), so that a row's scales are
// one thread's scalars.  Persistent CTAs, one per SM, walk over the tiles of all
// experts, token tiles fastest (they share the weights in L2).
//   warp 0: bulk copies of a channel group's eight packed row blocks (2 KB codes,
//     256 B signs, 64 B scales each) into the raw ring;
//   warp 2: TMA of the group's activation codes (rows in place order);
//   warps 4-11: (a) turn the raw row blocks into the two K-major, 128-byte-
//     swizzled int8 operands, codes and +-1 (0 outside the mask) trunk bytes;
//     (b) read each group's R from tensor memory and add s_g R to binary32
//     registers; (c) at the end of a tile read T, add the outlier channels and
//     write y.  Warps 4-7 hold the first half of the tile's tokens, 8-11 the
//     second;
//   warp 1 (one lane): per group, R of the first half, R of the second half
//     (each free again while the other MMAs run), then T over all tokens.
// What bounds it: shared-memory bandwidth.  Per group the copies write 19 + 32 KB,
// the operand warps read 16 and write 32 KB, the MMAs read the operands of R twice
// (one for each half) and of T once, 112 KB at 256 tokens; 128 bytes a clock
// give 1750 clocks for 128 x 256 x 128, twice that of the MMAs alone.  Hence
// the wide tile: 128 tokens would cost 1170.
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

constexpr int kThreads = 384;
constexpr int kComputeThreads = 256;
constexpr int kLaunchRegs = 168;    // registers a thread at launch, as 384 threads allow
constexpr int kProducerRegs = 40, kComputeRegs = 232;
constexpr int kRows = 128;          // weight rows per tile (MMA M)
constexpr int kTokens = 256;        // most tokens per tile (MMA N)
constexpr int kBlocks = kRows / kTileRows;
constexpr uint32_t kTmemCols = 512; // T [0, 256), R of half h from 256 + 128 h
constexpr int kMaxBufs = 4;         // R buffers per half (128 columns; small tiles hold several)
constexpr int kRawStages = 2, kAStages = 3, kBStages = 2;
constexpr int kABytes = kRows * kTileK;      // one operand: 16 KB
constexpr int kBBytes = kTokens * kTileK;    // 32 KB
constexpr int kScaleSlots = 4;
constexpr int kMaxOut = 128;        // outlier channels this kernel takes
constexpr uint64_t kWaitNs = 1000000000ull;

template <bool MASK>
struct Raw {
  static constexpr int kSign = kBlocks * 2048;
  static constexpr int kMask = kSign + kBlocks * 256;
  static constexpr int kScale = MASK ? kMask + kBlocks * 256 : kMask;
  static constexpr int kBytes = kScale + kBlocks * 64;
};

struct Aux {
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  uint64_t a_full[kAStages], a_empty[kAStages];
  uint64_t b_full[kBStages], b_empty[kBStages];
  uint64_t accf[2][kMaxBufs], acce[2][kMaxBufs];
  uint64_t t_full, t_empty, wo_full, wo_empty, drain;
  uint32_t tmem_base;
  int abort;
  int part[kThreads / 32];
  float scale[kScaleSlots][kRows];
};

struct Params {
  GroupedArgs a;
  const float* sxp;   // [n] token scales in place order
  const float* xop;   // [n][n8] outlier activations in place order
  int n8;             // n_out rounded up to 4
  float* wout;        // [CTAs][kMaxOut][kRows] outlier weights of the CTA's tile
  int rt;             // row tiles per expert
  int off_b, off_raw, off_aux, off_pre, off_ostart;  // shared-memory offsets
};

// D (s32) (+)= A (s8) B (s8), both K-major; M = 128, N = n.
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, int n, bool acc) {
  const uint32_t idesc =
      (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0));
}

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Aux* aux, const Params& p) {
  if (mbar_wait(bar, parity, kWaitNs)) return true;
  set_status(p.a.status, SQ_ERR_TIMEOUT);
  atomicExch(&aux->abort, 1);
  return false;
}
__device__ __forceinline__ bool aborted(const Aux* aux) {
  return *reinterpret_cast<const volatile int*>(&aux->abort) != 0;
}

__device__ __forceinline__ uint32_t sign_bytes(uint32_t x) {
  uint32_t d;
  asm("prmt.b32 %0, %1, 0, 0xBA98;" : "=r"(d) : "r"(x));
  return d;
}
template <bool MASK>
__device__ __forceinline__ uint32_t trunk_word(uint32_t sign, uint32_t mask, int w) {
  const uint32_t t = ~sign_bytes(sign << (7 - w)) | 0x01010101u;
  return MASK ? t & sign_bytes(mask << (7 - w)) : t;
}
__device__ __forceinline__ uint32_t swap_halves(uint32_t b) {
  return ((b >> 4) & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
}
// 16 consecutive TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, int (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// |r| < 2^22
__device__ __forceinline__ float small_int_to_float(int r) {
  return __fsub_rn(__int_as_float(r + 0x4B400000), 12582912.0f);
}

// One tile: an expert's 128 rows x up to 256 of its places.
struct Tile {
  int rb0;       // first row block in the stack
  int blocks;    // row blocks of the expert in this tile (1..8)
  int row0;      // first row in the expert
  int p0, cnt;   // first place, tokens
  int n;         // MMA N: cnt rounded up to 32
};
__device__ __forceinline__ Tile tile_at(const Params& p, const int* pre, int item) {
  const GroupedArgs& a = p.a;
  const int e = unit_expert(pre, a.E, item / p.rt);
  const int local = item - pre[e] * p.rt, ntt = pre[e + 1] - pre[e];
  const int tt = local % ntt, rt = local / ntt;
  const int2 seg = segment_bounds(a.offsets, a.n, e, nullptr);
  const int total = seg.y - seg.x;
  const int ts = ((total + ntt - 1) / ntt + 31) & ~31;  // <= 256, and (ntt - 1) ts < total
  Tile t;
  t.rb0 = e * a.rbe + rt * kBlocks;
  t.blocks = min(kBlocks, a.rbe - rt * kBlocks);
  t.row0 = rt * kRows;
  t.p0 = seg.x + tt * ts;
  t.cnt = min(ts, total - tt * ts);
  t.n = (t.cnt + 31) & ~31;
  return t;
}
// R buffers per half of a tile with MMA N = n: 128 columns hold that many n/2.
__device__ __forceinline__ int r_bufs(int n) { return n > 128 ? 1 : n > 64 ? 2 : kMaxBufs; }

template <bool MASK>
__global__ void __launch_bounds__(kThreads, 1)
    k_grouped_tc5(const __grid_constant__ CUtensorMap tmB, const Params p) {
  using RW = Raw<MASK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Aux* aux = reinterpret_cast<Aux*>(smem + p.off_aux);
  int* pre = reinterpret_cast<int*>(smem + p.off_pre);
  int* ostart = reinterpret_cast<int*>(smem + p.off_ostart);
  const GroupedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(&aux->raw_full[s], 1);
      mbar_init(&aux->raw_empty[s], kComputeThreads / 32);
    }
    for (int s = 0; s < kAStages; ++s) {
      mbar_init(&aux->a_full[s], kComputeThreads / 32);
      mbar_init(&aux->a_empty[s], 1);
    }
    for (int s = 0; s < kBStages; ++s) {
      mbar_init(&aux->b_full[s], 1);
      mbar_init(&aux->b_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h)
      for (int b = 0; b < kMaxBufs; ++b) {
        mbar_init(&aux->accf[h][b], 1);
        mbar_init(&aux->acce[h][b], 4);
      }
    mbar_init(&aux->t_full, 1);
    mbar_init(&aux->t_empty, kComputeThreads / 32);
    mbar_init(&aux->wo_full, kComputeThreads / 32);
    mbar_init(&aux->wo_empty, kComputeThreads / 32);
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
  for (int i = threadIdx.x; i < n_out; i += kThreads) {
    const int g0 = i > 0 ? (__ldg(a.idx + i - 1) >> 7) + 1 : 0, g1 = __ldg(a.idx + i) >> 7;
    for (int g = g0; g <= g1; ++g) ostart[g] = i;
  }
  for (int g = (n_out > 0 ? (__ldg(a.idx + n_out - 1) >> 7) + 1 : 0) + threadIdx.x; g <= a.tpr; g += kThreads)
    ostart[g] = n_out;
  pdl_wait();
  pdl_launch_dependents();
  const int units = segment_units<kThreads>(a.offsets, a.E, a.n, a.status, kTokens, pre, aux->part);
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
      int last[kRawStages];
#pragma unroll
      for (int s = 0; s < kRawStages; ++s) last[s] = -1;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const Tile t = tile_at(p, pre, item);
        // lane: row block lane % 8 of the array lane / 8 (blocks past the
        // expert repeat its last; their rows are not written)
        const int64_t rb = t.rb0 + min(lane & 7, t.blocks - 1);
        for (int kb = 0; kb < a.tpr; ++kb, ++g) {
          const int s = (int)(g % kRawStages);
          const uint32_t use = g / kRawStages;
          if (g >= kRawStages) ok = wait_or_abort(&aux->raw_empty[s], (use & 1u) ^ 1u, aux, p);
          ok = __all_sync(0xffffffffu, ok && !aborted(aux));
          if (!ok) break;
          uint8_t* st = smem + p.off_raw + s * RW::kBytes;
          if (lane == 0) mbar_arrive_expect_tx(&aux->raw_full[s], RW::kBytes);
          __syncwarp();
          const int64_t tile = rb * a.tpr + kb;
          const int b = lane & 7;
          if (lane < 8) tc05::bulk_load(st + b * 2048, a.res + tile * 2048, 2048, &aux->raw_full[s]);
          else if (lane < 16) tc05::bulk_load(st + RW::kSign + b * 256, a.sign + tile * 64, 256, &aux->raw_full[s]);
          else if (lane < 24) tc05::bulk_load(st + RW::kScale + b * 64, a.scale + tile * 16, 64, &aux->raw_full[s]);
          else if (MASK) tc05::bulk_load(st + RW::kMask + b * 256, a.mask + tile * 64, 256, &aux->raw_full[s]);
          last[s] = (int)use;
        }
      }
      if (aborted(aux)) {  // every requested stage must have landed
#pragma unroll
        for (int s = 0; s < kRawStages; ++s)
          if (last[s] >= 0) (void)mbar_wait(&aux->raw_full[s], (uint32_t)last[s] & 1u, kWaitNs);
      }
    } else if (warp == 2 && lane == 0) {
      // ---- activation producer: n rows of 128 codes per channel group
      uint32_t g = 0;
      int last[kBStages];
#pragma unroll
      for (int s = 0; s < kBStages; ++s) last[s] = -1;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const Tile t = tile_at(p, pre, item);
        for (int kb = 0; kb < a.tpr; ++kb, ++g) {
          const int s = (int)(g % kBStages);
          const uint32_t use = g / kBStages;
          if (g >= kBStages) ok = wait_or_abort(&aux->b_empty[s], (use & 1u) ^ 1u, aux, p);
          ok = ok && !aborted(aux);
          if (!ok) break;
          uint8_t* st = smem + p.off_b + s * kBBytes;
          mbar_arrive_expect_tx(&aux->b_full[s], (uint32_t)t.n * kTileK);
          for (int r = 0; r < t.n; r += 32)
            tc05::tma_load_2d(st + r * kTileK, &tmB, kb * kTileK, t.p0 + r, &aux->b_full[s]);
          last[s] = (int)use;
        }
      }
      if (aborted(aux)) {
#pragma unroll
        for (int s = 0; s < kBStages; ++s)
          if (last[s] >= 0) (void)mbar_wait(&aux->b_full[s], (uint32_t)last[s] & 1u, kWaitNs);
      }
    } else if (warp == 1 && lane == 0) {
      // ---- MMA issuer
      uint32_t g = 0, n_items = 0;
      uint32_t used[2] = {0u, 0u}, phase[2] = {0u, 0u};  // per half: buffers ever used, their acce parity
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x, ++n_items) {
        const Tile t = tile_at(p, pre, item);
        const int h = t.n / 2, bufs = r_bufs(t.n);
        for (int kb = 0; kb < a.tpr; ++kb, ++g) {
          const int sa = (int)(g % kAStages), sb = (int)(g % kBStages), b = kb % bufs;
          ok = wait_or_abort(&aux->a_full[sa], (g / kAStages) & 1u, aux, p) &&
               wait_or_abort(&aux->b_full[sb], (g / kBStages) & 1u, aux, p);
          // (R buffers lie differently in the next tile: all of this one's are free)
          if (ok && kb == 0 && n_items > 0) ok = wait_or_abort(&aux->t_empty, (n_items & 1u) ^ 1u, aux, p);
          if (!ok) break;
          fence_after();
          const uint32_t ca = smem_u32(smem + sa * 2 * kABytes), ta = ca + kABytes;
          const uint32_t xb = smem_u32(smem + p.off_b + sb * kBBytes);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if ((used[half] >> b) & 1u) {
              ok = wait_or_abort(&aux->acce[half][b], (phase[half] >> b) & 1u, aux, p);
              if (!ok) break;
              phase[half] ^= 1u << b;
              fence_after();
            }
            used[half] |= 1u << b;
            const uint32_t d = tmem + kTokens + 128 * half + b * h;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_i8(d, tc05::sw128_desc(ca + 32 * kk), tc05::sw128_desc(xb + half * h * kTileK + 32 * kk), h, kk > 0);
            tc05::mma_commit(&aux->accf[half][b]);
          }
          if (!ok) break;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_i8(tmem, tc05::sw128_desc(ta + 32 * kk), tc05::sw128_desc(xb + 32 * kk), t.n, kb > 0 || kk > 0);
          tc05::mma_commit(&aux->a_empty[sa]);
          tc05::mma_commit(&aux->b_empty[sb]);
        }
        if (ok) tc05::mma_commit(&aux->t_full);
      }
      if (aborted(aux)) {  // the MMAs issued must be done before the tensor memory is freed
        tc05::mma_commit(&aux->drain);
        (void)mbar_wait(&aux->drain, 0u, kWaitNs);
      }
    }
  } else {
    // ---- operands, promotion, epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
    const int cw = warp - 4;                 // row block that this warp turns into operands
    const int half = cw >> 2, q = warp & 3;  // tokens; tensor-memory lane quarter
    const int gid = lane >> 2, tid4 = lane & 3;
    const bool hi = tid4 >= 2;               // takes its two 8-channel pairs in the other order
    const int my_row = 32 * q + lane;
    float* wout = p.wout + (int64_t)blockIdx.x * kMaxOut * kRows;
    uint32_t gc = 0, gp = 0, n_items = 0;    // groups converted, promoted; tiles finished
    uint32_t accp = 0;                       // parity of accf[half][b]
    int citem = blockIdx.x, ckb = 0;         // the conversion runs one group ahead, across tiles
    bool ok = true;

    // this warp's row block of the next group into operand stage gc % kAStages
    auto convert = [&]() {
      if (citem >= items || !ok) return;
      const int sr = (int)(gc % kRawStages), sa = (int)(gc % kAStages);
      ok = wait_or_abort(&aux->raw_full[sr], (gc / kRawStages) & 1u, aux, p);
      if (ok && gc >= kAStages) ok = wait_or_abort(&aux->a_empty[sa], ((gc / kAStages) & 1u) ^ 1u, aux, p);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
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
      uint8_t* ao = smem + sa * 2 * kABytes + cw * 2048 + gid * 128;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = hi ? i ^ 1 : i;  // 16 channels: words 4c .. 4c + 3
        const uint4 u = *reinterpret_cast<const uint4*>(cb + 32 * c), v = *reinterpret_cast<const uint4*>(cb + 32 * c + 16);
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
      const float* sc = reinterpret_cast<const float*>(st + RW::kScale + cw * 64);
      if (lane < 16) aux->scale[gc % kScaleSlots][16 * cw + lane] = sc[lane];
      // outlier channels of this group: the dequantized weight of row `lane`
      const int o0 = ostart[ckb], o1 = ostart[ckb + 1];
      if (o0 < o1 && lane < 16) {
        const Tile t = tile_at(p, pre, citem);
        const float al = __ldg(a.alpha + (int64_t)(t.rb0 + min(cw, t.blocks - 1)) * kTileRows + lane);
        for (int o = o0; o < o1; ++o) {
          const int j = __ldg(a.idx + o) & 127, w = (j & 31) >> 2;
          const int own = (lane & 7) * 4 + (j >> 5), R = lane >> 3, bit = tiled_bit_of(j & 31);
          const int code = reinterpret_cast<const int8_t*>(st)[cw * 2048 + own * 64 + (w >> 1) * 16 +
                                                               ((w & 1) * 2 + R) * 4 + (j & 3)];
          const uint32_t sb = *reinterpret_cast<const uint32_t*>(st + RW::kSign + cw * 256 + own * 8 + 4 * R);
          float tr = ((sb >> bit) & 1u) ? al : -al;
          if constexpr (MASK) {
            const uint32_t mb = *reinterpret_cast<const uint32_t*>(st + RW::kMask + cw * 256 + own * 8 + 4 * R);
            if (!((mb >> bit) & 1u)) tr = 0.0f;
          }
          wout[o * kRows + 16 * cw + lane] = fmaf(sc[lane], (float)code, tr);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&aux->raw_empty[sr]);
        mbar_arrive(&aux->a_full[sa]);
      }
      ++gc;
      if (++ckb == a.tpr) {
        ckb = 0;
        citem += gridDim.x;
      }
    };

    convert();
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x, ++n_items) {
      const Tile t = tile_at(p, pre, item);
      const int h = t.n / 2, bufs = r_bufs(t.n);
      float F[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) F[i] = 0.0f;
      for (int kb = 0; kb < a.tpr; ++kb, ++gp) {
        // (the last group's successor belongs to the next tile, whose outlier
        // weights may only be written once this tile's are used)
        if (kb + 1 < a.tpr) convert();
        const int b = kb % bufs;
        if (ok)
          ok = wait_or_abort(&aux->a_full[gp % kAStages], (gp / kAStages) & 1u, aux, p) &&  // (the scales)
               wait_or_abort(&aux->accf[half][b], (accp >> b) & 1u, aux, p);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        accp ^= 1u << b;
        fence_after();
        const float s = aux->scale[gp % kScaleSlots][my_row];
        const uint32_t src = tmem + ((uint32_t)(32 * q) << 16) + kTokens + 128 * half + b * h;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (16 * c < h) {
            int r[16];
            tmem_ld16(src + 16 * c, r);
#pragma unroll
            for (int i = 0; i < 16; ++i) F[16 * c + i] = fmaf(s, small_int_to_float(r[i]), F[16 * c + i]);
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux->acce[half][b]);
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, wait_or_abort(&aux->t_full, n_items & 1u, aux, p));
      if (!ok) break;
      fence_after();
      const int row = t.row0 + my_row;
      const bool live = my_row < t.blocks * kTileRows && row < a.N;
      const float al = __ldg(a.alpha + (int64_t)t.rb0 * kTileRows + min(my_row, t.blocks * kTileRows - 1));
      const int t0 = half * h;                  // this half's tokens in the tile
      const int nt = max(0, min(h, t.cnt - t0));
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (16 * c < h) {
          int r[16];
          tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + t0 + 16 * c, r);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float sx = __ldg(p.sxp + t.p0 + min(t0 + 16 * c + i, t.cnt - 1));
            F[16 * c + i] = sx * fmaf(al, (float)r[i], F[16 * c + i]);
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&aux->t_empty);
      // the tile's outlier weights: written by every warp, then used, before the
      // next tile's are written
      __threadfence_block();
      __syncwarp();
      if (lane == 0) mbar_arrive(&aux->wo_full);
      ok = __all_sync(0xffffffffu, wait_or_abort(&aux->wo_full, n_items & 1u, aux, p));
      if (!ok) break;
      const float* xo = p.xop + (int64_t)(t.p0 + t0) * p.n8;
      for (int o0 = 0; o0 < n_out; o0 += 4) {
        float w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          w[u] = o0 + u < n_out ? *reinterpret_cast<volatile float*>(wout + (o0 + u) * kRows + my_row) : 0.0f;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          if (8 * c < nt) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int4 x = ldg_nc_v4(xo + (int64_t)min(8 * c + i, nt - 1) * p.n8 + o0);
              float f = F[8 * c + i];
              f = fmaf(w[3], __int_as_float(x.w), f);
              f = fmaf(w[2], __int_as_float(x.z), f);
              f = fmaf(w[1], __int_as_float(x.y), f);
              F[8 * c + i] = fmaf(w[0], __int_as_float(x.x), f);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&aux->wo_empty);
      if (live) {
        float* yr = a.y + (int64_t)(t.p0 + t0) * a.N + row;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i < nt) yr[(int64_t)(32 * c + i) * a.N] = F[32 * c + i];
        }
      }
      ok = __all_sync(0xffffffffu, wait_or_abort(&aux->wo_empty, n_items & 1u, aux, p));
      convert();  // the next tile's first group
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
// the TMA), scale and outlier values, one warp per place.
template <bool GATHER>
__global__ void __launch_bounds__(256) k_grouped_rows(const GroupedArgs a, int8_t* xs, float* sxp, float* xop, int n8) {
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
  const int live = min(max(__ldg(a.offsets + a.E), 0), a.n);
  for (int p = blockIdx.x * 8 + (threadIdx.x >> 5); p < live; p += gridDim.x * 8) {
    const int r = source_row(a, p);
    if (GATHER) {
      const int4* src = reinterpret_cast<const int4*>(a.xq + (int64_t)r * a.xs);
      int4* dst = reinterpret_cast<int4*>(xs + (int64_t)p * a.xs);
      for (int i = lane; i < a.xs / 16; i += 32) dst[i] = __ldg(src + i);
    }
    if (lane == 0) sxp[p] = __ldg(a.sx + r);
    for (int i = lane; i < n8; i += 32) xop[(int64_t)p * n8 + i] = i < a.n_out ? __ldg(a.xout + (int64_t)r * a.n_out + i) : 0.0f;
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
  c.xop = take((size_t)n * kMaxOut * 4);
  c.wout = take((size_t)sm_count * kMaxOut * kRows * 4);
  c.total = off;
  return c;
}

template <bool MASK>
cudaError_t launch_tiles(const CUtensorMap& mb, Params p, int grid, cudaStream_t stream) {
  p.off_b = kAStages * 2 * kABytes;
  p.off_raw = p.off_b + kBStages * kBBytes;
  p.off_aux = (int)round_up(p.off_raw + kRawStages * Raw<MASK>::kBytes, 16);
  p.off_pre = p.off_aux + (int)round_up(sizeof(Aux), 16);
  p.off_ostart = p.off_pre + (int)round_up(4 * (p.a.E + 1), 16);
  const int smem = p.off_ostart + (int)round_up(4 * (p.a.tpr + 1), 16) + 1024;
  if (smem > 227 * 1024) return cudaErrorInvalidValue;
  auto* fn = k_grouped_tc5<MASK>;
  // the register split of the warpgroups must add up to the launch's registers
  static_assert(128 * kProducerRegs + kComputeThreads * kComputeRegs == kThreads * kLaunchRegs, "register split");
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
  return cudaLaunchKernelEx(&cfg, fn, mb, p);
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
  p.xop = xop;
  p.n8 = (int)round_up(std::max(a.n_out, 1), 4);
  p.wout = reinterpret_cast<float*>(w + c.wout);
  p.rt = (int)ceil_div(a.rbe, kBlocks);
  // rows of the activation map: the places (in place order already without an
  // order), those past the last row read as zero
  CUtensorMap mb;
  const int64_t rows = a.order ? a.n : std::min(a.n, a.rows);
  if (!tc05::make_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.order ? xs : a.xq, (uint64_t)a.xs, (uint64_t)rows,
                      (uint64_t)a.xs, kTileK, 32, CU_TENSOR_MAP_SWIZZLE_128B))
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
  const cudaError_t e = a.order ? cudaLaunchKernelEx(&cfg, k_grouped_rows<true>, a, xs, sxp, xop, p.n8)
                                : cudaLaunchKernelEx(&cfg, k_grouped_rows<false>, a, xs, sxp, xop, p.n8);
  if (e != cudaSuccess) return e;
  const int64_t tiles = std::min<int64_t>(a.n, a.E + a.n / kTokens) * p.rt;
  if (tiles >= INT32_MAX) return cudaErrorInvalidValue;
  const int grid = (int)std::min<int64_t>(tiles, sm_count);
  return a.mask ? launch_tiles<true>(mb, p, grid, stream) : launch_tiles<false>(mb, p, grid, stream);
}

}  // namespace sq
