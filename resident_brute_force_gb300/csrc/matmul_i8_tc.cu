// matmul_i8_tc.cu -- the 8-bit integer product on the tensor cores
// (include/rbf_ops.h, matmul_i8_dev and linear_i8_dev):
//
//   out[i, j] = a_scale[i] * b_scale[j] * sum_k a[i, k] b[j, k] + bias[j]
//
// tcgen05 takes no 8-bit integers on sm_103a (kind::i8 does not assemble for
// it; the warp-level mma.sync of them does, at a rate that was not measured),
// but fp16 holds every 8-bit integer, and the product of two
// of them, up to 2^14, is exact in the fp32 accumulator as long as the running
// sum stays within 2^24: for 1,024 products whatever their values, and for as
// many stages of 128 as the largest sum of |a| over one of them allows (it is
// found while a is expanded; ordinary rows give 3,000 to 4,000 products). So
// the kernel multiplies in fp16 (kind::f16, the full 16-bit rate), and where
// the depth is larger than that it moves the accumulator into 32-bit integers
// in registers in between. The sums are exact for every input.
//
// The large operand (b: corpus rows or output channels) is read from memory as
// bytes and becomes fp16 on its way into the tensor memory, so it costs one
// byte a value everywhere outside the SM. The small one (a: queries or tokens)
// is expanded to fp16 once a call, into the handle's workspace.
//
// One kernel, clusters of two CTAs, one CTA per SM, tcgen05.mma.cta_group::2
// with M = 256 channels (128 per CTA, from TMEM) and N = NT tokens (half per
// CTA, from shared memory), K = 128 values a stage. The accumulator is the
// transposed tile: a TMEM lane is a channel, a column a token.
// Per CTA:
//   warp 0      loads the CTA's 128 channels x 128 bytes per stage (TMA, 128-
//               byte swizzle, 16 KB) into a ring of its own, deep enough to
//               cover HBM's latency at full rate;
//   warps 2-17  four groups of four; a group takes every fourth stage. A thread
//               reads its channel's 128 bytes (conflict-free: the swizzle),
//               turns four bytes into two fp16 pairs with two byte permutes
//               (0x6400 | b is 1024 + b) and two subtractions, and stores them
//               in its TMEM lane: 64 columns a stage, a ring of 4 to 7 in
//               the columns that the accumulator leaves;
//   warp 18     loads the CTA's tokens (TMA) into a ring of as many stages;
//   warp 1      one thread of the even CTA issues the pair's MMAs.
// At the end of a tile (and of an exact sum) warps 2-17 read the accumulator,
// after they have converted the next ring of stages, so that the MMAs of the next
// tile run while the last one's results are scaled and stored.
//
// Work is dealt out in tiles, or, where there are few tiles per pair and the
// exchange costs less than the idle pairs, in equal shares of all stages: a
// tile that several pairs share is summed from their integer partial sums (in
// any order: they are exact) by the pair that finishes last. No CTA waits for
// another pair.
//
// What bounds it, measured: with 32 to 64 tokens b's bytes (1M x 768 to bf16:
// 139 to 144 us, 114 for the bytes alone); with 128 and more the converting
// warps and the tensor pipe together (4096 x 8192 x 4096 from bf16 182 us of any
// bytes, 163 of the normally distributed ones, which draw less power: 1.51 and
// 1.69 PFLOP/s); with 256 tokens and a shallow depth the one accumulator that
// tensor memory has room for beside the ring, which is drained between tiles
// (256 x 1M x 768 to bf16 286 us back to back, 1.38 PFLOP/s, of a tile's 9,400 clocks some
// 3,200 from its last MMA to the next one's first).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "f32x2.cuh"
#include "ops_internal.h"
#include "pair_tiles.cuh"
#include "rbf_device.cuh"
#include "rbf_internal.h"
#include "tcgen05.cuh"

namespace rbf {
namespace {

constexpr int kDepth = 128;          // values of depth a stage
constexpr int kChannels = 128;       // channels per CTA and tile
constexpr int kPairChannels = 256;
constexpr int kWBytes = kChannels * kDepth;
constexpr int kExactStages = 1024 / kDepth;  // of any values
constexpr int kGroups = 4;           // of worker warps: a group takes every fourth stage
constexpr int kWorkers = 4 * kGroups;
constexpr int kXWarp = 2 + kWorkers;
constexpr int kThreads = (2 + kWorkers + 1) * 32;
constexpr int kTmemCols = 512;       // the accumulator first, then the ring of converted channels
constexpr int kStageCols = kDepth / 2;
constexpr int kRingBudget = 224 * 1024;
// Stages' time that an exchange of partial sums takes: with 16 tokens, 1024 x
// 8192 takes 18.5 us shared and 30.8 not, 4096 x 4096 18.1 and 18.6, 10007 x
// 1536 with 37 tokens 19.4 and 12.4; 4096 x 4096 with 100 tokens 22.9 and 20.6.
template <int NT>
constexpr int kSplitCost = NT <= 64 ? 20 : 32;

// OUT: what is stored: 0 the sums (int32), 1 fp32, 2 bf16, 3 fp16.
template <int NT, int OUT>
struct Shape {
  static constexpr int kXBytes = NT * kDepth;          // NT / 2 tokens x 128 fp16
  static constexpr int kAcc = NT <= 128 ? 2 : 1;       // accumulators
  static constexpr int kRing = (kTmemCols - kAcc * NT) / kStageCols;  // stages of the TMEM ring
  static constexpr int kXRing = NT == 256 ? 3 : kRing;                 // stages of the token ring
  static constexpr int kCols = NT / kGroups;           // accumulator columns (tokens) of one worker warp
  static constexpr int kSlab = kCols < 16 ? kCols : 16;  // of those, read at a time
  static constexpr int kStageOut = OUT >= 2 ? kCols * 64 : 0;  // a worker warp's results: 32 channels x 16 bits a token
  static constexpr int kOutBytes = kWorkers * kStageOut;
  static constexpr int kWStages = (kRingBudget - kXRing * kXBytes - kOutBytes) / kWBytes;
  static constexpr int kBars = 2 * kWStages + kXRing + 2 * kRing + 2 * kAcc + 2;
  static constexpr int kSmem = 1024 + kXRing * kXBytes + kWStages * kWBytes + kOutBytes + kBars * 8 + 16;
  static_assert(kRing >= kGroups && kWStages >= kGroups, "a group needs a slot of its own");
  static_assert(kSmem <= 227 * 1024, "shared memory of an SM");
};

struct Params {
  void* out;
  const float* a_scale;
  const float* b_scale;
  const float* bias;
  int64_t ld_out;
  int64_t m, n;
  int stages;        // per tile
  int token_tiles;
  int tiles;         // tiles x stages < 2^31
  int split;         // 1: equal shares of all stages, 0: whole tiles
  int tma_out;       // 1: 16-bit results may be stored by TMA
  int read_once;     // 1: the channels are read once (one token tile)
  int wait_channels; // 1: the kernel before this one writes them
  const unsigned* block_l1;  // the largest sum of |a| over a token's 128 values of a stage
  unsigned* block_l1_next;   // the next launch's, to be zero for it
  int* partial;      // split: two tiles of partial sums per CTA
  unsigned* arrived; // split: one counter per CTA, zero between launches
  int* err;
  uint64_t timeout_ns;
};

// D += A B with A in tensor memory (each CTA's 128 rows in its own).
__device__ __forceinline__ void umma_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Stages whose products one accumulator sums exactly: |b| <= 128 and
// sum |a| <= block_l1 a stage, so that many stages stay within 2^24.
// (block_l1 <= 128 * 128, which leaves kExactStages of them for any input.)
__device__ __forceinline__ int exact_stages(const Params& p) {
  const unsigned l1 = *reinterpret_cast<const volatile unsigned*>(p.block_l1);
  return max(kExactStages, static_cast<int>(min((1u << 17) / max(l1, 1u), static_cast<unsigned>(p.stages))));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four signed bytes to four fp16: with the sign bit flipped, byte b is the
// value + 128, and the fp16 pattern 0x6400 | b is 1024 + b, so subtracting
// 1152 leaves the value; every step is exact.
__device__ __forceinline__ void bytes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t f = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(f, 0x64646464u, 0x4140);
  const uint32_t b = __byte_perm(f, 0x64646464u, 0x4342);
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// A worker warp's part of a tile: 32 channels from j0 on, tokens i0 .. of which
// `live` exist. Its sums are in registers as the tensor memory gives them out:
//   OUT 0, 1: lane = channel, register = token;
//   OUT 2, 3: as the 8 x 8 blocks of a 16-bit matrix store: per 16 tokens, and for
//     each half of 16 channels, registers 4 j .. 4 j + 3 of a lane are tokens
//     8 j + 2 (lane % 4) + {0, 1} of channels lane / 4 and lane / 4 + 8.
// What they are multiplied by is read ahead of them.
template <int NT, int OUT>
struct Part {
  using S = Shape<NT, OUT>;
  static constexpr int kWords = (S::kCols + 31) / 32;
  static constexpr int kChan = OUT >= 2 ? 4 : 1;  // channels of a lane
  int64_t j0, i0;
  int live;
  float sa[kWords];  // tokens lane, 32 + lane
  float sb[kChan], add[kChan];

  __device__ __forceinline__ Part(const Params& p, int tile, int ch0, int col0, int lane) {
    j0 = static_cast<int64_t>(tile / p.token_tiles) * kPairChannels + ch0;
    i0 = static_cast<int64_t>(tile % p.token_tiles) * NT + col0;
    live = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(S::kCols), p.m - i0)));
    if constexpr (OUT != 0) {
#pragma unroll
      for (int q = 0; q < kChan; ++q) {
        const int64_t j = j0 + (OUT >= 2 ? 8 * q + lane / 4 : lane);
        sb[q] = p.b_scale && j < p.n ? p.b_scale[j] : 1.0f;
        add[q] = p.bias && j < p.n ? p.bias[j] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) sa[i] = p.a_scale && 32 * i + lane < live ? p.a_scale[i0 + 32 * i + lane] : 1.0f;
    }
  }
};

// 16-bit results go through shared memory, where 8 x 8 blocks are stored
// transposed (stmatrix): rows of one token's 32 channels, 64 bytes, in the
// 64-byte swizzle (16-byte piece q of row r at q ^ (r / 2 % 4)) that spreads a
// block's rows over all banks. From there one tiled TMA store a warp and tile
// writes them and clips them at the matrix' edges; where the output's rows are
// not on 16-byte boundaries, or end between them, the warp's lanes store them.

// The last tile's results have been read out of `buf`.
template <int OUT>
__device__ __forceinline__ void store_begin(int lane) {
  if constexpr (OUT >= 2) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
  }
}

template <int NT, int OUT>
__device__ __forceinline__ void store_end(const Params& p, const CUtensorMap* map, const Part<NT, OUT>& t, const uint8_t* buf,
                                          int lane) {
  if constexpr (OUT >= 2) {
    if (t.j0 >= p.n || t.live == 0) return;
    // The tensor store's clipping ends at 16 bytes, not at an element.
    if (p.tma_out && (t.j0 + 32 <= p.n || p.n % 8 == 0)) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                     "r"(static_cast<int>(t.j0)), "r"(static_cast<int>(t.i0)), "r"(smem_addr(buf))
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    } else {
      __syncwarp();
      uint16_t* o = static_cast<uint16_t*>(p.out) + t.i0 * p.ld_out + t.j0 + lane;
      const bool mine = t.j0 + lane < p.n;
#pragma unroll 8
      for (int i = 0; i < t.live; ++i) {
        const uint16_t v = *reinterpret_cast<const uint16_t*>(buf + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2);
        if (mine) o[i * p.ld_out] = v;
      }
      __syncwarp();
    }
  }
}

// Scale and store (16-bit types: put into `buf`) tokens c0 .. c0 + kSlab - 1 of
// the part: r holds their sums, integers for OUT 0 and fp32 numbers else.
template <int NT, int OUT>
__device__ __forceinline__ void store_slab(const Params& p, const Part<NT, OUT>& t, int c0, const uint32_t* r, uint8_t* buf,
                                           int lane) {
  using S = Shape<NT, OUT>;
  if (t.j0 >= p.n || c0 >= t.live) return;
  if constexpr (OUT == 0) {
    int* o = static_cast<int*>(p.out) + (t.i0 + c0) * p.ld_out + t.j0 + lane;
#pragma unroll
    for (int c = 0; c < S::kSlab; ++c)
      if (t.j0 + lane < p.n && c0 + c < t.live) o[c * p.ld_out] = static_cast<int>(r[c]);
  } else if constexpr (OUT == 1) {
    float* o = static_cast<float*>(p.out) + (t.i0 + c0) * p.ld_out + t.j0 + lane;
    const bool mine = t.j0 + lane < p.n;
#pragma unroll
    for (int c = 0; c < S::kSlab; ++c) {
      const float v = __fmaf_rn(__fmul_rn(__uint_as_float(r[c]), __shfl_sync(kFullMask, t.sa[c0 / 32], (c0 + c) & 31)), t.sb[0], t.add[0]);
      if (mine && c0 + c < t.live) o[c * p.ld_out] = v;
    }
  } else {
    constexpr int kBlocks = S::kSlab / 8;
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
      const int tok = c0 + 8 * j + 2 * (lane & 3);
      const uint64_t sa2 = pack2(__shfl_sync(kFullMask, t.sa[c0 / 32], tok & 31), __shfl_sync(kFullMask, t.sa[c0 / 32], (tok + 1) & 31));
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t* e = r + ((q / 2) * kBlocks + j) * 4 + (q & 1) * 2;
        const uint64_t v = fma2(mul2(pack2(__uint_as_float(e[0]), __uint_as_float(e[1])), sa2), pack2(t.sb[q], t.sb[q]), pack2(t.add[q], t.add[q]));
        if constexpr (OUT == 2) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(low2(v), high2(v));
          w[q] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(low2(v), high2(v));
          w[q] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      const int row = c0 + 8 * j + (lane & 7);
      const uint32_t at = smem_addr(buf) + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4);
      asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]),
                   "r"(w[2]), "r"(w[3])
                   : "memory");
    }
  }
}

template <int NT, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_i8_pair_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                          const __grid_constant__ CUtensorMap tmap_out, const Params p) {
  using S = Shape<NT, OUT>;
  constexpr int kCols = S::kCols;
  constexpr int kSlab = S::kSlab;
  constexpr int kRing = S::kRing;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* xring = smem;
  uint8_t* wring = smem + S::kXRing * S::kXBytes;
  uint8_t* outbuf = wring + S::kWStages * kWBytes;  // 16-bit results of each worker warp
  uint64_t* w_full = reinterpret_cast<uint64_t*>(outbuf + S::kOutBytes);
  uint64_t* w_empty = w_full + S::kWStages;
  uint64_t* x_full = w_empty + S::kWStages;  // the even CTA's are used: both CTAs' tokens
  uint64_t* c_full = x_full + S::kXRing;     // the even CTA's are used: both CTAs' converted channels
  uint64_t* done = c_full + kRing;           // the MMAs of a stage have read both rings
  uint64_t* acc_full = done + kRing;
  uint64_t* acc_empty = acc_full + S::kAcc;  // the even CTA's are used
  uint64_t* drain = acc_empty + S::kAcc;
  uint64_t* meet = drain + 1;                // the workers of this CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meet + 1);
  __shared__ int abort_flag;
  __shared__ unsigned last_flag[2];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int pairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < S::kWStages; ++s) {
      mbar_init(&w_full[s], 1);
      mbar_init(&w_empty[s], 4);
    }
    for (int s = 0; s < S::kXRing; ++s) mbar_init(&x_full[s], 1);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&c_full[s], 8);  // four worker warps of each CTA
      mbar_init(&done[s], 1);
    }
    for (int b = 0; b < S::kAcc; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kWorkers);
    }
    mbar_init(drain, 1);
    mbar_init(meet, kWorkers);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.block_l1_next = 0;

  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&abort_flag) != 0; };
  auto give_up = [&](int bit) {
    atomicOr(p.err, bit);
    *reinterpret_cast<volatile int*>(&abort_flag) = 1;
  };

  Walk walk(p, pair, pairs);
  int tile, k0, k1;

  if (warp == 0) {
    // ---------------------------------------------------- channels (bytes)
    // Where the kernel launched just before this one does not write them, their
    // loads start while that one still runs.
    if (lane == 0) {
      if (p.wait_channels) pdl_wait();
      const uint64_t policy = p.read_once ? l2_policy_evict_first() : l2_policy_evict_last();
      Slot<S::kWStages> s;
      int armed = 0;
      bool ok = true;
      while (ok && walk.next(tile, k0, k1)) {
        const int row = tile / p.token_tiles * kPairChannels + static_cast<int>(rank) * kChannels;
        for (int k = k0; k < k1; ++k) {
          if (!mbar_wait(&w_empty[s.i], s.phase ^ 1u, p.timeout_ns) || aborted()) {
            if (!aborted()) give_up(kErrProducerTimeout);
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&w_full[s.i], kWBytes);
          tma_load_2d(wring + s.i * kWBytes, &tmap_w, k * kDepth, row, &w_full[s.i], policy);
          s.advance();
          if (armed < S::kWStages) ++armed;
        }
      }
      // No load may be in flight when the CTA exits.
      if (!ok) {
        for (; armed > 0; --armed) {
          if (s.i == 0) {
            s.i = S::kWStages;
            s.phase ^= 1u;
          }
          --s.i;
          if (!mbar_wait(&w_full[s.i], s.phase, p.timeout_ns)) atomicOr(p.err, kErrDrainTimeout);
        }
      }
    }
    __syncwarp();
  } else if (warp == kXWarp) {
    // ------------------------------------------------------- tokens (fp16)
    if (lane == 0) {
      pdl_wait();  // the kernel before this one writes them
      const uint64_t policy = l2_policy_evict_last();
      Slot<S::kXRing> s;
      Slot<kRing> over;  // the stage whose tokens this one's overwrite
      int at = 0, armed = 0;
      bool ok = true;
      while (ok && walk.next(tile, k0, k1)) {
        const int row = tile % p.token_tiles * NT + static_cast<int>(rank) * (NT / 2);
        for (int k = k0; k < k1; ++k, ++at) {
          if (at >= S::kXRing) {
            if (!mbar_wait(&done[over.i], over.phase, p.timeout_ns) || aborted()) {
              if (!aborted()) give_up(kErrProducerTimeout);
              ok = false;
              break;
            }
            over.advance();
          }
          if (leader) mbar_arrive_expect_tx(&x_full[s.i], 2 * S::kXBytes);
          const uint32_t bar = cluster_addr(&x_full[s.i], 0);
          uint8_t* dst = xring + s.i * S::kXBytes;
          tma_load_2d_pair(dst, &tmap_x, k * kDepth, row, bar, policy);
          tma_load_2d_pair(dst + S::kXBytes / 2, &tmap_x, k * kDepth + kDepth / 2, row, bar, policy);
          s.advance();
          if (armed < S::kXRing) ++armed;
        }
      }
      if (!ok && leader) {
        for (; armed > 0; --armed) {
          if (s.i == 0) {
            s.i = S::kXRing;
            s.phase ^= 1u;
          }
          --s.i;
          if (!mbar_wait(&x_full[s.i], s.phase, p.timeout_ns)) atomicOr(p.err, kErrDrainTimeout);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    // The whole warp walks and waits, so that addresses and descriptors stay
    // in uniform registers, and one elected lane issues: 20 cycles an MMA of
    // 32 tokens instead of 45 from a branch on the lane's number.
    if (leader) {
      constexpr uint32_t idesc = make_idesc(kPairChannels, NT, 0u);
      const bool even = (lane & 1) == 0;  // even lanes wait for the channels while odd ones wait for the tokens
      Slot<kRing> s;
      Slot<S::kXRing> xs;
      Slot<S::kAcc> as;
      pdl_wait();
      const int exact = exact_stages(p);
      bool ok = true, ready = false;
      while (ok && walk.next(tile, k0, k1)) {
        for (int k = k0; k < k1 && ok; k += exact) {
          const int kend = min(k + exact, k1);
          ok = __all_sync(kFullMask, mbar_wait(&acc_empty[as.i], as.phase ^ 1u, p.timeout_ns));
          const uint32_t d = tmem_base + static_cast<uint32_t>(as.i * NT);
          tc_fence_after();
          for (int kk = k; kk < kend && ok; ++kk) {
            if (!ready) {
              ok = __all_sync(kFullMask, mbar_wait(even ? &c_full[s.i] : &x_full[xs.i], even ? s.phase : xs.phase, p.timeout_ns));
              if (!ok) break;
            }
            tc_fence_after();
            const uint64_t b0 = sw128_kmajor_desc(xring + xs.i * S::kXBytes);
            const uint64_t b1 = sw128_kmajor_desc(xring + xs.i * S::kXBytes + S::kXBytes / 2);
            const uint32_t c = tmem_base + S::kAcc * NT + static_cast<uint32_t>(s.i * kStageCols);
            Slot<kRing> next = s;
            next.advance();
            xs.advance();
            // Looked at now, and the answer used when this stage's MMAs are issued.
            const bool there = mbar_try_wait(even ? &c_full[next.i] : &x_full[xs.i], even ? next.phase : xs.phase);
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < kDepth / 16; ++i)
                umma_pair_ts(d, c + static_cast<uint32_t>(8 * i), (i < 4 ? b0 : b1) + static_cast<uint64_t>(2 * (i & 3)), idesc,
                             (kk != k) | (i != 0));
              umma_commit_pair(&done[s.i]);
            }
            __syncwarp();
            ready = __all_sync(kFullMask, there);
            s = next;
          }
          if (ok && elect_one()) umma_commit_pair(&acc_full[as.i]);
          __syncwarp();
          as.advance();
        }
      }
      if (!ok && lane == 0 && !aborted()) give_up(kErrConsumerTimeout);
      if (elect_one()) umma_commit_pair(drain);
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------------- workers
    const int group = (warp - 2) >> 2;
    const int quad = warp & 3;  // TMEM lanes that this warp may access
    const int ch = quad * 32 + lane;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t acc_empty_addr = cluster_addr(acc_empty, 0);
    uint8_t* outs = outbuf + (warp - 2) * S::kStageOut;
    const uint32_t c_full_addr = cluster_addr(c_full, 0);
    const int total = walk.total();
    bool ok = true;
    // Warp-uniform: whether every lane's wait has ended in time.
    auto fine = [&](bool in_time) { return __all_sync(kFullMask, in_time) != 0; };
    uint32_t meet_phase = 0;
    int flag = 0;
    auto workers_meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      const bool r = fine(mbar_wait(meet, meet_phase, p.timeout_ns));
      meet_phase ^= 1u;
      return r;
    };

    // Convert this group's stages up to (not including) stage `until`.
    int stage = group;
    Slot<S::kWStages> ws;
    ws.i = group;
    Slot<kRing> rs;
    rs.i = group;
    auto convert_until = [&](int until) {
      for (; ok && stage < until; stage += kGroups) {
        ok = fine(mbar_wait(&w_full[ws.i], ws.phase, p.timeout_ns));
        if (!ok) break;
        const uint8_t* row = wring + ws.i * kWBytes + ch * kDepth;
        const uint32_t dst = lane_base + S::kAcc * NT + rs.i * kStageCols;
        uint4 raw[2][2];  // 32 bytes, and the next 32
        auto fetch = [&](int h) {
#pragma unroll
          for (int c = 0; c < 2; ++c) raw[h & 1][c] = *reinterpret_cast<const uint4*>(row + (((2 * h + c) ^ (ch & 7)) << 4));
        };
        fetch(0);
        ok = fine(mbar_wait(&done[rs.i], rs.phase ^ 1u, p.timeout_ns));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (h < 3) fetch(h + 1);
          if (h == 3) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_empty[ws.i]);
          }
          uint32_t f[16];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 v = raw[h & 1][c];
            bytes_to_f16(v.x, f[8 * c + 0], f[8 * c + 1]);
            bytes_to_f16(v.y, f[8 * c + 2], f[8 * c + 3]);
            bytes_to_f16(v.z, f[8 * c + 4], f[8 * c + 5]);
            bytes_to_f16(v.w, f[8 * c + 6], f[8 * c + 7]);
          }
          tmem_st16(dst + 16 * h, f);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(c_full_addr + rs.i * 8);  // orders TMEM only, as for acc_empty
        ws.advance(kGroups);
        rs.advance(kGroups);
      }
    };

    int finished = 0;  // stages whose accumulator has been read
    Slot<S::kAcc> as;
    // The next accumulator is complete; its address for this warp.
    auto acc_ready = [&](uint32_t& from) {
      ok = fine(mbar_wait(&acc_full[as.i], as.phase, p.timeout_ns));
      tc_fence_after();
      from = lane_base + static_cast<uint32_t>(as.i * NT + group * kCols);
      return ok;
    };
    auto acc_release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty_addr + as.i * 8);
      as.advance();
    };
    auto ld = [&](uint32_t at, uint32_t* v) {  // kSlab columns of the warp's 32 lanes
      if constexpr (OUT >= 2) {
        constexpr uint32_t kHalf = 16u << 16;  // TMEM lanes 16-31 of the warp's
        if constexpr (kSlab == 16) {
          tmem_ld_blocks2(at, v);
          tmem_ld_blocks2(at + kHalf, v + 8);
        } else {
          tmem_ld_blocks1(at, v);
          tmem_ld_blocks1(at + kHalf, v + 4);
        }
      } else if constexpr (kSlab == 16) {
        tmem_ld16(at, v);
      } else {
        tmem_ld8(at, v);
      }
    };
    convert_until(min(kRing, total));  // before anything that the kernel before this one writes is needed
    pdl_wait();                        // it writes the scales, and may read `out`
    const int exact = exact_stages(p);
    while (ok && walk.next(tile, k0, k1)) {
      const int ch0 = static_cast<int>(rank) * kChannels + quad * 32;
      if (k0 == 0 && k1 == p.stages && p.stages <= exact) {
        // The sums are one accumulator's: from tensor memory to the output, a
        // slab at a time, the next one's load under way.
        finished += k1;
        convert_until(min(finished + kRing, total));
        if (!ok) break;
        const Part<NT, OUT> part(p, tile, ch0, group * kCols, lane);
        uint32_t from;
        if (!acc_ready(from)) break;
        // One accumulator: it is read at once and given back before its sums
        // are stored. Two: the next slab is read while this one is stored.
        constexpr int kAhead = S::kAcc == 1 ? kCols / kSlab : 2;
        uint32_t v[kAhead][kSlab];
        store_begin<OUT>(lane);
#pragma unroll
        for (int i = 0; i < kAhead - (S::kAcc == 2); ++i) ld(from + i * kSlab, v[i]);
#pragma unroll
        for (int i = 0; i < kCols / kSlab; ++i) {
          uint32_t(&now)[kSlab] = v[i % kAhead];
          tmem_wait_ld<kSlab>(now);
          if (S::kAcc == 2 && i + 1 < kCols / kSlab) ld(from + (i + 1) * kSlab, v[(i + 1) % kAhead]);
          if (i == (S::kAcc == 1 ? 0 : kCols / kSlab - 1)) acc_release();
          if constexpr (OUT == 0) {
#pragma unroll
            for (int c = 0; c < kSlab; ++c) now[c] = static_cast<uint32_t>(__float2int_rn(__uint_as_float(now[c])));
          }
          store_slab<NT, OUT>(p, part, i * kSlab, now, outs, lane);
        }
        store_end<NT, OUT>(p, &tmap_out, part, outs, lane);
        continue;
      }
      uint32_t acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0;
      for (int k = k0; k < k1; k += exact) {
        finished += min(exact, k1 - k);
        convert_until(min(finished + kRing, total));
        uint32_t from;
        if (!ok || !acc_ready(from)) break;
#pragma unroll
        for (int c = 0; c < kCols; c += kSlab) {
          uint32_t v[kSlab];
          ld(from + c, v);
          tmem_wait_ld<kSlab>(v);
#pragma unroll
          for (int i = 0; i < kSlab; ++i) acc[c + i] += static_cast<uint32_t>(__float2int_rn(__uint_as_float(v[i])));
        }
        acc_release();
      }
      if (!ok) break;
      if (k0 != 0 || k1 != p.stages) {
        // A shared tile: leave the partial sums, and finish it if all are there.
        const int64_t all = static_cast<int64_t>(p.tiles) * p.stages, first_stage = static_cast<int64_t>(tile) * p.stages;
        const int first = static_cast<int>(((first_stage + 1) * pairs - 1) / all);
        const int last = static_cast<int>(((first_stage + p.stages) * pairs - 1) / all);
        auto slot_of = [&](int who) {  // a register's 32 lanes side by side
          return p.partial + (static_cast<int64_t>(who * 2 + static_cast<int>(rank)) * 2 + (who == first ? 1 : 0)) * (kChannels * NT) +
                 group * kCols * kChannels + ch;
        };
        int* mine = slot_of(pair);
#pragma unroll
        for (int c = 0; c < kCols; ++c) __stcg(mine + c * kChannels, static_cast<int>(acc[c]));
        // One thread's fences order all of the CTA's: they have met before and meet after.
        ok = workers_meet();
        if (!ok) break;
        if (threadIdx.x == 64) {
          __threadfence();
          const unsigned n = atomicAdd(&p.arrived[first * 2 + static_cast<int>(rank)], 1u) + 1u;
          const bool fin = n == static_cast<unsigned>(last - first + 1);
          if (fin) p.arrived[first * 2 + static_cast<int>(rank)] = 0u;
          __threadfence();
          last_flag[flag] = fin ? 1u : 0u;
        }
        ok = workers_meet();
        if (!ok) break;
        const bool fin = *reinterpret_cast<volatile unsigned*>(&last_flag[flag]) != 0;
        flag ^= 1;  // the next tile's is another word: this one may still be read
        if (!fin) continue;
        for (int who = first; who <= last; ++who) {
          if (who == pair) continue;
          const int* theirs = slot_of(who);
#pragma unroll
          for (int c = 0; c < kCols; ++c) acc[c] += static_cast<uint32_t>(__ldcg(theirs + c * kChannels));
        }
      }
      const Part<NT, OUT> part(p, tile, ch0, group * kCols, lane);
      store_begin<OUT>(lane);
#pragma unroll
      for (int c = 0; c < kCols; c += kSlab) {
        if constexpr (OUT != 0) {
#pragma unroll
          for (int i = 0; i < kSlab; ++i) acc[c + i] = __float_as_uint(__int2float_rn(static_cast<int>(acc[c + i])));
        }
        store_slab<NT, OUT>(p, part, c, acc + c, outs, lane);
      }
      store_end<NT, OUT>(p, &tmap_out, part, outs, lane);
    }
    if (OUT >= 2 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok && lane == 0 && !aborted()) give_up(kErrConsumerTimeout);
  }

  tc_fence_before();
  __syncthreads();
  // Every MMA (they read both CTAs' memories) is done before either exits. The
  // wait's bound starts here, when the CTA's workers have seen the last sums:
  // from the kernel's start it would be one on the whole product's time.
  if (warp == 1) {
    if (!mbar_wait(drain, 0, p.timeout_ns)) atomicOr(p.err, kErrDrainTimeout);
    __syncwarp();
  }
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

// 8-bit rows to fp16, [m][pitch], zero past k: eight values a thread, and the
// largest sum of magnitudes of 128 values (16 threads') into block_l1.
__global__ void __launch_bounds__(256)
    expand_rows_kernel(const int8_t* __restrict__ a, int64_t ld_a, int64_t m, int k, __half* __restrict__ x, int pitch,
                       unsigned* __restrict__ block_l1) {
  pdl_launch_dependents();  // the product may become resident now; it waits for these rows
  const int per = pitch / 8;  // a multiple of 16
  const bool wide = (reinterpret_cast<uintptr_t>(a) & 7) == 0 && ld_a % 8 == 0;
  unsigned top = 0;
  const int64_t groups = m * per;
  for (int64_t g = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; g < (groups + 31) / 32 * 32;
       g += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    uint2 raw = make_uint2(0u, 0u);
    if (g < groups) {
      const int64_t i = g / per;
      const int c = static_cast<int>(g - i * per) * 8;
      const int8_t* src = a + i * ld_a + c;
      if (wide && c + 8 <= k) {
        raw = *reinterpret_cast<const uint2*>(src);
      } else if (c < k) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int b = 0; b < 8; ++b)
          if (c + b < k) w[b >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(src[b])) << (8 * (b & 3));
        raw = make_uint2(w[0], w[1]);
      }
      uint4 out;
      bytes_to_f16(raw.x, out.x, out.y);
      bytes_to_f16(raw.y, out.z, out.w);
      *reinterpret_cast<uint4*>(x + i * pitch + c) = out;
    }
    unsigned l1 = __dp4a(__vabs4(raw.x), 0x01010101u, __dp4a(__vabs4(raw.y), 0x01010101u, 0u));
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) l1 += __shfl_xor_sync(kFullMask, l1, d);
    top = max(top, l1);
  }
  __shared__ unsigned part[8];
  top = __reduce_max_sync(kFullMask, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) top = max(top, part[w]);
    atomicMax(block_l1, top);
  }
}

template <int NT, int OUT>
cudaError_t launch_t(const MatmulI8Launch& a, const MatmulI8Workspace& w, cudaStream_t st) {
  CUtensorMap mx, mw, mo;
  const int pitch = matmul_i8_pitch(a.k);
  if (!make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, w.rows_f16, pitch, a.m, int64_t(pitch) * 2, kDepth / 2, NT / 2) ||
      !make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.b, a.k, a.n, a.ld_b, kDepth, kChannels))
    return cudaErrorInvalidValue;
  Params p;
  p.tma_out = OUT >= 2 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.ld_out % 8 == 0 &&
              make_map(&mo, CU_TENSOR_MAP_DATA_TYPE_UINT16, a.out, a.n, a.m, a.ld_out * 2, 32, Shape<NT, OUT>::kCols,
                       CU_TENSOR_MAP_SWIZZLE_64B);
  if (!p.tma_out) mo = mx;
  p.out = a.out;
  p.a_scale = a.a_scale;
  p.b_scale = a.b_scale;
  p.bias = a.bias;
  p.ld_out = a.ld_out;
  p.m = a.m;
  p.n = a.n;
  p.stages = pitch / kDepth;
  p.token_tiles = static_cast<int>((a.m + NT - 1) / NT);
  p.tiles = static_cast<int>((a.n + kPairChannels - 1) / kPairChannels * p.token_tiles);
  p.read_once = p.token_tiles == 1;
  p.wait_channels = a.b_is_new;
  p.block_l1 = w.block_l1;
  p.block_l1_next = w.block_l1_next;
  p.partial = w.partial;
  p.arrived = w.arrived;
  p.err = w.err;
  p.timeout_ns = w.timeout_ns;
  const int64_t max_pairs = w.num_sms / 2;
  const int64_t total = static_cast<int64_t>(p.tiles) * p.stages;
  // Shares of all stages where the rounds of whole tiles take longer by more
  // than the exchange of partial sums does, in stages' time.
  const int64_t rounds = (p.tiles + max_pairs - 1) / max_pairs;
  p.split = rounds * p.stages > (total + max_pairs - 1) / max_pairs + kSplitCost<NT>;
  const int64_t pairs = p.split ? std::min(max_pairs, total) : std::min<int64_t>(max_pairs, p.tiles);

  auto fn = matmul_i8_pair_kernel<NT, OUT>;
  static PerDeviceOnce once;
  const cudaError_t limit = once.run(
      [fn] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NT, OUT>::kSmem); });
  if (limit != cudaSuccess) return limit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(Shape<NT, OUT>::kSmem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, mx, mw, mo, p);
}

template <int NT>
cudaError_t launch_out(const MatmulI8Launch& a, const MatmulI8Workspace& w, cudaStream_t st) {
  if (a.out_dtype == kI32) return launch_t<NT, 0>(a, w, st);
  if (a.out_dtype == kF32) return launch_t<NT, 1>(a, w, st);
  if (a.out_dtype == kBF16) return launch_t<NT, 2>(a, w, st);
  return launch_t<NT, 3>(a, w, st);
}

}  // namespace

int matmul_i8_pitch(int k) { return (k + kDepth - 1) / kDepth * kDepth; }

size_t matmul_i8_partial_bytes(int num_sms) { return static_cast<size_t>(num_sms) * 2 * kChannels * 256 * sizeof(int); }

int64_t matmul_i8_tc_rows(int64_t m, int k) {
  // The tensor map has 32-bit coordinates; the kernel counts stages in 32 bits.
  const double stages = (m / (m <= 128 ? 32.0 : 256.0) + 1) * (k / 128.0 + 1);  // of 256 rows
  return std::min<int64_t>(static_cast<int64_t>(2.0e9 / stages) - 1, INT32_MAX / kPairChannels - 1) * kPairChannels;
}

cudaError_t launch_expand_rows(const int8_t* a, int64_t ld_a, int64_t m, int k, const MatmulI8Workspace& w,
                               cudaStream_t st) {
  const int pitch = matmul_i8_pitch(k);
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((m * (pitch / 8) + 255) / 256, int64_t(w.num_sms) * 16));
  expand_rows_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(a, ld_a, m, k, static_cast<__half*>(w.rows_f16), pitch,
                                                                   w.block_l1);
  return cudaGetLastError();
}

cudaError_t launch_matmul_i8_tc(const MatmulI8Launch& a, const MatmulI8Workspace& w, cudaStream_t st) {
  if (a.m <= 32) return launch_out<32>(a, w, st);
  if (a.m <= 64) return launch_out<64>(a, w, st);
  if (a.m <= 128) return launch_out<128>(a, w, st);
  // A stage of 256 tokens takes 7/4 of one of 128 (0.40 us; the accumulator is
  // one and waits to be read): whichever needs less time for its rounds of
  // tiles. 256 x 8192 x 4096 takes 22.7 us with 128 and 33.0 with 256, 512
  // tokens 35.0 and 33.3, 1000 tokens 62.4 and 58.8, 4096 tokens 202 and 186.
  const int64_t pairs = w.num_sms / 2, channels = (a.n + kPairChannels - 1) / kPairChannels;
  const int64_t rounds_128 = ((a.m + 127) / 128 * channels + pairs - 1) / pairs;
  const int64_t rounds_256 = ((a.m + 255) / 256 * channels + pairs - 1) / pairs;
  return rounds_256 * 7 < rounds_128 * 4 ? launch_out<256>(a, w, st) : launch_out<128>(a, w, st);
}

}  // namespace rbf
