// matmul_f8.cu -- product of two 8-bit floating-point matrices with a scale for
// each 128 values of a row of a, and for each 128 values of a row or of 128 rows
// of b (include/rbf_ops.h, matmul_f8_dev), on the tensor cores:
//
//   out[i, j] = sum_c a_scale[i, c] b_scale[j / block_rows, c] sum_{k in block c} a[i, k] b[j, k] + bias[j]
//
// The tensor cores sum a block's 128 products (kind::f8f6f4, fp32 accumulator in
// tensor memory); the scales, which differ from block to block, are applied to each
// block's sums on their way into the running sums, which threads hold in registers.
// The two scales are multiplied first: one FMA a sum is left, and with a scale for 128
// channels that product is made once for all of them. (The sum times either
// scale would leave fp32's range for other scales, no fewer.)
//
// One kernel, clusters of two CTAs, one CTA per SM, tcgen05.mma.cta_group::2 with
// M = 256 channels (rows of b, 128 per CTA) and N = NT tokens (rows of a, half per
// CTA), K = 128 values a stage, both from shared memory. A TMEM lane is a channel,
// a column a token. Per CTA:
//   warp 0      loads its channels and its tokens of a stage (TMA, 128-byte swizzle);
//   warp 1      one thread of the even CTA issues the pair's MMAs, each stage's into
//               the next of kAcc accumulators;
//   warps 2, 3  put the scales of four blocks at a time into shared memory (with one
//               scale for 128 channels: the products of both);
//   warps 4 on  (sixteen from 128 tokens on, else eight) read an accumulator, 32
//               channels and a part of the tokens each, and add it, times its
//               scales, to their running sums, two numbers an instruction; at a
//               tile's end they add the bias, round and store.
// Work is dealt out in tiles, or, where there are few tiles per pair, in equal
// shares of all stages: a tile that several pairs share is summed from their
// partial sums, in the pairs' order, by the one that finishes last. No CTA waits
// for another pair.
//
// What bounds it. Few tokens: HBM, which b passes through once (1 x 1M x 768 at 6.7
// TB/s). Many: a stage of 256 tokens is 512 clocks of MMAs at the nominal rate, in which
// each of 16 warps reads 64 columns of sums and adds them; 4096 x 8192 x 4096 runs at 2.0 PFLOP/s,
// 137 us, of which 111 to 117 without the FMAs and 99 without the reads too, at the
// power limit by then. Tried there without gain: two accumulators of 128 tokens (135),
// tiles of 128 tokens (164), eight warps of 128 sums, suspending waits (208).
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

constexpr int kDepth = 128;     // values of depth a stage: a block
constexpr int kChannels = 128;  // channels per CTA and tile
constexpr int kPairChannels = 256;
constexpr int kWBytes = kChannels * kDepth;
constexpr int kFirstScale = 2;   // warps 2 and 3
constexpr int kFirstWorker = 4;  // from the second warpgroup on
constexpr int kScaleBlocks = 4;  // blocks whose scales are in a slot
constexpr int kScaleSlots = 2;
constexpr int kMaxSmem = 227 * 1024;
// Stages' time that an exchange of partial sums takes, measured at sizes of one round of
// tiles. With it, and never / always sharing, in us: 1 x 4096 x 4096 11.1 / 12.3, 1 x 8192 x 8192 16.4 / 21.0, 128 x 1024 x 8192
// 18.6 / 25.9 (it shares); 100 x 8192 x 4096 15.7, 17.8 shared, 256 x 4096 x 4096 14.6, 16.9 shared (it does not).
template <int NT>
constexpr int kSplitCost = NT <= 64 ? 20 : 32;

// OUT: what is stored: 1 fp32, 2 bf16, 3 fp16.
template <int NT, int OUT>
struct Shape {
  static constexpr int kGroups = NT >= 128 ? 4 : 2;        // of four workers: each takes a part of the tokens
  static constexpr int kWorkers = 4 * kGroups;
  static constexpr int kThreads = (kFirstWorker + kWorkers) * 32;
  // A worker with 64 sums needs more than an equal share of the registers: the
  // launch has kLaunchRegs a thread, 4 warps give some back and 16 take them.
  static constexpr bool kMoveRegs = NT == 256;
  static constexpr int kLaunchRegs = 96, kControlRegs = 56, kWorkerRegs = 104;
  static_assert(!kMoveRegs || kControlRegs * 128 + kWorkerRegs * kWorkers * 32 <= kLaunchRegs * kThreads, "registers of the launch");
  static constexpr int kXBytes = NT / 2 * kDepth;
  static constexpr int kStage = kWBytes + kXBytes;
  static constexpr int kAcc = NT == 256 ? 2 : 4;           // accumulators
  static constexpr int kCols = NT / kGroups;               // tokens of a worker
  static constexpr int kSlab = 16;                         // of those, read at a time
  static_assert(kCols % kSlab == 0, "whole slabs");
  static constexpr int kOutTokens = kCols < 32 ? kCols : 32;  // 16-bit results in shared memory at a time
  static constexpr int kStageOut = OUT >= 2 ? kOutTokens * 64 : 0;  // of a worker: 32 channels x 16 bits a token
  static constexpr int kOutBytes = kWorkers * kStageOut;
  static constexpr int kScaleFloats = kScaleBlocks * (NT + kChannels);  // of a slot
  static constexpr int kScaleBytes = kScaleSlots * kScaleFloats * 4;
  static constexpr int kMostBars = 2 * 16 + 2 * 4 + 2 * kScaleSlots + 2;
  static constexpr int kStages = (kMaxSmem - 1024 - kOutBytes - kScaleBytes - kMostBars * 8 - 16) / kStage < 12
                                     ? (kMaxSmem - 1024 - kOutBytes - kScaleBytes - kMostBars * 8 - 16) / kStage
                                     : 12;
  static constexpr int kSmem = 1024 + kStages * kStage + kOutBytes + kScaleBytes + kMostBars * 8 + 16;
  static_assert(kSmem <= kMaxSmem && kStages >= 4, "shared memory of an SM");
};

struct Params {
  void* out;
  const float* a_scale;
  const float* b_scale;
  const float* bias;
  int64_t ld_a_scale, ld_b_scale;
  int64_t ld_out;
  int64_t m, n;
  uint32_t formats;  // of the instruction descriptor
  int stages;        // per tile
  int token_tiles;
  int tiles;         // tiles x stages < 2^31
  int split;         // 1: equal shares of all stages, 0: whole tiles
  int tma_out;       // 1: 16-bit results may be stored by TMA
  int read_once;     // 1: the channels are read once (one token tile)
  float* partial;    // split: two tiles of partial sums per CTA
  unsigned* arrived; // split: one counter per CTA, zero between launches
  int* err;
  uint64_t timeout_ns;
};

// D (+)= A B, both operands from shared memory (each CTA's half of either in its own).
__device__ __forceinline__ void umma_pair_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 columns of the warp's 32 TMEM lanes, the load and its wait in one: a
// wait of its own would have to take all registers through itself, a move each.
// As 8 x 8 blocks: registers 4 j, 4 j + 1 are columns 8 j + 2 (lane % 4) + {0, 1} of TMEM lane lane / 4,
// 4 j + 2, 4 j + 3 of lane / 4 + 8, and 8 on the same of TMEM lanes 16 on.
__device__ __forceinline__ void tmem_read_blocks(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      :
        "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
}
// A register a column.
__device__ __forceinline__ void tmem_read_columns(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      :
        "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}

// A worker's part of a tile: 32 channels from j0 on, tokens i0 .. of which `live`
// exist. Its sums are in registers as the tensor memory gives them out:
//   OUT 1: lane = channel, register = token;
//   OUT 2, 3: as tmem_read_blocks gives them, the 8 x 8 blocks of a 16-bit matrix store:
//     tokens 8 j + 2 (lane % 4) + {0, 1} of channels lane / 4 + 8 q.
template <int NT, int OUT>
struct Part {
  using S = Shape<NT, OUT>;
  static constexpr int kChan = OUT >= 2 ? 4 : 1;  // channels of a lane
  int64_t j0, i0;
  int live;
  float add[kChan];

  __device__ __forceinline__ Part(const Params& p, int tile, int ch0, int col0, int lane) {
    j0 = static_cast<int64_t>(tile / p.token_tiles) * kPairChannels + ch0;
    i0 = static_cast<int64_t>(tile % p.token_tiles) * NT + col0;
    live = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(S::kCols), p.m - i0)));
#pragma unroll
    for (int q = 0; q < kChan; ++q) {
      const int64_t j = j0 + (OUT >= 2 ? 8 * q + lane / 4 : lane);
      add[q] = p.bias && j < p.n ? p.bias[j] : 0.0f;
    }
  }
};

// 16-bit results go through shared memory, where 8 x 8 blocks are stored
// transposed (stmatrix): rows of one token's 32 channels, 64 bytes, in the
// 64-byte swizzle that spreads a block's rows over all banks. From there a tiled
// TMA store writes them and clips them at the matrix' edges; where the output's
// rows are not on 16-byte boundaries, or end between them, the lanes store them.
template <int NT, int OUT>
__device__ __forceinline__ void store_tokens(const Params& p, const CUtensorMap* map, const Part<NT, OUT>& t, int c0, const float* acc,
                                             uint8_t* buf, int lane) {
  using S = Shape<NT, OUT>;
  constexpr int kTok = S::kOutTokens;
  if (t.j0 >= p.n || c0 >= t.live) return;
  if constexpr (OUT == 1) {
    float* o = static_cast<float*>(p.out) + (t.i0 + c0) * p.ld_out + t.j0 + lane;
    const bool mine = t.j0 + lane < p.n;
#pragma unroll
    for (int c = 0; c < kTok; ++c) {
      const float v = __fadd_rn(acc[c], t.add[0]);
      if (mine && c0 + c < t.live) o[c * p.ld_out] = v;
    }
  } else {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last results have been read out of `buf`
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kTok / 8; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float* of = acc + 8 * j / S::kSlab * S::kSlab + q / 2 * (S::kSlab / 2) + j % (S::kSlab / 8) * 4 + (q & 1) * 2;
        const float v0 = __fadd_rn(of[0], t.add[q]), v1 = __fadd_rn(of[1], t.add[q]);
        if constexpr (OUT == 2) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v0, v1);
          w[q] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(v0, v1);
          w[q] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      const int row = 8 * j + (lane & 7);
      const uint32_t at = smem_addr(buf) + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4);
      asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]),
                   "r"(w[2]), "r"(w[3])
                   : "memory");
    }
    // The tensor store's clipping ends at 16 bytes, not at an element.
    if (p.tma_out && (t.j0 + 32 <= p.n || p.n % 8 == 0)) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                     "r"(static_cast<int>(t.j0)), "r"(static_cast<int>(t.i0 + c0)), "r"(smem_addr(buf))
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    } else {
      __syncwarp();
      uint16_t* o = static_cast<uint16_t*>(p.out) + (t.i0 + c0) * p.ld_out + t.j0 + lane;
      const bool mine = t.j0 + lane < p.n;
      const int live = min(kTok, t.live - c0);
#pragma unroll 8
      for (int i = 0; i < live; ++i) {
        const uint16_t v = *reinterpret_cast<const uint16_t*>(buf + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2);
        if (mine) o[i * p.ld_out] = v;
      }
      __syncwarp();
    }
  }
}

// BY_CHANNEL: every channel has scales of its own.
template <int NT, int OUT, bool BY_CHANNEL>
__global__ void __launch_bounds__(Shape<NT, OUT>::kThreads, 1)
    matmul_f8_pair_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                          const __grid_constant__ CUtensorMap tmap_out, const Params p) {
  using S = Shape<NT, OUT>;
  constexpr int kCols = S::kCols;
  constexpr int kSlab = S::kSlab;
  constexpr int kStages = S::kStages;
  constexpr int kTmemCols = S::kAcc * NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* outbuf = ring + kStages * S::kStage;
  float* scales = reinterpret_cast<float*>(outbuf + S::kOutBytes);  // a slot: [block][tokens | channels]
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + kScaleSlots * S::kScaleFloats);  // the even CTA's are used: both CTAs' stage
  uint64_t* empty = full + kStages;           // the MMAs of a stage have read it
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + S::kAcc;   // the even CTA's are used
  uint64_t* sc_full = acc_empty + S::kAcc;
  uint64_t* sc_empty = sc_full + kScaleSlots;
  uint64_t* drain = sc_empty + kScaleSlots;
  uint64_t* meet = drain + 1;                 // the workers of this CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meet + 1);
  __shared__ int abort_flag;
  __shared__ unsigned last_flag[2];

  const int warp = __shfl_sync(kFullMask, static_cast<int>(threadIdx.x >> 5), 0);  // in a uniform register, and what follows from it
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int pairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < S::kAcc; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * S::kWorkers);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(&sc_full[s], 2);
      mbar_init(&sc_empty[s], S::kWorkers);
    }
    mbar_init(drain, 1);
    mbar_init(meet, S::kWorkers);
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
  const uint32_t tmem_base = __shfl_sync(kFullMask, *tmem_slot, 0);
  pdl_launch_dependents();

  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&abort_flag) != 0; };
  auto give_up = [&](int bit) {
    atomicOr(p.err, bit);
    *reinterpret_cast<volatile int*>(&abort_flag) = 1;
  };

  Walk walk(p, pair, pairs);
  int tile, k0, k1;

  if (warp < kFirstWorker) {
    if constexpr (S::kMoveRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kControlRegs));  // by the whole warpgroup at one place
    if (warp == 0) {
      // ------------------------------------------------- channels and tokens
      if (lane == 0) {
        pdl_wait();
        const uint64_t policy_w = p.read_once ? l2_policy_evict_first() : l2_policy_evict_last();
        const uint64_t policy_x = l2_policy_evict_last();
        Slot<kStages> s;
        int armed = 0;
        bool ok = true;
        while (ok && walk.next(tile, k0, k1)) {
          const int row_w = tile / p.token_tiles * kPairChannels + static_cast<int>(rank) * kChannels;
          const int row_x = tile % p.token_tiles * NT + static_cast<int>(rank) * (NT / 2);
          for (int k = k0; k < k1; ++k) {
            if (!mbar_wait(&empty[s.i], s.phase ^ 1u, p.timeout_ns) || aborted()) {
              if (!aborted()) give_up(kErrProducerTimeout);
              ok = false;
              break;
            }
            if (leader) mbar_arrive_expect_tx(&full[s.i], 2 * S::kStage);
            const uint32_t bar = cluster_addr(&full[s.i], 0);
            uint8_t* dst = ring + s.i * S::kStage;
            tma_load_2d_pair(dst, &tmap_w, k * kDepth, row_w, bar, policy_w);
            tma_load_2d_pair(dst + kWBytes, &tmap_x, k * kDepth, row_x, bar, policy_x);
            s.advance();
            if (armed < kStages) ++armed;
          }
        }
        // No load may be in flight when the CTA exits.
        if (!ok && leader) {
          for (; armed > 0; --armed) {
            if (s.i == 0) {
              s.i = kStages;
              s.phase ^= 1u;
            }
            --s.i;
            if (!mbar_wait(&full[s.i], s.phase, p.timeout_ns)) atomicOr(p.err, kErrDrainTimeout);
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ----------------------------------------------------------- MMA issuer
      // The whole warp walks and waits, so that addresses and descriptors stay in
      // uniform registers, and one elected lane issues.
      if (leader) {
        const uint32_t idesc = make_idesc(kPairChannels, NT, 0u) | p.formats;
        const bool even = (lane & 1) == 0;  // even lanes wait for the operands while odd ones wait for the accumulator
        Slot<kStages> s;
        Slot<S::kAcc> as;
        bool ok = true;
        while (ok && walk.next(tile, k0, k1)) {
          for (int k = k0; k < k1 && ok; ++k) {
            ok = __all_sync(kFullMask, mbar_wait(even ? &full[s.i] : &acc_empty[as.i], even ? s.phase : as.phase ^ 1u, p.timeout_ns));
            if (!ok) break;
            tc_fence_after();
            const uint64_t w = sw128_kmajor_desc(ring + s.i * S::kStage);
            const uint64_t x = sw128_kmajor_desc(ring + s.i * S::kStage + kWBytes);
            const uint32_t d = tmem_base + static_cast<uint32_t>(as.i * NT);
            if (elect_one()) {
  #pragma unroll
              for (int i = 0; i < kDepth / 32; ++i)
                umma_pair_f8(d, w + static_cast<uint64_t>(2 * i), x + static_cast<uint64_t>(2 * i), idesc, i != 0);
              umma_commit_pair(&empty[s.i]);
              umma_commit_pair(&acc_full[as.i]);
            }
            __syncwarp();
            s.advance();
            as.advance();
          }
        }
        if (!ok && lane == 0 && !aborted()) give_up(kErrConsumerTimeout);
        if (elect_one()) umma_commit_pair(drain);
        __syncwarp();
      }
    } else {
      // --------------------------------------------------------------- scales
      // A slot is four blocks, from a multiple of four on, half of it a warp. The
      // next one's scales are on their way while this one's are waited for and stored.
      const int half = warp - kFirstScale;
      pdl_wait();
      Slot<kScaleSlots> s;
      constexpr int kX = (NT + 63) / 64, kW = kChannels / 64;  // a lane's tokens and channels, 64 apart
      const int at = 32 * half + lane;
      const bool some = NT > 32 || half == 0;
      float x[kX][kScaleBlocks], w[kW][kScaleBlocks];
      const bool wide_a = (reinterpret_cast<uintptr_t>(p.a_scale) & 15) == 0 && p.ld_a_scale % 4 == 0;
      const bool wide_b = (reinterpret_cast<uintptr_t>(p.b_scale) & 15) == 0 && p.ld_b_scale % 4 == 0;
      auto fetch = [&](const float* row, bool there, int k, bool wide, float (&v)[kScaleBlocks]) {
        if (wide && k + kScaleBlocks <= p.stages) {
          const float4 f = there ? *reinterpret_cast<const float4*>(row + k) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          v[0] = f.x;
          v[1] = f.y;
          v[2] = f.z;
          v[3] = f.w;
        } else {
#pragma unroll
          for (int q = 0; q < kScaleBlocks; ++q) v[q] = there && k + q < p.stages ? row[k + q] : 0.0f;
        }
      };
      auto fetch_all = [&](int k) {
        const int64_t j0 = static_cast<int64_t>(tile / p.token_tiles) * kPairChannels + static_cast<int64_t>(rank) * kChannels;
        const int64_t i0 = static_cast<int64_t>(tile % p.token_tiles) * NT + at;
#pragma unroll
        for (int t = 0; t < kX; ++t) fetch(p.a_scale + (i0 + 64 * t) * p.ld_a_scale, some && i0 + 64 * t < p.m, k, wide_a, x[t]);
        if (BY_CHANNEL) {
#pragma unroll
          for (int t = 0; t < kW; ++t) fetch(p.b_scale + (j0 + 64 * t + at) * p.ld_b_scale, j0 + 64 * t + at < p.n, k, wide_b, w[t]);
        } else {
          fetch(p.b_scale + j0 / kChannels * p.ld_b_scale, j0 < p.n, k, wide_b, w[0]);
        }
      };
      int k = 0;
      auto next_slot = [&]() {  // the first block of the next one, or none
        k += kScaleBlocks;
        if (k < k1) return true;
        if (!walk.next(tile, k0, k1)) return false;
        k = k0 / kScaleBlocks * kScaleBlocks;
        return true;
      };
      k1 = 0;
      bool more = next_slot();
      if (more) fetch_all(k);
      while (more) {
        const bool ok = mbar_wait(&sc_empty[s.i], s.phase ^ 1u, p.timeout_ns) && !aborted();
        if (!__all_sync(kFullMask, ok)) {
          if (lane == 0 && !aborted()) give_up(kErrProducerTimeout);
          break;
        }
        float* to = scales + s.i * S::kScaleFloats + at;
#pragma unroll
        for (int q = 0; q < kScaleBlocks; ++q) {
#pragma unroll
          for (int t = 0; t < kX; ++t)
            if (some) to[q * (NT + kChannels) + 64 * t] = BY_CHANNEL ? x[t][q] : __fmul_rn(x[t][q], w[0][q]);
          if (BY_CHANNEL) {
#pragma unroll
            for (int t = 0; t < kW; ++t) to[q * (NT + kChannels) + NT + 64 * t] = w[t][q];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[s.i]);
        s.advance();
        more = next_slot();
        if (more) fetch_all(k);
      }
    }
  } else {
    // -------------------------------------------------------------- workers
    if constexpr (S::kMoveRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kWorkerRegs));
    const int group = (warp - kFirstWorker) >> 2;
    const int quad = warp & 3;  // TMEM lanes that this warp may access
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(group * kCols);
    const uint32_t acc_empty_addr = cluster_addr(acc_empty, 0);
    uint8_t* outs = outbuf + (warp - kFirstWorker) * S::kStageOut;
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
    pdl_wait();  // the kernel before it may read `out`, and writes the bias
    Slot<S::kAcc> as;
    Slot<kScaleSlots> ss;
    while (ok && walk.next(tile, k0, k1)) {
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.0f;
      for (int k = k0; k < k1;) {
        ok = fine(mbar_wait(&sc_full[ss.i], ss.phase, p.timeout_ns));
        if (!ok) break;
        const float* sx = scales + ss.i * S::kScaleFloats + k % kScaleBlocks * (NT + kChannels);
        const int last = min(k1, (k / kScaleBlocks + 1) * kScaleBlocks);
#pragma unroll 1
        for (; k < last; ++k, sx += NT + kChannels) {
          // One scale for all channels is in the tokens' already.
          float sw[Part<NT, OUT>::kChan];
          if constexpr (BY_CHANNEL) {
#pragma unroll
            for (int c = 0; c < Part<NT, OUT>::kChan; ++c) sw[c] = sx[NT + quad * 32 + (OUT >= 2 ? 8 * c + lane / 4 : lane)];
          }
          const float* st = sx + group * kCols + (OUT >= 2 ? 2 * (lane & 3) : 0);
          ok = fine(mbar_wait(&acc_full[as.i], as.phase, p.timeout_ns));
          if (!ok) break;
          tc_fence_after();
          const uint32_t from = lane_base + static_cast<uint32_t>(as.i * NT);
          constexpr int kF = OUT >= 2 ? kSlab / 8 : kSlab / 2;
#pragma unroll
          for (int i = 0; i < kCols / kSlab; ++i) {
            u64 f[kF];
#pragma unroll
            for (int j = 0; j < kF; ++j) f[j] = *reinterpret_cast<const u64*>(st + i * kSlab + (OUT >= 2 ? 8 * j : 2 * j));
            float v[kSlab];
            if constexpr (OUT >= 2)
              tmem_read_blocks(from + i * kSlab, v);
            else
              tmem_read_columns(from + i * kSlab, v);
            if (i + 1 == kCols / kSlab) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(acc_empty_addr + as.i * 8);
            }
#pragma unroll
            for (int e = 0; e < kSlab; e += 2) {
              u64 s = f[OUT >= 2 ? (e >> 2) % (kSlab / 8) : e >> 1];
              if constexpr (BY_CHANNEL) {
                const float c = sw[OUT >= 2 ? 2 * (e / (kSlab / 2)) + (e >> 1 & 1) : 0];
                s = mul2(s, pack2(c, c));
              }
              float* to = acc + i * kSlab + e;
              const u64 r = fma2(pack2(v[e], v[e + 1]), s, pack2(to[0], to[1]));
              to[0] = low2(r);
              to[1] = high2(r);
            }
          }
          as.advance();
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_empty[ss.i]);
        ss.advance();
      }
      if (!ok) break;
      if (k0 != 0 || k1 != p.stages) {
        // A shared tile: leave the partial sums, and finish it if all are there.
        const int64_t all = static_cast<int64_t>(p.tiles) * p.stages, first_stage = static_cast<int64_t>(tile) * p.stages;
        const int first = static_cast<int>(((first_stage + 1) * pairs - 1) / all);
        const int last = static_cast<int>(((first_stage + p.stages) * pairs - 1) / all);
        auto slot_of = [&](int who) {  // a register's 32 lanes side by side
          return reinterpret_cast<u64*>(p.partial + (static_cast<int64_t>(who * 2 + static_cast<int>(rank)) * 2 + (who == first ? 1 : 0)) * (kChannels * NT)) +
                 (warp - kFirstWorker) * (kCols / 2 * 32) + lane;
        };
        u64* mine = slot_of(pair);
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) __stcg(mine + c * 32, pack2(acc[2 * c], acc[2 * c + 1]));
        // One thread's fences order all of the CTA's: they have met before and meet after.
        ok = workers_meet();
        if (!ok) break;
        if (threadIdx.x == kFirstWorker * 32) {
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
        // In the pairs' order, whoever finishes: the same sums every time.
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] = 0.0f;
        for (int who = first; who <= last; ++who) {
          const u64* theirs = slot_of(who);
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {
            const u64 v = __ldcg(theirs + c * 32);
            acc[2 * c] += low2(v);
            acc[2 * c + 1] += high2(v);
          }
        }
      }
      const Part<NT, OUT> part(p, tile, static_cast<int>(rank) * kChannels + quad * 32, group * kCols, lane);
#pragma unroll
      for (int c = 0; c < kCols; c += S::kOutTokens) store_tokens<NT, OUT>(p, &tmap_out, part, c, acc + c, outs, lane);
    }
    if (OUT >= 2 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok && lane == 0 && !aborted()) give_up(kErrConsumerTimeout);
  }

  tc_fence_before();
  __syncthreads();
  // Every MMA (they read both CTAs' memories) is done before either exits. The
  // wait's bound starts here, when the CTA's workers have seen the last sums.
  if (warp == 1) {
    if (!mbar_wait(drain, 0, p.timeout_ns)) atomicOr(p.err, kErrDrainTimeout);
    __syncwarp();
  }
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

template <int NT, int OUT, bool BY_CHANNEL>
cudaError_t launch_t(const MatmulF8Launch& a, const MatmulF8Workspace& w, cudaStream_t st) {
  using S = Shape<NT, OUT>;
  CUtensorMap mx, mw, mo;
  if (!make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a, a.k, a.m, a.ld_a, kDepth, NT / 2) ||
      !make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.b, a.k, a.n, a.ld_b, kDepth, kChannels))
    return cudaErrorInvalidValue;
  Params p;
  p.tma_out = OUT >= 2 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.ld_out % 8 == 0 &&
              make_map(&mo, CU_TENSOR_MAP_DATA_TYPE_UINT16, a.out, a.n, a.m, a.ld_out * 2, 32, S::kOutTokens, CU_TENSOR_MAP_SWIZZLE_64B);
  if (!p.tma_out) mo = mx;
  p.out = a.out;
  p.a_scale = a.a_scale;
  p.b_scale = a.b_scale;
  p.bias = a.bias;
  p.ld_a_scale = a.ld_a_scale;
  p.ld_b_scale = a.ld_b_scale;
  p.ld_out = a.ld_out;
  p.m = a.m;
  p.n = a.n;
  // A is b's rows, B is a's: 0 e4m3, 1 e5m2.
  p.formats = (a.b_dtype == kE5M2 ? 1u << 7 : 0u) | (a.a_dtype == kE5M2 ? 1u << 10 : 0u);
  p.stages = (a.k + kDepth - 1) / kDepth;
  p.token_tiles = static_cast<int>((a.m + NT - 1) / NT);
  p.tiles = static_cast<int>((a.n + kPairChannels - 1) / kPairChannels * p.token_tiles);
  p.read_once = p.token_tiles == 1;
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

  auto fn = matmul_f8_pair_kernel<NT, OUT, BY_CHANNEL>;
  static PerDeviceOnce once;
  const cudaError_t limit = once.run([fn] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem); });
  if (limit != cudaSuccess) return limit;
  if (S::kMoveRegs) {  // the workers would wait for registers that the launch does not have
    static const int regs = [fn] {
      cudaFuncAttributes attr;
      return cudaFuncGetAttributes(&attr, fn) == cudaSuccess ? attr.numRegs : 0;
    }();
    if (regs < S::kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(S::kSmem);
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

template <int NT, int OUT>
cudaError_t launch_blocks(const MatmulF8Launch& a, const MatmulF8Workspace& w, cudaStream_t st) {
  return a.block_rows == 1 ? launch_t<NT, OUT, true>(a, w, st) : launch_t<NT, OUT, false>(a, w, st);
}

template <int NT>
cudaError_t launch_out(const MatmulF8Launch& a, const MatmulF8Workspace& w, cudaStream_t st) {
  if (a.out_dtype == kF32) return launch_blocks<NT, 1>(a, w, st);
  if (a.out_dtype == kBF16) return launch_blocks<NT, 2>(a, w, st);
  return launch_blocks<NT, 3>(a, w, st);
}

}  // namespace

int64_t matmul_f8_rows(int64_t m, int k) {
  // The tensor map has 32-bit coordinates; the kernel counts stages in 32 bits.
  const double stages = (m / (m <= 128 ? 32.0 : 256.0) + 1) * (k / 128.0 + 1);  // of 256 rows
  return std::min<int64_t>(static_cast<int64_t>(2.0e9 / stages) - 1, INT32_MAX / kPairChannels - 1) * kPairChannels;
}

cudaError_t launch_matmul_f8(const MatmulF8Launch& a, const MatmulF8Workspace& w, cudaStream_t st) {
  if (a.m <= 32) return launch_out<32>(a, w, st);
  if (a.m <= 64) return launch_out<64>(a, w, st);
  if (a.m <= 128) return launch_out<128>(a, w, st);
  // A round of tiles of 256 tokens takes 7/4 of one of 128 (it has twice the MMAs, and
  // the scales and its start once). In us, as 128 / 256: 256 x 8192 x 4096 16.0 / 25.6,
  // 1000 x 8192 x 4096 50.0 / 47.5, 384 x 8192 x 4096 25.4 / 22.7, 700 x 4096 x 4096 25.5 / 22.5, 2048 x 8192 x 4096 78 / 78.
  const int64_t pairs = w.num_sms / 2, channels = (a.n + kPairChannels - 1) / kPairChannels;
  const int64_t rounds_128 = ((a.m + 127) / 128 * channels + pairs - 1) / pairs;
  const int64_t rounds_256 = ((a.m + 255) / 256 * channels + pairs - 1) / pairs;
  return rounds_256 * 7 < rounds_128 * 4 ? launch_out<256>(a, w, st) : launch_out<128>(a, w, st);
}

}  // namespace rbf
