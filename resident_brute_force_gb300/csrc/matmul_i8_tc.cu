// matmul_i8_tc.cu -- the 8-bit integer product on the tensor cores
// (include/rbf_ops.h, matmul_i8_dev and linear_i8_dev):
//
//   out[i, j] = a_scale[i] * b_scale[j] * sum_k a[i, k] b[j, k] + bias[j]
//
// sm_103a has no 8-bit integer tensor instruction (tcgen05 kind::i8 does not
// assemble for it), but fp16 holds every 8-bit integer, and the product of two
// of them, up to 2^14, is exact in the fp32 accumulator as long as the running
// sum stays within 2^24: for 1,024 products whatever their values. So the
// kernel multiplies in fp16 (kind::f16, the full 16-bit rate), and where the
// depth is larger it moves the accumulator into 32-bit integers in registers
// every 1,024 values. The sums are exact for every input.
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
// At the end of a tile (and every 1,024 values) warps 2-17 read the accumulator,
// after they have converted the next ring of stages, so that the MMAs of the next
// tile run while the last one's results are scaled and stored.
//
// Work is dealt out in tiles, or, where there are few tiles per pair, in equal
// shares of all stages: a tile that several pairs share is summed from their
// integer partial sums (in any order: they are exact) by the pair that
// finishes last. No CTA waits for another pair.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_internal.h"
#include "rbf_device.cuh"
#include "tcgen05.cuh"

namespace rbf {
namespace {

constexpr int kDepth = 128;          // values of depth a stage
constexpr int kChannels = 128;       // channels per CTA and tile
constexpr int kPairChannels = 256;
constexpr int kWBytes = kChannels * kDepth;
constexpr int kExactStages = 1024 / kDepth;
constexpr int kGroups = 4;           // of worker warps: a group takes every fourth stage
constexpr int kWorkers = 4 * kGroups;
constexpr int kXWarp = 2 + kWorkers;
constexpr int kThreads = (2 + kWorkers + 1) * 32;
constexpr int kTmemCols = 512;       // the accumulator first, then the ring of converted channels
constexpr int kStageCols = kDepth / 2;
constexpr int kRingBudget = 224 * 1024;

template <int NT>
struct Shape {
  static constexpr int kXBytes = NT * kDepth;  // NT / 2 tokens x 128 fp16
  static constexpr int kRing = (kTmemCols - NT) / kStageCols;  // stages of the token ring and of the TMEM ring
  static constexpr int kCols = NT / kGroups;   // accumulator columns of one worker thread
  static constexpr int kWStages = (kRingBudget - kRing * kXBytes) / kWBytes;
  static constexpr int kSmem = 1024 + kRing * kXBytes + kWStages * kWBytes + (2 * kWStages + 3 * kRing + 4) * 8 + 16;
  static_assert(kRing >= kGroups && kWStages >= kGroups, "a group needs a slot of its own");
};

struct Params {
  void* out;
  const float* a_scale;
  const float* b_scale;
  const float* bias;
  int64_t ld_out;
  int64_t m, n;
  int out_dtype;
  int stages;        // per tile
  int token_tiles;
  int tiles;         // tiles x stages < 2^31
  int split;         // 1: equal shares of all stages, 0: whole tiles
  int read_once;     // 1: the channels are read once (one token tile)
  int* partial;      // split: two tiles of partial sums per CTA
  unsigned* arrived; // split: one counter per CTA, zero between launches
  int* err;
  uint64_t timeout_ns;
};

// The pair's part of the work, one tile's stages [k0, k1) at a time.
struct Walk {
  int at, end, stages, step;
  bool split;

  __device__ __forceinline__ Walk(const Params& p, int pair, int pairs) : stages(p.stages), step(pairs), split(p.split) {
    at = split ? share_start(p, pair, pairs) : pair;
    end = split ? share_start(p, pair + 1, pairs) : p.tiles;
  }
  static __device__ __forceinline__ int share_start(const Params& p, int pair, int pairs) {
    return static_cast<int>(static_cast<int64_t>(p.tiles) * p.stages * pair / pairs);
  }
  __device__ __forceinline__ int total() const {
    return split ? end - at : (at < end ? (end - at + step - 1) / step * stages : 0);
  }
  __device__ __forceinline__ bool next(int& tile, int& k0, int& k1) {
    if (at >= end) return false;
    if (split) {
      tile = at / stages;
      k0 = at - tile * stages;
      k1 = min(stages, k0 + (end - at));
      at += k1 - k0;
    } else {
      tile = at;
      k0 = 0;
      k1 = stages;
      at += step;
    }
    return true;
  }
};

// A position in a ring of S slots; `phase` is the parity of its full barrier.
template <int S>
struct Slot {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance(int by = 1) {
    i += by;
    if (i >= S) {
      i -= S;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

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

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
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

// What a worker warp multiplies its part of a tile by, read ahead of the sums:
// lane l has the scale and bias of channel ch0 + l, and the scales of tokens
// col0 + l, col0 + 32 + l ...
template <int NT>
struct Scales {
  static constexpr int kWords = (Shape<NT>::kCols + 31) / 32;
  float sa[kWords];
  float sb, add;
  int64_t j0, i0;
  int live;    // tokens of this part that exist
  bool mine;   // this lane's channel exists

  __device__ __forceinline__ void read(const Params& p, int tile, int ch0, int col0, int lane) {
    j0 = static_cast<int64_t>(tile / p.token_tiles) * kPairChannels + ch0;
    i0 = static_cast<int64_t>(tile % p.token_tiles) * NT + col0;
    live = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(Shape<NT>::kCols), p.m - i0)));
    mine = j0 + lane < p.n;
    sb = p.b_scale && mine ? p.b_scale[j0 + lane] : 1.0f;
    add = p.bias && mine ? p.bias[j0 + lane] : 0.0f;
#pragma unroll
    for (int i = 0; i < kWords; ++i) sa[i] = p.a_scale && 32 * i + lane < live ? p.a_scale[i0 + 32 * i + lane] : 1.0f;
  }
};

// Scale and store a worker warp's part of a tile, fp32 sums as they are. 16-bit
// results are exchanged between neighbouring lanes, so that a lane holds two
// channels of one token: one 4-byte store for two results.
template <int NT, bool OUT16>
__device__ __forceinline__ void store_tile(const Params& p, const Scales<NT>& s, const uint32_t (&acc)[Shape<NT>::kCols], int lane) {
  constexpr int kCols = Shape<NT>::kCols;
  constexpr int kSlab = kCols < 16 ? kCols : 16;
  if (s.j0 >= p.n || s.live == 0) return;
  const int odd = lane & 1;
  const bool paired = OUT16 && s.j0 + 32 <= p.n && p.ld_out % 2 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 3) == 0;
#pragma unroll
  for (int c0 = 0; c0 < kCols; c0 += kSlab) {
    if (c0 >= s.live) break;
    float v[kSlab];
#pragma unroll
    for (int c = 0; c < kSlab; ++c)
      v[c] = __fmaf_rn(__fmul_rn(__uint_as_float(acc[c0 + c]), __shfl_sync(kFullMask, s.sa[c0 / 32], (c0 + c) & 31)), s.sb, s.add);
    if constexpr (!OUT16) {
      float* o = static_cast<float*>(p.out) + (s.i0 + c0) * p.ld_out + s.j0 + lane;
#pragma unroll
      for (int c = 0; c < kSlab; ++c)
        if (s.mine && c0 + c < s.live) o[c * p.ld_out] = v[c];
    } else {
      uint32_t two[kSlab / 2];  // tokens c and c + 1 of this lane's channel
#pragma unroll
      for (int c = 0; c < kSlab; c += 2) {
        if (p.out_dtype == kBF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[c], v[c + 1]);
          two[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(v[c], v[c + 1]);
          two[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      if (paired) {
        const uint32_t pick = odd ? 0x3276u : 0x5410u;
        uint32_t* o = static_cast<uint32_t*>(p.out) + ((s.i0 + c0 + odd) * p.ld_out + s.j0 + lane - odd) / 2;
#pragma unroll
        for (int c = 0; c < kSlab; c += 2) {
          const uint32_t other = __shfl_xor_sync(kFullMask, two[c / 2], 1);
          if (c0 + c + odd < s.live) o[c / 2 * p.ld_out] = __byte_perm(two[c / 2], other, pick);
        }
      } else {
        uint16_t* o = static_cast<uint16_t*>(p.out) + (s.i0 + c0) * p.ld_out + s.j0 + lane;
#pragma unroll
        for (int c = 0; c < kSlab; ++c)
          if (s.mine && c0 + c < s.live) o[c * p.ld_out] = static_cast<uint16_t>(two[c / 2] >> (16 * (c & 1)));
      }
    }
  }
}

// The integer sums themselves.
template <int NT>
__device__ __forceinline__ void store_sums(const Params& p, const Scales<NT>& s, const uint32_t (&acc)[Shape<NT>::kCols], int lane) {
  int* o = static_cast<int*>(p.out) + s.i0 * p.ld_out + s.j0 + lane;
#pragma unroll
  for (int c = 0; c < Shape<NT>::kCols; ++c)
    if (s.mine && c < s.live) o[c * p.ld_out] = static_cast<int>(acc[c]);
}

// OUT: what is stored: 0 the sums (int32), 1 fp32, 2 a 16-bit type.
template <int NT, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_i8_pair_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                          const Params p) {
  using S = Shape<NT>;
  constexpr int kCols = S::kCols;
  constexpr int kDrain = kCols < 16 ? kCols : 16;  // columns read at a time
  constexpr int kRing = S::kRing;
  constexpr bool kSums = OUT == 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* xring = smem;
  uint8_t* wring = smem + kRing * S::kXBytes;
  uint64_t* w_full = reinterpret_cast<uint64_t*>(wring + S::kWStages * kWBytes);
  uint64_t* w_empty = w_full + S::kWStages;
  uint64_t* x_full = w_empty + S::kWStages;  // the even CTA's are used: both CTAs' tokens
  uint64_t* c_full = x_full + kRing;         // the even CTA's are used: both CTAs' converted channels
  uint64_t* done = c_full + kRing;           // the MMAs of a stage have read both rings
  uint64_t* acc_full = done + kRing;
  uint64_t* acc_empty = acc_full + 1;        // the even CTA's is used
  uint64_t* drain = acc_empty + 1;
  uint64_t* meet = drain + 1;                // the workers of this CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meet + 1);
  __shared__ int abort_flag;
  __shared__ unsigned last_flag;

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
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&x_full[s], 1);
      mbar_init(&c_full[s], 8);  // four warps of each CTA
      mbar_init(&done[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * kWorkers);
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

  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&abort_flag) != 0; };
  auto give_up = [&](int bit) {
    atomicOr(p.err, bit);
    *reinterpret_cast<volatile int*>(&abort_flag) = 1;
  };

  Walk walk(p, pair, pairs);
  int tile, k0, k1;

  if (warp == 0) {
    // ---------------------------------------------------- channels (bytes)
    // They are never written by the kernel launched just before this one, so
    // their loads start while that one still runs.
    if (lane == 0) {
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
      Slot<kRing> s;
      int armed = 0;
      bool ok = true;
      while (ok && walk.next(tile, k0, k1)) {
        const int row = tile % p.token_tiles * NT + static_cast<int>(rank) * (NT / 2);
        for (int k = k0; k < k1; ++k) {
          if (!mbar_wait(&done[s.i], s.phase ^ 1u, p.timeout_ns) || aborted()) {
            if (!aborted()) give_up(kErrProducerTimeout);
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&x_full[s.i], 2 * S::kXBytes);
          const uint32_t bar = cluster_addr(&x_full[s.i], 0);
          uint8_t* dst = xring + s.i * S::kXBytes;
          tma_load_2d_pair(dst, &tmap_x, k * kDepth, row, bar, policy);
          tma_load_2d_pair(dst + S::kXBytes / 2, &tmap_x, k * kDepth + kDepth / 2, row, bar, policy);
          s.advance();
          if (armed < kRing) ++armed;
        }
      }
      if (!ok && leader) {
        for (; armed > 0; --armed) {
          if (s.i == 0) {
            s.i = kRing;
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
    // 32 tokens instead of 45 from a branch on the lane's number. An MMA of
    // 256 tokens takes 130, and few are queued, so the next stage's barriers
    // are looked at while the second half of this one's is still to be issued.
    if (leader) {
      constexpr uint32_t idesc = make_idesc(kPairChannels, NT, 0u);
      Slot<kRing> s;
      uint32_t acc_phase = 0;
      bool ok = true, ready = false;
      while (ok && walk.next(tile, k0, k1)) {
        for (int k = k0; k < k1 && ok; k += kExactStages) {
          const int kend = min(k + kExactStages, k1);
          ok = __all_sync(kFullMask, mbar_wait(acc_empty, acc_phase ^ 1u, p.timeout_ns)) && !aborted();
          tc_fence_after();
          for (int kk = k; kk < kend && ok; ++kk) {
            if (!ready) {
              ok = __all_sync(kFullMask, mbar_wait(&x_full[s.i], s.phase, p.timeout_ns) &&
                                             mbar_wait(&c_full[s.i], s.phase, p.timeout_ns));
              if (!ok) break;
            }
            tc_fence_after();
            const uint64_t b0 = sw128_kmajor_desc(xring + s.i * S::kXBytes);
            const uint64_t b1 = sw128_kmajor_desc(xring + s.i * S::kXBytes + S::kXBytes / 2);
            const uint32_t c = tmem_base + NT + static_cast<uint32_t>(s.i * kStageCols);
            const bool one_lane = elect_one();
            if (one_lane) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                umma_pair_ts(tmem_base, c + static_cast<uint32_t>(8 * i), b0 + static_cast<uint64_t>(2 * i), idesc,
                             (kk != k) | (i != 0));
            }
            __syncwarp();
            Slot<kRing> next = s;
            next.advance();
            ready = __all_sync(kFullMask, mbar_try_wait(&x_full[next.i], next.phase) &&
                                              mbar_try_wait(&c_full[next.i], next.phase));
            if (one_lane) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                umma_pair_ts(tmem_base, c + static_cast<uint32_t>(8 * (i + 4)), b1 + static_cast<uint64_t>(2 * i), idesc, 1u);
              umma_commit_pair(&done[s.i]);
            }
            __syncwarp();
            s = next;
          }
          if (ok && elect_one()) umma_commit_pair(acc_full);
          __syncwarp();
          acc_phase ^= 1u;
        }
      }
      if (!ok && lane == 0 && !aborted()) give_up(kErrConsumerTimeout);
      // Every MMA (they read both CTAs' memories) is done before either exits.
      if (elect_one()) umma_commit_pair(drain);
      __syncwarp();
    }
    if (!mbar_wait(drain, 0, p.timeout_ns)) atomicOr(p.err, kErrDrainTimeout);
    __syncwarp();
  } else {
    // -------------------------------------------------------------- workers
    const int group = (warp - 2) >> 2;
    const int quad = warp & 3;  // TMEM lanes that this warp may access
    const int ch = quad * 32 + lane;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t acc_empty_addr = cluster_addr(acc_empty, 0);
    const uint32_t c_full_addr = cluster_addr(c_full, 0);
    const int total = walk.total();
    bool ok = true;
    // Warp-uniform: whether every lane's wait has ended in time.
    auto fine = [&](bool in_time) { return __all_sync(kFullMask, in_time) != 0; };
    uint32_t meet_phase = 0;
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
        const uint32_t dst = lane_base + NT + rs.i * kStageCols;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint4 raw[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) raw[c] = *reinterpret_cast<const uint4*>(row + (((2 * h + c) ^ (ch & 7)) << 4));
          if (h == 0) {
            ok = fine(mbar_wait(&done[rs.i], rs.phase ^ 1u, p.timeout_ns));
            if (!ok) break;
            tc_fence_after();
          }
          if (h == 3) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_empty[ws.i]);
          }
          uint32_t f[16];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            bytes_to_f16(raw[c].x, f[8 * c + 0], f[8 * c + 1]);
            bytes_to_f16(raw[c].y, f[8 * c + 2], f[8 * c + 3]);
            bytes_to_f16(raw[c].z, f[8 * c + 4], f[8 * c + 5]);
            bytes_to_f16(raw[c].w, f[8 * c + 6], f[8 * c + 7]);
          }
          tmem_st16(dst + 16 * h, f);
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(c_full_addr + rs.i * 8);  // orders TMEM only, as for acc_empty
        ws.advance(kGroups);
        rs.advance(kGroups);
      }
    };

    int finished = 0;  // stages whose accumulator has been read
    uint32_t acc_phase = 0;
    bool waited = false;
    while (ok && walk.next(tile, k0, k1)) {
      if (!waited) {  // the scales may come from the kernel before this one, which may also read `out`
        pdl_wait();
        waited = true;
      }
      Scales<NT> scales;
      scales.read(p, tile, static_cast<int>(rank) * kChannels + quad * 32, group * kCols, lane);
      uint32_t acc[kCols];
      // The whole sum is one accumulator's and fp32 holds it.
      const bool one = k1 - k0 <= kExactStages && k0 == 0 && k1 == p.stages && !kSums;
      for (int k = k0; k < k1 && ok; k += kExactStages) {
        finished += min(kExactStages, k1 - k);
        convert_until(min(finished + kRing, total));
        if (!ok) break;
        ok = fine(mbar_wait(acc_full, acc_phase, p.timeout_ns));
        if (!ok) break;
        acc_phase ^= 1u;
        tc_fence_after();
        auto ld = [&](int c, uint32_t* v) {
          if constexpr (kDrain == 16)
            tmem_ld16(lane_base + group * kCols + c, v);
          else
            tmem_ld8(lane_base + group * kCols + c, v);
        };
        if (one) {
#pragma unroll
          for (int c = 0; c < kCols; c += kDrain) ld(c, acc + c);
          tmem_wait_ld();
        } else {
          if (k == k0) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) acc[c] = 0;
          }
#pragma unroll
          for (int c = 0; c < kCols; c += kDrain) {
            uint32_t v[kDrain];
            ld(c, v);
            tmem_wait_ld();
#pragma unroll
            for (int d = 0; d < kDrain; ++d) acc[c + d] += static_cast<uint32_t>(__float2int_rn(__uint_as_float(v[d])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_addr);
      }
      if (!ok) break;
      if (k0 != 0 || k1 != p.stages) {
        // A shared tile: leave the partial sums, and finish it if all are there.
        const int64_t all = static_cast<int64_t>(p.tiles) * p.stages, first_stage = static_cast<int64_t>(tile) * p.stages;
        const int first = static_cast<int>(((first_stage + 1) * pairs - 1) / all);
        const int last = static_cast<int>(((first_stage + p.stages) * pairs - 1) / all);
        auto slot_of = [&](int who) {
          return p.partial + (static_cast<int64_t>(who * 2 + static_cast<int>(rank)) * 2 + (who == first ? 1 : 0)) * (kChannels * NT);
        };
        int* mine = slot_of(pair) + group * kCols * kChannels + ch;
#pragma unroll
        for (int c = 0; c < kCols; ++c) __stcg(mine + c * kChannels, static_cast<int>(acc[c]));
        __threadfence();
        ok = workers_meet();
        if (!ok) break;
        if (threadIdx.x == 64) {
          const unsigned n = atomicAdd(&p.arrived[first * 2 + static_cast<int>(rank)], 1u) + 1u;
          const bool fin = n == static_cast<unsigned>(last - first + 1);
          if (fin) p.arrived[first * 2 + static_cast<int>(rank)] = 0u;
          __threadfence();
          last_flag = fin ? 1u : 0u;
        }
        ok = workers_meet();
        if (!ok) break;
        const bool fin = *reinterpret_cast<volatile unsigned*>(&last_flag) != 0;
        __threadfence();
        ok = workers_meet();  // last_flag may be written again
        if (!ok) break;
        if (!fin) continue;
        for (int who = first; who <= last; ++who) {
          if (who == pair) continue;
          const int* theirs = slot_of(who) + group * kCols * kChannels + ch;
#pragma unroll
          for (int c = 0; c < kCols; ++c) acc[c] += static_cast<uint32_t>(__ldcg(theirs + c * kChannels));
        }
      }
      if constexpr (kSums) {
        store_sums<NT>(p, scales, acc, lane);
      } else {
        if (!one) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) acc[c] = __float_as_uint(__int2float_rn(static_cast<int>(acc[c])));
        }
        store_tile<NT, OUT == 2>(p, scales, acc, lane);
      }
    }
    if (!ok && lane == 0 && !aborted()) give_up(kErrConsumerTimeout);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

// 8-bit rows to fp16, [m][pitch], zero past k: eight values a thread.
__global__ void __launch_bounds__(256)
    expand_rows_kernel(const int8_t* __restrict__ a, int64_t ld_a, int64_t m, int k, __half* __restrict__ x, int pitch) {
  pdl_launch_dependents();  // the product may become resident now; it waits for these rows
  const int per = pitch / 8;
  const bool wide = (reinterpret_cast<uintptr_t>(a) & 7) == 0 && ld_a % 8 == 0;
  for (int64_t g = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; g < m * per;
       g += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t i = g / per;
    const int c = static_cast<int>(g - i * per) * 8;
    const int8_t* src = a + i * ld_a + c;
    uint2 raw = make_uint2(0u, 0u);
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
}

bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols, int64_t rows, int64_t pitch_bytes,
              int box_cols, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, int OUT>
cudaError_t launch_t(const MatmulI8Launch& a, const MatmulI8Workspace& w, cudaStream_t st) {
  CUtensorMap mx, mw;
  const int pitch = matmul_i8_pitch(a.k);
  if (!make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, w.rows_f16, pitch, a.m, int64_t(pitch) * 2, kDepth / 2, NT / 2) ||
      !make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.b, a.k, a.n, a.ld_b, kDepth, kChannels))
    return cudaErrorInvalidValue;
  Params p;
  p.out = a.out;
  p.a_scale = a.a_scale;
  p.b_scale = a.b_scale;
  p.bias = a.bias;
  p.ld_out = a.ld_out;
  p.m = a.m;
  p.n = a.n;
  p.out_dtype = a.out_dtype;
  p.stages = pitch / kDepth;
  p.token_tiles = static_cast<int>((a.m + NT - 1) / NT);
  p.tiles = static_cast<int>((a.n + kPairChannels - 1) / kPairChannels * p.token_tiles);
  p.read_once = p.token_tiles == 1;
  p.partial = w.partial;
  p.arrived = w.arrived;
  p.err = w.err;
  p.timeout_ns = w.timeout_ns;
  const int64_t max_pairs = w.num_sms / 2;
  const int64_t total = static_cast<int64_t>(p.tiles) * p.stages;
  // Whole tiles from four rounds on (the last round then costs a fifth at
  // most), or where they come out even.
  p.split = !(p.tiles >= 4 * max_pairs || p.tiles % max_pairs == 0);
  const int64_t pairs = p.split ? std::min(max_pairs, total) : std::min<int64_t>(max_pairs, p.tiles);

  auto fn = matmul_i8_pair_kernel<NT, OUT>;
  static PerDeviceOnce once;
  const cudaError_t limit = once.run(
      [fn] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NT>::kSmem); });
  if (limit != cudaSuccess) return limit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(Shape<NT>::kSmem);
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
  return cudaLaunchKernelEx(&cfg, fn, mx, mw, p);
}

template <int NT>
cudaError_t launch_out(const MatmulI8Launch& a, const MatmulI8Workspace& w, cudaStream_t st) {
  if (a.out_dtype == kI32) return launch_t<NT, 0>(a, w, st);
  if (a.out_dtype == kF32) return launch_t<NT, 1>(a, w, st);
  return launch_t<NT, 2>(a, w, st);
}

}  // namespace

int matmul_i8_pitch(int k) { return (k + kDepth - 1) / kDepth * kDepth; }

size_t matmul_i8_partial_bytes(int num_sms) { return static_cast<size_t>(num_sms) * 2 * kChannels * 256 * sizeof(int); }

bool matmul_i8_tc_fits(const MatmulI8Launch& a) {
  // The tensor map wants 16-byte boundaries and 32-bit coordinates; the kernel counts stages in 32 bits.
  const double stages = (a.n / 256.0 + 1) * (a.m / (a.m <= 128 ? 32.0 : 256.0) + 1) * (a.k / 128.0 + 1);
  return a.k > 0 && (reinterpret_cast<uintptr_t>(a.b) & 15) == 0 && a.ld_b % 16 == 0 && a.n <= INT32_MAX - kPairChannels &&
         stages < 2.0e9;
}

cudaError_t launch_expand_rows(const int8_t* a, int64_t ld_a, int64_t m, int k, void* rows_f16, int num_sms,
                               cudaStream_t st) {
  const int pitch = matmul_i8_pitch(k);
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((m * (pitch / 8) + 255) / 256, int64_t(num_sms) * 16));
  expand_rows_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(a, ld_a, m, k, static_cast<__half*>(rows_f16), pitch);
  return cudaGetLastError();
}

cudaError_t launch_matmul_i8_tc(const MatmulI8Launch& a, const MatmulI8Workspace& w, cudaStream_t st) {
  if (a.m <= 32) return launch_out<32>(a, w, st);
  if (a.m <= 64) return launch_out<64>(a, w, st);
  if (a.m <= 128) return launch_out<128>(a, w, st);
  return launch_out<256>(a, w, st);
}

}  // namespace rbf
