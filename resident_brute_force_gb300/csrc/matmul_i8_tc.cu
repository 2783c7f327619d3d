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
//   warps 2-9   two groups of four; a group takes every other stage. A thread
//               reads its channel's 128 bytes (conflict-free: the swizzle),
//               turns four bytes into two fp16 pairs with two byte permutes
//               (0x6400 | b is 1024 + b) and two subtractions, and stores them
//               in its TMEM lane: 64 columns a stage, a ring of four;
//   warp 10     loads the CTA's tokens (TMA) into a ring of four stages;
//   warp 1      one thread of the even CTA issues the pair's MMAs.
// At the end of a tile (and every 1,024 values) warps 2-9 read the accumulator,
// after they have converted the next four stages, so that the MMAs of the next
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
constexpr int kRing = 4;             // stages of the token ring and of the TMEM ring
constexpr int kExactStages = 1024 / kDepth;
constexpr int kWorkers = 8;          // warps 2-9
constexpr int kThreads = (2 + kWorkers + 1) * 32;
constexpr int kTmemCols = 512;       // accumulator: columns 0-255; converted channels: 256-511
constexpr int kTmemRing = 256;
constexpr int kStageCols = kDepth / 2;
constexpr int kRingBudget = 224 * 1024;

template <int NT>
struct Shape {
  static constexpr int kXBytes = NT * kDepth;  // NT / 2 tokens x 128 fp16
  static constexpr int kWStages = (kRingBudget - kRing * kXBytes) / kWBytes;
  static constexpr int kSmem = 1024 + kRing * kXBytes + kWStages * kWBytes + (2 * kWStages + 3 * kRing + 4) * 8 + 16;
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
  int64_t tiles;
  int split;         // 1: equal shares of all stages, 0: whole tiles
  int read_once;     // 1: the channels are read once (one token tile)
  int* partial;      // split: two tiles of partial sums per CTA
  unsigned* arrived; // split: one counter per CTA, zero between launches
  int* err;
  uint64_t timeout_ns;
};

// The pair's part of the work, one tile's stages [k0, k1) at a time.
struct Walk {
  int64_t at, end;
  int stages, step;
  bool split;

  __device__ __forceinline__ Walk(const Params& p, int pair, int pairs) : stages(p.stages), step(pairs), split(p.split) {
    if (split) {
      const int64_t total = p.tiles * stages;
      at = total * pair / pairs;
      end = total * (pair + 1) / pairs;
    } else {
      at = pair;
      end = p.tiles;
    }
  }
  __device__ __forceinline__ int64_t total() const {
    return split ? end - at : (at < end ? (end - at + step - 1) / step * stages : 0);
  }
  __device__ __forceinline__ bool next(int64_t& tile, int& k0, int& k1) {
    if (at >= end) return false;
    if (split) {
      tile = at / stages;
      k0 = static_cast<int>(at - tile * stages);
      k1 = static_cast<int>(min(static_cast<int64_t>(stages), k0 + (end - at)));
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

// Arrive on the even CTA's barrier once this warp's stores to TMEM are done.
__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// mbar_wait for a barrier that the other CTA's threads arrive on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint64_t timeout_ns) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait_cluster(bar, parity)) return true;
    if (global_timer_ns() - t0 > timeout_ns) return false;
  }
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
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
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

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_i8_pair_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                          const Params p) {
  using S = Shape<NT>;
  constexpr int kCols = NT / 2;  // accumulator columns of one worker thread
  constexpr int kDrain = kCols < 32 ? kCols : 32;  // of those, read at a time
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
      mbar_init(&w_empty[s], kWorkers / 2);
    }
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&x_full[s], 1);
      mbar_init(&c_full[s], kWorkers);  // four warps of each CTA
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
  int64_t tile;
  int k0, k1;

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
        const int row = static_cast<int>(tile / p.token_tiles * kPairChannels) + static_cast<int>(rank) * kChannels;
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
  } else if (warp == 10) {
    // ------------------------------------------------------- tokens (fp16)
    if (lane == 0) {
      pdl_wait();  // the kernel before this one writes them
      const uint64_t policy = l2_policy_evict_last();
      Slot<kRing> s;
      int armed = 0;
      bool ok = true;
      while (ok && walk.next(tile, k0, k1)) {
        const int row = static_cast<int>(tile % p.token_tiles) * NT + static_cast<int>(rank) * (NT / 2);
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
    if (lane == 0) {
      if (leader) {
        constexpr uint32_t idesc = make_idesc(kPairChannels, NT, 0u);
        Slot<kRing> s;
        uint32_t acc_phase = 0;
        bool ok = true;
        while (ok && walk.next(tile, k0, k1)) {
          for (int k = k0; k < k1 && ok; k += kExactStages) {
            const int kend = min(k + kExactStages, k1);
            if (!mbar_wait_cluster(acc_empty, acc_phase ^ 1u, p.timeout_ns) || aborted()) ok = false;
            tc_fence_after();
            for (int kk = k; kk < kend && ok; ++kk) {
              if (!mbar_wait(&x_full[s.i], s.phase, p.timeout_ns) ||
                  !mbar_wait_cluster(&c_full[s.i], s.phase, p.timeout_ns) || aborted()) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint64_t b0 = sw128_kmajor_desc(xring + s.i * S::kXBytes);
              const uint64_t b1 = sw128_kmajor_desc(xring + s.i * S::kXBytes + S::kXBytes / 2);
              const uint32_t c = tmem_base + kTmemRing + static_cast<uint32_t>(s.i * kStageCols);
#pragma unroll
              for (int i = 0; i < kDepth / 16; ++i)
                umma_pair_ts(tmem_base, c + static_cast<uint32_t>(8 * i),
                             (i < 4 ? b0 : b1) + static_cast<uint64_t>(2 * (i & 3)), idesc, (kk != k) | (i != 0));
              umma_commit_pair(&done[s.i]);
              s.advance();
            }
            if (ok) umma_commit_pair(acc_full);
            acc_phase ^= 1u;
          }
        }
        if (!ok && !aborted()) give_up(kErrConsumerTimeout);
        // Every MMA (they read both CTAs' memories) is done before either exits.
        umma_commit_pair(drain);
      }
      if (!mbar_wait(drain, 0, p.timeout_ns)) atomicOr(p.err, kErrDrainTimeout);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- workers
    const int group = (warp - 2) >> 2;
    const int quad = warp & 3;  // TMEM lanes that this warp may access
    const int ch = quad * 32 + lane;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t acc_empty_addr = cluster_addr(acc_empty, 0);
    const int64_t total = walk.total();
    bool ok = true;
    // Warp-uniform: whether every lane's wait has ended in time.
    auto fine = [&](bool in_time) { return __all_sync(kFullMask, in_time && !aborted()); };
    uint32_t meet_phase = 0;
    auto workers_meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      const bool r = fine(mbar_wait(meet, meet_phase, p.timeout_ns));
      meet_phase ^= 1u;
      return r;
    };

    // Convert this group's stages up to (not including) stage `until`.
    int64_t stage = group;
    Slot<S::kWStages> ws;
    ws.advance(group);
    uint32_t ring_slot = static_cast<uint32_t>(group);
    uint32_t ring_phase = 0;
    auto convert_until = [&](int64_t until) {
      for (; ok && stage < until; stage += 2) {
        ok = fine(mbar_wait(&w_full[ws.i], ws.phase, p.timeout_ns));
        if (!ok) break;
        const uint8_t* row = wring + ws.i * kWBytes + ch * kDepth;
        const uint32_t dst = lane_base + kTmemRing + ring_slot * kStageCols;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 raw[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) raw[c] = *reinterpret_cast<const uint4*>(row + (((4 * h + c) ^ (ch & 7)) << 4));
          if (h == 0) {
            ok = fine(mbar_wait(&done[ring_slot], ring_phase ^ 1u, p.timeout_ns));
            if (!ok) break;
            tc_fence_after();
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_empty[ws.i]);
          }
          uint32_t f[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            bytes_to_f16(raw[c].x, f[8 * c + 0], f[8 * c + 1]);
            bytes_to_f16(raw[c].y, f[8 * c + 2], f[8 * c + 3]);
            bytes_to_f16(raw[c].z, f[8 * c + 4], f[8 * c + 5]);
            bytes_to_f16(raw[c].w, f[8 * c + 6], f[8 * c + 7]);
          }
          tmem_st32(dst + 32 * h, f);
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_release_cluster(cluster_addr(&c_full[ring_slot], 0));
        ws.advance(2);
        ring_slot ^= 2u;
        if (ring_slot == static_cast<uint32_t>(group)) ring_phase ^= 1u;
      }
    };

    int64_t finished = 0;  // stages whose accumulator has been read
    uint32_t acc_phase = 0;
    bool waited = false;
    while (ok && walk.next(tile, k0, k1)) {
      uint32_t acc[kCols];
      const bool one = k1 - k0 <= kExactStages && k0 == 0 && k1 == p.stages;  // a whole sum that fp32 holds
      for (int k = k0; k < k1 && ok; k += kExactStages) {
        finished += min(kExactStages, k1 - k);
        convert_until(min(finished + kRing, total));
        if (!ok) break;
        ok = fine(mbar_wait(acc_full, acc_phase, p.timeout_ns));
        if (!ok) break;
        acc_phase ^= 1u;
        tc_fence_after();
        if (one) {
#pragma unroll
          for (int c = 0; c < kCols; c += 16) tmem_ld16(lane_base + group * kCols + c, acc + c);
          tmem_wait_ld();
        } else {
          if (k == k0) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) acc[c] = 0;
          }
#pragma unroll
          for (int c = 0; c < kCols; c += kDrain) {
            uint32_t v[kDrain];
#pragma unroll
            for (int d = 0; d < kDrain; d += 16) tmem_ld16(lane_base + group * kCols + c + d, v + d);
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
      if (!waited) {  // the scales may come from the kernel before this one, which may also read `out`
        pdl_wait();
        waited = true;
      }
      if (k0 != 0 || k1 != p.stages) {
        // A shared tile: leave the partial sums, and finish it if all are there.
        const int64_t all = p.tiles * p.stages, first_stage = tile * p.stages;
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
      const int64_t j = tile / p.token_tiles * kPairChannels + static_cast<int>(rank) * kChannels + ch;
      const int64_t i0 = tile % p.token_tiles * NT + group * kCols;
      if (j < p.n && i0 < p.m) {
        const int live = static_cast<int>(min(static_cast<int64_t>(kCols), p.m - i0));
        const float sb = p.b_scale ? p.b_scale[j] : 1.0f;
        const float add = p.bias ? p.bias[j] : 0.0f;
        const float* sa = p.a_scale ? p.a_scale + i0 : nullptr;
        auto value = [&](int c) {
          float f = one ? __uint_as_float(acc[c]) : __int2float_rn(static_cast<int>(acc[c]));
          if (sa) f = __fmul_rn(f, sa[c]);
          return __fadd_rn(__fmul_rn(f, sb), add);
        };
        const int64_t at = i0 * p.ld_out + j;
        if (p.out_dtype == kI32) {
          int* o = static_cast<int*>(p.out) + at;
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (c < live) o[c * p.ld_out] = one ? __float2int_rn(__uint_as_float(acc[c])) : static_cast<int>(acc[c]);
        } else if (p.out_dtype == kF32) {
          float* o = static_cast<float*>(p.out) + at;
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (c < live) o[c * p.ld_out] = value(c);
        } else if (p.out_dtype == kBF16) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (c < live) o[c * p.ld_out] = __float2bfloat16_rn(value(c));
        } else {
          __half* o = static_cast<__half*>(p.out) + at;
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (c < live) o[c * p.ld_out] = __float2half_rn(value(c));
        }
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

template <int NT>
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
  p.tiles = (a.n + kPairChannels - 1) / kPairChannels * p.token_tiles;
  p.read_once = p.token_tiles == 1;
  p.partial = w.partial;
  p.arrived = w.arrived;
  p.err = w.err;
  p.timeout_ns = w.timeout_ns;
  const int64_t max_pairs = w.num_sms / 2;
  const int64_t total = p.tiles * p.stages;
  // Whole tiles from four rounds on (the last round then costs a fifth at
  // most), or where they come out even.
  p.split = !(p.tiles >= 4 * max_pairs || p.tiles % max_pairs == 0);
  const int64_t pairs = p.split ? std::min(max_pairs, total) : std::min(max_pairs, p.tiles);

  auto fn = matmul_i8_pair_kernel<NT>;
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

}  // namespace

int matmul_i8_pitch(int k) { return (k + kDepth - 1) / kDepth * kDepth; }

size_t matmul_i8_partial_bytes(int num_sms) { return static_cast<size_t>(num_sms) * 2 * kChannels * 256 * sizeof(int); }

bool matmul_i8_tc_fits(const MatmulI8Launch& a) {
  // The tensor map wants 16-byte boundaries; a row of the map's coordinates is 32 bits.
  return a.k > 0 && (reinterpret_cast<uintptr_t>(a.b) & 15) == 0 && a.ld_b % 16 == 0 && a.n <= INT32_MAX - kPairChannels;
}

cudaError_t launch_expand_rows(const int8_t* a, int64_t ld_a, int64_t m, int k, void* rows_f16, int num_sms,
                               cudaStream_t st) {
  const int pitch = matmul_i8_pitch(k);
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((m * (pitch / 8) + 255) / 256, int64_t(num_sms) * 16));
  expand_rows_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(a, ld_a, m, k, static_cast<__half*>(rows_f16), pitch);
  return cudaGetLastError();
}

cudaError_t launch_matmul_i8_tc(const MatmulI8Launch& a, const MatmulI8Workspace& w, cudaStream_t st) {
  if (a.m <= 32) return launch_t<32>(a, w, st);
  if (a.m <= 64) return launch_t<64>(a, w, st);
  if (a.m <= 128) return launch_t<128>(a, w, st);
  return launch_t<256>(a, w, st);
}

}  // namespace rbf
